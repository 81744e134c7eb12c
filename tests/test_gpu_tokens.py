"""GPU tests of the token operators against their definitions in 64 bits, at
the sizes, types, strides and masks where they can go wrong."""
import math

import pytest
import torch

import token_oracle as o
from token_oracle import TYPES, U32, close, rounding

pytestmark = pytest.mark.gpu


def _api():
    import recsys_table_embedding_gb300 as tbe
    return tbe


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(seed, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=TYPES[dtype], device="cuda").normal_(0, std, generator=_gen(seed))


def _strided(t, extra, shift=0):
    """The same values in a buffer with longer rows that starts `shift` elements in."""
    big = torch.full((t.shape[0] * (t.shape[1] + extra) + shift,), 7.0, dtype=t.dtype, device=t.device)
    v = big[shift:].view(t.shape[0], t.shape[1] + extra)[:, :t.shape[1]]
    v.copy_(t)
    return v


def _ids(seed, n, V, bad=0.1, dtype=torch.int64):
    g = _gen(seed)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    mask = torch.rand(n, generator=g, device="cuda") < bad
    wrong = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -1 - ids, V + ids)
    return torch.where(mask, wrong, ids).to(dtype)


# ---------------------------------------------------------------------------
# token embedding

@pytest.mark.parametrize("D", [1, 2, 3, 8, 12, 33, 64, 100, 256, 257, 1000, 2050])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_lookup(D, types):
    t, out = types
    for i, N in enumerate((1, 2, 31, 700)):
        table = _rand(D + i, (501, D), t)
        ids = _ids(i, N, 501, dtype=torch.int32 if i % 2 else torch.int64)
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        got = _api().tbe_token_forward(table, ids, scale=1.7, dtype=TYPES[out], status=status)
        want = o.token_forward(table, ids, float(torch.tensor(1.7)))
        assert got.dtype == TYPES[out] and got.shape == (N, D)
        close(got, want, 2 * U32 * want.abs() + rounding(want, TYPES[out]))
        assert int(status[0]) == int(((ids < 0) | (ids >= 501)).sum())
        assert status[1:].tolist() == [0, 0, 0]


@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8), (3, 2)])
def test_lookup_strided(extra, shift):
    table = _strided(_rand(1, (300, 40), "bf16"), extra, shift)
    ids = _ids(2, 130, 300, bad=0)
    out = _strided(torch.zeros(130, 40, dtype=torch.bfloat16, device="cuda"), extra, shift)
    ref = out._base.clone()
    got = _api().tbe_token_forward(table, ids, out=out)
    assert got is out
    assert torch.equal(out, table[ids])
    # nothing between the rows was written
    between = torch.ones_like(ref, dtype=torch.bool)
    between[shift:].view(130, 40 + extra)[:, :40] = False
    assert torch.equal(out._base[between], ref[between])


def test_lookup_shapes_and_empty():
    table = _rand(0, (50, 24), "f32")
    ids = _ids(1, 12, 50, bad=0).view(3, 4)
    got = _api().tbe_token_forward(table, ids)
    assert torch.equal(got, table[ids])
    assert torch.equal(_api().tbe_token_forward(table, ids[0, 0]), table[ids[0, 0]])
    assert _api().tbe_token_forward(table, ids[:0]).shape == (0, 4, 24)


def _check_backward(grad, ids, V, scale=1.0, padding=None, dtype=None, base=None, status=None):
    dt = dtype or grad.dtype
    if base is None:
        got = _api().tbe_token_backward(grad, ids, V, scale=scale, padding_id=padding, dtype=dt, status=status)
    else:
        got = base.clone()
        _api().tbe_token_backward(grad, ids, scale=scale, padding_id=padding, grad_table=got,
                                  accumulate=True, status=status)
    want, mag, n = o.token_backward(grad, ids, V, scale, padding)
    bound = (n + 2) * U32 * mag
    if base is not None:
        want = want + base.double()
        bound = bound + 2 * U32 * (mag + base.double().abs()) + rounding(want, dt) + U32 * bound
        untouched = (n == 0).expand_as(want)
        assert torch.equal(got[untouched], base[untouched])
    else:
        bound = bound + rounding(want, dt) * (1 + 2.0 ** -7)
        bound = torch.where(n == 0, torch.zeros_like(bound), bound)
    close(got, want, bound)
    return got


@pytest.mark.parametrize("D", [1, 2, 3, 8, 12, 33, 64, 100, 256, 257, 1000, 2050])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_gradient(D, types):
    t, out = types
    for i, (N, V) in enumerate(((1, 7), (40, 100), (5000, 300), (3000, 9000))):
        ids = _ids(i + D, N, V, dtype=torch.int32 if i % 2 else torch.int64)
        grad = _rand(3 * i + D, (N, D), t, 0.3)
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        _check_backward(grad, ids, V, scale=0.5, dtype=TYPES[out], status=status)
        assert int(status[0]) == int(((ids < 0) | (ids >= V)).sum()) and int(status[1]) == 0
        base = _rand(9 + i, (V, D), out)
        _check_backward(grad, ids, V, scale=0.5, padding=3, dtype=TYPES[out], base=base)


RUNS = [[1], [31], [32], [33], [34], [63, 1], [64, 64], [65], [1] * 70, [33] * 20, [32] * 20, [5, 300, 2, 1000, 7],
        [2500], [1, 31, 33, 31, 1, 96, 97, 3], [16, 48, 17, 15], [8, 9, 40, 7, 200]]


@pytest.mark.parametrize("D,t", [(4, "f32"), (1, "f32"), (24, "f32"), (40, "bf16"), (128, "f32"), (300, "f16"), (17, "bf16"), (1100, "f32")])
@pytest.mark.parametrize("runs", RUNS, ids=[str(r)[:24] for r in RUNS])
def test_gradient_run_lengths(runs, D, t):
    V = 3 * len(runs) + 2
    ids = torch.cat([torch.full((n,), 3 * i + 1, dtype=torch.int64) for i, n in enumerate(runs)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(D))].cuda()
    grad = _rand(D, (len(ids), D), t)
    a = _check_backward(grad, ids, V)
    # the order of the sum does not depend on the launch
    assert torch.equal(a, _api().tbe_token_backward(grad, ids, V))
    # padding and ids that are left out, spread among them
    mixed = ids.clone()
    mixed[::3] = -1
    mixed[1::5] = 1
    _check_backward(grad, mixed, V, padding=1)


@pytest.mark.parametrize("N,V", [(1023, 5000), (1024, 3), (1025, 40), (2047, 50), (2047, 100_003), (2048, 50), (2049, 50), (4096, 70000), (4097, 3), (20000, 1), (65536, 65535),
                                 (70001, 65536), (140000, 131072), (300000, 2000)])
def test_gradient_sizes(N, V):
    g = _gen(N)
    rank = torch.rand(N, generator=g, device="cuda").pow(4)
    ids = (rank * V).long().clamp(max=V - 1)
    grad = _rand(N, (N, 24), "bf16")
    _check_backward(grad, ids, V, dtype=torch.float32)


@pytest.mark.parametrize("N,V,D", [(3, 70_000, 1), (50, 40_001, 3), (700, 9001, 5), (2000, 20_000, 37), (40, 5, 9001), (2048, 30, 2050)])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
def test_gradient_of_few_tokens(N, V, D, types):
    t, out = types
    grad = _rand(N, (N, D), t)
    for seed in (1, 2):
        g = _gen(seed)
        ids = (torch.rand(N, generator=g, device="cuda").pow(3 * seed) * V).long().clamp(max=V - 1)
        a = _check_backward(grad, ids, V, dtype=TYPES[out], padding=0)
        _check_backward(grad, ids, V, dtype=TYPES[out], base=_rand(5, (V, D), out))
        assert torch.equal(a, _api().tbe_token_backward(grad, ids, V, padding_id=0, dtype=TYPES[out]))


def test_gradient_nothing_to_sum():
    grad = _rand(0, (64, 20), "f32")
    for ids in (torch.full((64,), -1, device="cuda"), torch.full((64,), 5, device="cuda")):
        got = _api().tbe_token_backward(grad, ids, 9, padding_id=5)
        assert torch.equal(got, torch.zeros_like(got))
        base = _rand(1, (9, 20), "f32")
        kept = base.clone()
        _api().tbe_token_backward(grad, ids, grad_table=base, padding_id=5, accumulate=True)
        assert torch.equal(base, kept)
    got = _api().tbe_token_backward(grad[:0], ids[:0], 9)
    assert torch.equal(got, torch.zeros_like(got)) and got.shape == (9, 20)


def test_gradient_infinities_stay_in_their_row():
    ids = torch.tensor([2, 4, 2, -1, 6], device="cuda")
    grad = torch.ones(5, 16, device="cuda")
    grad[0, 3], grad[3], grad[4, 5] = math.inf, math.nan, math.nan
    got = _api().tbe_token_backward(grad, ids, 8, padding_id=4)
    want = torch.zeros(8, 16, device="cuda")
    want[2], want[6] = 2, 1
    want[2, 3], want[6, 5] = math.inf, math.nan
    assert torch.equal(torch.nan_to_num(got, nan=-5), torch.nan_to_num(want, nan=-5))


@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_strided(extra, shift, accumulate):
    ids = _ids(5, 900, 60)
    grad = _rand(6, (900, 40), "bf16")
    base = _rand(7, (60, 40), "f32")
    out = _strided(base, extra, shift)
    before = out._base.clone()
    _api().tbe_token_backward(_strided(grad, extra, shift), ids, grad_table=out, accumulate=accumulate)
    want = base.clone() if accumulate else torch.empty_like(base)
    _api().tbe_token_backward(grad, ids, grad_table=want, accumulate=accumulate)
    want64, mag, n = o.token_backward(grad, ids, 60, 1.0)
    close(out, want.double(), 2 * (n + 4) * U32 * (mag + base.double().abs()))
    between = torch.ones_like(before, dtype=torch.bool)
    between[shift:].view(60, 40 + extra)[:, :40] = False
    assert torch.equal(out._base[between], before[between])


def test_gradient_of_one_row_for_all_tokens():
    # an expanded gradient (stride 0): every token has the same row
    ids = _ids(8, 500, 40, bad=0)
    grad = _rand(9, (1, 32), "f32").expand(500, 32)
    _check_backward(grad, ids, 40)


def test_lookup_and_gradient_are_adjoint():
    # the lookup is linear in the table: <G, E(W + h) - E(W)> = <E'(G), h>
    W, h = _rand(1, (90, 36), "f32"), _rand(2, (90, 36), "f32")
    ids = _ids(3, 800, 90)
    G = _rand(4, (800, 36), "f32")
    api = _api()
    lhs = (G.double() * (api.tbe_token_forward(W + h, ids, scale=3.0).double() -
                         api.tbe_token_forward(W, ids, scale=3.0).double())).sum()
    dW = api.tbe_token_backward(G, ids, 90, scale=3.0)
    rhs = (dW.double() * ((W + h) - W).double()).sum()
    size = (G.double().abs() * api.tbe_token_forward((W.abs() + h.abs()), ids, scale=3.0).double()).sum()
    assert abs(float(lhs - rhs)) <= float(size) * U32 * (800 / 90 * 4 + 8)


def test_offsets_beyond_32_bits():
    V, D = 40_000_000, 64                      # 2.56e9 elements
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, 33_554_432, V - 2, V - 1], device="cuda")
    table[ids] = torch.arange(1, 6, device="cuda", dtype=torch.bfloat16)[:, None]
    got = _api().tbe_token_forward(table, ids)
    assert torch.equal(got, table[ids])
    grad = _rand(0, (5, D), "bf16")
    dW = _api().tbe_token_backward(grad, ids, V, scale=1.0)
    want = (grad[0].float() + grad[4].float()).bfloat16()
    assert torch.equal(dW[V - 1], want) and torch.equal(dW[33_554_432], grad[2]) and torch.equal(dW[V - 2], grad[3])
    assert torch.equal(dW[0], grad[1])
    dW[ids] = 0
    assert int(torch.count_nonzero(dW)) == 0


# ---------------------------------------------------------------------------
# routing

def _experts(seed, T, K, E, drop, dtype=torch.int32, skew=False):
    g = _gen(seed)
    u = torch.rand((T, K), generator=g, device="cuda")
    ids = ((u * u if skew else u) * E).long().clamp(max=E - 1)
    gone = torch.rand((T, K), generator=g, device="cuda") < drop
    wrong = torch.where(torch.rand((T, K), generator=g, device="cuda") < 0.5, -1, E + 3)
    return torch.where(gone, wrong, ids).to(dtype)


ROUTES = [(1, 1, 1), (1, 8, 64), (2, 3, 5), (7, 2, 300), (64, 4, 16), (341, 3, 37), (512, 2, 8), (513, 2, 8), (1025, 1, 1),
          (1000, 8, 1000), (4096, 2, 4096), (2048, 2, 9), (4097, 1, 4), (3000, 6, 128), (20000, 8, 7)]


@pytest.mark.parametrize("T,K,E", ROUTES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_route_sort(T, K, E, drop):
    for dtype, skew in ((torch.int32, False), (torch.int64, True)):
        ids = _experts(T + K, T, K, E, drop, dtype, skew)
        slot, source, offset = o.route(ids.cpu(), E)
        r = _api().tbe_route_sort(ids, E)
        assert torch.equal(r.offset.cpu(), offset)
        assert torch.equal(r.slot.cpu(), slot)
        assert torch.equal(r.source.cpu(), source)
        x = _rand(1, (T, 20), "bf16")
        rows, r2 = _api().tbe_route_sort_dispatch(x, ids, E)
        assert torch.equal(r2.slot, r.slot) and torch.equal(r2.source, r.source) and torch.equal(r2.offset, r.offset)
        assert torch.equal(rows, _api().tbe_route_dispatch(x, r))
        want = torch.where((r.source >= 0)[:, None], x[r.source.clamp(min=0).long() // K], 0)
        assert torch.equal(rows, want)


@pytest.mark.parametrize("H", [1, 2, 5, 8, 36, 64, 100, 501, 1024, 2056])
@pytest.mark.parametrize("t,wt", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_route_rows(H, t, wt):
    for T, K, E, drop in ((1, 1, 3, 0.0), (1, 8, 16, 0.2), (37, 3, 5, 0.3), (260, 9, 12, 0.1), (9, 2, 4, 1.0)):
        ids = _experts(H + T, T, K, E, drop)
        r = _api().tbe_route_sort(ids, E)
        M = int(r.offset[-1])
        y, w = _rand(1, (T * K, H), t), _rand(2, (T, K), wt)
        y[M:] = math.nan                                   # rows without a pair are not read
        w[r.slot < 0] = math.nan                           # nor are dropped pairs' weights
        out = _api().tbe_route_combine(y, r, w)
        want, mag = o.combine(y, r.slot, w)
        close(out, want, (K + 2) * U32 * mag + rounding(want, TYPES[t]) * (1 + 2.0 ** -7))
        dx = _api().tbe_route_dispatch_backward(y, r)
        want, mag = o.combine(y, r.slot)
        close(dx, want, (K + 2) * U32 * mag + rounding(want, TYPES[t]) * (1 + 2.0 ** -7))
        dout = _rand(3, (T, H), t)
        dy, dw = _api().tbe_route_combine_backward(dout, y, r, w)
        wy, ww, mag = o.combine_backward(dout, y, r.slot, w)
        close(dy, wy, 2 * U32 * wy.abs() + rounding(wy, TYPES[t]))
        close(dw, ww, (H + 2) * U32 * mag + rounding(ww, TYPES[wt]) * (1 + 2.0 ** -7))
        assert torch.equal(dy[M:], torch.zeros_like(dy[M:])) and dw.dtype == TYPES[wt]


@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8)])
def test_route_strided(extra, shift):
    T, K, E, H = 75, 4, 6, 48
    ids = _experts(1, T, K, E, 0.2)
    x, y = _rand(2, (T, H), "f16"), _rand(3, (T * K, H), "f16")
    w, dout = _rand(4, (T, K), "f32"), _rand(5, (T, H), "f16")
    api = _api()
    r = api.tbe_route_sort(ids, E)
    s = lambda v: _strided(v, extra, shift)  # noqa: E731
    z = lambda n: _strided(torch.zeros(n, H, dtype=torch.float16, device="cuda"), extra, shift)  # noqa: E731
    assert torch.equal(api.tbe_route_dispatch(s(x), r, rows=z(T * K)), api.tbe_route_dispatch(x, r))
    assert torch.equal(api.tbe_route_combine(s(y), r, w, out=z(T)), api.tbe_route_combine(y, r, w))
    assert torch.equal(api.tbe_route_dispatch_backward(s(y), r, grad_x=z(T)), api.tbe_route_dispatch_backward(y, r))
    dy, dw = api.tbe_route_combine_backward(s(dout), s(y), r, w, grad_rows=z(T * K))
    ey, ew = api.tbe_route_combine_backward(dout, y, r, w)
    want, ww, mag = o.combine_backward(dout, y, r.slot, w)
    assert torch.equal(dy, ey)
    close(dw, ww, (H + 2) * U32 * mag + rounding(ww, torch.float32))
    close(ew, ww, (H + 2) * U32 * mag + rounding(ww, torch.float32))


def test_route_no_tokens():
    api = _api()
    ids = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 16, device="cuda")
    rows, r = api.tbe_route_sort_dispatch(x, ids, 9)
    assert rows.shape == (0, 16) and r.offset.tolist() == [0] * 10
    w = torch.zeros(0, 4, device="cuda")
    assert api.tbe_route_combine(rows, r, w).shape == (0, 16)
    assert [t.shape for t in api.tbe_route_combine_backward(x, rows, r, w)] == [(0, 16), (0, 4)]


def test_route_gradients_are_adjoint():
    # dispatch is linear, combine is linear in rows and in weights
    api = _api()
    T, K, E, H = 130, 3, 9, 40
    r = api.tbe_route_sort(_experts(3, T, K, E, 0.2), E)
    x, G = _rand(1, (T, H), "f32"), _rand(2, (T * K, H), "f32")
    rows = api.tbe_route_dispatch(x, r)
    size = float((rows.double().abs() * G.double().abs()).sum())
    assert abs(float((rows.double() * G.double()).sum() -
                     (x.double() * api.tbe_route_dispatch_backward(G, r).double()).sum())) <= size * U32 * 16
    y, w, dout = _rand(3, (T * K, H), "f32"), _rand(4, (T, K), "f32"), _rand(5, (T, H), "f32")
    out = api.tbe_route_combine(y, r, w)
    dy, dw = api.tbe_route_combine_backward(dout, y, r, w)
    f = float((out.double() * dout.double()).sum())
    size = float((api.tbe_route_combine(y.abs(), r, w.abs()).double() * dout.double().abs()).sum())
    assert abs(f - float((dy.double() * y.double()).sum())) <= size * U32 * 16
    assert abs(f - float((dw.double() * w.double()).sum())) <= size * U32 * (H + 16)


def test_route_rows_beyond_32_bits():
    T, K, E, H = 70_000, 8, 4, 4096                       # 2.3e9 elements
    ids = _experts(1, T, K, E, 0.01)
    x = _rand(2, (T, H), "bf16")
    api = _api()
    rows, r = api.tbe_route_sort_dispatch(x, ids, E)
    s = torch.randint(0, T * K, (2000,), device="cuda", generator=_gen(3))
    s[:3] = torch.tensor([T * K - 1, int(r.offset[-1]) - 1, 0])
    src = r.source[s].long()
    want = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // K], 0)
    assert torch.equal(rows[s], want)
    back = api.tbe_route_dispatch_backward(rows, r)
    n = (r.slot >= 0).sum(1, keepdim=True).float()
    assert torch.equal(back, (x.float() * n).bfloat16())


# ---------------------------------------------------------------------------
# distillation

def _distill_case(seed, N, V, K, t, tt="f32", short=True, idx=torch.int32):
    g = _gen(seed)
    z = _rand(seed, (N, V), t, 2.0)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] if V >= K else
                       torch.randint(0, V, (K,), generator=g, device="cuda") for _ in range(N)])
    top = (torch.randn((N, K), generator=g, device="cuda") * 2 + 3).to(TYPES[tt])
    if short:
        kept = torch.randint(0, K + 1, (N, 1), generator=g, device="cuda")
        ids = torch.where(torch.arange(K, device="cuda") < kept, ids, -1)
    gl = torch.rand(N, generator=g, device="cuda") + 0.1
    return z, ids.to(idx), top, gl


def _check_distill(z, ids, top, gl, c, **kw):
    api = _api()
    want = o.distill(z, ids, top, gl, c)
    for stored in (False, True):
        if stored:
            loss, lse = api.tbe_distill_forward(z, ids, top, temperature=c)
            grad = api.tbe_distill_backward(z, ids, top, lse, gl, temperature=c)
        else:
            loss, lse, grad = api.tbe_distill_loss_grad(z, ids, top, gl, temperature=c)
        bl, bs, bg = o.distill_bounds(z, ids, top, gl, c, want, True)
        close(loss, want[0], bl)
        close(lse, want[1], bs)
        close(grad, want[2], bg)
        empty = (want[3].sum(1) == 0)
        assert not grad[empty].any() and not loss[empty].any() and not lse[empty].any()


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 100, 257, 1000, 4097, 8192, 8200, 16389, 50021, 131072, 200003])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_distill(V, t):
    for i, (N, K, c) in enumerate(((1, 1, 1.0), (3, 5, 2.0), (9, 64, 0.7))):
        case = _distill_case(V + i, N, V, K, t, "f32" if i % 2 else t, idx=torch.int64 if i else torch.int32)
        _check_distill(*case, c)


@pytest.mark.parametrize("K", [1, 2, 31, 33, 256, 1000, 1024])
def test_distill_entries(K):
    _check_distill(*_distill_case(K, 70, 2001, K, "f16"), 1.0)        # more rows than share a launch with their teacher
    _check_distill(*_distill_case(K, 6, 3001, K, "f32", short=False), 1.5)
    _check_distill(*_distill_case(K, 6, 501, K, "bf16"), 3.0)


@pytest.mark.parametrize("V", [700_003, 1_000_000])
def test_distill_long_rows(V):
    _check_distill(*_distill_case(1, 2, V, 40, "f32"), 1.0)
    _check_distill(*_distill_case(2, 2, V, 40, "bf16"), 2.0)


def test_distill_repeated_ids():
    z, ids, top, gl = _distill_case(4, 8, 300, 48, "f32", short=False)
    ids = ids % 7
    ids[:, ::5] = -1
    _check_distill(z, ids, top, gl, 2.0)


@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("t", ["f32", "f16"])
def test_distill_strided(extra, shift, t):
    api = _api()
    z, ids, top, gl = _distill_case(5, 7, 9001, 20, t)
    zs = _strided(z, extra, shift)
    want = o.distill(z, ids, top, gl, 1.0)
    bound = o.distill_bounds(z, ids, top, gl, 1.0, want, True)
    for oe, os in ((extra, shift), (0, 0), (1, 3)):
        for two in (False, True):
            out = _strided(torch.zeros_like(z), oe, os)
            before = out._base.clone()
            if two:
                loss, lse = api.tbe_distill_forward(zs, ids, top)
                api.tbe_distill_backward(zs, ids, top, lse, gl, grad_logits=out)
            else:
                loss, lse, _ = api.tbe_distill_loss_grad(zs, ids, top, gl, grad_logits=out)
            close(loss, want[0], bound[0])
            close(out, want[2], bound[2])
            between = torch.ones_like(before, dtype=torch.bool)
            between[os:].view(7, 9001 + oe)[:, :9001] = False
            assert torch.equal(out._base[between], before[between])


@pytest.mark.parametrize("V", [50, 9001, 40000, 800_001])
def test_distill_in_place(V):
    api = _api()
    z, ids, top, gl = _distill_case(6, 5, V, 30, "bf16")
    _, lse, want = api.tbe_distill_loss_grad(z, ids, top, gl)
    two = z.clone()
    api.tbe_distill_backward(two, ids, top, lse, gl, grad_logits=two)
    one = z.clone()
    _, _, got = api.tbe_distill_loss_grad(one, ids, top, gl, grad_logits=one)
    assert got is one and torch.equal(one, want)
    assert torch.equal(two, api.tbe_distill_backward(z, ids, top, lse, gl))


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [600, 20000])
def test_distill_masked_logits(t, V):
    # masked columns: -inf and the type's lowest value have probability 0
    z, ids, top, gl = _distill_case(7, 6, V, 16, t, short=False)
    lowest = torch.finfo(TYPES[t]).min
    free = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids.long(), True)
    mask = (torch.rand(z.shape, generator=_gen(8), device="cuda") < 0.5) & ~free
    z = torch.where(mask, torch.where(torch.arange(V, device="cuda") % 2 == 0, -math.inf, lowest).to(z.dtype), z)
    top[0, 3:] = -math.inf                                  # entries without probability
    _check_distill(z, ids, top, gl, 1.0)
    _check_distill(z, ids, top, gl, 2.5)
    # a teacher entry on a masked column: infinite loss, finite gradient
    z[1, ids[1, 0].long()] = -math.inf
    loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, gl)
    assert float(loss[1]) == math.inf and bool(torch.isfinite(grad).all()) and bool(torch.isfinite(lse).all())
    # ... unless its own probability is 0
    z[0, ids[0, 5].long()] = -math.inf
    loss, _, _ = _api().tbe_distill_loss_grad(z, ids, top, gl)
    assert math.isfinite(float(loss[0]))


@pytest.mark.parametrize("V", [600, 20000])
def test_distill_rows_without_entries(V):
    # padding positions: zeros whatever the row holds, and no other row changes
    z, ids, top, gl = _distill_case(9, 6, V, 10, "f32", short=False)
    loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, gl)
    ids2, top2, z2, gl2 = ids.clone(), top.clone(), z.clone(), gl.clone()
    ids2[1], top2[3], z2[1], z2[3] = -1, -math.inf, math.nan, math.inf
    gl2[1] = math.nan
    for two in (False, True):
        if two:
            a, b = _api().tbe_distill_forward(z2, ids2, top2)
            c = _api().tbe_distill_backward(z2, ids2, top2, b, gl2)
        else:
            a, b, c = _api().tbe_distill_loss_grad(z2, ids2, top2, gl2)
        for r in range(6):
            if r in (1, 3):
                assert float(a[r]) == 0 and float(b[r]) == 0 and not c[r].any()
            elif not two:
                assert a[r] == loss[r] and b[r] == lse[r] and torch.equal(c[r], grad[r])


def test_distill_nan_reaches_its_row_only():
    for where in ("logit", "teacher"):
        z, ids, top, gl = _distill_case(10, 4, 5000, 10, "f32", short=False)
        if where == "logit":
            z[2, 77] = math.nan
        else:
            top[2, 1] = math.nan
        loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, gl)
        assert math.isnan(float(loss[2])) and bool(torch.isnan(grad[2, ids[2].long()]).all())
        assert bool(torch.isfinite(loss[[0, 1, 3]]).all()) and bool(torch.isfinite(grad[[0, 1, 3]]).all())


def test_distill_counts_ids_beyond_the_columns():
    z, ids, top, gl = _distill_case(11, 5, 100, 8, "f32", short=False)
    clean = ids.clone()
    ids[0, 2], ids[3, 0], ids[3, 1], ids[4, 4] = 100, 2 ** 31 - 1, 101, -9
    clean[0, 2], clean[3, 0], clean[3, 1], clean[4, 4] = -1, -1, -1, -1
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = _api().tbe_distill_loss_grad(z, ids, top, gl, status=status)
    assert status.tolist() == [3, 0, 0, 0]
    _api().tbe_distill_forward(z, ids, top, status=status)
    assert status.tolist() == [6, 0, 0, 0]
    b = _api().tbe_distill_loss_grad(z, clean, top, gl)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_distill_gradient_against_differences():
    # (loss(z + h e_j) - loss(z - h e_j)) / 2h; the third derivative of the
    # loss is below 1 / c, each loss is off by at most its bound
    c, h = 2.0, 0.05
    z, ids, top, _ = _distill_case(12, 1, 40, 6, "f32", short=False)
    one = torch.ones(1, device="cuda")
    _, _, grad = _api().tbe_distill_loss_grad(z, ids, top, one, temperature=c)
    steps = torch.eye(40, device="cuda") * h
    many = lambda x: _api().tbe_distill_forward(  # noqa: E731
        x.contiguous(), ids.expand(40, -1).contiguous(), top.expand(40, -1).contiguous(), temperature=c)[0].double()
    plus, minus = z + steps, z - steps
    width = (plus - minus).double().diagonal()
    numeric = (many(plus) - many(minus)) / width
    want = o.distill(z, ids, top, one, c)
    b_loss = float(o.distill_bounds(z, ids, top, one, c, want, False)[0])
    assert float((numeric - grad[0].double()).abs().max()) <= h * h / 6 / c + 2 * b_loss / (2 * h)


@pytest.mark.parametrize("gl", [None, 0.25])
def test_distill_one_factor_for_all_rows(gl):
    z, ids, top, _ = _distill_case(13, 5, 700, 9, "f32")
    full = torch.full((5,), 1.0 if gl is None else gl, device="cuda")
    a = _api().tbe_distill_loss_grad(z, ids, top, gl)
    b = _api().tbe_distill_loss_grad(z, ids, top, full)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    lse = a[1]
    assert torch.equal(_api().tbe_distill_backward(z, ids, top, lse, gl), _api().tbe_distill_backward(z, ids, top, lse, full))


def test_distill_leading_dimensions_and_no_rows():
    z, ids, top, gl = _distill_case(14, 6, 333, 5, "bf16")
    a = _api().tbe_distill_loss_grad(z, ids, top, gl)
    b = _api().tbe_distill_loss_grad(z.view(2, 3, 333), ids.view(2, 3, 5), top.view(2, 3, 5), gl.view(2, 3))
    assert b[0].shape == (2, 3) and b[2].shape == (2, 3, 333)
    assert all(torch.equal(x.reshape(-1), y.reshape(-1)) for x, y in zip(a, b))
    n = _api().tbe_distill_loss_grad(z[:0], ids[:0], top[:0], gl[:0])
    assert [t.shape for t in n] == [(0,), (0,), (0, 333)]


def test_distill_offsets_beyond_32_bits():
    N, V = 17_000, 131_072                                  # 2.2e9 elements
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    last = _distill_case(15, 3, V, 8, "bf16", short=False)
    z[-3:] = last[0]
    ids = torch.full((N, 8), -1, dtype=torch.int32, device="cuda")
    ids[-3:] = last[1]
    top = torch.zeros(N, 8, device="cuda")
    top[-3:] = last[2]
    want = _api().tbe_distill_loss_grad(*last[:3], 1.0)
    loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, 1.0, grad_logits=z)
    assert torch.equal(loss[-3:], want[0]) and torch.equal(grad[-3:], want[2])
    assert int(torch.count_nonzero(grad[:-3])) == 0
    loss, lse = _api().tbe_distill_forward(z, ids, top)
    grad = _api().tbe_distill_backward(z, ids, top, lse, 1.0)
    assert int(torch.count_nonzero(grad[:-3])) == 0 and int(torch.count_nonzero(grad[-3:])) > 0


# ---------------------------------------------------------------------------
# streams, graphs, refusals

def _step(api, x, ids, eids, w, top_ids, top, stream=None):
    """One of everything, tied through its results."""
    h = api.tbe_token_forward(x, ids, scale=2.0, stream=stream)
    rows, r = api.tbe_route_sort_dispatch(h, eids, 5, stream=stream)
    out = api.tbe_route_combine(rows, r, w, stream=stream)
    loss, lse, dout = api.tbe_distill_loss_grad(out, top_ids, top, 0.5, stream=stream)
    drows, dw = api.tbe_route_combine_backward(dout, rows, r, w, stream=stream)
    dh = api.tbe_route_dispatch_backward(drows, r, stream=stream)
    dx = api.tbe_token_backward(dh, ids, x.shape[0], scale=2.0, stream=stream)
    return loss, lse, dout, drows, dw, dh, dx


def _step_inputs():
    x = _rand(1, (400, 64), "f32")
    return (x, _ids(2, 3000, 400), _experts(3, 3000, 2, 5, 0.1), _rand(4, (3000, 2), "f32"),
            _ids(5, 3000 * 4, 64).view(3000, 4), _rand(6, (3000, 4), "f32"))


def test_other_stream():
    api = _api()
    args = _step_inputs()
    want = _step(api, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for form in (s, s.cuda_stream):
        got = _step(api, *args, stream=form)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        got = _step(api, *args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_capture():
    api = _api()
    args = _step_inputs()
    want = _step(api, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(api, *args)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _step(api, *args)
    for _ in range(2):
        for t in got:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    api = _api()
    E = api.TbeError
    table, ids = _rand(0, (10, 16), "f32"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(E, match="int32 or int64"):
        api.tbe_token_forward(table, ids.float())
    with pytest.raises(E, match="not contiguous"):
        api.tbe_token_forward(table, ids[::2])
    with pytest.raises(E, match="columns are not contiguous"):
        api.tbe_token_forward(table.t(), ids)
    with pytest.raises(E, match="CUDA"):
        api.tbe_token_forward(table.cpu(), ids.cpu())
    with pytest.raises(E, match="one device"):
        api.tbe_token_forward(table, ids.cpu())
    with pytest.raises(E, match="float32, float16 or bfloat16"):
        api.tbe_token_forward(table.double(), ids)
    with pytest.raises(E, match="status 4"):
        api.tbe_token_forward(table, ids, dtype=torch.float16)
    with pytest.raises(E, match="out is"):
        api.tbe_token_forward(table, ids, out=torch.empty(4, 15, device="cuda"))
    g = _rand(1, (4, 16), "f32")
    with pytest.raises(E, match="rows come from"):
        api.tbe_token_backward(g, ids)
    with pytest.raises(E, match="rows come from"):
        api.tbe_token_backward(g, ids, 10, accumulate=True)
    with pytest.raises(E, match="grad_out is"):
        api.tbe_token_backward(g[:3], ids, 10)
    with pytest.raises(E, match="status 7"):
        api.tbe_token_backward(_rand(1, (3000, 16), "f32"), torch.zeros(3000, dtype=torch.int64, device="cuda"), 10,
                               workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E, match="status 2"):                # overlapping rows of a result
        api.tbe_token_backward(g, ids, grad_table=torch.empty(1, 16, device="cuda").expand(10, 16))
    eids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(E, match="at least one expert"):
        api.tbe_route_sort(eids, 0)
    with pytest.raises(E, match="status 2"):
        api.tbe_route_sort(eids, 5000)
    with pytest.raises(E, match="T, K"):
        api.tbe_route_sort(eids.view(-1), 5)
    r = api.tbe_route_sort(eids, 5)
    with pytest.raises(E, match="status 2"):
        api.tbe_route_dispatch(_rand(0, (5, 8), "f32"), r)
    with pytest.raises(E, match="weights has shape"):
        api.tbe_route_combine(_rand(0, (8, 8), "f32"), r, _rand(0, (4, 3), "f32"))
    with pytest.raises(E, match="status 4"):
        api.tbe_route_combine_backward(_rand(0, (4, 8), "f16"), _rand(0, (8, 8), "f32"), r, _rand(0, (4, 2), "f32"))
    with pytest.raises(E, match="other sizes"):
        api.tbe_route_sort(eids, 6, route=r)
    z, tid, top = _rand(0, (4, 30), "f32"), torch.zeros(4, 3, dtype=torch.int32, device="cuda"), _rand(1, (4, 3), "f32")
    for c in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(E, match="status 2"):
            api.tbe_distill_forward(z, tid, top, temperature=c)
    with pytest.raises(E, match="status 2"):
        api.tbe_distill_forward(z, tid.repeat(1, 400), top.repeat(1, 400))
    with pytest.raises(E, match="teacher_ids are"):
        api.tbe_distill_forward(z, tid[:3], top[:3])
    with pytest.raises(E, match="teacher_logits has shape"):
        api.tbe_distill_forward(z, tid, top[:, :2].contiguous())
    with pytest.raises(E, match="grad_loss is"):
        api.tbe_distill_loss_grad(z, tid, top, torch.ones(3, device="cuda"))
    big = _rand(0, (5, 30), "f32")
    with pytest.raises(E, match="status 2"):                # a gradient that overlaps other rows' logits
        api.tbe_distill_loss_grad(big[:4], tid, top, 1.0, grad_logits=big[1:])
