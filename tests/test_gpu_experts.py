"""GPU tests of the experts' products against their definitions in 64 bits, at
the sizes, types, strides and groups where they can go wrong."""
import pytest
import torch

import layer_oracle as o
from layer_oracle import close, rounded
from token_oracle import TYPES

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


def _route(counts, dropped=0):
    """A route of one expert a token with `counts` tokens of each expert, in a mixed order."""
    ids = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)] + [torch.full((dropped,), -1)]).long()
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))]
    return _api().tbe_route_sort(ids.int().cuda().view(-1, 1), len(counts))


# groups of rows: (rows of each expert, dropped rows); None: one group of 150 rows
GROUPS = {"one": None, "ragged": ([5, 0, 130, 1, 64], 9), "empty ends": ([0, 0, 33, 0], 0), "none left": ([0, 0], 7),
          "single row": ([0, 1, 0], 0), "many": ([1, 2, 3, 0, 7, 31, 32, 33, 127, 128, 129, 0, 4, 255, 257], 40),
          "one each": ([1] * 40, 0), "few": ([3, 0, 5, 1, 6], 1), "few of one": ([0, 16, 0], 0)}
# (N, K) of a weight
SIZES = [(1, 1), (3, 5), (16, 16), (64, 64), (128, 256), (72, 200), (130, 65), (257, 129), (99, 501), (320, 1000)]


def _rows(name):
    return 150 if GROUPS[name] is None else sum(GROUPS[name][0]) + GROUPS[name][1]


def _setup(name):
    """(route, offsets or None, experts, rows)"""
    if GROUPS[name] is None:
        return None, None, 1, 150
    route = _route(*GROUPS[name])
    return route, route.offset, len(GROUPS[name][0]), _rows(name)


def _poison(x, offset):
    """Rows behind the last group hold what no result may depend on."""
    if offset is not None:
        x[int(offset[-1]):] = float("nan")
    return x


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", GROUPS)
def test_products(name, dtype, size):
    route, offset, E, P = _setup(name)
    N, K = size
    x, w = _poison(_rand(1, (P, K), dtype), offset), _rand(2, (E, N, K), dtype, K ** -0.5)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = _api().tbe_expert_forward(x, w, route, status=status)
    want, bound = o.product(x, w, offset)
    assert got.shape == (P, N) and got.dtype == TYPES[dtype]
    close(got, want, rounded(bound, want, got.dtype))
    dy = _poison(_rand(3, (P, N), dtype, 0.3), offset)
    got = _api().tbe_expert_backward(dy, w, route, status=status)
    want, bound = o.product(dy, w, offset, transposed=True)
    assert got.shape == (P, K)
    close(got, want, rounded(bound, want, got.dtype))
    for out in {dtype, "f32"}:
        got = _api().tbe_expert_weight_backward(dy, x, route, dtype=TYPES[out], status=status)
        want, bound = o.weight_gradient(dy, x, offset, E)
        assert got.shape == ((E, N, K) if route is not None else (N, K)) and got.dtype == TYPES[out]
        close(got.view(E, N, K), want, rounded(bound, want, got.dtype))
        base = _rand(4, (E, N, K), out)
        got = _api().tbe_expert_weight_backward(dy, x, route, grad_weight=base.clone(), accumulate=True, status=status)
        total = want + base.double()
        close(got, total, rounded(bound + 2 * o.U32 * (want.abs() + base.double().abs()), total, got.dtype))
        if offset is not None:
            idle = torch.diff(offset) == 0
            assert torch.equal(got[idle], base[idle])
    assert status.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("size", [(1, 1), (3, 5), (32, 64), (64, 128), (36, 200), (65, 99), (200, 501), (520, 264)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_block(name, dtype, size, kind):
    route, offset, E, P = _setup(name)
    F, H = size
    x, w = _poison(_rand(1, (P, H), dtype), offset), _rand(2, (E, 2 * F, H), dtype, 2 * H ** -0.5)
    hidden, gate_up = _api().tbe_expert_gated_forward(x, w, route, activation=kind, keep=True)
    z, bz = o.product(x, w, offset)
    close(gate_up, z, rounded(bz, z, gate_up.dtype))
    want, bound = o.gated(z, bz, kind)
    close(hidden, want, rounded(bound, want, hidden.dtype))
    alone, none = _api().tbe_expert_gated_forward(x, w, route, activation=kind)
    assert none is None and torch.equal(alone, hidden)
    # the gradient of the gate, through a second layer's weight
    w2, dy = _rand(5, (E, 40, F), dtype, 0.15), _poison(_rand(6, (P, 40), dtype), offset)
    kept = _poison(gate_up.clone(), offset)
    got = _api().tbe_expert_backward(dy, w2, route, gate_up=kept, activation=kind)
    dh, bh = o.product(dy, w2, offset, transposed=True)
    want, bound = o.gate_gradient(dh, bh, gate_up, kind)
    assert got.shape == (P, 2 * F)
    close(got, want, rounded(bound, want, got.dtype))


def _strided(t, extra, shift):
    """The same values in rows that lie `extra` elements further apart, `shift` elements into a buffer."""
    rows = t.numel() // t.shape[-1]
    big = torch.full((rows * (t.shape[-1] + extra) + shift,), 7.0, dtype=t.dtype, device=t.device)
    v = big[shift:].view(*t.shape[:-1], t.shape[-1] + extra)[..., :t.shape[-1]]
    v.copy_(t)
    return v


@pytest.mark.parametrize("extra,shift", [(0, 1), (8, 8), (3, 2), (5, 0), (16, 0), (1, 4)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strides_and_places(dtype, extra, shift):
    route, offset, E, P = _setup("ragged")
    N, K = 72, 136
    plain = [_rand(1, (P, K), dtype), _rand(2, (E, N, K), dtype, 0.1), _rand(3, (P, N), dtype)]
    x, w, dy = (_strided(t, extra, shift) for t in plain)
    t = _api()

    def both(fn, shape, **kw):
        """A call on strided operands, its result in a strided place: nothing around it is written."""
        name = kw.pop("name")
        out = _strided(torch.zeros(shape, dtype=TYPES[dtype], device="cuda"), extra, shift)
        before = out._base.clone()
        got = fn(**{name: out}, **kw)
        got = got[0] if isinstance(got, tuple) else got
        assert got is out
        around = torch.ones_like(before, dtype=torch.bool)
        around[shift:].view(*shape[:-1], shape[-1] + extra)[..., :shape[-1]] = False
        assert torch.equal(out._base[around], before[around])
        return out

    want, bound = o.product(plain[0], plain[1], offset)
    got = both(t.tbe_expert_forward, (P, N), rows=x, weight=w, route=route, name="out")
    close(got, want, rounded(bound, want, got.dtype))
    hid, bh = o.gated(want, bound, "silu")
    got = both(t.tbe_expert_gated_forward, (P, N // 2), rows=x, weight=w, route=route, name="hidden")
    close(got, hid, rounded(bh, hid, got.dtype))
    want, bound = o.product(plain[2], plain[1], offset, transposed=True)
    got = both(t.tbe_expert_backward, (P, K), grad_out=dy, weight=w, route=route, name="grad_rows")
    close(got, want, rounded(bound, want, got.dtype))
    z = _strided(_rand(4, (P, 2 * K), dtype), extra, shift)
    want, bound = o.gate_gradient(want, bound, z, "gelu")
    want, bound = (torch.where(torch.arange(P, device="cuda")[:, None] < offset[-1], v, 0.0) for v in (want, bound))
    got = both(t.tbe_expert_backward, (P, 2 * K), grad_out=dy, weight=w, route=route, gate_up=z, activation="gelu",
               name="grad_rows")
    close(got, want, rounded(bound, want, got.dtype))
    want, bound = o.weight_gradient(plain[2], plain[0], offset, E)
    got = both(t.tbe_expert_weight_backward, (E, N, K), grad_out=dy, rows=x, route=route, name="grad_weight")
    close(got, want, rounded(bound, want, got.dtype))


def test_one_row_for_all_and_one_weight_for_all():
    # stride 0: broadcast rows, and experts that share one matrix
    route, offset, E, P = _setup("ragged")
    x, w = _rand(1, (1, 64), "bf16").expand(P, 64), _rand(2, (1, 48, 64), "bf16").expand(E, 48, 64)
    want, bound = o.product(x, w, offset)
    close(_api().tbe_expert_forward(x, w, route), want, rounded(bound, want, torch.bfloat16))
    dy = _rand(3, (1, 48), "bf16").expand(P, 48)
    want, bound = o.weight_gradient(dy, x, offset, E)
    close(_api().tbe_expert_weight_backward(dy, x, route), want, rounded(bound, want, torch.bfloat16))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_infinities_stay_in_their_rows_and_experts(dtype):
    # a row of infinities, NaN and largest values next to rows of other experts in one tile
    route, offset, E, P = _setup("ragged")
    x, w = _rand(1, (P, 72), dtype), _rand(2, (E, 80, 72), dtype, 0.1)
    clean = _api().tbe_expert_forward(x, w, route), _api().tbe_expert_weight_backward(_rand(3, (P, 80), dtype), x, route)
    bad = int(offset[3])                    # the single row of expert 3
    y = x.clone()
    y[bad, ::3], y[bad, 1::3] = float("inf"), float("nan")
    got = _api().tbe_expert_forward(y, w, route), _api().tbe_expert_weight_backward(_rand(3, (P, 80), dtype), y, route)
    others = torch.arange(P, device="cuda") != bad
    assert torch.equal(got[0][others], clean[0][others]) and not torch.isfinite(got[0][bad]).any()
    e = torch.arange(E, device="cuda") != 3
    assert torch.equal(got[1][e], clean[1][e])
    # an expert's bad weight stays with its rows
    v = w.clone()
    v[2, 5] = float("nan")
    got = _api().tbe_expert_forward(x, v, route)
    a, b = int(offset[2]), int(offset[3])
    assert torch.isnan(got[a:b, 5]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[a:b, 5] = False
    assert torch.equal(got[keep], clean[0][keep])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,K,shift", [(72, 200, 0), (1000, 328, 0), (99, 131, 0), (520, 264, 3)])
def test_long_groups(N, K, shift, dtype):
    # more tiles than CTAs, sums over many steps, the weights' gradient in slices of rows
    t, P = _api(), 5001
    x, dy = _strided(_rand(1, (P, K), dtype), shift, 0), _strided(_rand(2, (P, N), dtype, 0.3), shift, 0)
    w = _rand(3, (N, K), dtype, K ** -0.5)
    want, bound = o.product(x, w[None], None)
    got = t.tbe_expert_forward(x, w)
    close(got, want, rounded(bound, want, got.dtype))
    want, bound = o.product(dy, w[None], None, transposed=True)
    got = t.tbe_expert_backward(dy, w)
    close(got, want, rounded(bound, want, got.dtype))
    want, bound = o.weight_gradient(dy, x, None, 1)
    from recsys_table_embedding_gb300.layers import _lib
    assert _lib().tbe_expert_workspace_bytes(P, 1, N, K) > 0
    for out in {dtype, "f32"}:
        got = t.tbe_expert_weight_backward(dy, x, dtype=TYPES[out])
        close(got[None], want, rounded(bound, want, got.dtype))
        base = _rand(4, (N, K), out)
        both = t.tbe_expert_weight_backward(dy, x, grad_weight=base.clone(), accumulate=True)
        total = want + base.double()
        close(both[None], total, rounded(bound + 2 * o.U32 * (want.abs() + base.double().abs()), total, both.dtype))
    again = t.tbe_expert_weight_backward(dy, x, dtype=TYPES[out])
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_experts_most_without_rows(dtype):
    E = 1000
    counts = [0] * E
    for e in (0, 3, 500, 501, 999):
        counts[e] = 40 + e % 7
    route = _route(counts, 11)
    P = sum(counts) + 11
    x, w = _poison(_rand(1, (P, 40), dtype), route.offset), _rand(2, (E, 24, 40), dtype, 0.2)
    want, bound = o.product(x, w, route.offset)
    got = _api().tbe_expert_forward(x, w, route)
    close(got, want, rounded(bound, want, got.dtype))
    dy = _poison(_rand(3, (P, 24), dtype), route.offset)
    want, bound = o.weight_gradient(dy, x, route.offset, E)
    got = _api().tbe_expert_weight_backward(dy, x, route)
    close(got, want, rounded(bound, want, got.dtype))


@pytest.mark.parametrize("shift", [0, 1])
def test_offsets_beyond_32_bits(shift):
    # 2^31 elements and more of rows and of results: the last rows like a call of theirs alone
    t = _api()
    P, K = (1 << 31) // 1024 + 700, 1024 + shift
    x = torch.empty(P, K, dtype=torch.bfloat16, device="cuda")
    x[-600:] = _rand(1, (600, K), "bf16")
    x[:-600] = 0
    w = _rand(2, (72, K), "bf16", 0.03)
    got = t.tbe_expert_forward(x, w)
    want, bound = o.product(x[-600:], w[None], None)
    close(got[-600:], want, rounded(bound, want, got.dtype))
    assert not got[:-600].any()
    dy = torch.zeros(P, 72, dtype=torch.bfloat16, device="cuda")
    dy[-600:] = _rand(3, (600, 72), "bf16")
    got = t.tbe_expert_backward(dy, w)
    want, bound = o.product(dy[-600:], w[None], None, transposed=True)
    close(got[-600:], want, rounded(bound, want, got.dtype))
    assert not got[-1200:-600].any()
    got = t.tbe_expert_weight_backward(dy, x, dtype=torch.float32)
    want, bound = o.weight_gradient(dy[-600:], x[-600:], None, 1)
    close(got[None], want, rounded(bound, want, got.dtype))


def test_offsets_that_leave_the_rows_are_held_to_them():
    route = _route([3, 60, 5])
    route.offset.copy_(torch.tensor([-5, 3, 500, 68], device="cuda"))       # the second beyond, the third before it
    x, w = _rand(1, (68, 64), "bf16"), _rand(2, (3, 64, 64), "bf16", 0.1)
    got = _api().tbe_expert_forward(x, w, route)
    want, bound = o.product(x[:3], w[:1], None)
    close(got[:3], want, rounded(bound, want, got.dtype))
    want, bound = o.product(x[3:], w[1:2], None)
    close(got[3:], want, rounded(bound, want, got.dtype))


def test_no_rows():
    t = _api()
    w = _rand(1, (3, 8, 16), "f32")
    route = t.tbe_route_sort(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 3)
    assert t.tbe_expert_forward(_rand(1, (0, 16), "f32"), w, route).shape == (0, 8)
    assert t.tbe_expert_backward(_rand(1, (0, 8), "f32"), w, route).shape == (0, 16)
    dw = t.tbe_expert_weight_backward(_rand(1, (0, 8), "f32"), _rand(1, (0, 16), "f32"), route)
    assert dw.shape == (3, 8, 16) and not dw.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_calls_give_equal_bits(dtype):
    route, offset, E, P = _setup("many")
    x, w, dy = _rand(1, (P, 264), dtype), _rand(2, (E, 136, 264), dtype), _rand(3, (P, 136), dtype)
    t = _api()
    for fn in (lambda: t.tbe_expert_forward(x, w, route), lambda: t.tbe_expert_backward(dy, w, route),
               lambda: t.tbe_expert_weight_backward(dy, x, route, dtype=torch.float32),
               lambda: t.tbe_expert_gated_forward(x, w, route)[0]):
        assert torch.equal(fn(), fn())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_calls_follow_the_routes(dtype):
    # a captured graph of the calls, replayed with another routing of other rows
    t = _api()
    E, T, K = 6, 200, 2
    ids = torch.randint(0, E, (T, K), generator=_gen(1), device="cuda", dtype=torch.int32)
    x, w1, w2 = _rand(1, (T, 64), dtype), _rand(2, (E, 96, 64), dtype, 0.2), _rand(3, (E, 64, 48), dtype, 0.2)

    def calls():
        rows, route = t.tbe_route_sort_dispatch(x, ids, E)
        hidden, z = t.tbe_expert_gated_forward(rows, w1, route, keep=True)
        out = t.tbe_expert_forward(hidden, w2, route)
        dz = t.tbe_expert_backward(out, w2, route, gate_up=z)
        return out, t.tbe_expert_backward(dz, w1, route), t.tbe_expert_weight_backward(dz, rows, route)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for seed in (5, 6):
        ids.copy_(torch.randint(-1, E, (T, K), generator=_gen(seed), device="cuda"))
        x.copy_(_rand(seed, (T, 64), dtype))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, calls()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    t = _api()
    route, offset, E, P = _setup("many")
    x, w = _rand(1, (P, 512), "bf16"), _rand(2, (E, 512, 512), "bf16", 0.05)
    alone = t.tbe_expert_forward(x, w, route)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[t.tbe_expert_forward(x, w, route, stream=s) for _ in range(4)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, alone) for gs in got for g in gs)


def test_refusals():
    t = _api()
    route, offset, E, P = _setup("ragged")
    x, w = _rand(1, (P, 64), "bf16"), _rand(2, (E, 32, 64), "bf16")
    for bad in (lambda: t.tbe_expert_forward(x, w), lambda: t.tbe_expert_forward(x[:-1], w, route),
                lambda: t.tbe_expert_forward(x, w[:-1], route), lambda: t.tbe_expert_forward(x[:, :63], w, route),
                lambda: t.tbe_expert_forward(x, w.half(), route), lambda: t.tbe_expert_forward(x, w.double(), route),
                lambda: t.tbe_expert_forward(x, w.transpose(1, 2), route), lambda: t.tbe_expert_forward(x, w.cpu(), route),
                lambda: t.tbe_expert_forward(x, w, route, out=torch.empty(P, 31, device="cuda", dtype=torch.bfloat16)),
                lambda: t.tbe_expert_gated_forward(x, w[:, :31], route),
                lambda: t.tbe_expert_gated_forward(x, w, route, activation="tanh"),
                lambda: t.tbe_expert_backward(x, w, route),
                lambda: t.tbe_expert_backward(x[:, :32], w, route, gate_up=x),
                lambda: t.tbe_expert_weight_backward(x, x[:-1], route),
                lambda: t.tbe_expert_weight_backward(x, x, route, accumulate=True),
                lambda: t.tbe_expert_weight_backward(x, x, route, dtype=torch.float16),
                lambda: t.tbe_expert_weight_backward(x, x, route, grad_weight=torch.empty(E, 64, 63, device="cuda")),
                lambda: t.tbe_expert_forward(x.detach().requires_grad_(), w, route)):
        with pytest.raises(t.TbeError):
            bad()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_in_the_columns_of_one_buffer(dtype):
    # rows of the results in between one another, and between those they are made from; shared elements are refused
    t = _api()
    route, _, E, P = _setup("ragged")
    H, F = 64, 48
    w, down = _rand(2, (E, 2 * F, H), dtype, 0.1), _rand(3, (E, H, F), dtype, 0.1)
    buf = torch.zeros(P, H + 3 * F + H, dtype=w.dtype, device="cuda")
    x, z, h, y = buf[:, :H], buf[:, H:H + 2 * F], buf[:, H + 2 * F:H + 3 * F], buf[:, H + 3 * F:]
    x.copy_(_rand(1, (P, H), dtype))
    want_h, want_z = t.tbe_expert_gated_forward(x.clone(), w, route, keep=True)
    t.tbe_expert_gated_forward(x, w, route, hidden=h, gate_up=z)
    t.tbe_expert_forward(h, down, route, out=y)
    assert torch.equal(h, want_h) and torch.equal(z, want_z) and torch.equal(y, t.tbe_expert_forward(want_h, down, route))
    dz = t.tbe_expert_backward(y.clone(), down, route, gate_up=z)
    for call in (lambda: t.tbe_expert_forward(x, w[:, :H], route, out=x), lambda: t.tbe_expert_forward(x, w[:, :H], route, out=buf[:, 8:8 + H]),
                 lambda: t.tbe_expert_gated_forward(x, w, route, hidden=z[:, :F], gate_up=z),
                 lambda: t.tbe_expert_backward(y, down, route, gate_up=z, grad_rows=z),
                 lambda: t.tbe_layer_norm_forward(x, out=x)):
        with pytest.raises(RuntimeError):
            call()
    assert torch.equal(z, want_z) and torch.equal(dz, t.tbe_expert_backward(y, down, route, gate_up=z))
