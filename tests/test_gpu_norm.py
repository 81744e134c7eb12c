"""GPU tests of layer norm and its gradients against their definitions in 64
bits, at the sizes, types, strides and values where they can go wrong."""
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


def _rand(seed, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=_gen(seed)).to(TYPES[dtype])


def _strided(t, extra, shift):
    big = torch.full((t.shape[0] * (t.shape[1] + extra) + shift,), 7.0, dtype=t.dtype, device=t.device)
    v = big[shift:].view(t.shape[0], t.shape[1] + extra)[:, :t.shape[1]]
    v.copy_(t)
    return v


def _check(x, dy, w, b, eps=1e-5, dtype=None, **kw):
    t = _api()
    out, mean, rstd = t.tbe_layer_norm_forward(x, w, b, eps=eps, **kw)
    want, bound = o.norm(x, w, b, eps)
    assert out.dtype == x.dtype and mean.dtype == rstd.dtype == torch.float32
    close(out, want[0], rounded(bound[0], want[0], out.dtype))
    close(mean, want[1], bound[1] + 2.0 ** -140)
    close(rstd, want[2], bound[2])
    got = t.tbe_layer_norm_backward(dy, x, mean, rstd, w, dtype=dtype)
    want, bound = o.norm_backward(dy, x, mean, rstd, w)
    for g, v, e in zip(got, want, bound):
        close(g, v, rounded(e, v, g.dtype))
    kind = dtype or (w.dtype if w is not None else torch.float32)
    assert got[0].dtype == x.dtype and got[1].dtype == got[2].dtype == kind
    return (out, mean, rstd), got


@pytest.mark.parametrize("D", [1, 2, 3, 8, 31, 64, 100, 256, 257, 501, 512, 1000, 1024, 2050, 4096, 6001, 8192, 8200,
                               16_384, 32_768, 33_000, 70_001])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f32", "bf16")])
def test_sizes(D, types):
    for i, N in enumerate((1, 2, 9, 700)):
        if N * D > 8_000_000:
            N = 40
        x, dy = _rand(D + i, (N, D), types[0], 2.0, 0.5), _rand(D + i + 1, (N, D), types[0], 0.3)
        w, b = _rand(3, (D,), types[1], 0.3, 1.0), _rand(4, (D,), types[1], 0.3)
        _check(x, dy, w, b)


@pytest.mark.parametrize("N,D", [(5000, 64), (20_000, 40), (3000, 1024), (2500, 4096), (1300, 8192), (600, 10_000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(N, D, dtype):
    x, dy = _rand(1, (N, D), dtype, 1.5, -0.2), _rand(2, (N, D), dtype, 0.1)
    a = _check(x, dy, _rand(3, (D,), "f32", 0.3, 1.0), None)
    b = _check(x, dy, _rand(3, (D,), "f32", 0.3, 1.0), None)
    assert all(torch.equal(p, q) for u, v in zip(a, b) for p, q in zip(u, v))     # equal calls, equal bits


@pytest.mark.parametrize("w,b", [(None, None), ("f32", None), (None, "bf16"), ("f16", "f16")])
def test_without_weight_or_bias(w, b):
    x, dy = _rand(1, (50, 96), "bf16"), _rand(2, (50, 96), "bf16")
    make = lambda s, k: None if k is None else _rand(s, (96,), k, 0.3, 1.0)  # noqa: E731
    _check(x, dy, make(3, w), make(4, b))
    _check(x, dy, make(3, w), make(4, b), dtype=torch.float32)


@pytest.mark.parametrize("offset,spread", [(1e4, 1.0), (-3e5, 0.5), (1e-3, 1e-6), (0.0, 1e-12), (1e15, 1e14)])
def test_offsets_and_spreads(offset, spread):
    # a row's offset far above its spread; spreads below sqrt(eps); squares near the range's end
    for D in (60, 3000, 40_000):
        x = _rand(1, (20, D), "f32", spread, offset)
        _check(x, _rand(2, (20, D), "f32"), _rand(3, (D,), "f32", 0.3, 1.0), None)


def test_constant_rows():
    x = torch.full((3, 200), 5.0, device="cuda")
    out, mean, rstd = _api().tbe_layer_norm_forward(x, eps=1e-5)
    assert not out.any() and (mean == 5).all()
    close(rstd, torch.full((3,), 1e-5 ** -0.5, dtype=torch.float64, device="cuda"), 8 * o.U32 * 320 * torch.ones(3, device="cuda", dtype=torch.float64))


@pytest.mark.parametrize("D", [100, 5000, 40_000])
def test_infinities_stay_in_their_rows(D):
    x = _rand(1, (30, D), "f32")
    clean = _api().tbe_layer_norm_forward(x)
    y = x.clone()
    y[7, 3], y[9, 5], y[11] = float("nan"), float("inf"), 3e38
    got = _api().tbe_layer_norm_forward(y)
    keep = torch.ones(30, dtype=torch.bool, device="cuda")
    keep[[7, 9, 11]] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert torch.isnan(got[0][7]).all() and torch.isnan(got[0][9, 5]) and torch.isnan(got[2][7])
    # a NaN gradient of one row reaches that row's gradient and the sums only
    dy = _rand(2, (30, D), "f32")
    a = _api().tbe_layer_norm_backward(dy, x, clean[1], clean[2])
    dy[4, 0] = float("nan")
    b = _api().tbe_layer_norm_backward(dy, x, clean[1], clean[2])
    keep = torch.arange(30, device="cuda") != 4
    assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][4]).all()
    assert torch.isnan(b[1][0]) and torch.isnan(b[2][0]) and torch.equal(a[1][1:], b[1][1:])


@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8), (3, 2), (4, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_places(extra, shift, dtype):
    t = _api()
    D = 72
    plain = [_rand(1, (90, D), dtype), _rand(2, (90, D), dtype)]
    x, dy = (_strided(v, extra, shift) for v in plain)
    w = torch.zeros(D + 1, dtype=TYPES[dtype], device="cuda")[1:]        # at an odd place
    w.copy_(_rand(3, (D,), dtype, 0.2, 1.0))
    out, dx = (_strided(torch.zeros_like(plain[0]), extra, shift) for _ in range(2))
    before = out._base.clone()
    got, mean, rstd = t.tbe_layer_norm_forward(x, w, w, out=out)
    assert got is out
    want, bound = o.norm(plain[0], w, w, 1e-5)
    close(out, want[0], rounded(bound[0], want[0], out.dtype))
    r = t.tbe_layer_norm_backward(dy, x, mean, rstd, w, grad_x=dx)
    want, bound = o.norm_backward(plain[1], plain[0], mean, rstd, w)
    for g, v, e in zip(r, want, bound):
        close(g, v, rounded(e, v, g.dtype))
    around = torch.ones_like(before, dtype=torch.bool)
    around[shift:].view(90, D + extra)[:, :D] = False
    assert torch.equal(out._base[around], before[around]) and torch.equal(dx._base[around], before[around])


def test_one_row_for_all_and_empty():
    t = _api()
    x = _rand(1, (1, 64), "f32").expand(33, 64)
    _check(x, _rand(2, (1, 64), "f32").expand(33, 64), None, None)
    none = x[:0]
    out, mean, rstd = t.tbe_layer_norm_forward(none)
    assert out.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dx, dw, db = t.tbe_layer_norm_backward(none, none, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    y = _rand(1, (3, 5, 64), "f32")
    assert torch.equal(t.tbe_layer_norm_forward(y)[0], t.tbe_layer_norm_forward(y.view(15, 64))[0].view(3, 5, 64))
    assert t.tbe_layer_norm_forward(y)[1].shape == (3, 5)


def test_gradients_against_differences():
    # the loss sum(out c) of a small problem, differenced in 64 bits by the oracle
    x, c = _rand(1, (6, 40), "f32"), _rand(2, (6, 40), "f32")
    w, b = _rand(3, (40,), "f32", 0.3, 1.0), _rand(4, (40,), "f32")
    _, mean, rstd = _api().tbe_layer_norm_forward(x, w, b)
    dx, dw, db = _api().tbe_layer_norm_backward(c, x, mean, rstd, w)
    loss = lambda x, w, b: float((o.norm(x, w, b, 1e-5)[0][0] * c.double()).sum())  # noqa: E731
    h = 1e-6
    for t, g in ((x, dx), (w, dw), (b, db)):
        d = torch.randn(t.shape, generator=_gen(9), device="cuda", dtype=torch.float64)
        above, below = ([v.double() + (s * h * d if v is t else 0.0) for v in (x, w, b)] for s in (1, -1))
        slope = (loss(*above) - loss(*below)) / (2 * h)
        # differences: h^2 of third derivatives and 1e-16 / h of the loss; the gradient's 32-bit sums
        assert abs(slope - float((g.double() * d).sum())) <= 1e-4 * float((g.double() * d).abs().sum())


def test_offsets_beyond_32_bits():
    # 2^31 elements and more: the last rows like a call of theirs alone
    t = _api()
    D = 4096
    N = (1 << 31) // D + 50
    x = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    x[-40:] = _rand(1, (40, D), "bf16")
    w = _rand(3, (D,), "f32", 0.3, 1.0)
    out, mean, rstd = t.tbe_layer_norm_forward(x, w)
    want, bound = o.norm(x[-40:], w, None, 1e-5)
    close(out[-40:], want[0], rounded(bound[0], want[0], out.dtype))
    close(mean[-40:], want[1], bound[1])
    assert not out[:-40].any() and not mean[:-40].any()
    dx, dw, db = t.tbe_layer_norm_backward(x, x, mean, rstd, w)
    want, bound = o.norm_backward(x[-40:], x[-40:], mean[-40:], rstd[-40:], w)
    close(dx[-40:], want[0], rounded(bound[0], want[0], dx.dtype))
    close(dw, want[1], rounded(bound[1], want[1], dw.dtype))
    close(db, want[2], rounded(bound[2], want[2], db.dtype))


@pytest.mark.parametrize("D", [96, 640, 3000, 20_000])
def test_single_results(D):
    # the sums alone, the rows' gradient alone: through the C entry point
    from recsys_table_embedding_gb300 import layers
    from recsys_table_embedding_gb300.tokens import _matrix
    L = layers._lib()
    x, dy, w = _rand(1, (1500, D), "bf16"), _rand(2, (1500, D), "bf16"), _rand(3, (D,), "f32", 0.2, 1.0)
    _, mean, rstd = _api().tbe_layer_norm_forward(x, w)
    want, bound = o.norm_backward(dy, x, mean, rstd, w)
    dx = torch.empty_like(x)
    dw = torch.empty(D, device="cuda")
    n = L.tbe_layer_norm_workspace_bytes(1500, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    call = lambda gx, gw: L.tbe_layer_norm_backward(_matrix(dy, "dy"), _matrix(x, "x"), w.data_ptr(), 0, mean.data_ptr(),  # noqa: E731
                                                    rstd.data_ptr(), gx, gw, None, 0, ws.data_ptr(), n, None, stream)
    assert call(_matrix(dx, "dx"), None) == 0 and call(None, dw.data_ptr()) == 0
    close(dx, want[0], rounded(bound[0], want[0], dx.dtype))
    close(dw, want[1], rounded(bound[1], want[1], dw.dtype))


def test_captured_and_on_another_stream():
    t = _api()
    x, dy, w = _rand(1, (300, 256), "bf16"), _rand(2, (300, 256), "bf16"), _rand(3, (256,), "f32", 0.2, 1.0)

    def calls(stream=None):
        out, mean, rstd = t.tbe_layer_norm_forward(x, w, w, stream=stream)
        return (out, *t.tbe_layer_norm_backward(dy, x, mean, rstd, w, stream=stream))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    x.copy_(_rand(7, (300, 256), "bf16"))
    graph.replay()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = calls(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(got, calls(), other))


def test_refusals():
    t = _api()
    x, w = _rand(1, (10, 64), "bf16"), _rand(2, (64,), "f32")
    _, mean, rstd = t.tbe_layer_norm_forward(x)
    for bad in (lambda: t.tbe_layer_norm_forward(x, w[:-1]), lambda: t.tbe_layer_norm_forward(x, w, w.half()),
                lambda: t.tbe_layer_norm_forward(x, w.double()), lambda: t.tbe_layer_norm_forward(x.t()),
                lambda: t.tbe_layer_norm_forward(x, eps=-1.0), lambda: t.tbe_layer_norm_forward(x, eps=float("nan")),
                lambda: t.tbe_layer_norm_forward(x, out=torch.empty(10, 64, device="cuda")),
                lambda: t.tbe_layer_norm_forward(x, mean=mean[:-1]), lambda: t.tbe_layer_norm_forward(x.double()),
                lambda: t.tbe_layer_norm_forward(x[0]), lambda: t.tbe_layer_norm_forward(x, w.cpu()),
                lambda: t.tbe_layer_norm_backward(x.float(), x, mean, rstd), lambda: t.tbe_layer_norm_backward(x[:5], x, mean, rstd),
                lambda: t.tbe_layer_norm_backward(x, x, mean[:5], rstd), lambda: t.tbe_layer_norm_backward(x, x, mean.half(), rstd),
                lambda: t.tbe_layer_norm_backward(x, x, mean, rstd, grad_weight=w, grad_bias=w.half()),
                lambda: t.tbe_layer_norm_backward(x, x, mean, rstd, dtype=torch.float64),
                lambda: t.tbe_layer_norm_forward(x.detach().requires_grad_())):
        with pytest.raises(t.TbeError):
            bad()


@pytest.mark.parametrize("N", [609, 1216])
@pytest.mark.parametrize("D", [1032, 2048, 4104, 8200, 16_384])
@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "f32")])
def test_two_rows_a_block(N, D, types):
    # an odd number of rows too, rows apart, and nothing written behind the last or beside a row
    t = _api()
    x, w, b = _rand(D, (N, D), types[0], 2.0, 0.5), _rand(3, (D,), types[1], 0.3, 1.0), _rand(4, (D,), types[1], 0.3)
    (out, mean, rstd), _ = _check(x, _rand(D + 1, (N, D), types[0], 0.3), w, b)
    big = torch.full((N + 2, D + 8), 5.0, dtype=x.dtype, device="cuda")
    stats = torch.full((2, N + 2), 5.0, device="cuda")
    got = t.tbe_layer_norm_forward(_strided(x, 24, 8), w, b, out=big[1:N + 1, :D], mean=stats[0, 1:N + 1], rstd=stats[1, 1:N + 1])
    assert all(torch.equal(p, q) for p, q in zip(got, (out, mean, rstd)))
    big[1:N + 1, :D], stats[:, 1:N + 1] = 5.0, 5.0
    assert (big == 5.0).all() and (stats == 5.0).all()
    # a row of infinities or a NaN stays by itself
    y = x.clone()
    y[N - 1], y[6, 3] = float("inf"), float("nan")
    got = t.tbe_layer_norm_forward(y, w, b)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[N - 1] = keep[6] = False
    for p, q in zip(got, (out, mean, rstd)):
        assert torch.equal(p[keep], q[keep]) and torch.isnan(p[~keep]).any(-1).all()
