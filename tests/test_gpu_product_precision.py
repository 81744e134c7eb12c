"""GPU tests of how precise the experts' products' sums are, beyond what a bound that
grows with every term can see: operands of one sign, whose sums the tensor core's
cutting off makes smaller with every term, and whose errors do not cancel.

Bounds.  A tensor core's FP32 sum loses 2^-27 of itself a term at most (16 terms are
added at once, and 2^-23 of the sum is what its last bit can be worth), and the sums
leave it after so many terms that this stays below a fifth of the result's smallest
half step: after 8192 of FP16 (2^-14 of 2^-12), after 65,536 of BF16 (2^-11 of 2^-9).
What leaves, every 2048 terms at the most (512 where rows have no vectors), is added in
FP32: 2^-24 an addition.  Then the result is rounded once."""
import pytest
import torch

import layer_oracle as o
from layer_oracle import close, rounded
from token_oracle import TYPES

pytestmark = pytest.mark.gpu

MOST = {"f16": 8192, "bf16": 65_536}


def _api():
    import recsys_table_embedding_gb300 as tbe
    return tbe


def _positive(seed, rows, cols, dtype, scale, odd):
    """[rows, cols] in scale * [0.5, 1.5]; odd: rows that no vector fits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    big = torch.empty(rows, cols + odd, dtype=TYPES[dtype], device="cuda")
    big.copy_((torch.rand(rows, cols + odd, device="cuda", generator=g) + 0.5) * scale)
    return big[:, :cols]


def _loss(K, dtype, odd):
    """What the sums of K positive terms may lack, relative to them."""
    return min(K, MOST[dtype]) * 2.0 ** -27 + (K // (512 if odd else 2048) + 2) * 2.0 ** -24


def _scales(K):
    """Of two operands, so that sums of K of their products are between 1 and 2."""
    bits = (K - 1).bit_length()
    return 2.0 ** -(bits // 2), 2.0 ** -(bits - bits // 2)


LONG = [("f16", 8192), ("f16", 8264), ("f16", 40_000), ("f16", 1 << 20), ("bf16", 65_536), ("bf16", 66_000), ("bf16", 1 << 20)]


@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("dtype,K", LONG)
def test_long_sums_of_rows(dtype, K, odd):
    P, N = 300, 264
    a, b = _scales(K)
    x, w = _positive(1, P, K, dtype, a, odd), _positive(2, N, K, dtype, b, odd)
    want, loss = x.double() @ w.double().t(), _loss(K, dtype, odd)
    got = _api().tbe_expert_forward(x, w)
    close(got, want, rounded(loss * want, want, got.dtype))
    hidden, z = _api().tbe_expert_gated_forward(x, w, keep=True)
    close(z, want, rounded(loss * want, want, z.dtype))
    h, bound = o.gated(want, loss * want, "silu")
    close(hidden, h, rounded(bound, h, hidden.dtype))


@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("dtype,K", LONG)
def test_long_sums_of_the_rows_gradient(dtype, K, odd):
    P, N = 300, 136
    a, b = _scales(K)
    dy, w = _positive(1, P, K, dtype, a, odd), _positive(2, K, N, dtype, b, odd)
    want, loss = dy.double() @ w.double(), _loss(K, dtype, odd)
    got = _api().tbe_expert_backward(dy, w)
    close(got, want, rounded(loss * want, want, got.dtype))
    z = torch.empty(P, 2 * N, dtype=got.dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    got = _api().tbe_expert_backward(dy, w, gate_up=z, activation="gelu")
    want, bound = o.gate_gradient(want, loss * want, z, "gelu")
    close(got, want, rounded(bound, want, got.dtype))


@pytest.mark.parametrize("dtype,K", [("f16", 9000), ("bf16", 70_000)])
def test_long_sums_by_expert(dtype, K):
    # groups that end inside tiles, experts without rows, rows of no expert that hold NaN
    from test_gpu_experts import _poison, _route
    t = _api()
    route = _route([5, 0, 290, 1, 64], 9)
    P, E, N = 369, 5, 72
    a, b = _scales(K)
    x, w = _poison(_positive(1, P, K, dtype, a, 0), route.offset), _positive(2, E * N, K, dtype, b, 0).view(E, N, K)
    rel, n = _loss(K, dtype, 0), int(route.offset[-1])
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    want, _ = o.product(x, w, route.offset)
    got = t.tbe_expert_forward(x, w, route, status=status)
    close(got, want, rounded(rel * want, want, got.dtype))
    hidden, z = t.tbe_expert_gated_forward(x, w, route, activation="gelu", keep=True, status=status)
    h, bound = o.gated(want, rel * want, "gelu")
    close(z, want, rounded(rel * want, want, z.dtype))
    close(hidden, h, rounded(bound, h, hidden.dtype))
    assert not hidden[n:].any() and not z[n:].any() and not got[n:].any()
    down = _positive(4, E * K, N, dtype, b, 0).view(E, K, N)
    want, _ = o.product(x, down, route.offset, transposed=True)
    got = t.tbe_expert_backward(x, down, route, status=status)
    close(got, want, rounded(rel * want, want, got.dtype))
    z = _poison(torch.empty(P, 2 * N, dtype=x.dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5)),
                route.offset)
    got = t.tbe_expert_backward(x, down, route, gate_up=z, status=status)
    want, bound = o.gate_gradient(want[:n], rel * want[:n], z[:n], "silu")
    close(got[:n], want, rounded(bound, want, got.dtype))
    assert not got[n:].any() and status.tolist() == [0, 0, 0, 0]
    again = t.tbe_expert_backward(x, down, route, gate_up=z)
    assert torch.equal(got, again)


def _residuals(seed, rows, cols, odd=0):
    """FP32 numbers between 1 and 1 + 2^-8: their first BF16 piece is 1, and all others
    are above it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (1 + torch.rand(rows, cols + odd, device="cuda", generator=g).clamp(2.0 ** -10, 0.999) * 2.0 ** -8)[:, :cols]


def pieces_above(seed, rows, cols, odd=0, device="cuda"):
    """FP32 numbers of three BF16 pieces of one sign: 1, a second between 2^-9 and 2^-8 and
    a third below 2^-17, which a sum without them lacks by 2^-7.4 and 2^-17 of itself."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    second = torch.randint(128, 256, (rows, cols + odd), device=device, generator=g)
    third = torch.randint(1, 64, (rows, cols + odd), device=device, generator=g)
    return (1 + second * 2.0 ** -16 + third * 2.0 ** -23)[:, :cols]


def third_pieces_close(got, want, n):
    """What is left out, the products of a second with a third piece: 2 * 2^-8 * 2^-17.
    The rest as in _pieces_close, sums of fewer terms cut off less often."""
    lost = 2.0 ** -24 + 5 * min(n, 2048) / 16 * 2.0 ** -23 * 2.0 ** -7
    off = (got.double() - want) / want
    assert off.abs().max() <= lost + (n // 128 + n // 2048 + 4) * 2.0 ** -24
    assert off.mean().abs() <= lost + 2.0 ** -26


def _pieces_close(got, want, n):
    """The pieces' products beside the first, 2^-8 of the sum here, are five in 16 terms,
    each cut off at 2^-23 of their sum so far at most, and leave the tensor core after
    2048 terms: 5 * 128 * 2^-23 * 2^-8 = 2^-21.7 of the sum, at most and in one direction.
    All other errors are roundings, to the nearest, of additions that differ from element
    to element: they add up to 2^-24 each, n / 128 + n / 2048 of them, at most, and to
    nothing in the mean of 79,200 elements (below 2^-24 64 / sqrt(79,200) = 2^-26)."""
    lost = 640 * 2.0 ** -31 * (1 + 2.0 ** -6)
    off = (got.double() - want) / want
    assert off.abs().max() <= lost + (n // 128 + n // 2048 + 4) * 2.0 ** -24
    assert off.mean().abs() <= lost + 2.0 ** -26


@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "odd"])
def test_the_pieces_of_long_f32_sums(odd):
    P, N, K = 300, 264, 1 << 17
    x, w = _residuals(1, P, K, odd), _residuals(2, N, K, odd)
    want = x.double() @ w.double().t()
    _pieces_close(_api().tbe_expert_forward(x, w), want, K)
    hidden, z = _api().tbe_expert_gated_forward(x, w, keep=True)
    _pieces_close(z, want, K)
    back = torch.empty(K, N + odd, device="cuda")[:, :N]
    back.copy_(w.t())
    _pieces_close(_api().tbe_expert_backward(x, back), want, K)


def test_the_pieces_of_a_long_f32_weights_gradient():
    # so many tiles that the rows are not cut into slices
    from recsys_table_embedding_gb300.layers import _lib
    P, N, K = 1 << 17, 4608, 4352
    assert _lib().tbe_expert_workspace_bytes(P, 1, N, K) == 0
    dy, x = _residuals(1, P, N), _residuals(2, P, K)
    got = _api().tbe_expert_weight_backward(dy, x)
    _pieces_close(got[-300:, -264:], dy[:, -300:].double().t() @ x[:, -264:].double(), P)


@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("K", [16, 64, 501, 2048, 5001, 8192])
def test_no_piece_of_f32_is_lost(K, odd):
    t, P, N = _api(), 300, 264
    x, w = pieces_above(1, P, K, odd), pieces_above(2, N, K, odd)
    want = x.double() @ w.double().t()
    third_pieces_close(t.tbe_expert_forward(x, w), want, K)
    third_pieces_close(t.tbe_expert_gated_forward(x, w, keep=True)[1], want, K)
    back, dy = torch.empty(K, N + odd, device="cuda")[:, :N], torch.empty(K, P + odd, device="cuda")[:, :P]
    back.copy_(w.t())
    dy.copy_(x.t())
    third_pieces_close(t.tbe_expert_backward(x, back), want, K)
    third_pieces_close(t.tbe_expert_weight_backward(dy, back), want, K)
    # few rows, which are not cut into pieces: two roundings a term at most
    few = t.tbe_expert_forward(x[:4], w)
    assert ((few.double() - want[:4]) / want[:4]).abs().max() <= (K // 32 + 8) * 2.0 ** -24


@pytest.mark.parametrize("N,K", [(72, 200), (99, 131), (4608, 4352)], ids=["slices", "odd slices", "one slice"])
@pytest.mark.parametrize("P", [512, 5001, 8192, 1 << 17])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_sums_of_the_weights_gradient(dtype, P, N, K):
    """Of 16-bit operands: FP32 results lose 2^-27 a term over 512 terms, 16-bit ones over
    2048, and 2^-24 for each of these sums (at most 292 and 36 of them, rounded to the
    nearest: 0.29 * 2^-24 sqrt(292) each, below 2^-24 / 8 in the mean of 13,000 elements)."""
    t = _api()
    a, b = _scales(P)
    dy, x = _positive(1, P, N, dtype, a, 0), _positive(2, P, K, dtype, b, 0)
    rows, cols = slice(max(0, N - 300), N), slice(max(0, K - 264), K)
    want = dy[:, rows].double().t() @ x[:, cols].double()
    got = t.tbe_expert_weight_backward(dy, x, dtype=torch.float32)[rows, cols]
    off = (got.double() - want) / want
    lost = min(P, 512) * 2.0 ** -27
    assert off.abs().max() <= lost + (P // 512 + 36) * 2.0 ** -24
    assert off.mean().abs() <= lost + 2.0 ** -24 / 8
    got = t.tbe_expert_weight_backward(dy, x)[rows, cols]
    close(got, want, rounded((min(P, 2048) * 2.0 ** -27 + (P // 512 + 36) * 2.0 ** -24) * want, want, got.dtype))


@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -112, 2.0 ** -120, 2.0 ** -126, 2.0 ** -140])
def test_small_f32_operands(size, odd):
    """The third piece is a multiple of BF16's smallest number, 2^-133: an operand is taken
    to within 2^-134, whatever it is multiplied with."""
    t, P, N, K = _api(), 300, 136, 200
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(P, K + odd, device="cuda", generator=g)[:, :K] * size
    w = torch.randn(N, K + odd, device="cuda", generator=g)[:, :K] * 2.0 ** 20
    want, bound = o.product(x, w[None], None)
    bound = bound + 2.0 ** -134 * w.double().abs().sum(1) + 2.0 ** -149
    close(t.tbe_expert_forward(x, w), want, rounded(bound, want, torch.float32))
    dy = torch.randn(P, N, device="cuda", generator=g) * 2.0 ** 20
    want, bound = o.weight_gradient(dy, x, None, 1)
    bound = bound + 2.0 ** -134 * dy.double().abs().sum(0)[:, None] + 2.0 ** -149
    close(t.tbe_expert_weight_backward(dy, x)[None], want, rounded(bound, want, torch.float32))
