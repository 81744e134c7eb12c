"""The bounds that the GPU tests hold the experts' products to see what they are made
for: planted here are products that leave a piece of an FP32 operand out, and sums that
are cut off too often, in the oracle, on the CPU."""
import pytest
import torch

from test_gpu_product_precision import MOST, _loss, pieces_above, third_pieces_close


def _pieces(x):
    parts, left = [], x.double()
    for _ in range(3):
        parts.append(left.bfloat16().double())
        left = left - parts[-1]
    return parts


def _product(x, w, without=()):
    """The sum of the six products of pieces that the kernels form, in 64 bits, rounded once."""
    a, b = _pieces(x), _pieces(w)
    return sum(a[i] @ b[j].t() for i in range(3) for j in range(3) if i + j < 3 and (i, j) not in without).float()


@pytest.mark.parametrize("K", [16, 501, 5001])
def test_pieces_that_are_left_out_are_seen(K):
    x, w = pieces_above(1, 100, K, device="cpu"), pieces_above(2, 80, K, device="cpu")
    assert torch.equal(sum(_pieces(x)), x.double()) and bool((_pieces(x)[2] > 0).all())
    want = x.double() @ w.double().t()
    third_pieces_close(_product(x, w), want, K)
    for without in ((0, 1), (1, 0), (0, 2), (2, 0), (1, 1)):
        with pytest.raises(AssertionError):
            third_pieces_close(_product(x, w, [without]), want, K)


@pytest.mark.parametrize("dtype,K", [("f16", 32_768), ("bf16", 1 << 20)])
def test_sums_that_are_not_cut_into_segments_are_seen(dtype, K):
    # what such sums were measured to lack (2^-27.3 of themselves a term) is beyond the bound
    # that is added to the result's rounding
    assert K > MOST[dtype] and K * 2.0 ** -27.3 > 2 * _loss(K, dtype, 0)
