"""The time limit of the products' waits: where operands do not arrive the result is
NaN, the flag is set and the context stays usable.  The self-test waits for copies
that are never issued; nothing faults or hangs."""
import pytest
import torch

import layer_oracle as o

pytestmark = pytest.mark.gpu


def test_products_of_operands_that_do_not_arrive_are_nan():
    import recsys_table_embedding_gb300 as api
    from recsys_table_embedding_gb300 import tbe
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = tbe.tbe_selftest_wait_limit(tbe.SELFTEST_PRODUCT_COPY, status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, tbe.FLAG_MMA_TIMEOUT, 0, 0]
    assert bool(ws[:2 * 2 * 8 * 64].view(torch.bfloat16).isnan().all())
    x, w = torch.randn(300, 64, device="cuda").bfloat16(), torch.randn(72, 64, device="cuda").bfloat16()
    got = api.tbe_expert_forward(x, w, status=status)
    want, bound = o.product(x, w[None], None)
    o.close(got, want, o.rounded(bound, want, got.dtype))
