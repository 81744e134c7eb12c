"""The time limit of the distillation's copy waits: a slice that does not arrive
makes its row NaN, whether or not the caller reads status words, and a row that
needs no slice is right.  The self-test waits for copies that are never issued;
nothing faults or hangs, the context stays usable."""
import math

import pytest
import torch

from test_gpu_tokens import _check_distill, _distill_case

pytestmark = pytest.mark.gpu


def test_late_slices_are_nan():
    from recsys_table_embedding_gb300 import tbe
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = tbe.tbe_selftest_wait_limit(tbe.SELFTEST_DISTILL_COPY, status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, tbe.FLAG_COPY_TIMEOUT, 0, 0]
    got = ws[:4 * 132].view(torch.float32)
    loss, lse, grad = got[:2], got[2:4], got[4:].view(2, 64)
    assert math.isnan(float(loss[0])) and math.isnan(float(lse[0])) and bool(grad[0].isnan().all())
    assert float(loss[1]) == 0 and float(lse[1]) == 0 and not grad[1].any()
    _check_distill(*_distill_case(3, 5, 700, 9, "f32"), 1.0)
