"""GPU test of a product that takes longer than its waits' limit of a second: what
is waited for is the next step, not the call's end."""
import pytest
import torch

import layer_oracle as o
from layer_oracle import close, rounded

pytestmark = pytest.mark.gpu


def test_a_ragged_group_behind_a_second_of_whole_ones():
    # 4608 steps of 64 rows in each of the first expert's 65,536 tiles, 2.5e15 operations
    # (1.3 s at 1.89 PFLOP/s), and one row of a second: only its step is cleared
    import recsys_table_embedding_gb300 as api
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 60 GB of the device")
    P, N = 294_912, 65_536
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(P + 1, N, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    route = api.tbe_route_sort((torch.arange(P + 1, device="cuda") == P).int().view(-1, 1), 2)
    assert route.offset.tolist() == [0, P, P + 1]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    got = api.tbe_expert_weight_backward(x, x, route, status=status)
    end.record()
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, 0]
    assert start.elapsed_time(end) > 1000      # (otherwise nothing has been shown)
    row = x[P].double()
    assert torch.equal(got[1][:256], (row[:256, None] * row[None]).bfloat16()) and not got[1].isnan().any()
    for a, b in ((0, 0), (N - 40, 777), (31_000, N - 264)):
        want, bound = o.weight_gradient(x[:P, a:a + 40], x[:P, b:b + 264], None, 1)
        close(got[0, a:a + 40, b:b + 264], want[0], rounded(bound[0], want[0], got.dtype))
    del x, got, row
    torch.cuda.empty_cache()
