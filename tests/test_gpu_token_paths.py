"""The table gradient by sorted tokens at the sizes where its launches are the
sort, the sums of runs and the join, not the one launch of few tokens: run
lengths around the long-run limit, rows with gaps between them, gradients of
one row for all tokens, batches without a token that counts, tables beyond two
digits and beyond 32 bits.  Every case says which launches it means to run."""
import ctypes
import math

import pytest
import torch

import token_oracle as o
from test_gpu_tokens import RUNS, _api, _gen, _ids, _rand, _strided
from token_oracle import TYPES, U32, close, rounding

pytestmark = pytest.mark.gpu


class Launches:
    """The timing hook of a call: names of its kernel launches."""

    def __init__(self, most=32):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * most)]
        for e in self.events:
            e.record()
        self.handles = (ctypes.c_void_p * (2 * most))(*[e.cuda_event for e in self.events])
        self.raw = (ctypes.c_char_p * most)()
        self.used = ctypes.c_int32(0)
        self.cfg = _api().config()
        self.cfg.kernel_events, self.cfg.kernel_names = ctypes.addressof(self.handles), ctypes.addressof(self.raw)
        self.cfg.n_kernel_events, self.cfg.kernel_events_used = most, ctypes.addressof(self.used)

    def names(self):
        return [self.raw[i].decode().removeprefix("tbe_token_") for i in range(self.used.value)]


def _gradient(grad, ids, V, want_launches, scale=1.0, padding=None, dtype=None, out=None, accumulate=False):
    """The gradient, within its bound of the definition, by the launches given."""
    dt = dtype or grad.dtype
    base = out.clone() if accumulate else None
    launches = Launches()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = _api().tbe_token_backward(grad, ids, V, scale=scale, padding_id=padding, dtype=dt if out is None else None,
                                    grad_table=out, accumulate=accumulate, status=status, cfg=launches.cfg)
    assert launches.names() == want_launches
    assert status.tolist() == [int(((ids < 0) | (ids >= V)).sum()), 0, 0, 0]
    want, mag, n = o.token_backward(grad, ids, V, scale, padding)
    bound = (n + 2) * U32 * mag
    if accumulate:
        want = want + base.double()
        bound = bound + 2 * U32 * (mag + base.double().abs()) + rounding(want, got.dtype) + U32 * bound
        untouched = (n == 0).expand_as(want)
        assert torch.equal(got[untouched], base[untouched])
    else:
        bound = torch.where(n == 0, 0.0, bound + rounding(want, got.dtype) * (1 + 2.0 ** -7))
    close(got, want, bound)
    return got


SORTED = ["sort", "reduce", "join"]                      # one CTA's sort, zeros beside it
TILES = ["count", "place"]


@pytest.mark.parametrize("D,t", [(1, "f32"), (4, "f32"), (17, "bf16"), (24, "f32"), (40, "bf16"), (128, "f32"), (300, "f16")])
@pytest.mark.parametrize("runs", RUNS, ids=[str(r)[:24] for r in RUNS])
def test_run_lengths(runs, D, t):
    # filler tokens in rows of their own behind the runs, in one token each and
    # in longer ones, move the call to the sort without moving the runs
    V, filler = 3 * len(runs) + 2, 2500
    ids = torch.cat([torch.full((n,), 3 * i + 1, dtype=torch.int64) for i, n in enumerate(runs)] +
                    [V + torch.arange(filler // 2), V + filler // 2 + torch.arange(filler // 2) // 7])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(D))].cuda()
    V += filler
    grad = _rand(D, (len(ids), D), t)
    a = _gradient(grad, ids, V, SORTED)
    assert torch.equal(a, _api().tbe_token_backward(grad, ids, V))
    b = _rand(D + 1, (V, D), t)
    _gradient(grad, ids, V, SORTED, out=b, accumulate=True)
    mixed = ids.clone()
    mixed[::3] = -1
    mixed[1::5] = 1
    _gradient(grad, mixed, V, SORTED, padding=1)


@pytest.mark.parametrize("N,sort", [(3000, ["sort"]), (20_000, TILES)])
@pytest.mark.parametrize("extra,shift", [(0, 1), (5, 0), (8, 8), (3, 2)])
@pytest.mark.parametrize("t,out", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_strided(N, sort, extra, shift, t, out):
    # rows with gaps, or off 16 bytes, are zeroed by a launch of their own
    V, D = 700, 40
    ids = _ids(N + extra, N, V)
    ids = torch.where(ids % 11 == 3, 3, ids)              # one long run
    grad = _rand(6, (N, D), t)
    for accumulate in (False, True):
        table = _strided(_rand(7, (V, D), out), extra, shift)
        before = table._base.clone()
        launches = ([] if accumulate else ["zero"]) + sort + ["reduce", "join"]
        _gradient(_strided(grad, extra, shift), ids, V, launches, scale=0.5, out=table, accumulate=accumulate)
        between = torch.ones_like(before, dtype=torch.bool)
        between[shift:].view(V, D + extra)[:, :D] = False
        assert torch.equal(table._base[between], before[between])


@pytest.mark.parametrize("N,sort", [(3000, ["sort"]), (9000, TILES)])
def test_one_row_for_all_tokens(N, sort):
    ids = _ids(8, N, 40, bad=0.1)
    grad = _rand(9, (1, 32), "f32").expand(N, 32)
    _gradient(grad, ids, 40, sort + ["reduce", "join"])


@pytest.mark.parametrize("N,sort", [(3000, ["sort"]), (9000, TILES)])
@pytest.mark.parametrize("D", [7, 64])
def test_nothing_to_sum(N, sort, D):
    grad = torch.full((N, D), math.nan, device="cuda")
    for ids in (torch.full((N,), -1, device="cuda"), torch.full((N,), 9, device="cuda"),
                torch.full((N,), 5, dtype=torch.int32, device="cuda")):
        got = _gradient(grad, ids, 9, sort + ["reduce", "join"], padding=5)
        assert not got.any()
        base = _rand(1, (9, D), "f32")
        kept = base.clone()
        _gradient(grad, ids, 9, sort + ["reduce", "join"], padding=5, out=base, accumulate=True)
        assert torch.equal(base, kept)


@pytest.mark.parametrize("N,sort", [(3000, ["sort"]), (9000, TILES)])
def test_infinities_stay_in_their_row(N, sort):
    V, D = 500, 36
    ids = _ids(2, N, V, bad=0.05)
    ids[100:400] = 17                                     # a long run with one infinity
    grad = _rand(3, (N, D), "f32")
    left_out = (ids < 0) | (ids >= V) | (ids == 4)
    grad[left_out] = math.nan
    kept = torch.nonzero(~left_out)[:, 0]
    grad[kept[0], 3], grad[kept[5], 7], grad[200, 11] = math.inf, math.nan, -math.inf
    launches = Launches()
    got = _api().tbe_token_backward(grad, ids, V, padding_id=4, cfg=launches.cfg)
    assert launches.names() == sort + ["reduce", "join"]
    want, mag, n = o.token_backward(grad, ids, V, 1.0, 4)
    close(got, want, torch.nan_to_num((n + 4) * U32 * mag, nan=0.0, posinf=0.0))
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[ids[[int(kept[0]), int(kept[5]), 200]]] = True
    assert bool(torch.isfinite(got[~touched]).all())


@pytest.mark.parametrize("V", [(1 << 20) - 1, 1 << 20, 1 << 21])
@pytest.mark.parametrize("N,sort", [(3000, 1), (30_000, 2)])
def test_three_digits(V, N, sort):
    g = _gen(N + V)
    ids = (torch.rand(N, generator=g, device="cuda").pow(5) * V).long().clamp(max=V - 1)
    ids[::7] = V - 1 - torch.arange(len(ids[::7]), device="cuda") % 50
    ids[3::11] = -5
    passes = 2 if V < 1 << 20 else 3
    _gradient(_rand(N, (N, 12), "bf16"), ids, V, (["sort"] if sort == 1 else TILES * passes) + ["reduce", "join"],
              dtype=torch.float32)


@pytest.mark.parametrize("N,sort", [(3000, ["sort"]), (9000, TILES * 3)])
def test_offsets_beyond_32_bits(N, sort):
    V, D = 40_000_000, 64                                 # 2.56e9 elements
    ids = torch.randint(0, V, (N,), generator=_gen(N), device="cuda")
    ids[:40] = V - 1
    ids[40:44] = torch.tensor([0, 33_554_431, 33_554_432, V - 2], device="cuda")
    ids[50:60] = -1
    grad = _rand(0, (N, D), "bf16")
    launches = Launches()
    dW = _api().tbe_token_backward(grad, ids, V, cfg=launches.cfg)
    assert launches.names() == sort + ["reduce", "join"]
    rows, at = torch.unique(ids[ids >= 0], return_inverse=True)
    want, mag, n = o.token_backward(grad[ids >= 0], at, len(rows), 1.0)
    close(dW[rows], want, (n + 2) * U32 * mag + rounding(want, torch.bfloat16) * (1 + 2.0 ** -7))
    dW[rows] = 0
    assert int(torch.count_nonzero(dW)) == 0


def test_grad_rows_beyond_32_bits():
    N, D = 1_100_000, 2050                                # 2.26e9 elements
    grad = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    pick = torch.randint(0, N, (5000,), generator=_gen(1), device="cuda").unique()
    pick = torch.cat([pick, torch.tensor([N - 1], device="cuda")]).unique()
    ids[pick] = torch.arange(len(pick), dtype=torch.int32, device="cuda") % 90
    grad[pick] = _rand(2, (len(pick), D), "bf16")
    launches = Launches()
    got = _api().tbe_token_backward(grad, ids, 90, dtype=torch.float32, cfg=launches.cfg)
    assert launches.names() == TILES + ["reduce", "join"]
    want, mag, n = o.token_backward(grad[pick], ids[pick], 90, 1.0)
    close(got, want, (n + 2) * U32 * mag + rounding(want, torch.float32))
