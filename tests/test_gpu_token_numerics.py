"""The distillation loss where its numbers are hard to hold: logits of any
size (rows of masked columns only, large offsets, the smallest and the largest
temperatures), in every form of launch: rows held on chip, rows too long for
that, gradients whose rows lie at another place within 16 bytes, few rows and
many, loss and gradient at once or from a stored lse."""
import math

import pytest
import torch

import token_oracle as o
from test_gpu_tokens import _api, _distill_case, _strided
from token_oracle import TYPES, U, U32, close

pytestmark = pytest.mark.gpu

# rows, columns (16-bit types twice that: as many bytes), a gradient at another phase
FORMS = {"held": (5, 9001, False), "long": (2, 450_001, False), "other phase": (5, 9001, True),
         "many": (70, 2100, False), "many, other phase": (70, 2100, True)}


def _definition(z, ids, top, gl, c):
    """(loss, lse, grad, p per column) in 64 bits, by logits as differences from
    their row's largest: 64 bits do not hold a log of a sum beside 1e20 either."""
    m = z.double().max(1).values
    m = torch.where(torch.isinf(m) | torch.isnan(m), torch.zeros_like(m), m)
    loss, low, grad, dense = o.distill(z.double() - m[:, None], ids, top, gl, c)
    return loss, torch.where(dense.sum(1) > 0, m / c + low, 0.0), grad, dense


def _bounds(z, ids, top, gl, c, want, stored):
    """Bounds of (loss, lse, grad).  A sum of exponentials is a chain of at most
    V/256 + 64 additions of terms that are off by 2^-21; an exponent of size d
    carries its scale's two roundings and its own (4 U32 d is more), 40 being
    the largest that counts in a sum.  A stored lse below 64 is off by half its
    last place; beyond, it is not used.  2^x below 2^-126 is 0."""
    loss, lse, grad, dense = want
    K, V = ids.shape[1], z.shape[1]
    m = z.double().max(1, keepdim=True).values
    d = torch.nan_to_num((m - z.double()) / c, nan=0.0, posinf=0.0)
    total = torch.log((-d).exp().sum(1))                       # log of the sum, without the maximum
    rel_sum = (V / 256 + 64 + 160) * U32 + 2.0 ** -21
    b_lse = rel_sum + 4 * U32 * ((m[:, 0] / c).abs() + lse.abs())
    valid = (ids >= 0) & (ids < V)
    t = torch.where(valid & torch.isfinite(top), top.double() / c, torch.nan)
    spread = (torch.nan_to_num(t, nan=-1e30).max(1).values - torch.nan_to_num(t, nan=1e30).min(1).values).clamp(0, 1e4)
    b_p = (K + 64) * U32 + 8 * U32 * spread[:, None] + 2.0 ** -21
    size = torch.where(valid, d.gather(1, ids.clamp(0, V - 1).long()), 0.0).max(1).values + total + spread + math.log(K + 1)
    b_loss = c * c * (b_p[:, 0] * size + rel_sum + 8 * U32 * size + (K + 8) * U32 * size)
    q = torch.where(dense.sum(1, keepdim=True) > 0, (-d - total[:, None]).exp(), 0.0)
    rel_q = rel_sum + 4 * U32 * d + (2 * U32 * lse.abs().clamp(max=64)[:, None] if stored else 0.0)
    b = (gl.double() * c).abs()[:, None] * (q * rel_q + dense * b_p + 4 * U32 * (q + dense) + 2.0 ** -125)
    return b_loss, b_lse, b + o.rounding(grad, z.dtype) + b * U[z.dtype] + 2.0 ** -125


def _check(z, ids, top, gl, c, other, lse_fits=True):
    api = _api()
    c = float(torch.tensor(c, dtype=torch.float32))
    want = _definition(z, ids, top, gl, c)
    for two in (False, True):
        out = _strided(torch.zeros_like(z), 16 // z.element_size(), 1) if other else torch.empty_like(z)
        if two:
            loss, lse = api.tbe_distill_forward(z, ids, top, temperature=c)
            grad = api.tbe_distill_backward(z, ids, top, lse, gl, temperature=c, grad_logits=out)
        else:
            loss, lse, grad = api.tbe_distill_loss_grad(z, ids, top, gl, temperature=c, grad_logits=out)
        bl, bs, bg = _bounds(z, ids, top, gl, c, want, two)
        close(loss, want[0], bl)
        if lse_fits:
            close(lse, want[1], bs)
        close(grad, want[2], bg)
    if other:
        return
    # in the logits' place: the same numbers
    for two in (False, True):
        zz = z.clone()
        if two:
            _, lse = api.tbe_distill_forward(zz, ids, top, temperature=c)
            api.tbe_distill_backward(zz, ids, top, lse, gl, temperature=c, grad_logits=zz)
        else:
            api.tbe_distill_loss_grad(zz, ids, top, gl, temperature=c, grad_logits=zz)
        close(zz, want[2], _bounds(z, ids, top, gl, c, want, two)[2])


def _case(form, t, K=12, seed=1):
    N, V, other = FORMS[form]
    return _distill_case(seed, N, V if t == "f32" else 2 * V, K, t, short=False), other


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("value", [-1e10, -7e11, -1e15, -1e20, -1e28])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_masked_stretches(form, t, value):
    # whole stretches of a row at a mask's value, the rest ordinary
    (z, ids, top, gl), other = _case(form, t)
    V = z.shape[1]
    free = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids.long(), True)
    at = torch.arange(V, device="cuda")
    mask = ((at >= V // 3) | (at % 4 == 1)) & ~free
    z = torch.where(mask, torch.tensor(value, device="cuda").to(z.dtype), z)
    _check(z, ids, top, gl, 1.0, other)


@pytest.mark.parametrize("form", ["held", "many"])
@pytest.mark.parametrize("t,value", [("f32", -1e9), ("f32", -1e10), ("f32", 3e12), ("f32", -1e20), ("f32", "lowest"),
                                     ("bf16", -1e10), ("bf16", "lowest"), ("f16", "lowest")])
def test_loss_and_gradient_of_rows_of_one_value(form, t, value):
    (z, ids, top, gl), _ = _case(form, t)
    z.fill_(torch.finfo(TYPES[t]).min if value == "lowest" else value)
    want = _definition(z, ids, top, gl, 1.0)
    loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, gl)
    for got, w, b in zip((loss, lse, grad), want, _bounds(z, ids, top, gl, 1.0, want, False)):
        close(got, w, b)


@pytest.mark.parametrize("form", ["held", "many"])
@pytest.mark.parametrize("c", [1.0, 0.01])
def test_loss_and_gradient_of_parts_on_both_sides_of_a_size(form, c):
    # ascending rows around powers of two of max / c log2 e: the parts of a row
    # that are summed apart lie on both sides, and all of them count
    c = float(torch.tensor(c))
    for e in (12, 20, 21, 24, 31, 34):
        (z, ids, top, gl), _ = _case(form, "f32", seed=e)
        z = (2.0 ** e * math.log(2.0) * c + z.double().sort(1).values * c).float()
        want = _definition(z, ids, top, gl, c)
        loss, lse, grad = _api().tbe_distill_loss_grad(z, ids, top, gl, temperature=c)
        for got, w, b in zip((loss, lse, grad), want, _bounds(z, ids, top, gl, c, want, False)):
            close(got, w, b)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("t,value", [("f32", -1e9), ("f32", -1e10), ("f32", 3e12), ("f32", -1e20), ("f32", "lowest"),
                                     ("bf16", -1e10), ("bf16", "lowest"), ("f16", "lowest")])
def test_rows_of_one_value(form, t, value):
    # every column masked alike, or nearly: the softmax is uniform whatever the value
    (z, ids, top, gl), other = _case(form, t)
    z.fill_(torch.finfo(TYPES[t]).min if value == "lowest" else value)
    _check(z, ids, top, gl, 1.0, other)
    _check(z, ids, top, gl, 0.25, other, lse_fits=value != "lowest")   # below the lowest 32-bit number


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("t,offset", [("f32", 300.0), ("f32", -20_000.0), ("f32", 1e6), ("bf16", 900.0), ("f16", -60_000.0)])
def test_offset_logits(form, t, offset):
    (z, ids, top, gl), other = _case(form, t)
    z = (z.float() + offset).to(z.dtype)
    _check(z, ids, top, gl, 1.0, other)
    _check(z, ids, top, gl, 0.3, other)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("c,centre,step", [(1e-6, 5.0, 2.0 ** -21), (1e-6, 2000.0, 0.0), (1e-6, -3e4, 0.0), (1e-3, 40.0, 2.0 ** -10),
                                           (1e6, 0.0, 1e5), (1e6, 1e12, 2.0 ** 17)])
def test_temperatures(form, c, centre, step):
    (z, ids, top, gl), other = _case(form, "f32")
    z = torch.round(z) * step + centre
    top = (torch.round(top) * min(c, 1.0)).float()
    _check(z, ids, top, gl, c, other)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("c", [1.0, 0.01])
def test_parts_on_both_sides_of_a_size(form, c):
    # ascending rows around powers of two of max / c log2 e: the parts of a row
    # that are summed apart lie on both sides, and all of them count
    for e in (12, 20, 21, 24):
        (z, ids, top, gl), other = _case(form, "f32", seed=e)
        z = (2.0 ** e * math.log(2.0) * c + z.double().sort(1).values * c).float()
        _check(z, ids, top, gl, c, other)


@pytest.mark.parametrize("K", [300, 1024])
def test_offset_logits_many_entries(K):
    # the teacher of a row is a whole block's
    z, ids, top, gl = _distill_case(K, 9, 5003, K, "f32", short=False)
    _check(z + 5000.0, ids, top, gl, 1.0, False)
    _check(torch.full_like(z, -1e10), ids, top, gl, 1.0, False)


@pytest.mark.parametrize("V", [450_001, 800_001])
def test_long_rows_in_place_of_many(V):
    # more clusters than run at once, every row its own values
    z, ids, top, gl = _distill_case(V, 40, V, 5, "bf16" if V > 500_000 else "f32", short=True)
    _check(z, ids, top, gl, 1.0, False)


@pytest.mark.parametrize("N,K", [(70, 5), (3, 300)])
@pytest.mark.parametrize("t,V", [("f32", 450_001), ("bf16", 900_003)])
@pytest.mark.parametrize("shift", [0.0, 3000.0])
def test_long_rows_with_their_teachers_apart(N, K, t, V, shift):
    # more rows, or entries, than share a launch with their teachers
    z, ids, top, gl = _distill_case(V + K, N, V, K, t)
    ids[1] = -1
    _check((z.float() + shift).to(z.dtype), ids, top, gl, 1.0, False)


@pytest.mark.parametrize("form", FORMS)
def test_rows_without_entries_in_every_form(form):
    (z, ids, top, gl), other = _case(form, "f32")
    ids[1] = -1
    z[1] = math.nan
    top[0] = -math.inf
    want = _definition(z, ids, top, gl, 1.0)
    assert not want[2][:2].any()
    for two in (False, True):
        out = _strided(torch.ones_like(z), 4, 1) if other else torch.empty_like(z)
        before = out._base.clone() if other else None
        if two:
            loss, lse = _api().tbe_distill_forward(z, ids, top)
            _api().tbe_distill_backward(z, ids, top, lse, gl, grad_logits=out)
        else:
            loss, lse, _ = _api().tbe_distill_loss_grad(z, ids, top, gl, grad_logits=out)
        assert not loss[:2].any() and not lse[:2].any() and not out[:2].any()
        if z.shape[0] > 2:
            bound = _bounds(z[2:], ids[2:], top[2:], gl[2:], 1.0, [w[2:] for w in want], two)
            close(out[2:], want[2][2:], bound[2])
        if other:
            between = torch.ones_like(before, dtype=torch.bool)
            between[1:].view(z.shape[0], -1)[:, :z.shape[1]] = False
            assert torch.equal(out._base[between], before[between])


@pytest.mark.parametrize("N", [5, 70])
@pytest.mark.parametrize("V,gap", [(2100, 0), (2101, 3), (2100, 2), (900_004, 0)])
def test_gradient_between_the_logits_rows(N, V, gap):
    # halves of one buffer's columns; nothing but the gradient's is written
    if N > 5 and V > 10_000:
        pytest.skip("covered by the few rows")
    z, ids, top, gl = _distill_case(V, N, V, 9, "bf16", short=False)
    both = torch.full((N, 2 * V + gap), 3.0, dtype=torch.bfloat16, device="cuda")
    both[:, :V] = z
    out = both[:, V + gap:]
    want = _definition(z, ids, top, gl, 1.0)
    for two in (False, True):
        out.fill_(5.0)
        if two:
            _, lse = _api().tbe_distill_forward(both[:, :V], ids, top)
            _api().tbe_distill_backward(both[:, :V], ids, top, lse, gl, grad_logits=out)
        else:
            _api().tbe_distill_loss_grad(both[:, :V], ids, top, gl, grad_logits=out)
        close(out, want[2], _bounds(z, ids, top, gl, 1.0, want, two)[2])
        assert torch.equal(both[:, :V], z) and bool((both[:, V:V + gap] == 3).all())
