"""GPU tests of the AdamW step against its definition in 64 bits, with states in
32 and in 8 bits, at the sizes, types, places and values where it can go wrong."""
import math

import pytest
import torch

import layer_oracle as o
from layer_oracle import close, rounded
from token_oracle import TYPES

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _api():
    import recsys_table_embedding_gb300 as tbe
    return tbe


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(seed, n, dtype, std=1.0):
    return torch.empty(n, dtype=torch.float32, device="cuda").normal_(0, std, generator=_gen(seed)).to(TYPES[dtype])


SIZES = [1, 2, 3, 31, 255, 256, 257, 1000, 2047, 2048, 2049, 5000, 70_003]


class State:
    """Tensors of the given sizes; packed: back to back, so at odd places."""

    def __init__(self, sizes, param="f32", grad="f32", copy=None, state="f32", packed=False, seed=0):
        total = sum(sizes) if packed else sum(-(-n // 64) * 64 for n in sizes)
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += n if packed else -(-n // 64) * 64
        cut = lambda flat: [flat[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        self.sizes, self.state = sizes, state
        self.p, self.g = cut(_rand(seed, total, param, 0.1)), cut(_rand(seed + 1, total, grad, 0.01))
        self.copies = cut(torch.zeros(total, dtype=TYPES[copy], device="cuda")) if copy else None
        self.scales = None
        if state == "f32":
            self.m, self.v = cut(_rand(seed + 2, total, "f32", 0.01)), cut(_rand(seed + 3, total, "f32", 0.01).square())
        else:
            self.m = cut(_rand(seed + 2, total, "f32", 90).clamp(-448, 448).to(F8))
            self.v = cut(_rand(seed + 3, total, "f32", 90).abs().clamp(2.0 ** -9, 448).to(F8))
            self.scales = [torch.rand(-(-n // 256), 2, generator=_gen(seed + 4), device="cuda").mul_(1e-4).add_(1e-5)
                           for n in sizes]

    def values(self):
        """(m, v) of each tensor in 64 bits"""
        if self.state == "f32":
            return [x.double() for x in self.m], [x.double() for x in self.v]
        wide = [s.double().repeat_interleave(256, 0)[:n] for s, n in zip(self.scales, self.sizes)]
        return ([x.double() * s[:, 0] for x, s in zip(self.m, wide)],
                [(x.double() * s[:, 1]).square() for x, s in zip(self.v, wide)])

    def copy(self):
        c = object.__new__(State)
        c.sizes, c.state = self.sizes, self.state
        for n in ("p", "g", "m", "v", "scales", "copies"):
            x = getattr(self, n)
            setattr(c, n, None if x is None else [t.clone() for t in x])
        return c

    def tensors(self):
        return self.p + self.m + self.v + (self.scales or []) + (self.copies or [])

    def step(self, t=3, **kw):
        _api().tbe_adamw_step(self.p, self.g, self.m, self.v, t, scales=self.scales, copies=self.copies, **kw)


HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-7, weight_decay=0.05)


def _check(s, t=3, seed=0, scale=1.0, hyper=HYPER, step=None, **kw):
    m0, v0 = s.values()
    p0 = [x.double() for x in s.p]
    s.step(step if step is not None else t, **hyper, seed=seed, **kw)
    h = hyper
    m1, v1 = s.values()
    for i, n in enumerate(s.sizes):
        g = s.g[i].double() * scale
        want, bound = o.adamw(p0[i], g, m0[i], v0[i], t, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"])
        # decoded states carry a rounding each (two of v: r and its square)
        more = 0.0
        if s.state != "f32" or scale != 1:
            change = (want[0] - p0[i]).abs() + h["lr"] * h["weight_decay"] * p0[i].abs()
            parts = h["beta1"] * m0[i].abs() + (1 - h["beta1"]) * g.abs()
            more = 8 * o.U32 * change + 4 * o.U32 * h["lr"] / (1 - h["beta1"] ** t) * parts / \
                (want[2].sqrt() / math.sqrt(1 - h["beta2"] ** t) + h["eps"])
        close(s.p[i], want[0], rounded(bound[0] + more, want[0], s.p[i].dtype))
        if s.copies is not None:
            assert torch.equal(s.copies[i], s.p[i].to(s.copies[i].dtype))
        if s.state == "f32":
            close(s.m[i], want[1], bound[1] + 2 * o.U32 * g.abs() + 2.0 ** -140)
            close(s.v[i], want[2], 2 * bound[2] + 2.0 ** -140)
            continue
        bits = o.random16(seed, t, i, n, "cuda")
        # (the states before the step are decoded with a rounding, v with two more)
        bm = bound[1] + o.U32 * h["beta1"] * m0[i].abs() + 2 * o.U32 * g.abs()
        br = 12 * o.U32 * want[2].sqrt()
        for k, (codes, x, b) in enumerate(((s.m[i], want[1], bm), (s.v[i], want[2].sqrt(), br))):
            q, sc, sure = o.encode(x, b, bits[k], k == 1)
            close(s.scales[i][:, k], sc, 4 * o.U32 * sc + o.in_blocks(b).amax(1) / 448)
            assert float(sure.double().mean()) > 0.98 or n < 100
            assert torch.equal(codes.double()[sure], q[sure])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"),
                                             ("bf16", "bf16", None), ("f16", "f16", None), ("f32", "f32", "bf16"),
                                             ("bf16", "f32", None)])
def test_step(packed, state, param, grad, copy):
    _check(State(SIZES, param, grad, copy, state, packed), seed=77)


@pytest.mark.parametrize("t", [1, 2, 10, 1000, 10_000_000])
@pytest.mark.parametrize("state", ["f32", "f8"])
def test_steps_far_and_near(t, state):
    _check(State([300, 5000], state=state), t=t)
    _check(State([300, 5000], state=state), t=t, hyper=dict(lr=1e-3, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0))


def test_more_tensors_than_a_launch_takes():
    sizes = [1 + (i * 37) % 900 for i in range(1000)]
    for state in ("f32", "f8"):
        _check(State(sizes, state=state, packed=True), seed=5)


def test_mixed_states_and_left_out_tensors():
    # states of both kinds in one call, tensors without a gradient and empty ones among them
    a, b = State(SIZES, state="f32"), State(SIZES, state="f8", seed=9)
    want = [x.copy() for x in (a, b)]
    n = len(SIZES)
    args = [x for pair in zip(a.p, b.p) for x in pair], [x for pair in zip(a.g, b.g) for x in pair]
    ms, vs = [x for pair in zip(a.m, b.m) for x in pair], [x for pair in zip(a.v, b.v) for x in pair]
    scales = [x for s in b.scales for x in (None, s)]
    args[1][4] = None
    before = [x.clone() for x in (args[0][4], ms[4], vs[4])]
    empty = torch.empty(0, device="cuda")
    lists = [x + [empty] for x in (args[0], args[1], ms, vs)]
    _api().tbe_adamw_step(*lists, 3, scales=scales + [None], seed=1, **HYPER)
    assert all(torch.equal(x, y) for x, y in zip(before, (args[0][4], ms[4], vs[4])))
    want[0].step(seed=1, **HYPER)
    for i in range(n):
        if i != 2:
            assert torch.equal(want[0].p[i], a.p[i]) and torch.equal(want[0].m[i], a.m[i])
    # the random numbers go by the place in the call's lists
    _api().tbe_adamw_step([x for p in want[1].p for x in (empty, p)], [x for p in want[1].g for x in (empty, p)],
                          [x for p in want[1].m for x in (empty, p)], [x for p in want[1].v for x in (empty, p)], 3,
                          scales=scales_of(want[1]), seed=1, **HYPER)
    for i in range(n):
        assert torch.equal(want[1].m[i].view(torch.uint8), b.m[i].view(torch.uint8))
        assert torch.equal(want[1].p[i], b.p[i])


def scales_of(s):
    return [x for c in s.scales for x in (None, c)]


def test_numbers_on_the_device():
    for state in ("f32", "f8"):
        s = State([3000, 17], state=state)
        step, lr = torch.tensor([4], device="cuda"), torch.tensor(0.25, device="cuda")
        _check(s, t=4, step=step, hyper=HYPER | dict(lr=0.25))
        s = State([3000, 17], state=state)
        same = s.copy()
        s.step(step, **(HYPER | dict(lr=lr)))
        same.step(4, **(HYPER | dict(lr=0.25)))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s.tensors(), same.tensors()))


def test_scaled_gradients():
    scale = torch.tensor(0.37, device="cuda")
    for state in ("f32", "f8"):
        _check(State(SIZES, grad="bf16", state=state), scale=float(scale), grad_scale=scale)


def test_captured_step_counts_on():
    a = State([4000, 300], state="f8")
    b = a.copy()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    warm = a.copy()
    warm.step(torch.ones(1, dtype=torch.int64, device="cuda"), **HYPER)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        a.step(step, seed=3, **HYPER)
    for t in (1, 2, 3):
        graph.replay()
        b.step(t, seed=3, **HYPER)
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.tensors(), b.tensors()))


def test_8_bit_states_follow_a_slow_average():
    # v under beta2 = 0.999 moves by less than a code a step: at random, it still
    # moves by the right amount on average.  After 400 steps of gradient 2 from
    # v = 1, v is 4 - 3 * 0.999^400 = 1.99.
    n = 1 << 16
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 2.0, device="cuda")
    m, v = torch.zeros(n, device="cuda", dtype=F8), torch.full((n,), 448.0, device="cuda").to(F8)
    scales = torch.full((n // 256, 2), 1 / 448, device="cuda")
    # every 256th element holds the scale up
    g[::256], scales[:, 1] = 8.0, 8 / 448
    v.view(torch.uint8).copy_(torch.full((n,), 56.0, device="cuda").to(F8).view(torch.uint8))
    v[::256] = torch.full((n // 256,), 448.0, device="cuda").to(F8)
    for t in range(1, 401):
        _api().tbe_adamw_step([p], [g], [m], [v], t, lr=0.0, scales=[scales], seed=11)
    r = v.float() * scales[:, 1].repeat_interleave(256)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::256] = False
    mean = float(r[keep].double().square().mean())
    want = 4 - 3 * 0.999 ** 400
    # sqrt(v) moves by dx = (4 - v) 0.001 / (2 sqrt(v)) <= 1.5e-3 a step, off a code
    # whose neighbour is h <= 8 * 8 / 448 away: rounded without bias, its square
    # gains the variance dx h (1 - dx / h) <= 2.2e-4 a step, 0.09 in 400 steps.
    # The mean of 65,000 values that spread by less than 1 is off by 0.02 at most.
    assert want - 0.02 <= mean <= want + 0.09 + 0.02


def test_roundings_are_unbiased():
    n = 1 << 18
    s = State([n], state="f8", seed=4)
    m0, v0 = s.values()
    s.step(3, seed=5, **HYPER)
    m1, v1 = s.values()
    for x, y in ((HYPER["beta1"] * m0[0] + (1 - HYPER["beta1"]) * s.g[0].double(), m1[0]),
                 ((HYPER["beta2"] * v0[0] + (1 - HYPER["beta2"]) * s.g[0].double() ** 2).sqrt(), v1[0].sqrt())):
        e = (y - x) / x.abs().clamp(min=1e-30)
        e = e[x.abs() > x.abs().mean() / 4]
        assert float(e.abs().max()) <= 2.0 ** -3 + 1e-5                     # a code's neighbours
        assert abs(float(e.mean())) <= 6 * float(e.std()) / math.sqrt(e.numel())


def test_offsets_beyond_32_bits():
    # a tensor of 2^31 elements and more: its last ones like a call of theirs
    n, k = (1 << 31) + 1000, 5000
    new = lambda dt: torch.zeros(n, dtype=torch.uint8 if dt is F8 else dt, device="cuda").view(dt)  # noqa: E731
    p, g, m, v = new(torch.bfloat16), new(torch.bfloat16), new(F8), new(F8)
    scales = torch.zeros(-(-n // 256), 2, device="cuda")
    p[-k:], g[-k:] = _rand(1, k, "bf16"), _rand(2, k, "bf16")
    before = p[-k:].clone()
    _api().tbe_adamw_step([p], [g], [m], [v], 1, scales=[scales], seed=3, **HYPER)
    zero = torch.zeros(k, device="cuda")
    h = HYPER
    want, bound = o.adamw(before, g[-k:], zero, zero, 1, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"])
    close(p[-k:], want[0], rounded(2 * bound[0], want[0], torch.bfloat16))
    assert not p[:-k].any() and not m[:-k].view(torch.uint8).any()
    b = n // 256 - 3
    low, high = (torch.stack([x]) for x in (scales[b:b + 2, 0], scales[b:b + 2, 1]))
    got = m[b * 256:(b + 2) * 256].float() * low.flatten().repeat_interleave(256)
    part = 0.1 * g[b * 256:(b + 2) * 256].float()
    assert float((got - part).abs().max()) <= 2.0 ** -3 * float(part.abs().max()) and bool((high > 0).all())


def test_values_out_of_range():
    n = 600
    for bad in (float("nan"), float("inf"), -float("inf")):
        s = State([n], state="f8")
        clean = s.copy()
        clean.step(seed=2, **HYPER)
        s.g[0][300] = bad
        s.step(seed=2, **HYPER)
        keep = torch.arange(n, device="cuda") // 256 != 1
        assert torch.equal(s.p[0][keep], clean.p[0][keep])
        others = torch.arange(n, device="cuda") != 300
        assert torch.equal(s.p[0][others], clean.p[0][others])
        assert torch.isnan(s.m[0][300].float()) and torch.isnan(s.v[0][300].float())
        assert torch.isfinite(s.m[0].float()[others]).all() and torch.isfinite(s.scales[0]).all()
    # all zero bytes are zero states; a block without anything stays zero
    s = State([n], state="f8")
    s.m[0].view(torch.uint8).zero_(), s.v[0].view(torch.uint8).zero_(), s.scales[0].zero_(), s.g[0].zero_()
    s.step(1, **HYPER)
    assert not s.m[0].float().any() and not s.v[0].float().any() and not s.scales[0].any()
    assert torch.isfinite(s.p[0]).all()
    # a small second moment keeps a code
    s.g[0].fill_(1e-12)
    s.g[0][::256] = 1.0
    s.step(1, **HYPER)
    assert (s.v[0].float() > 0).all()


def test_other_stream_and_versions():
    s = State([5000], copy="bf16")
    same = s.copy()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    versions = [x._version for x in s.tensors()]
    s.step(stream=stream, **HYPER)
    torch.cuda.synchronize()
    same.step(**HYPER)
    assert all(torch.equal(a, b) for a, b in zip(s.tensors(), same.tensors()))
    assert all(x._version > v for x, v in zip(s.tensors(), versions))


def test_refusals():
    t = _api()
    p, g, m, v = (torch.zeros(600, device="cuda") for _ in range(4))
    codes, sc = torch.zeros(600, device="cuda").to(F8), torch.zeros(3, 2, device="cuda")
    call = lambda p=p, g=g, m=m, v=v, step=1, **kw: t.tbe_adamw_step([p], [g], [m], [v], step, **kw)  # noqa: E731
    call()
    call(m=codes, v=codes.clone(), scales=[sc])
    for bad in (lambda: call(step=0), lambda: call(lr=-1.0), lambda: call(lr=float("nan")), lambda: call(beta1=1.0),
                lambda: call(beta2=-0.1), lambda: call(eps=-1.0), lambda: call(weight_decay=float("inf")),
                lambda: call(g=g[:-1]), lambda: call(m=m.half()), lambda: call(m=codes), lambda: call(m=codes, v=codes),
                lambda: call(m=codes, v=codes, scales=[sc[:2]]), lambda: call(m=codes, v=codes, scales=[sc.double()]),
                lambda: call(p=p.double()), lambda: call(g=g.cpu()), lambda: call(copies=[p.clone()]),
                lambda: call(copies=[p.half()[:-1]]), lambda: call(p=p[::2], g=g[:300], m=m[:300], v=v[:300]),
                lambda: call(step=torch.ones(1, device="cuda")), lambda: call(grad_scale=torch.ones(2, device="cuda")),
                lambda: call(p=p.clone().requires_grad_()), lambda: t.tbe_adamw_step([p], [], [m], [v], 1)):
        with pytest.raises(t.TbeError):
            bad()
    with torch.no_grad():
        q = p.clone().requires_grad_()
        call(p=q)


def test_copies_that_require_a_gradient_and_tensors_listed_twice_are_refused():
    from recsys_table_embedding_gb300 import layers
    p, g, m, v = (torch.ones(300, device="cuda") for _ in range(4))
    copy = p.to(torch.bfloat16).requires_grad_()
    with pytest.raises(RuntimeError, match="requires a gradient"):
        layers.tbe_adamw_step([p], [g], [m], [v], 1, copies=[copy])
    q, n, u = (torch.ones(300, device="cuda") for _ in range(3))
    for twice in (([p, p], [m, n], [v, u]), ([p, q], [m, m], [v, u]), ([p, q], [m, n], [v, v])):
        with pytest.raises(RuntimeError):
            layers.tbe_adamw_step(twice[0], [g, g], twice[1], twice[2], 1)
    assert torch.equal(p, m) and torch.equal(p, q)
    with torch.no_grad():
        layers.tbe_adamw_step([p, q], [g, g], [m, n], [v, u], 1, copies=[copy, None])
    assert torch.equal(p, q) and torch.equal(copy, p.to(torch.bfloat16)) and not torch.equal(p, g)
