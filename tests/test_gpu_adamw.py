"""AdamW over many tensors (adamw_plan / _grad_norm / _step / _state_values) against 64 bits.

Tolerances, derived before any run, with u = 2^-24: m and v are two products and a sum, each
rounded once, on coefficients rounded once: 4 u of the sum of the terms' magnitudes.  The update
m / (sqrt(v) k + eps) carries 4 u of m's terms, 4 u of v's through the root, and at most 12 u for
the bias corrections (an fp32 expm1 and a root), the root, the product, the sum and the quotient,
taken as 20 u lr (|m terms| / denominator); p adds 2 u |p| and, in bf16, half a unit in the last
of 8 bits.  A rounded code equals floor(x + u16 / 2^16) of the exact x; where x + u16 / 2^16 lies
within 2^-10 of a whole number (the fp32 error of x is below 128 steps times 2^-20) the code
next to it is allowed too."""
import numpy as np
import pytest
import torch

import adamw_ref as ref
from mxfp8_block_scaled_rowwise_gb300 import binding as mx
from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
SIZES = [1, 7, 31, 32, 33, 100, 2047, 2048, 2049, 5000, 40001]
BF, F32 = torch.bfloat16, torch.float32


class Params:
    """Tensors of the given sizes with random contents, and their plan."""

    def __init__(self, dev, sizes, bits, pdt, gdt, seed=0, copy=False, wd=0.1, lr_mult=1.0, shift=0):
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        self.sizes, self.bits = sizes, bits

        def rnd(n, std):
            mag = torch.exp(1.5 * torch.randn(-(-n // 32), 1, generator=gen, device=dev))
            return (torch.randn(-(-n // 32), 32, generator=gen, device=dev) * mag * std).reshape(-1)[:n]

        def own(t):   # `shift` bytes past an allocation's start
            k = shift // t.element_size()
            b = torch.zeros(t.numel() + k, dtype=t.dtype, device=dev)
            b[k:] = t
            return b[k:]
        self.p = [own((torch.randn(n, generator=gen, device=dev) * 0.02).to(pdt)) for n in sizes]
        self.g = [own(rnd(n, 1e-3).to(gdt)) for n in sizes]
        self.copy = [own(torch.zeros(n, dtype=BF, device=dev)) for n in sizes] if copy else None
        self.sm = self.sr = None
        if bits == 32:
            self.m = [own(rnd(n, 3e-4)) for n in sizes]
            self.v = [own(rnd(n, 1e-3).square()) for n in sizes]
        else:   # random codes under random scales (E4M3's NaN codes left out)
            nb = [-(-n // 32) for n in sizes]
            self.m = [own(torch.randint(0, 256, (n,), generator=gen, device=dev).to(torch.uint8)) for n in sizes]
            for m in self.m:
                m[(m & 127) == 127] = 0x35
            self.v = [own(torch.randint(0, 256, (n,), generator=gen, device=dev).to(torch.uint8)) for n in sizes]
            self.sm = [torch.randint(100, 108, (n + 1,), generator=gen, device=dev).to(torch.uint8)[1:] for n in nb]
            self.sr = [torch.randint(110, 118, (n + 1,), generator=gen, device=dev).to(torch.uint8)[1:] for n in nb]
        self.wd = wd
        self.plan = mx.adamw_plan(self.p, self.g, self.m, self.v, self.sm, self.sr, self.copy, wd, lr_mult)
        self.step = torch.zeros(1, dtype=torch.int64, device=dev)

    def np(self, ts):
        return [t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy() for t in ts]

    def moments(self):
        if self.bits == 32:
            return [m.astype(np.float64) for m in self.np(self.m)], [v.astype(np.float64) for v in self.np(self.v)]
        m = [ref.decode(c, s, ref.E4M3) for c, s in zip(self.np(self.m), self.np(self.sm))]
        r = [ref.decode(c, s, ref.ROOT) for c, s in zip(self.np(self.v), self.np(self.sr))]
        return m, [x * x for x in r]

    def bytes(self):
        ts = self.p + self.m + self.v + (self.sm or []) + (self.sr or []) + (self.copy or []) + [self.step]
        return [t.clone() for t in ts]


def _param_slack(p0, g, m0, v0, t, scale, wd, h):
    b1, b2 = h["beta1"], h["beta2"]
    terms = b1 * np.abs(m0) + (1 - b1) * np.abs(g * scale)
    v = b2 * v0 + (1 - b2) * (g * scale) ** 2
    den = np.sqrt(v / (1 - b2 ** t)) + h["eps"]
    return 20 * U * h["lr"] / (1 - b1 ** t) * terms / den + 2 * U * np.abs(p0)


def _check_codes(x, got, u16, top, mantissa, low, least):
    """got: decoded values; x: exact magnitudes; every value the stochastic rounding of x."""
    steps, one, e = ref.grid(x, top, mantissa, low)
    y = steps + u16 / 65536.0
    want = np.floor(y) * one
    unit = np.repeat(np.exp2(e), 32)[:x.size]
    want = np.where((x > 0) & (want < least * unit), least * unit, want)
    near = np.abs(y - np.round(y)) < 2.0 ** -10
    diff = np.abs(got - want)
    assert (diff[~near] == 0).all(), (diff[~near].max(), int((diff[~near] > 0).sum()))
    assert (diff[near] <= 2 * one[near]).all()
    assert near.mean() < 0.02 or x.size < 2000


@pytest.mark.parametrize("bits,pdt,gdt,copy,stochastic", [
    (32, BF, BF, False, False), (32, BF, F32, False, True), (32, F32, F32, True, False), (32, F32, BF, False, False),
    (8, BF, F32, False, True), (8, BF, BF, False, False), (8, F32, F32, True, False), (8, F32, BF, True, True)])
@pytest.mark.parametrize("shift", [0, 16])
def test_steps_match_64_bit(dev, bits, pdt, gdt, copy, stochastic, shift):
    s = Params(dev, SIZES, bits, pdt, gdt, seed=bits + 3 * copy, copy=copy, wd=[0.1 * (i % 2) for i in range(len(SIZES))], shift=shift)
    norm = torch.zeros(2, device=dev)
    for t in (1, 2, 3):
        p0, g, (m0, v0) = s.np(s.p), s.np(s.g), s.moments()
        mx.adamw_grad_norm(s.plan, 1e-2, norm)
        mx.adamw_step(s.plan, s.step, grad_scale=norm[1:], seed=77, stochastic=stochastic, **HYPER)
        torch.cuda.synchronize()
        want = np.sqrt(sum((x.astype(np.float64) ** 2).sum() for x in g))
        got_norm, scale = norm.cpu().numpy().astype(np.float64)
        assert abs(got_norm - want) <= 1e-6 * want and abs(scale - min(1.0, 1e-2 / want)) <= 1e-6 * scale
        assert int(s.step) == t
        p1, (m1, v1) = s.np(s.p), s.moments()
        codes = s.np(s.m)
        for i, n in enumerate(s.sizes):
            x0, gi = p0[i].astype(np.float64), g[i].astype(np.float64)
            pe, me, ve = ref.step(x0, gi, m0[i], v0[i], t, HYPER["lr"], 0.9, 0.999, 1e-8, s.wd[i], scale)
            slack = _param_slack(x0, gi, m0[i], v0[i], t, scale, s.wd[i], HYPER)
            pos = s.plan.starts[i] + np.arange(n)
            um, ur, up = ref.random_bits(pos, 77, t)
            if pdt == BF and stochastic:
                ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(pe), 2.0 ** -126))) - 7)
                y = np.abs(pe) / ulp + up / 65536.0
                near = np.abs(y - np.round(y)) < slack / ulp + 2.0 ** -12
                diff = np.abs(np.abs(p1[i]) - np.floor(y) * ulp)
                assert (diff[~near] == 0).all() and (diff[near] <= 2 * ulp[near]).all()
            else:
                half = 2.0 ** -8 * np.abs(pe) if pdt == BF else 0.0
                assert (np.abs(p1[i] - pe) <= slack + half).all()
            if copy:
                assert torch.equal(s.copy[i], s.p[i].to(BF))
            if bits == 32:
                terms = 0.9 * np.abs(m0[i]) + 0.1 * np.abs(gi * scale)
                assert (np.abs(m1[i] - me) <= 4 * U * terms + 1e-45).all()
                assert (np.abs(v1[i] - ve) <= 5 * U * ve + 1e-45).all()
            else:
                _check_codes(np.abs(me), np.abs(m1[i]), um, 448.0, 3, -6, 0.0)
                assert (np.sign(m1[i])[m1[i] != 0] == np.sign(me)[m1[i] != 0]).all()
                _check_codes(np.sqrt(ve), np.sqrt(v1[i]), ur, 31 / 16, 4, -15, 17 / 16 * 2.0 ** -15)
                assert ((codes[i] & 127) != 127).all()


def test_state_values_are_the_codes_values(dev):
    s = Params(dev, SIZES, 8, BF, BF, seed=5)
    mom, root = (torch.full((s.plan.positions,), 9.0, dtype=BF, device=dev) for _ in range(2))
    mx.adamw_state_values(s.plan, mom, root)
    m, v = s.moments()
    for i, n in enumerate(s.sizes):
        a = s.plan.starts[i]
        assert np.array_equal(mom[a:a + n].double().cpu().numpy(), m[i])
        assert np.array_equal(root[a:a + n].double().cpu().numpy(), np.sqrt(v[i]))
        end = s.plan.starts[i + 1] if i + 1 < len(s.sizes) else s.plan.positions
        assert bool((mom[a + n:end] == 9.0).all()) and bool((root[a + n:end] == 9.0).all())


def _one(dev, n, bits, g, pdt=F32, p=None, **kw):
    z = torch.zeros
    p = z(n, dtype=pdt, device=dev) if p is None else p
    if bits == 8:
        m, v, sm, sr = z(n, dtype=torch.uint8, device=dev), z(n, dtype=torch.uint8, device=dev), z(-(-n // 32), dtype=torch.uint8, device=dev), z(-(-n // 32), dtype=torch.uint8, device=dev)
        plan = mx.adamw_plan([p], [g], [m], [v], [sm], [sr], **kw)
    else:
        m, v, sm, sr = z(n, device=dev), z(n, device=dev), None, None
        plan = mx.adamw_plan([p], [g], [m], [v], **kw)
    return plan, p, m, v, sm, sr, torch.zeros(1, dtype=torch.int64, device=dev)


@pytest.mark.parametrize("bits", [8, 32])
def test_zero_gradients_from_the_initial_state(dev, bits):
    """Nothing but weight decay happens; no NaN from a zero second moment; zero blocks stay zero."""
    n = 3000
    p = torch.linspace(-1, 1, n, device=dev)
    p0 = p.clone()
    plan, p, m, v, sm, sr, step = _one(dev, n, bits, torch.zeros(n, device=dev), p=p, weight_decay=0.5)
    for _ in range(3):
        mx.adamw_step(plan, step, lr=0.1)
    assert not m.any() and not v.any() and (bits == 32 or not (sm.any() or sr.any()))
    assert torch.allclose(p, p0 * 0.95 ** 3, rtol=1e-6)


def test_range_inside_a_block(dev):
    """Gradients 2^-30 apart in one block: the small ones' second moment never becomes zero, and
    their first moment, below E4M3's range under the block's scale, is zero or its smallest code."""
    n = 64
    g = torch.exp2(torch.linspace(0, -62, n, device=dev))
    plan, p, m, v, sm, sr, step = _one(dev, n, 8, g)
    for _ in range(5):
        mx.adamw_step(plan, step, lr=1e-3)
    mom, root = (torch.zeros(n, dtype=BF, device=dev) for _ in range(2))
    mx.adamw_state_values(plan, mom, root)
    assert bool((root > 0).all()) and bool(torch.isfinite(p).all()) and bool(torch.isfinite(mom).all())
    assert float(p.abs().max()) <= 5 * 1e-3 * 11    # no step above lr b1-corrected m over the root of its own v


def test_eight_bit_moments_follow_small_changes(dev):
    """Constant gradients for 3000 steps: each step moves r by less than 0.05 %, far below a code
    (3 to 6 %).  Stochastic rounding follows; rounding to nearest would stop where it started."""
    n, g0 = 8192, 0.01
    g = torch.full((n,), g0, device=dev)
    plan, p, m, v, sm, sr, step = _one(dev, n, 8, g)
    for _ in range(3000):
        mx.adamw_step(plan, step, lr=0.0, seed=3)
    mom, root = (torch.zeros(n, dtype=BF, device=dev) for _ in range(2))
    mx.adamw_state_values(plan, mom, root)
    want = g0 * (1 - 0.999 ** 3000) ** 0.5
    # one value's spread is below a code (6 %); the mean over 8192 is held to 2 %
    assert abs(float(root.float().mean()) / want - 1) < 0.02
    assert abs(float(mom.float().mean()) / g0 - 1) < 0.02


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite_skip_the_step(dev, bits, bad):
    s = Params(dev, [100, 5000, 33], bits, BF, F32, seed=8)
    s.g[1][4321] = bad
    norm = torch.zeros(2, device=dev)
    before = s.bytes()
    mx.adamw_grad_norm(s.plan, 1.0, norm)
    mx.adamw_step(s.plan, s.step, grad_scale=norm[1:], seed=1, stochastic=True, **HYPER)
    torch.cuda.synchronize()
    assert not torch.isfinite(norm[0]) and torch.isnan(norm[1])
    assert all(torch.equal(a, b) for a, b in zip(before, s.bytes()))
    s.g[1][4321] = 0.0
    mx.adamw_grad_norm(s.plan, 1.0, norm)
    mx.adamw_step(s.plan, s.step, grad_scale=norm[1:], seed=1, stochastic=True, **HYPER)
    assert int(s.step) == 1 and bool(torch.isfinite(norm).all())
    assert not any(torch.equal(a, b) for a, b in zip(before[:3], s.bytes()[:3]))


def test_nan_without_clipping_stays_in_its_element_and_block(dev):
    n = 2080
    g = torch.full((n,), 0.5, device=dev)
    g[70] = float("nan")
    for bits in (8, 32):
        plan, p, m, v, sm, sr, step = _one(dev, n, bits, g, pdt=BF)
        mx.adamw_step(plan, step, lr=1e-2, stochastic=True)
        bad = torch.isnan(p)
        assert bool(bad[70]) and int(bad.sum()) == 1
        if bits == 8:
            assert int(sm[2]) == 255 and int(sr[2]) == 255 and int((sm == 255).sum()) == 1 and int((sr == 255).sum()) == 1
            mom, root = (torch.zeros(plan.positions, dtype=BF, device=dev) for _ in range(2))
            mx.adamw_state_values(plan, mom, root)
            for x in (mom, root):
                assert bool(torch.isnan(x[64:96]).all()) and int(torch.isnan(x).sum()) == 32


def test_norm_options(dev):
    s = Params(dev, SIZES, 32, F32, BF, seed=9)
    out = torch.zeros(2, device=dev)
    mx.adamw_grad_norm(s.plan, 0.0, out)
    want = float(torch.cat(s.g).double().norm())
    assert abs(float(out[0]) - want) <= 1e-6 * want and float(out[1]) == 1.0
    mx.adamw_grad_norm(s.plan, 10 * want, out)
    assert float(out[1]) == 1.0
    first = out.clone()
    mx.adamw_grad_norm(s.plan, 10 * want, out)
    assert torch.equal(first, out)
    for g in s.g:
        g.zero_()
    mx.adamw_grad_norm(s.plan, 1.0, out)
    assert out.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bits", [8, 32])
def test_same_bytes_on_another_stream_and_in_a_graph(dev, bits):
    """Three steps eagerly, on another stream, and as graph replays (the step count and the learning
    rate live on the device, so a replay is the next step) end in the same bytes."""
    lr = torch.tensor([1e-3], device=dev)
    norm = torch.zeros(2, device=dev)

    def one(s):
        mx.adamw_grad_norm(s.plan, 1e-2, norm)
        mx.adamw_step(s.plan, s.step, lr=123.0, lr_dev=lr, grad_scale=norm[1:], seed=4, stochastic=True)

    def fresh():
        return Params(dev, SIZES, bits, BF, F32, seed=10)
    a = fresh()
    for k in range(3):
        lr.fill_(1e-3 / (k + 1))
        one(a)
    b = fresh()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for k in range(3):
            lr.fill_(1e-3 / (k + 1))
            one(b)
    torch.cuda.synchronize()
    c = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(c)
    assert int(c.step) == 0
    for k in range(3):
        lr.fill_(1e-3 / (k + 1))
        graph.replay()
    torch.cuda.synchronize()
    assert int(a.step) == int(c.step) == 3
    for x, y, z in zip(a.bytes(), b.bytes(), c.bytes()):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_lr_mult_and_many_tensors(dev):
    """A thousand tensors of one to a few elements, each with its own factor on the rate."""
    n = 1000
    sizes = [1 + i % 5 for i in range(n)]
    s = Params(dev, sizes, 32, F32, F32, seed=11, wd=0.0, lr_mult=[(i % 7) / 4 for i in range(n)])
    p0, g, (m0, v0) = s.np(s.p), s.np(s.g), s.moments()
    mx.adamw_step(s.plan, s.step, **HYPER)
    p1 = s.np(s.p)
    for i in range(n):
        h = dict(HYPER, lr=HYPER["lr"] * (i % 7) / 4)
        pe = ref.step(p0[i].astype(np.float64), g[i], m0[i], v0[i], 1, h["lr"], 0.9, 0.999, 1e-8, 0.0)[0]
        assert (np.abs(p1[i] - pe) <= _param_slack(p0[i], g[i].astype(np.float64), m0[i], v0[i], 1, 1.0, 0.0, h) + 1e-12).all()


def test_elements_past_32_bits(dev):
    n = (1 << 32) + 45
    p = torch.zeros(n, dtype=BF, device=dev)
    g = torch.zeros(n, dtype=BF, device=dev)
    g[-50:] = 0.25
    plan, p, m, v, sm, sr, step = _one(dev, n, 8, g, p=p)
    norm = torch.zeros(2, device=dev)
    mx.adamw_grad_norm(plan, 0.0, norm)
    mx.adamw_step(plan, step, lr=0.5, seed=6)
    torch.cuda.synchronize()
    assert abs(float(norm[0]) - 0.25 * 50 ** 0.5) < 1e-5
    assert not p[:-50].any() and bool((p[-50:] == -0.5).all())
    assert int((m[-64:] > 0).sum()) == 50 and int((sm > 0).sum()) == 3   # 5 + 32 + 13 elements
    um, ur, up = ref.random_bits(np.arange(n - 45, n), 6, 1)
    x = np.full(45, 0.025)
    # the last block is ragged (13 elements) and the one before whole: both hold equal values
    got = ref.decode(m[-45:].cpu().numpy(), sm[-2:].cpu().numpy(), ref.E4M3)
    steps, one, e = ref.grid(x, 448.0, 3, -6)
    assert np.array_equal(got, np.floor(steps + um / 65536.0) * one)


def test_binding_refuses(dev):
    z = torch.zeros
    p, g, m, v = (z(40, device=dev) for _ in range(4))
    u8 = z(40, dtype=torch.uint8, device=dev)
    s8 = z(2, dtype=torch.uint8, device=dev)
    bad = [lambda: mx.adamw_plan([], [], [], []),
           lambda: mx.adamw_plan([p], [g, g], [m], [v]),
           lambda: mx.adamw_plan([p], [g[:39]], [m], [v]),
           lambda: mx.adamw_plan([p.half()], [g], [m], [v]),
           lambda: mx.adamw_plan([p], [g.half()], [m], [v]),
           lambda: mx.adamw_plan([p], [g], [m], [u8]),
           lambda: mx.adamw_plan([p], [g], [u8], [u8]),
           lambda: mx.adamw_plan([p], [g], [u8], [u8], [s8], [s8[:1]]),
           lambda: mx.adamw_plan([p], [g], [m], [v], copies=[p]),
           lambda: mx.adamw_plan([p.bfloat16()], [g], [m], [v], copies=[p.bfloat16()]),
           lambda: mx.adamw_plan([p], [g.cpu()], [m], [v]),
           lambda: mx.adamw_plan([z(80, device=dev)[::2]], [g], [m], [v]),
           lambda: mx.adamw_plan([z(44, device=dev)[1:41]], [g], [m], [v]),
           lambda: mx.adamw_plan([p], [g], [m], [v], weight_decay=-1.0),
           lambda: mx.adamw_plan([p], [g], [m], [v], weight_decay=[0.1, 0.1]),
           lambda: mx.adamw_plan([z(0, device=dev)], [z(0, device=dev)], [z(0, device=dev)], [z(0, device=dev)])]
    for i, f in enumerate(bad):
        with pytest.raises(mx.MxError):
            f()
            pytest.fail("case %d was taken" % i)
    plan = mx.adamw_plan([p], [g], [m], [v])
    step = z(1, dtype=torch.int64, device=dev)
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=0.1, beta1=1.0), dict(lr=0.1, beta2=-0.1),
               dict(lr=0.1, eps=0.0), dict(lr=0.1, grad_scale=step)):
        with pytest.raises(mx.MxError):
            mx.adamw_step(plan, step, **kw)
    with pytest.raises(mx.MxError):
        mx.adamw_step(plan, step.int(), lr=0.1)
    with pytest.raises(mx.MxError):
        mx.adamw_grad_norm(plan, -1.0, z(2, device=dev))
    with pytest.raises(mx.MxError):
        mx.adamw_state_values(plan, z(64, dtype=BF, device=dev), z(64, dtype=BF, device=dev))
    assert int(step) == 0 and not p.any()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_learning_rate_that_is_not_finite_shows(dev, bits):
    """NaN on the device as learning rate makes bf16 parameters NaN, whichever way they are rounded: never
    a value whose bits a rounding carry has changed."""
    for stochastic in (False, True):
        p = torch.full((4096,), 0.5, dtype=BF, device=dev)
        g = torch.full((4096,), 0.25, device=dev)
        plan, p, m, v, sm, sr, step = _one(dev, 4096, bits, g, p=p)
        mx.adamw_step(plan, step, lr=0.0, lr_dev=torch.tensor([float("nan")], device=dev), stochastic=stochastic)
        assert bool(torch.isnan(p).all())
