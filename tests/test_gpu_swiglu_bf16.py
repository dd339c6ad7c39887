"""moe_swiglu_fwd / moe_swiglu_bwd against the formulas in 64 bits and against differences.

Tolerances, derived before any run.  sigmoid in fp32 from the special-function unit is within
(1.1 |g| + 20) 2^-24 of the true value; the products add at most 4 roundings of 2^-24 each; the
result rounds once to bf16 (half a unit in the last of 8 bits, at most 2^-8 of its magnitude).  The gate gradient's factor 1 + g (1 - s) can
cancel: its absolute error is at most (1 + |g|) (|g| + 24) 2^-23, scaled by |dh up s|."""
import pytest
import torch

from mxfp8_block_scaled_rowwise_gb300 import binding as mx
from mxfp8_block_scaled_rowwise_gb300 import synth
from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(1, 8), (3, 16), (7, 2040), (1, 2048), (129, 264), (64, 1536), (1000, 40), (5, 8200)]


def _forward(gate, up):
    return gate * torch.sigmoid(gate) * up


def _rel(gate):
    return (1.1 * gate.abs() + 20) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -8


@pytest.mark.parametrize("R,I", SIZES)
@pytest.mark.parametrize("scale", [1.0, 12.0])
def test_matches_64_bit(dev, R, I, scale):
    g = synth.generator(R + I)
    a = synth.randn_bf16((R, 2 * I), g, std=scale).to(dev)
    dh = synth.randn_bf16((R, I), g).to(dev)
    h = torch.empty(R, I, dtype=torch.bfloat16, device=dev)
    da = torch.empty(R, 2 * I, dtype=torch.bfloat16, device=dev)
    mx.moe_swiglu_fwd(a, R, I, h)
    mx.moe_swiglu_bwd(dh, a, R, I, da)
    gate, up, d = a[:, :I].double(), a[:, I:].double(), dh.double()
    s = torch.sigmoid(gate)
    tiny = 2.0 ** -126
    ref = _forward(gate, up)
    assert bool(((h.double() - ref).abs() <= _rel(gate) * ref.abs() + tiny).all())
    ref = d * gate * s
    assert bool(((da[:, I:].double() - ref).abs() <= _rel(gate) * ref.abs() + tiny).all())
    ref = d * up * s * (1 + gate * (1 - s))
    slack = (d * up * s).abs() * (1 + gate.abs()) * (gate.abs() + 24) * 2.0 ** -23
    assert bool(((da[:, :I].double() - ref).abs() <= _rel(gate) * ref.abs() + slack + tiny).all())
    # in place: da over a
    mx.moe_swiglu_bwd(dh, a, R, I, a)
    torch.cuda.synchronize()
    assert torch.equal(a, da)


def test_gradient_is_the_difference_of_the_forward(dev):
    R, I, step = 17, 24, 1e-6
    g = synth.generator(3)
    a = synth.randn_bf16((R, 2 * I), g, std=2.0).to(dev)
    dh = synth.randn_bf16((R, I), g).to(dev)
    da = torch.empty_like(a)
    mx.moe_swiglu_bwd(dh, a, R, I, da)
    gate, up, d = a[:, :I].double(), a[:, I:].double(), dh.double()
    for col, num in ((0, (_forward(gate + step, up) - _forward(gate - step, up)) / (2 * step)),
                     (I, (_forward(gate, up + step) - _forward(gate, up - step)) / (2 * step))):
        got = da[:, col:col + I].double()
        # bf16 rounding, the fp32 slack of the cancelling factor, and the difference's own error
        assert bool(((got - d * num).abs() <= 2.0 ** -8 * (d * num).abs() + 1e-5 * (d * up).abs() + 1e-7).all())


def test_extreme_values(dev):
    """Gates whose exponential over- or underflows, zeros of both signs, infinities and NaN."""
    big = 3.0e38
    gates = [0.0, -0.0, 90.0, -90.0, 1e4, -1e4, big, -big, float("inf"), float("nan"), 1e-38, -1e-38, 30.0, -30.0, 5.0, -5.0]
    gate = torch.tensor(gates, dtype=torch.float32).bfloat16()
    up = torch.full_like(gate, 0.5)
    a = torch.cat([gate, up]).view(1, -1).to(dev)
    dh = torch.ones(1, 16, dtype=torch.bfloat16, device=dev)
    h, da = torch.empty(1, 16, dtype=torch.bfloat16, device=dev), torch.empty(1, 32, dtype=torch.bfloat16, device=dev)
    mx.moe_swiglu_fwd(a, 1, 16, h)
    mx.moe_swiglu_bwd(dh, a, 1, 16, da)
    h, du = h[0].cpu(), da[0, 16:].cpu()
    assert h[8] == float("inf") and torch.isnan(h[9]) and torch.isnan(da[0, 9])
    finite = [i for i in range(16) if i not in (8, 9)]
    x = gate[finite].double()
    ref = x * torch.sigmoid(x)
    for got, want in ((h[finite], 0.5 * ref), (du[finite], ref)):
        ok = (got.double() - want).abs() <= _rel(x.clamp(-100, 100)) * want.abs() + 2.0 ** -120
        assert bool(ok.all()), (got, want)
    dg = da[0, :16].cpu()[[0, 1, 2, 3, 4, 5, 6]].double()
    assert torch.allclose(dg, torch.tensor([0.25, 0.25, 0.5, 0.0, 0.5, 0.0, 0.5], dtype=torch.float64), atol=1e-6)


def test_no_rows_and_large_offsets(dev):
    e = torch.empty(0, 16, dtype=torch.bfloat16, device=dev)
    mx.moe_swiglu_fwd(e, 0, 8, torch.empty(0, 8, dtype=torch.bfloat16, device=dev))
    mx.moe_swiglu_bwd(torch.empty(0, 8, dtype=torch.bfloat16, device=dev), e, 0, 8, e)
    R, I = 160000, 7168                      # 2 I R = 2.3e9 elements
    a = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device=dev)
    a[-1] = 1.0
    h = torch.ones(R, I, dtype=torch.bfloat16, device=dev)
    mx.moe_swiglu_fwd(a, R, I, h)
    assert not h[:-1].any()
    assert bool((h[-1] == torch.sigmoid(torch.tensor(1.0)).bfloat16().to(dev)).all())
