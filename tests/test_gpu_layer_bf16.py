"""The bf16 MoE FFN layer step against the same layer in 64 bits, its CUDA graph, and training both
layers with AdamW.

Tolerances, derived before any run: every stage rounds its output to bf16 once (at most 2^-8 of a
value, 2^-8 / sqrt(3) rms over many), and what it adds to a stage's output is bounded in the relative
2-norm.  A value that passes n roundings is within n 2^-8 of its norm times the amplification of the
maps between, which is near 1 for products with random weights; out passes 4 stages, dx and dw1 8, so
8 * 2^-8 = 3 % bounds all of them."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from mxfp8_block_scaled_rowwise_gb300 import synth
from mxfp8_block_scaled_rowwise_gb300.layer import MoEFFNStepBf16
from gpu_util import check_dev_err, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _fill(st, seed):
    g = synth.generator(seed)
    st.x.copy_(synth.randn_bf16(st.x.shape, g))
    logits = torch.randn(st.T, st.E, generator=g)
    ids = synth.topk_ids(logits, st.k)
    st.ids.copy_(ids)
    st.gate.copy_(torch.softmax(logits.gather(1, ids.long()), dim=1))
    st.w1.copy_(synth.randn_bf16(st.w1.shape, g, std=st.H ** -0.5))
    st.w2.copy_(synth.randn_bf16(st.w2.shape, g, std=st.I ** -0.5))
    st.dout.copy_(synth.randn_bf16(st.dout.shape, g, std=1e-2))


def _reference(st):
    x, gate, w1, w2 = (t.double().clone().requires_grad_() for t in (st.x, st.gate, st.w1, st.w2))
    out = torch.zeros(st.T, st.H, dtype=torch.float64, device=st.dev)
    ids = st.ids.long()
    for e in range(st.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        a = x[t] @ w1[e].t()
        h = torch.nn.functional.silu(a[:, :st.I]) * a[:, st.I:]
        out = out.index_add(0, t, gate[t, j, None] * (h @ w2[e].t()))
    out.backward(st.dout.double())
    return dict(out=out.detach(), dx=x.grad, dgate=gate.grad, dw1=w1.grad, dw2=w2.grad)


@pytest.mark.parametrize("T,E,k,H,I", [(384, 8, 3, 256, 128), (1, 16, 4, 264, 72), (77, 5, 2, 520, 200), (700, 3, 1, 128, 392)])
def test_step_matches_64_bit(dev, T, E, k, H, I):
    st = MoEFFNStepBf16(T, E, k, H, I, device=dev)
    _fill(st, 5 + T)
    st.step()
    check_dev_err(st.dev_err)
    for name, want in _reference(st).items():
        got = getattr(st, name).double()
        assert float((got - want).norm()) <= 8 * 2.0 ** -8 * float(want.norm()), name


def test_graph_replay_matches_eager_step(dev):
    st = MoEFFNStepBf16(200, 6, 2, 264, 136, device=dev)
    _fill(st, 71)
    st.step()
    check_dev_err(st.dev_err)
    names = ("out", "dx", "dgate", "dw1", "dw2")
    graph = st.capture()
    _fill(st, 72)
    graph.replay()
    check_dev_err(st.dev_err)
    replayed = {n: getattr(st, n).clone() for n in names}
    st.step()
    check_dev_err(st.dev_err)
    for n in names:
        assert torch.equal(replayed[n], getattr(st, n)), n


def _example():
    spec = importlib.util.spec_from_file_location("train_moe_ffn", os.path.join(ROOT, "examples", "train_moe_ffn.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def _training_in_64_bit(steps, T=512, E=8, k=2, H=256, I=256, lr=2e-3, seed=1):
    """The example's losses with layer, teacher and AdamW in 64 bits, on the example's numbers."""
    g = synth.generator(seed)

    class Layer:
        pass
    both = []
    for _ in range(2):
        st = Layer()
        st.T, st.E, st.k, st.H, st.I, st.dev = T, E, k, H, I, "cuda"
        st.w1 = synth.randn_bf16((E, 2 * I, H), g, std=H ** -0.5).double().cuda()
        st.w2 = synth.randn_bf16((E, H, I), g, std=I ** -0.5).double().cuda()
        both.append(st)
    teacher, layer = both
    m = {n: 0.0 for n in ("w1", "w2")}
    v = {n: 0.0 for n in ("w1", "w2")}
    losses = []
    for t in range(1, steps + 1):
        x = synth.randn_bf16((T, H), g).cuda()
        logits = torch.randn(T, E, generator=g)
        ids = synth.topk_ids(logits, k)
        for st in both:
            st.x, st.ids, st.dout = x, ids.cuda(), torch.zeros(T, H, device="cuda")
            st.gate = torch.softmax(logits.gather(1, ids.long()), dim=1).cuda()
        diff = _reference(layer)["out"] - _reference(teacher)["out"]
        losses.append(float(diff.square().mean()))
        layer.dout = diff * (2.0 / diff.numel())
        grads = _reference(layer)
        norm = (grads["dw1"].square().sum() + grads["dw2"].square().sum()).sqrt()
        for n in ("w1", "w2"):
            d = grads["d" + n] * torch.clamp(1.0 / norm, max=1.0)
            m[n] = 0.9 * m[n] + 0.1 * d
            v[n] = 0.999 * v[n] + 0.001 * d.square()
            w = getattr(layer, n)
            w -= lr * (m[n] / (1 - 0.9 ** t)) / ((v[n] / (1 - 0.999 ** t)).sqrt() + 1e-8)
    return losses


@pytest.mark.parametrize("precision,states", [("bf16", 32), ("bf16", 8), ("mxfp8", 32)])
def test_training_example_follows_64_bit(dev, precision, states):
    """The example's losses over 20 steps against the same training in 64 bits.  Output and target each
    carry 4 bf16 roundings, 1.6 % of their norm, and while the loss is above half of its start their
    difference is at least their norm: 2 * (1.6 + 1.6) % of the loss at most, 10 % with what the
    parameters' own rounding adds.  MXFP8 rounds operands to 4 significant bits, up to 2^-4 of a value
    (a third of that rms over a product) in each of the layer's 4 quantized operands: 20 %."""
    losses = _example().train(precision, states, steps=20)
    want = _training_in_64_bit(20)
    tol = 0.10 if precision == "bf16" else 0.20
    assert want[-1] < want[0]
    assert all(abs(a - b) <= tol * b for a, b in zip(losses, want)), list(zip(losses, want))


def test_training_example_captured_or_eager(dev):
    """A captured step does what an eager one does, byte for byte."""
    ex = _example()
    assert ex.train("bf16", 8, steps=8, graph=False) == ex.train("bf16", 8, steps=8, graph=True)
