"""Trains one MoE FFN layer to reproduce another one's outputs on random tokens.

    python examples/train_moe_ffn.py --precision bf16 --states 8 --steps 200
    python examples/train_moe_ffn.py --precision mxfp8 --states 32

Every step is the layer's forward and backward pass (MoEFFNStepBf16 or MoEFFNStep) and an AdamW step
over its expert weights, captured once as a CUDA graph and replayed.  Prints the loss every tenth of
the way.  Needs a GB300 and the built library.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mxfp8_block_scaled_rowwise_gb300 import synth  # noqa: E402
from mxfp8_block_scaled_rowwise_gb300.layer import AdamW, MoEFFNStep, MoEFFNStepBf16  # noqa: E402


def train(precision="bf16", states=8, steps=200, tokens=512, experts=8, topk=2, hidden=256, inter=256, lr=2e-3, seed=1,
          graph=True):
    """Losses (mean squared error, one per step) of the run."""
    dev = torch.device("cuda")
    cls = {"bf16": MoEFFNStepBf16, "mxfp8": MoEFFNStep}[precision]
    g = synth.generator(seed)
    teacher, layer = (c(tokens, experts, topk, hidden, inter, device=dev) for c in (MoEFFNStepBf16, cls))
    for t in (teacher, layer):
        t.w1.copy_(synth.randn_bf16(t.w1.shape, g, std=hidden ** -0.5))
        t.w2.copy_(synth.randn_bf16(t.w2.shape, g, std=inter ** -0.5))
    opt = AdamW([layer.w1, layer.w2], [layer.dw1, layer.dw2], state_bits=states, lr=lr, weight_decay=0.0, max_norm=1.0,
                stochastic=True, seed=seed)
    target = torch.empty_like(layer.out)

    def one():
        layer.forward()
        layer.dout.copy_((layer.out.float() - target.float()) * (2.0 / layer.out.numel()))
        layer.backward()
        opt.step()
    losses, replay = [], None
    for _ in range(steps):
        x = synth.randn_bf16((tokens, hidden), g)
        logits = torch.randn(tokens, experts, generator=g)
        ids = synth.topk_ids(logits, topk)
        for t in (teacher, layer):
            t.x.copy_(x)
            t.ids.copy_(ids)
            t.gate.copy_(torch.softmax(logits.gather(1, ids.long()), dim=1))
        teacher.forward()
        target.copy_(teacher.out)
        if replay is None:
            one()                     # the first step runs eagerly: it warms up what a capture cannot hold
            if graph:
                replay = torch.cuda.CUDAGraph()
                with torch.cuda.graph(replay):
                    one()
            else:
                replay = type("Eager", (), {"replay": staticmethod(one)})
        else:
            replay.replay()
        losses.append((layer.out.float() - target.float()).square().mean().item())
    torch.cuda.synchronize()
    assert int(layer.dev_err.item()) == 0 and int(teacher.dev_err.item()) == 0 and int(opt.steps.item()) == steps
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--precision", choices=("bf16", "mxfp8"), default="bf16")
    ap.add_argument("--states", type=int, choices=(8, 32), default=8)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    losses = train(a.precision, a.states, a.steps)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print("step %4d  loss %.4f" % (i, losses[i]))
    print("step %4d  loss %.4f" % (a.steps - 1, losses[-1]))


if __name__ == "__main__":
    main()
