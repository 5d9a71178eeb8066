"""Trains one small MoE block (norms, router, experts, gate, residual) towards another one with AdamW,
its moments in 8 bits, and prints the loss.

    python examples/train_block.py [--steps 20] [--bits 8]
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_grouped_gemm_gb300 as moe  # noqa: E402
import synth  # noqa: E402
from combine_grouped_gemm_gb300.train import AdamW, MoETrainBlock  # noqa: E402


def make(cfg, seed):
    inp = synth.make_router_inputs(cfg.with_seed(seed), "cuda")
    W = {k: v for k, v in synth.make_expert_weights(cfg.with_seed(seed), "cuda").items()
         if v is not None and not k.endswith("_s")}
    ones = torch.ones(cfg.d, device="cuda")
    return MoETrainBlock(cfg, inp["w_gate"], inp["bias"], W, ones.clone(), ones.clone(), ones * 0.5)


def main(steps=20, lr=2e-3, bits=8):
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=256, d_ff_shared=128, R=1)
    x = synth.make_router_inputs(cfg, "cuda")["x"]
    target = make(cfg, cfg.seed).forward(x).float()
    block = make(cfg, cfg.seed + 1)
    opt = AdamW(block.parameters(), lr=lr, weight_decay=0.0, max_norm=1.0, state_bits=bits)
    losses = []
    for step in range(steps):
        diff = block.forward(x).float() - target
        losses.append(float(diff.square().mean() / target.square().mean()))
        # dh of the loss sum((h - target)^2) / (2 T)
        block.backward((diff / cfg.T).to(torch.bfloat16))
        opt.step()
        print(f"step {step}: relative squared error {losses[-1]:.4f}, gradient norm "
              f"{float(opt.norm):.4f}")
    if moe.read_status(opt.state) or moe.read_status(block.layer.bufs["ws"]):
        raise RuntimeError("device status word set")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    main(a.steps, bits=a.bits)
