"""Trains the experts of one small MoE layer towards those of another (same router) and prints
the loss: forward with 8-bit activation checkpoints, backward, and plain gradient descent.

    python examples/train_experts.py [--steps 20]
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_grouped_gemm_gb300 as moe  # noqa: E402
import synth  # noqa: E402
from combine_grouped_gemm_gb300.train import MoETrainLayer  # noqa: E402


def main(steps=20, lr=4.0):
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=256, d_ff_shared=128, R=1)
    inp = synth.make_router_inputs(cfg, "cuda")
    target_w = synth.make_expert_weights(cfg, "cuda")
    target = MoETrainLayer(cfg, inp["w_gate"], inp["bias"], target_w).forward(inp["x"]).float()
    W = synth.make_expert_weights(cfg.with_seed(cfg.seed + 1), "cuda")
    names = ("w13", "w2", "ws13", "ws2")
    master = {n: W[n].float() for n in names}
    layer = MoETrainLayer(cfg, inp["w_gate"], inp["bias"], W)
    losses = []
    for step in range(steps):
        diff = layer.forward(inp["x"]).float() - target
        losses.append(float(diff.square().mean() / target.square().mean()))
        # dy of the loss sum((y - target)^2) / (2 T)
        grads = layer.backward((diff / cfg.T).to(torch.bfloat16))
        for n in names:
            master[n] -= lr * grads["d" + n].view_as(master[n])
            W[n].copy_(master[n])
        print(f"step {step}: relative squared error {losses[-1]:.4f}")
    if moe.read_status(layer.bufs["ws"]) or moe.read_status(layer.routed.ws):
        raise RuntimeError("device status word set")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
