"""Experts in 4 bits, from gate logits to the layer's output.

Takes binary16 expert weights W1[E][2I][K] (gate and up) and W2[E][K][I], lays them out once as
MXFP4 blocks, and runs a batch of tokens through the router and the expert layer:

    python examples/mxfp4_experts.py [--tokens M] [--hidden K] [--intermediate I] [--experts E] [--topk k]

It prints the weights' sizes, the time of a router and layer call, and how far the output is from
the same layer with the weights and activations in 32 bits (what four bits cost).  With random
weights and activations that is about 0.3 of the output's norm.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import moe_expert_layer_gb300 as moe


class Mxfp4Experts:
    """MXFP4 weights of one layer, and the buffers of up to `max_tokens` tokens."""

    def __init__(self, w1, w2, topk, max_tokens):
        self.E, two_i, self.K = w1.shape
        self.I, self.topk, self.max_tokens = two_i // 2, topk, max_tokens
        dev = w1.device
        self.w1 = torch.empty(moe.moe_mxfp4_weights_bytes(self.E, two_i, self.K), dtype=torch.uint8, device=dev)
        self.w2 = torch.empty(moe.moe_mxfp4_weights_bytes(self.E, self.K, self.I), dtype=torch.uint8, device=dev)
        moe.moe_mxfp4_quant_weights(w1, self.w1, gate_up=True)
        moe.moe_mxfp4_quant_weights(w2, self.w2)
        size = moe.moe_mxfp4_layer_workspace_size(self.dims(max_tokens))  # enough for fewer tokens too
        self.workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        self.expert_idx = torch.empty(max_tokens, topk, dtype=torch.int32, device=dev)
        self.probs = torch.empty(max_tokens, topk, dtype=torch.float32, device=dev)

    def dims(self, m):
        return moe.dims(m, self.K, self.I, self.E, self.topk)

    def __call__(self, x, logits, out):
        """out [M][K] (binary16) = the experts' mixture for tokens x [M][K] (binary16) by logits [M][E]."""
        m = x.shape[0]
        idx, probs = self.expert_idx[:m], self.probs[:m]
        moe.moe_route_topk(logits, idx, probs)
        moe.moe_mxfp4_layer_fwd(self.dims(m), x, idx, probs, self.w1, self.w2, out, self.workspace)
        return out


def plain(x, w1, w2, idx, probs):
    """The layer in 32 bits, expert by expert."""
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    for e in range(w1.shape[0]):
        token, slot = (idx == e).nonzero(as_tuple=True)
        if len(token):
            g, u = (x[token].float() @ w1[e].float().T).chunk(2, dim=1)
            h = torch.nn.functional.silu(g) * u
            out.index_add_(0, token, probs[token, slot, None] * (h @ w2[e].float().T))
    return out


def run(tokens=128, hidden=4096, intermediate=1408, experts=64, topk=6, steps=20, seed=1):
    """-> (microseconds of a router and layer call, distance from 32 bits over the output's norm)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float16)

    x, logits = normal(tokens, hidden), normal(tokens, experts)
    w1 = normal(experts, 2 * intermediate, hidden) * hidden ** -0.5
    w2 = normal(experts, hidden, intermediate) * intermediate ** -0.5
    layer = Mxfp4Experts(w1, w2, topk, tokens)
    out = torch.empty_like(x)
    layer(x, logits, out)
    ref = plain(x, w1, w2, layer.expert_idx, layer.probs)
    status = moe.moe_workspace_status(layer.workspace)
    if status != 0:
        raise RuntimeError("device status %d" % status)
    distance = ((out.float() - ref).norm() / ref.norm()).item()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        layer(x, logits, out)
    start.record()
    for _ in range(steps):
        layer(x, logits, out)
    end.record()
    torch.cuda.synchronize()
    print("weights %.1f MB as MXFP4, %.1f MB as binary16" %
          ((layer.w1.numel() + layer.w2.numel()) / 1e6, 2 * (w1.numel() + w2.numel()) / 1e6))
    us = start.elapsed_time(end) / steps * 1e3
    print("%d tokens: router and layer %.1f us, distance from 32 bits %.3f" % (tokens, us, distance))
    return us, distance


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 128), ("hidden", 4096), ("intermediate", 1408), ("experts", 64), ("topk", 6)):
        p.add_argument("--" + name, type=int, default=value)
    run(**vars(p.parse_args()))
