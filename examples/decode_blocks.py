"""Decodes a few steps through a small stack of routed blocks on one GPU: the experts
served from a slot cache, the router with a balance bias, expert groups and the adapters
of two tenants.  Random weights.

    python examples/decode_blocks.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_offload_router_gb300 as M  # noqa: E402
from synth import configs, gen  # noqa: E402


def main(layers=3, steps=4, T=6):
    wl = configs.scaled(configs.TINY, E=32, k=4, S=48, T=T)
    torch.manual_seed(0)
    dev = torch.device("cuda")
    size = M.moe_fp4_expert_bytes(wl.H, wl.I)
    bank = torch.empty(layers * wl.E * size, dtype=torch.uint8, pin_memory=True)
    for layer in range(layers):
        for e in range(wl.E):
            at = (layer * wl.E + e) * size
            bank[at:at + size] = torch.from_numpy(gen.fp4_expert(wl, layer, e))
    slots = torch.empty(wl.S * size, dtype=torch.uint8, device=dev)
    cache = M.moe_cache(wl.S, layers, wl.E, size, slots, bank)
    views = M.make_views(wl.H, wl.I, slots, wl.S)
    load = torch.zeros(layers, wl.E, dtype=torch.int32, device=dev)
    bias = [torch.zeros(wl.E, device=dev) for _ in range(layers)]
    routing = M.Routing(score=M.MOE_SCORE_SIGMOID, bias=bias, n_group=4, topk_group=2, scale=1.5, load=load)
    runner = M.DecodeLayerRunner(cache, views, wl.E, wl.k, T, copy="device", routing=routing)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, device=dev) * by)
    ones = torch.ones(wl.H, device=dev)
    blocks = [M.BlockWeights(router=normal(wl.E, wl.H, by=wl.H ** -0.5).bfloat16(), pre=ones, post=ones, gate=0.3 * ones,
                             lora_a=normal(2, 8, wl.H, by=wl.H ** -0.5).bfloat16(),
                             lora_b=normal(2, wl.E, 8, by=0.3).bfloat16()) for _ in range(layers)]
    stack = M.RoutedBlocks(runner, blocks)
    tenants = torch.tensor([0, 0, 1, 1, -1, -1][:T], dtype=torch.int32, device=dev)   # the last two use no adapter
    x = normal(T, wl.H)
    for step in range(steps):
        stack.run(x, tenants)
        stack.synchronize()
        for b, n in zip(bias, load):    # towards balance, as in training
            b += 0.01 * torch.sign(n.float().mean() - n)
        print(f"step {step}: |x| = {x.square().mean().sqrt().item():.3f}, experts used per layer "
              f"{(load > 0).sum(1).tolist()}, misses {runner.stats['misses']}")
        load.zero_()
    cache.close()
    return x


if __name__ == "__main__":
    main()
