"""A stack of blocks around the routed experts: norm, router projection (with the
requests' adapters), routing, experts, and the norm, gate and residual after them.

    h = n(x) * next_weight                                   (before the first block)
    logits = W_router h + scale[a] B[a] (A[a] h)             (moe_adapter_linear)
    ids, w = route(logits)                                   (the runner's Routing)
    y = experts(h, ids, w)                                   (the runner)
    x, h = residual_scale x + gate n(y) post_weight, n(x) next_weight of the next block

Every step is a kernel of the library on one stream; this file sequences calls
and owns buffers.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import _lib as L


@dataclass
class BlockWeights:
    """One block's weights on the device.

    ``router`` [E, H] bf16; ``pre`` [H] the norm before the experts; ``post`` [H]
    the norm after them (None: none); ``gate`` [H] (None: none); the norms' and the
    gate's weights of one type.  ``lora_a`` [n, R, H], ``lora_b`` [n, E, R] bf16 and
    ``lora_scale`` [n] fp32: the router's adapters (None: none)."""
    router: torch.Tensor
    pre: torch.Tensor
    post: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    lora_a: Optional[torch.Tensor] = None
    lora_b: Optional[torch.Tensor] = None
    lora_scale: Optional[torch.Tensor] = None


class RoutedBlocks:
    """Blocks over one layer runner (its ``routing`` says how logits become experts).

    ``run(x, adapter_ids)`` takes the residual stream x [T, H] (fp32 or bf16)
    through every block in place.  Buffers are kept for up to T_max tokens; a
    device error of the projections is raised by ``synchronize``."""

    def __init__(self, runner, blocks: Sequence[BlockWeights], residual_scale: float = 1.0, eps: float = 1e-6):
        self.runner, self.blocks = runner, list(blocks)
        self.residual_scale, self.eps = residual_scale, eps
        T, H, E, dev = runner.T_max, runner.views.H, runner.E, runner.dev
        for b in self.blocks:
            if b.router.shape != (E, H) or b.router.dtype is not torch.bfloat16:
                raise ValueError(f"router must be [{E}, {H}] of torch.bfloat16, got {tuple(b.router.shape)} of "
                                 f"{b.router.dtype}")
        self.h = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        need = max((L.moe_adapter_linear_workspace(t, H, E, b.lora_a.shape[0], b.lora_a.shape[1])
                    for b in self.blocks if b.lora_a is not None for t in {1, T}), default=0)
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, x, adapter_ids=None, stream=None):
        """x [T, H] through every block, in place; returns x.  adapter_ids: device int32 [T]
        (negative: none) for the blocks that have adapters."""
        T = x.shape[0]
        if T > self.runner.T_max:
            raise ValueError(f"{T} tokens, and buffers for {self.runner.T_max}")
        stream = stream or torch.cuda.current_stream(self.runner.dev)
        h, y, logits = self.h[:T], self.y[:T], self.logits[:T]
        bits = torch.int16   # the experts' calls take bf16 bits
        L.moe_block_norm(x, next_weight=self.blocks[0].pre, eps=self.eps, h=h, stream=stream)
        for i, b in enumerate(self.blocks):
            lora = b.lora_a is not None and adapter_ids is not None
            L.moe_adapter_linear(h, b.router, b.lora_a if lora else None, b.lora_b, adapter_ids, b.lora_scale,
                                 out=logits, workspace=self.ws, d_error=self.err, stream=stream)
            self.runner.run(i, logits, h.view(bits), y.view(bits), stream=stream)
            after = self.blocks[i + 1].pre if i + 1 < len(self.blocks) else None
            L.moe_block_norm(x, y, b.post, b.gate, self.residual_scale, after, self.eps, x_out=x,
                             h=None if after is None else h, stream=stream)
        return x

    def synchronize(self, stream=None):
        """Waits for `stream` and raises what the device reported: the runner's errors, or an
        adapter id that names no adapter."""
        self.runner.synchronize(stream)
        stream = stream or torch.cuda.current_stream(self.runner.dev)
        with torch.cuda.stream(stream):
            e = int(self.err.item())
            self.err.zero_()
        if e != L.MOE_OK:
            raise L.MoeError(e, "the router's projection reported a failure on the device")
