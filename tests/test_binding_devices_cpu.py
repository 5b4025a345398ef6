"""Tensors that are not on a GPU are refused by the compiled entry points, each argument by its name, before
anything is launched: a kernel would read a host address as its own.  (CPU only: nothing here reaches a device.)"""
import pytest
import torch

f = torch.zeros
b = torch.bfloat16
i32 = torch.int32


@pytest.fixture(scope="module")
def L():
    from moe_expert_offload_router_gb300 import build
    build.build()
    from moe_expert_offload_router_gb300 import _lib
    return _lib


def _calls(L):
    return {
        "logits": lambda: L.moe_route(f(8, 4), 2),
        "logits, all given": lambda: L.moe_route(f(8, 4), 2, bias=f(4), token_mask=f(8, dtype=torch.bool),
                                                 topk_ids=f(8, 2, dtype=i32), topk_w=f(8, 2), load=f(4, dtype=i32)),
        "logits, a stream": lambda: L.moe_route(f(8, 4), 2, stream=0),
        "logits, backward": lambda: L.moe_route_backward(f(8, 4), f(8, 2, dtype=i32), f(8, 2)),
        "x": lambda: L.moe_block_norm(f(8, 4), f(8, 4), f(4), f(4), 1.0, f(4)),
        "x, backward": lambda: L.moe_block_norm_backward(f(8, 4), f(8, 4), f(8, 4), f(8, 4), f(4), f(4), 1.0, f(4)),
        "x, linear": lambda: L.moe_adapter_linear(f(8, 16, dtype=b), f(4, 16, dtype=b), f(2, 8, 16, dtype=b),
                                                  f(2, 4, 8, dtype=b), f(8, dtype=i32), f(2)),
        "x, linear with a stream": lambda: L.moe_adapter_linear(f(8, 16, dtype=b), f(4, 16, dtype=b), stream=0),
        "x, no tokens": lambda: L.moe_block_norm(f(0, 4), f(0, 4)),
    }


@pytest.mark.parametrize("name", ["logits", "logits, all given", "logits, a stream", "logits, backward", "x", "x, backward",
                                  "x, linear", "x, linear with a stream", "x, no tokens"])
def test_tensors_off_the_gpu_are_refused(L, name):
    with pytest.raises(L.MoeError, match=name.split(",")[0] + " is not on a GPU") as e:
        _calls(L)[name]()
    assert e.value.status == L.MOE_ERR_INVALID
