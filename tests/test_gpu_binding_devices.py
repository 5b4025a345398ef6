"""Among tensors on the GPU, one that was left on the host is refused by its name before any launch."""
import pytest
import torch

from tests.helpers import load_lib

pytestmark = pytest.mark.gpu


def _calls(M):
    """{call: (function, positional names, arguments)} of good calls, every tensor argument given."""
    def z(*s, dtype=torch.float32):
        return torch.ones(*s, dtype=dtype, device="cuda")
    i, b = torch.int32, torch.bfloat16
    T, E, H, N = 8, 16, 64, 24
    return {
        "route": (M.moe_route, dict(logits=z(T, E), k=2, bias=z(E), token_mask=z(T, dtype=torch.uint8),
                                    topk_ids=z(T, 2, dtype=i), topk_w=z(T, 2), load=z(E, dtype=i))),
        "route_backward": (M.moe_route_backward, dict(logits=z(T, E), topk_ids=z(T, 2, dtype=i) * 0 - 1, d_w=z(T, 2),
                                                      token_mask=z(T, dtype=torch.uint8), d_logits=z(T, E))),
        "block_norm": (M.moe_block_norm, dict(x=z(T, H), y=z(T, H), post_weight=z(H), gate=z(T, 1), next_weight=z(H),
                                              x_out=z(T, H), h=z(T, H))),
        "block_norm_backward": (M.moe_block_norm_backward,
                                dict(x=z(T, H), y=z(T, H), d_x_out=z(T, H), d_h=z(T, H), post_weight=z(H), gate=z(H),
                                     next_weight=z(H), d_x=z(T, H), d_y=z(T, H), d_post_weight=z(H), d_gate=z(H),
                                     d_next_weight=z(H), workspace=z(1 << 20, dtype=torch.uint8))),
        "adapter_linear": (M.moe_adapter_linear,
                           dict(x=z(T, H, dtype=b), weight=z(N, H, dtype=b), lora_a=z(2, 8, H, dtype=b),
                                lora_b=z(2, N, 8, dtype=b), adapter_ids=z(T, dtype=i) * 0, lora_scale=z(2),
                                out=z(T, N), workspace=z(1 << 16, dtype=torch.uint8), d_error=z(1, dtype=i))),
    }


@pytest.mark.parametrize("name", ["route", "route_backward", "block_norm", "block_norm_backward", "adapter_linear"])
def test_one_tensor_left_on_the_host(name):
    M = load_lib()
    f, good = _calls(M)[name]
    f(**good)
    for key, v in good.items():
        if not isinstance(v, torch.Tensor):
            continue
        for host in (v.cpu(), v.cpu().pin_memory()):
            with pytest.raises(M.MoeError, match=key + r".* is (not on a GPU|on another GPU)") as e:
                f(**dict(good, **{key: host}))
            assert e.value.status == M.MOE_ERR_INVALID
    f(**good)
    torch.cuda.synchronize()


def test_a_result_that_does_not_fit_raises_torchs_error():
    # 4 TB of fp32 results
    M = load_lib()
    x, W = (torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda") for n in (1 << 20, 1 << 20))
    with pytest.raises(torch.OutOfMemoryError):
        M.moe_adapter_linear(x, W, out_dtype=torch.float32)
