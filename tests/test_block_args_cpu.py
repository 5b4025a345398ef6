"""Refusals of the routing, block norm and adapter projection calls: every bad
argument is refused before any device work (CPU only)."""
import pytest
import torch

ONE = 16   # stands for a device pointer in calls that are refused before it is used


@pytest.fixture(scope="module")
def L():
    from moe_expert_offload_router_gb300 import build
    build.build()
    from moe_expert_offload_router_gb300 import _lib
    return _lib


def _refused(L, name, good, **bad):
    """The call `name` with the arguments `good` (a dict in order), some replaced, is refused with a message."""
    for key, values in bad.items():
        for v in values if isinstance(values, list) else [values]:
            assert key in good, key
            rc = getattr(L.raw(), name)(*dict(good, **{key: v}).values())
            assert rc == L.MOE_ERR_INVALID, (name, key, v)
            assert L.raw().moe_last_error(), (name, key, v)


ROUTE = dict(logits=ONE, dtype=0, ld=64, T=4, E=64, k=6, score=0, bias=None, n_group=8, topk_group=4, group_score=1,
             renorm=1, scale=1.0, mask=None, ids=ONE, w=ONE, load=None, stream=None)


def test_route_refusals(L):
    _refused(L, "moe_route", ROUTE, logits=None, dtype=[3, -1], ld=63, T=-1, E=[0, 2049], k=[0, 33, 65], score=[2, -1],
             n_group=[0, 7, 64], topk_group=[0, 9], group_score=[2, -1], ids=None, w=None)
    assert L.raw().moe_route(*dict(ROUTE, T=0, logits=None).values()) == L.MOE_OK
    back = dict(logits=ONE, dtype=0, ld=64, T=4, E=64, k=6, score=0, renorm=1, scale=1.0, mask=None, ids=ONE, dw=ONE,
                d=2 * ONE, ld_d=64, stream=None)
    _refused(L, "moe_route_backward", back, logits=None, dtype=3, ld=63, T=-1, E=0, k=33, score=2, ids=None, dw=None,
             d=[None, ONE], ld_d=63)


NORM = dict(T=4, H=64, xd=1, yd=1, wd=0, x=ONE, ld_x=64, y=ONE, ld_y=64, post=ONE, gate=ONE, mode=1, alpha=1.0,
            nxt=ONE, eps=1e-6, x_out=ONE, ld_xo=64, h=ONE, ld_h=64, stream=None)


def test_block_norm_refusals(L):
    _refused(L, "moe_block_norm", NORM, T=-1, H=[0, 16385], xd=[2, 3], yd=[0, 5], wd=4, x=None, ld_x=63, y=None,
             ld_y=63, gate=None, mode=[0, 3], nxt=None, ld_xo=63, h=None, ld_h=63)
    _refused(L, "moe_block_norm", dict(NORM, x_out=None, h=None, nxt=None), T=4)      # nothing to write
    _refused(L, "moe_block_norm", dict(NORM, y=None, gate=None, mode=0), T=4)         # a post weight without y
    _refused(L, "moe_block_norm", NORM, ld_xo=72)                                     # in place, another distance
    assert L.raw().moe_block_norm(*dict(NORM, T=0, x=None).values()) == L.MOE_OK


def test_block_norm_backward_refusals(L):
    good = dict(T=4, H=64, xd=1, yd=1, wd=0, x=ONE, ld_x=64, y=ONE, ld_y=64, du=2 * ONE, ld_du=64, dh=3 * ONE,
                ld_dh=64, post=ONE, gate=ONE, mode=1, alpha=1.0, nxt=ONE, eps=1e-6, dx=4 * ONE, ld_dx=64, dy=5 * ONE,
                ld_dy=64, dpost=ONE, dgate=ONE, dnext=ONE, ws=ONE, bytes=1 << 40, stream=None)
    _refused(L, "moe_block_norm_backward", good, T=-1, H=[0, 16385], xd=2, wd=4, x=None, ld_x=63, y=None, ld_y=63,
             ld_du=63, dh=None, ld_dh=63, post=None, gate=None, mode=0, nxt=None, dx=None, ld_dx=63, dy=None,
             ld_dy=63, ws=[None, 8], bytes=0)
    _refused(L, "moe_block_norm_backward", dict(good, du=None, dh=None, nxt=None, dnext=None), T=4)
    _refused(L, "moe_block_norm_backward", dict(good, dx=2 * ONE), ld_dx=72)
    _refused(L, "moe_block_norm_backward", dict(good, dy=3 * ONE), ld_dy=72)
    assert L.moe_block_norm_backward_workspace(0, 64) == 0


def test_adapter_linear_refusals(L):
    good = dict(T=4, H=64, N=48, dtype=1, out_dtype=1, x=ONE, ld_x=64, W=ONE, ld_w=64, n=3, R=16, A=ONE, B=ONE,
                ids=ONE, scale=None, out=ONE, ld_out=48, ws=ONE, bytes=1 << 40, err=None, stream=None)
    _refused(L, "moe_adapter_linear", good, T=-1, H=[0, 60], N=0, dtype=[0, 3], out_dtype=[2, 3], x=[None, 8],
             ld_x=[56, 68], W=[None, 24], ld_w=[56, 68], n=-1, R=[0, 4, 12, 136], A=[None, 8], B=[None, 8], ids=None,
             out=None, ld_out=47, ws=[None, 8], bytes=0)
    assert L.raw().moe_adapter_linear(*dict(good, T=0, x=None).values()) == L.MOE_OK
    assert L.moe_adapter_linear_workspace(0, 64, 48, 3, 16) == 0


def test_binding_refusals(L):
    f = torch.zeros
    with pytest.raises(ValueError, match="adjacent"):
        L.moe_route(f(8, 4).t(), 2)
    with pytest.raises(ValueError, match="rows overlap"):
        L.moe_route(f(1, 4).expand(8, 4), 2)
    with pytest.raises(ValueError, match="bias"):
        L.moe_route(f(8, 4), 2, bias=f(3))
    with pytest.raises(ValueError, match="bias"):
        L.moe_route(f(8, 4), 2, bias=f(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="topk_ids"):
        L.moe_route(f(8, 4), 2, topk_ids=f(8, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="unsupported"):
        L.moe_route(f(8, 4, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="d_logits"):
        L.moe_route_backward(f(8, 4), f(8, 2, dtype=torch.int32), f(8, 2), d_logits=f(8, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="one type"):
        L.moe_block_norm(f(8, 4), f(8, 4), f(4), f(4, dtype=torch.float16))
    with pytest.raises(ValueError, match="gate"):
        L.moe_block_norm(f(8, 4), f(8, 4), f(4), f(8))
    with pytest.raises(ValueError, match="y must be"):
        L.moe_block_norm(f(8, 4), f(7, 4))
    with pytest.raises(ValueError, match="x_out"):
        L.moe_block_norm(f(8, 4), f(8, 4), x_out=f(8, 4, dtype=torch.bfloat16))
    b = torch.bfloat16
    with pytest.raises(ValueError, match="weight"):
        L.moe_adapter_linear(f(8, 16, dtype=b), f(4, 16))
    with pytest.raises(ValueError, match="lora_b"):
        L.moe_adapter_linear(f(8, 16, dtype=b), f(4, 16, dtype=b), f(2, 8, 16, dtype=b), f(2, 8, 4, dtype=b),
                             f(8, dtype=torch.int32))
    with pytest.raises(L.MoeError):
        L.moe_adapter_linear(f(8, 12, dtype=b), f(4, 12, dtype=b), stream=0)
