"""Refusals of the calls around sorted rows and 4-bit products, before any device work (CPU only)."""
import pytest
import torch

from tests.test_block_args_cpu import L, ONE, _refused   # noqa: F401  (L: the fixture)


def test_sort_rows_refusals(L):   # noqa: F811
    good = dict(T=4, k=2, E=8, H=64, dtype=1, x=ONE, ld_x=64, ids=ONE, rows=ONE, ld_rows=64, offsets=ONE, pos=ONE,
                err=None, stream=None)
    _refused(L, "moe_sort_rows", good, T=[-1, 1 << 30], k=[0, 65], E=[0, 2049], H=0, dtype=[3, -1], x=None, ld_x=63,
             ids=None, rows=None, ld_rows=63, offsets=None, pos=None)
    back = dict(T=4, k=2, n_rows=8, H=64, dtype=1, d_rows=ONE, ld=64, pos=ONE, d_x=2 * ONE, ld_dx=64, stream=None)
    _refused(L, "moe_sort_rows_backward", back, T=-1, k=[0, 65], n_rows=-1, H=0, dtype=[3, -1], d_rows=None, ld=63,
             pos=None, d_x=None, ld_dx=63)
    assert L.raw().moe_sort_rows_backward(*dict(back, T=0, d_rows=None, pos=None, d_x=None).values()) == L.MOE_OK


def test_combine_rows_refusals(L):   # noqa: F811
    good = dict(T=4, k=2, n_rows=8, H=64, rd=0, yd=1, rows=ONE, ld_rows=64, pos=ONE, w=ONE, base=ONE, ld_base=64,
                y=2 * ONE, ld_y=64, stream=None)
    _refused(L, "moe_combine_rows", good, T=[-1, 1 << 30], k=[0, 65], n_rows=-1, H=0, rd=[2, 3], yd=[3, -1], rows=None,
             ld_rows=63, pos=None, ld_base=63, y=None, ld_y=63)
    _refused(L, "moe_combine_rows", dict(good, rd=1), yd=[0, 2])
    _refused(L, "moe_combine_rows", dict(good, base=2 * ONE), ld_base=72)          # in place, another distance
    assert L.raw().moe_combine_rows(*dict(good, T=0, rows=None, pos=None, y=None).values()) == L.MOE_OK
    back = dict(T=4, k=2, n_rows=8, H=64, rd=0, yd=1, dy=ONE, ld_dy=64, rows=2 * ONE, ld_rows=64, pos=ONE, w=ONE,
                d_rows=3 * ONE, ld_dr=64, dw=ONE, stream=None)
    _refused(L, "moe_combine_rows_backward", back, T=-1, k=[0, 65], n_rows=-1, H=0, rd=[2, 3], yd=[3, -1], dy=None,
             ld_dy=63, rows=None, ld_rows=63, pos=None, d_rows=None, ld_dr=63)
    _refused(L, "moe_combine_rows_backward", dict(back, d_rows=2 * ONE), ld_dr=72)
    assert L.raw().moe_combine_rows_backward(*dict(back, T=0, dy=None).values()) == L.MOE_OK


def test_w4_linear_refusals(L):   # noqa: F811
    good = dict(P=4, N=48, K=256, E=3, g=128, dtype=1, out_dtype=1, x=ONE, ld_x=256, codes=ONE, scales=ONE, zeros=None,
                offsets=ONE, swiglu=0, out=ONE, ld_out=48, err=None, stream=None)
    _refused(L, "moe_w4_linear", good, P=[-1, (1 << 30) + 1], N=[0, 1 << 25], K=[0, 64, 192, 1 << 25], E=[0, 2049],
             g=[0, 16, 96, 256], dtype=[0, 3], out_dtype=[2, 3], x=[None, 8], ld_x=[255, 260], codes=[None, 8],
             scales=None, offsets=None, out=None, ld_out=47)
    _refused(L, "moe_w4_linear", dict(good, swiglu=1, ld_out=24), N=47, ld_out=23)
    _refused(L, "moe_w4_linear", dict(good, E=2048), N=1 << 20)
    assert L.raw().moe_w4_linear(*dict(good, P=0, x=None, codes=None, out=None).values()) == L.MOE_OK


def test_binding_refusals_of_rows(L):   # noqa: F811
    f, i, u, b = torch.zeros, torch.int32, torch.uint8, torch.bfloat16
    with pytest.raises(ValueError, match="topk_ids"):
        L.moe_sort_rows(f(8, 4), f(7, 2, dtype=i), 4)
    with pytest.raises(ValueError, match="topk_ids"):
        L.moe_sort_rows(f(8, 4), f(8, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="rows"):
        L.moe_sort_rows(f(8, 4), f(8, 2, dtype=i), 4, rows=f(15, 4))
    with pytest.raises(ValueError, match="rows"):
        L.moe_sort_rows(f(8, 4), f(8, 2, dtype=i), 4, rows=f(16, 4, dtype=b))
    with pytest.raises(ValueError, match="offsets"):
        L.moe_sort_rows(f(8, 4), f(8, 2, dtype=i), 4, offsets=f(4, dtype=i))
    with pytest.raises(ValueError, match="adjacent"):
        L.moe_sort_rows(f(4, 8).t(), f(8, 2, dtype=i), 4)
    with pytest.raises(L.MoeError, match="GPU"):
        L.moe_sort_rows(f(8, 4), f(8, 2, dtype=i), 4)
    with pytest.raises(ValueError, match="d_x"):
        L.moe_sort_rows_backward(f(8, 4), f(4, 2, dtype=i), d_x=f(5, 4))
    with pytest.raises(ValueError, match="w must"):
        L.moe_combine_rows(f(8, 4), f(4, 2, dtype=i), f(4, 3))
    with pytest.raises(ValueError, match="base"):
        L.moe_combine_rows(f(8, 4), f(4, 2, dtype=i), None, f(4, 4), f(4, 4, dtype=b))
    with pytest.raises(ValueError, match="rows overlap"):
        L.moe_combine_rows(f(1, 4).expand(8, 4), f(4, 2, dtype=i))
    with pytest.raises(TypeError, match="out_dtype"):
        L.moe_combine_rows(f(8, 4), f(4, 2, dtype=i), out_dtype="bf16")
    with pytest.raises(ValueError, match="d_y"):
        L.moe_combine_rows_backward(f(3, 4), f(8, 4), f(4, 2, dtype=i))
    with pytest.raises(ValueError, match="d_w"):
        L.moe_combine_rows_backward(f(4, 4), f(8, 4), f(4, 2, dtype=i), d_w=f(4, 3))
    with pytest.raises(ValueError, match="codes"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(4, 30, dtype=u), f(4, 2, dtype=b))
    with pytest.raises(ValueError, match="codes"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(1, 1, 4, 32, dtype=u), f(4, 2, dtype=b))
    with pytest.raises(ValueError, match="scales"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(4, 32, dtype=u), f(4, 2))
    with pytest.raises(ValueError, match="zeros"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(4, 32, dtype=u), f(4, 2, dtype=b), f(4, 2, dtype=i))
    with pytest.raises(ValueError, match="offsets"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(3, 4, 32, dtype=u), f(3, 4, 2, dtype=b), None, f(3, dtype=i))
    with pytest.raises(L.MoeError, match="GPU"):
        L.moe_w4_linear(f(2, 64, dtype=b), f(4, 32, dtype=u), f(4, 2, dtype=b))
