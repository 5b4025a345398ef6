"""Products with 4-bit weights whose scales and zero points start and end anywhere (any even address, any address), between
values that must not be taken. Tolerances as in test_gpu_w4_linear."""
import numpy as np
import pytest
import torch

from tests.helpers import load_lib
from tests.test_gpu_w4_linear import check, normal, weights

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def inside(t, at, fill):
    """t's values `at` elements into a buffer, with `fill` on both sides."""
    room = torch.full((at + t.numel() + 9,), fill, dtype=t.dtype, device="cuda")
    v = room[at:at + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# N, K, group: one group to a row, three, five, eight; all of them a multiple of four or not
SIZES = [(130, 128, 128), (33, 96, 32), (258, 384, 128), (514, 320, 64), (256, 1024, 128), (1, 2176, 64)]


@pytest.mark.parametrize("P", [1, 12, 100, 300])
@pytest.mark.parametrize("N,K,group", SIZES)
@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_dense(P, N, K, group, at):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(P + N + K)
    x = normal(g, P, K, BF16)
    codes, scales, z = (t[0] for t in weights(g, 1, N, K, group, BF16))
    s, zz = inside(scales, at, float("nan")), inside(z, 3 * at + 1, 255)
    for swiglu in ([False, True] if N % 2 == 0 else [False]):
        got = M.moe_w4_linear(x, codes, s, zz, swiglu=swiglu, out_dtype=F32)
        check(got, x, codes, scales, z, None, swiglu)
    got = M.moe_w4_linear(x, codes, s, out_dtype=F32)
    check(got, x, codes, scales, None, None, False)


@pytest.mark.parametrize("N,K,group,dtype", [(2050, 1056, 32, BF16), (2050, 1088, 64, F16), (2050, 1152, 128, BF16)])
def test_wide_tiles(N, K, group, dtype):
    """600 rows: tiles of 128, whose rows an array's end cuts only in the first and the last of them."""
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(K)
    x = normal(g, 600, K, dtype)
    codes, scales, z = (t[0] for t in weights(g, 1, N, K, group, dtype))
    first = {}
    for at in (0, 1, 3):
        s, zz = inside(scales, at, float("nan")), inside(z, 3 * at, 255)
        for swiglu in (False, True):
            got = M.moe_w4_linear(x, codes, s, zz, swiglu=swiglu, out_dtype=F32)
            check(got, x, codes, scales, z, None, swiglu, rows=[0, 127, 128, 300, 599])
            assert torch.isfinite(got).all()
            assert torch.equal(first.setdefault(swiglu, got), got)   # the same sums in the same order


@pytest.mark.parametrize("counts", [[3, 0, 1], [70, 5, 150], [40, 41, 0, 30], [200] + [0] * 40 + [3] * 15])
@pytest.mark.parametrize("N,K,group", [(130, 128, 128), (66, 96, 32), (300, 320, 64)])
def test_experts(counts, N, K, group):
    M = load_lib()
    E, P = len(counts), sum(counts) + 2
    g = torch.Generator(device="cuda").manual_seed(P + N)
    x = normal(g, P, K, F16)
    codes, scales, z = weights(g, E, N, K, group, F16)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    for at in (1, 2):
        got = torch.full((P, N), 7.0, dtype=F32, device="cuda")
        M.moe_w4_linear(x, codes, inside(scales, at, float("nan")), inside(z, at, 255), offsets, out=got)
        check(got, x, codes, scales, z, offsets, False)
        assert (got[P - 2:] == 7).all()
