"""The routes of the 4-bit products that large matrices and many experts take. Tolerances as in test_gpu_w4_linear."""
import numpy as np
import pytest
import torch

from tests.helpers import load_lib
from tests.test_gpu_w4_linear import BF16, F16, F32, check, normal, weights

pytestmark = pytest.mark.gpu


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def some_rows(counts, n=40):
    """First and last rows of the largest and of other experts."""
    off = np.concatenate([[0], np.cumsum(counts)])
    used = [e for e in np.argsort(-np.asarray(counts), kind="stable") if counts[e]]
    chosen = used[:6] + used[6::max(1, len(used) // 12)] + [max(used), min(used)]
    return sorted({int(r) for e in chosen for r in (off[e], off[e + 1] - 1, off[e] + counts[e] // 2)})


@pytest.mark.parametrize("K", [4224, 8320])
@pytest.mark.parametrize("group,dtype,out,swiglu", [(32, BF16, F32, False), (64, F16, F16, True), (128, BF16, BF16, False)])
def test_few_rows_of_long_matrices(K, group, dtype, out, swiglu):
    """Blocks enough for every SM, none shared: x comes in several parts of 4096 columns."""
    M = load_lib()
    E, N = torch.cuda.get_device_properties(0).multi_processor_count + 8, 128
    counts = [e * 7 % 9 for e in range(E)]                                          # 0 to 8, at least E in all
    counts[3], counts[E - 1] = 24, 13                                               # codes read three and two times
    P = sum(counts) + 2
    g = torch.Generator(device="cuda").manual_seed(K + group)
    x = normal(g, P, K, dtype)
    x[P - 2:] = float("nan")
    codes, scales, z = weights(g, E, N, K, group, dtype)
    got = torch.full((P, N // 2 if swiglu else N), 7.0, dtype=out, device="cuda")
    M.moe_w4_linear(x, codes, scales, z, offsets_of(counts), swiglu=swiglu, out=got)
    check(got, x, codes, scales, z, offsets_of(counts), swiglu, rows=some_rows(counts))
    assert (got[P - 2:] == 7).all() and torch.isfinite(got[:P - 2]).all()
    again = torch.full_like(got, 7.0)
    M.moe_w4_linear(x, codes, scales, z, offsets_of(counts), swiglu=swiglu, out=again)
    assert torch.equal(again, got)


@pytest.mark.parametrize("P", [1, 3, 8])
@pytest.mark.parametrize("group", [32, 128])
def test_few_rows_of_a_large_matrix(P, group):
    M = load_lib()
    N, K = torch.cuda.get_device_properties(0).multi_processor_count * 128 + 17, 4480
    g = torch.Generator(device="cuda").manual_seed(P + group)
    x = normal(g, P, K, BF16)
    codes, scales, z = (t[0] for t in weights(g, 1, N, K, group, BF16))
    got = M.moe_w4_linear(x, codes, scales, z, out_dtype=F32)
    for lo in (0, 1000, N - 200):                                                    # the oracle over parts of the matrix
        part = slice(lo, lo + 200)
        check(got[:, part], x, codes[part], scales[part], z[part], None, False)


# rows of the experts that have any; E, N, K, group.  Means that take each width of the tiles, and skewed batches of many
# experts: the tiles of all experts are counted in several rounds of the block's threads.
MANY = [(1000, "few", 64, 128, 128), (2048, "few", 66, 128, 64), (2048, "few", 34, 96, 32), (1000, "12", 64, 128, 128),
        (1500, "40", 48, 128, 64), (1000, "70", 64, 128, 128), (900, "70", 130, 96, 32)]


@pytest.mark.parametrize("E,kind,N,K,group", MANY)
def test_tiles_of_many_experts(E, kind, N, K, group):
    M = load_lib()
    counts = np.zeros(E, dtype=np.int64)
    if kind == "few":
        for e, n in ((0, 25), (5, 24), (6, 300), (639, 26), (640, 70), (641, 3), (E - 2, 64), (E - 1, 129)):
            counts[e] = n
    else:
        counts[:] = np.random.default_rng(E).integers(0, 2 * int(kind) + 1, size=E)
        counts[7], counts[E - 1] = 0, 3 * int(kind)
        counts[11] += max(0, int(kind) * E - counts.sum())
    P = int(counts.sum()) + 3
    g = torch.Generator(device="cuda").manual_seed(E + N)
    x = normal(g, P, K, BF16)
    x[P - 3:] = float("nan")
    codes, scales, z = weights(g, E, N, K, group, BF16)
    got = torch.full((P, N), 7.0, dtype=F32, device="cuda")
    M.moe_w4_linear(x, codes, scales, z, offsets_of(counts), out=got)
    check(got, x, codes, scales, z, offsets_of(counts), False, rows=some_rows(counts))
    assert (got[P - 3:] == 7).all() and torch.isfinite(got[:P - 3]).all()
    # every row against the products in 64 bits
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double().unflatten(-1, (-1, group))
    W = ((q - z.double()[..., None]) * scales.double()[..., None]).flatten(-2)
    of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.from_numpy(counts).cuda())
    rel = (group / 16 * 4 + K / group + 8) * 2.0 ** -24
    for a in range(0, P - 3, 4096):
        b = min(P - 3, a + 4096)
        xs, ws = x[a:b].double(), W[of[a:b]]
        ref, size = torch.einsum("rk,rnk->rn", xs, ws), torch.einsum("rk,rnk->rn", xs.abs(), ws.abs())
        assert ((got[a:b].double() - ref).abs() <= (1 + 2.0 ** -24) * rel * size + 2.0 ** -24 * ref.abs()).all()


@pytest.mark.parametrize("P,N,K,group,dtype,out,zeros,swiglu", [
    (128, 2816, 4096, 128, BF16, F32, True, False), (101, 2816, 8192, 64, F16, F32, False, False),
    (128, 2690, 4608, 32, BF16, BF16, True, False), (127, 2816, 8192, 128, F16, F16, True, True)])
def test_wide_tiles_that_four_pairs_share(P, N, K, group, dtype, out, zeros, swiglu):
    """Ten to fifteen tiles of 128 rows of x: clusters of four pairs at that width."""
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(P + K)
    x = normal(g, P, K, dtype)
    codes, scales, z = (t if t is None else t[0] for t in weights(g, 1, N, K, group, dtype, zeros))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out, d_error=err)
    check(got, x, codes, scales, z, None, swiglu, rows=[0, 1, 31, 32, 33, 63, 64, 95, 96, P - 2, P - 1])
    for _ in range(10):
        again = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out)
    assert torch.equal(again, got) and int(err) == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("P", [1, 40, 300])
def test_zero_points_of_the_whole_byte(P, dtype):
    """Scales that are powers of two, one product a row: exact results."""
    M = load_lib()
    K, N = 128, 256
    q = torch.arange(N * K, device="cuda").view(N, K) * 7 % 16
    codes = (q[:, 0::2] + 16 * q[:, 1::2]).to(torch.uint8)
    z = (torch.arange(N * 2, device="cuda").view(N, 2) * 129 % 256).to(torch.uint8)
    scales = (2.0 ** (torch.arange(N * 2, device="cuda").view(N, 2) % 5 - 2)).to(dtype)
    x = torch.zeros(P, K, device="cuda", dtype=dtype)
    at = torch.arange(P, device="cuda") * 37 % K
    x[torch.arange(P, device="cuda"), at] = 1
    W = (q - z.long().repeat_interleave(64, 1)) * scales.float().repeat_interleave(64, 1)
    assert torch.equal(M.moe_w4_linear(x, codes, scales, z, out_dtype=F32), W.T[at])
