"""Products with 4-bit weights against the fp64 oracle.

Tolerance: products are exact. A step of the tensor cores adds 16 of them to a sum in fp32, truncating: off by at most
2^-22 of the magnitudes it adds, so a group's sum by (g / 16) 2^-22 of its magnitudes; scaled and added to at most
K / g others by fused multiply-adds, each off by 2^-24 of all magnitudes; eight parts of a row may be added up at the
end. One rounding to the result's type."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.double().cpu().numpy()


def weights(g, E, N, K, group, dtype, zeros=True):
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = ((0.5 + torch.rand(E, N, K // group, device="cuda", generator=g)) * (0.25 * K ** -0.5)).to(dtype)
    z = torch.randint(0, 16, scales.shape, dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return codes, scales, z


def normal(g, P, K, dtype, wide=0):
    return torch.randn(P, K + wide, device="cuda", generator=g).to(dtype)[:, :K]


def tolerance(ref, size, K, group, out, swiglu):
    u = torch.finfo(out).eps / 2
    rel = (group / 16 * 4 + K / group + 8) * 2.0 ** -24 + (8 * 2.0 ** -24 if swiglu else 0)
    return rel * size + u * (np.abs(ref) + rel * size) + torch.finfo(out).tiny * u


def check(got, x, codes, scales, zeros, offsets, swiglu, rows=None):
    """Every row (or `rows`) of got against the oracle."""
    K, group = x.shape[1], x.shape[1] // scales.shape[-1]
    off = None if offsets is None else offsets.cpu().numpy()
    xs, gs = f64(x), f64(got)
    if rows is not None:   # the oracle over some rows alone
        for r in rows:
            e = 0 if off is None else int(np.searchsorted(off, r, side="right")) - 1
            ref, size = R.w4_linear(xs[r:r + 1], codes.view(-1, *codes.shape[-2:])[e].cpu().numpy(),
                                    f64(scales.view(-1, *scales.shape[-2:])[e]),
                                    None if zeros is None else zeros.view(-1, *zeros.shape[-2:])[e].cpu().numpy(), None, swiglu)
            assert (np.abs(gs[r] - ref[0]) <= tolerance(ref[0], size[0], K, group, got.dtype, swiglu)).all(), r
        return
    ref, size = R.w4_linear(xs, codes.cpu().numpy(), f64(scales), None if zeros is None else zeros.cpu().numpy(), off, swiglu)
    for r in ref:
        assert (np.abs(gs[r] - ref[r]) <= tolerance(ref[r], size[r], K, group, got.dtype, swiglu)).all(), r


DENSE = [   # P, N, K, group, dtype, out, zeros, swiglu, columns between rows
    (1, 256, 512, 128, BF16, BF16, True, False, 0), (1, 17, 128, 128, F16, F16, False, False, 0),
    (3, 33, 96, 32, BF16, F32, True, False, 64), (8, 40, 64, 64, F16, F32, True, True, 0),
    (9, 130, 320, 64, BF16, BF16, False, True, 8), (16, 16, 32, 32, F16, F16, True, False, 0),
    (57, 200, 1024, 64, F16, F32, False, False, 0), (64, 1, 256, 128, BF16, BF16, True, False, 0),
    (65, 258, 384, 128, BF16, BF16, True, True, 0), (128, 300, 640, 32, F16, F16, True, False, 0),
    (200, 515, 256, 64, BF16, F32, True, False, 64), (300, 128, 4224, 128, BF16, BF16, False, False, 0),
    (31, 384, 8192, 128, F16, F32, True, False, 0), (2, 2, 8320, 64, BF16, F32, True, True, 0),
    (1000, 144, 160, 32, BF16, BF16, True, True, 0), (130, 2050, 128, 128, F16, F16, True, False, 0),
    (5, 2000, 2048, 32, BF16, BF16, True, False, 0), (24, 2000, 2048, 32, BF16, BF16, True, False, 0)]


@pytest.mark.parametrize("P,N,K,group,dtype,out,zeros,swiglu,wide", DENSE)
def test_dense(P, N, K, group, dtype, out, zeros, swiglu, wide):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(P * N + K)
    x = normal(g, P, K, dtype, wide)
    codes, scales, z = (t if t is None else t[0] for t in weights(g, 1, N, K, group, dtype, zeros))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out, d_error=err)
    assert got.dtype is out and got.shape == (P, N // 2 if swiglu else N)
    check(got, x, codes, scales, z, None, swiglu)
    assert torch.equal(M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out), got)   # the same bits
    room = torch.full((P, got.shape[1] + 5), 7.0, dtype=out, device="cuda")                      # strided results
    M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out=room[:, :got.shape[1]])
    assert torch.equal(room[:, :got.shape[1]], got) and (room[:, got.shape[1]:] == 7).all()
    assert int(err) == 0


GROUPED = [   # rows of each expert, N, K, group, dtype, out, zeros, swiglu
    ([1, 0, 2, 0, 0, 1], 48, 256, 128, BF16, BF16, True, False), ([0, 9, 1], 40, 128, 64, F16, F32, True, True),
    ([8, 16, 24, 0, 7], 130, 320, 32, BF16, F32, False, False), ([0] * 30 + [3] + [0] * 225, 64, 128, 128, BF16, BF16, True, True),
    ([1] * 40, 66, 256, 64, F16, F16, True, False), ([64, 1, 65], 129, 256, 128, BF16, BF16, True, False),
    ([200, 0, 3, 130, 17], 260, 512, 128, BF16, F32, True, True), ([33] * 12, 100, 192, 64, F16, F16, True, False),
    ([100, 150, 90, 128], 384, 256, 32, BF16, BF16, False, False), ([0, 0, 0], 32, 128, 128, BF16, BF16, True, False),
    ([2000, 1, 0, 50], 136, 128, 64, BF16, BF16, True, False)]


@pytest.mark.parametrize("counts,N,K,group,dtype,out,zeros,swiglu", GROUPED)
def test_experts(counts, N, K, group, dtype, out, zeros, swiglu):
    M = load_lib()
    E, tail = len(counts), 5
    P = sum(counts) + tail
    g = torch.Generator(device="cuda").manual_seed(P * N + K)
    x = normal(g, P, K, dtype)
    x[P - tail:] = float("nan")                       # rows behind the last expert's
    codes, scales, z = weights(g, E, N, K, group, dtype, zeros)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    outs = N // 2 if swiglu else N
    got = torch.full((P, outs), 7.0, dtype=out, device="cuda")
    M.moe_w4_linear(x, codes, scales, z, offsets, swiglu=swiglu, out=got)
    assert (got[P - tail:] == 7).all()                # left as they were
    check(got, x, codes, scales, z, offsets, swiglu)
    # one expert's rows on their own: the neighbours do not matter beyond the way that is taken
    e = int(np.argmax(counts))
    if counts[e]:
        a, b = int(offsets[e]), int(offsets[e + 1])
        alone = M.moe_w4_linear(x[a:b], codes[e], scales[e], None if z is None else z[e], swiglu=swiglu, out_dtype=out)
        check(alone, x[a:b], codes[e], scales[e], None if z is None else z[e], None, swiglu)


def test_a_rows_values_stay_in_its_row():
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(3)
    for P in (4, 20, 100, 300):
        x = normal(g, P, 256, BF16)
        codes, scales, z = (t[0] for t in weights(g, 1, 144, 256, 64, BF16))
        want = M.moe_w4_linear(x, codes, scales, z)
        x[1], x[P - 1, 7] = float("nan"), float("inf")
        got = M.moe_w4_linear(x, codes, scales, z)
        assert torch.isnan(got[1]).all() and not torch.isfinite(got[P - 1]).any()
        keep = [r for r in range(P) if r not in (1, P - 1)]
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("P", [1, 40, 300])
def test_codes_and_zero_points_one_by_one(P, dtype):
    """Every code with zero points of the whole range, scales that are powers of two: exact results."""
    M = load_lib()
    K, N = 128, 128
    q = torch.arange(N * K, device="cuda").view(N, K) * 7 % 16
    codes = (q[:, 0::2] + 16 * q[:, 1::2]).to(torch.uint8)
    z = (torch.arange(N * 2, device="cuda").view(N, 2) % 128).to(torch.uint8)
    scales = (2.0 ** (torch.arange(N * 2, device="cuda").view(N, 2) % 5 - 2)).to(dtype)
    x = torch.zeros(P, K, device="cuda", dtype=dtype)
    at = torch.arange(P, device="cuda") * 37 % K
    x[torch.arange(P, device="cuda"), at] = 1
    W = (q - z.long().repeat_interleave(64, 1)) * scales.float().repeat_interleave(64, 1)
    got = M.moe_w4_linear(x, codes, scales, z, out_dtype=F32)
    assert torch.equal(got, W.T[at])


@pytest.mark.parametrize("P", [1, 12, 96, 256])
def test_scales_at_the_ends_of_their_type(P):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(2)
    for dtype, low, high in ((BF16, 2.0 ** -120, 2.0 ** 100), (F16, 2.0 ** -24, 2.0 ** 15)):
        codes, scales, z = (t[0] for t in weights(g, 1, 64, 256, 128, dtype))
        scales[:, 0], scales[::2, 1] = low, high
        scales[1::2, 1] = 0
        x = normal(g, P, 256, dtype)
        got = M.moe_w4_linear(x, codes, scales, z, out_dtype=F32)
        check(got, x, codes, scales, z, None, False)


def test_swiglu_of_large_gates():
    M = load_lib()
    K = 128
    codes = torch.full((4, K // 2), 0x99, dtype=torch.uint8, device="cuda")            # q - 8 = 1
    scales = torch.tensor([[1000.0], [-1000.0], [1.0], [1.0]], device="cuda").to(BF16)
    x = torch.ones(2, K, device="cuda", dtype=BF16)
    for P in (1, 2):
        got = M.moe_w4_linear(x[:P], codes, scales, swiglu=True, out_dtype=F32)
        assert (got[:, 0] == 128000.0 * 128).all() and (got[:, 1] == 0).all()


def test_a_large_matrix_and_many_rows():
    """The sizes of a prompt: rows picked from both ends and in between."""
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = normal(g, 2051, 4096, BF16)
    codes, scales, z = (t[0] for t in weights(g, 1, 4096, 4096, 128, BF16))
    got = M.moe_w4_linear(x, codes, scales, z)
    check(got, x, codes, scales, z, None, False, rows=[0, 1, 127, 128, 1000, 2047, 2048, 2050])
    E = 64
    counts = np.random.default_rng(0).multinomial(3000, np.random.default_rng(1).dirichlet(np.ones(E)))
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    x = normal(g, 3000, 2048, F16)
    codes, scales, z = weights(g, E, 1024, 2048, 64, F16)
    got = M.moe_w4_linear(x, codes, scales, z, offsets, swiglu=True)
    check(got, x, codes, scales, z, offsets, True, rows=list(range(0, 3000, 171)) + [2999])


def test_offsets_past_32_bits():
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(6)
    E, N, K = 520, 4096, 4096                        # 4.4 GB of codes
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((E, N, K // 128), 2.0 ** -8, dtype=BF16, device="cuda")
    for rows in (1, 40):
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[E] = rows
        x = normal(g, rows, K, BF16)
        got = M.moe_w4_linear(x, codes, scales, None, offsets)
        check(got, x, codes[E - 1], scales[E - 1], None, None, False, rows=[0, rows - 1])


@pytest.mark.parametrize("P,N,K", [(2, 96, 256), (48, 320, 512), (300, 256, 256)])
def test_other_stream_and_graph(P, N, K):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(8)
    x = normal(g, P, K, BF16)
    codes, scales, z = weights(g, 3, N, K, 64, BF16)
    offsets = torch.tensor([0, P // 2, P // 2, P], dtype=torch.int32, device="cuda")
    want = M.moe_w4_linear(x, codes, scales, z, offsets).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.moe_w4_linear(x, codes, scales, z, offsets, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    M.moe_w4_linear(x, codes, scales, z, offsets, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        M.moe_w4_linear(x, codes, scales, z, offsets, out=out)
    x.copy_(normal(g, P, K, BF16)), offsets.copy_(torch.tensor([0, P, P, P], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, M.moe_w4_linear(x, codes, scales, z, offsets))
    check(out, x, codes, scales, z, offsets, False)
