"""Tokens sorted by expert and back, and the gradients of both, against the fp64 oracle.

Tolerances, u the half step of the result's type: a sum of n products by fused multiply-adds in fp32 is off by at most
n 2^-24 of the magnitudes it adds (each partial sum is at most those), its rounding by u of it, or half the smallest
step near 0."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2   # half a step of the subnormal numbers


def f64(t):
    return t.double().cpu().numpy()


def normal(g, *shape, dtype=F32, by=1.0, wide=0):
    t = torch.randn(*shape[:-1], shape[-1] + wide, device="cuda", generator=g) * by
    return t.to(dtype)[..., :shape[-1]]


def routing(g, T, k, E, out=0.0):
    """Distinct experts for each token; `out`: share of the pairs without one."""
    ids = torch.topk(torch.rand(T, E, device="cuda", generator=g), k, dim=1)[1].to(torch.int32)
    return torch.where(torch.rand(T, k, device="cuda", generator=g) < out, -1, ids)


def sorted_on_host(ids, E):
    """offsets, pos by numpy's stable sort."""
    flat = ids.reshape(-1).astype(np.int64)
    in_ = (flat >= 0) & (flat < E)
    order = np.nonzero(in_)[0][np.argsort(flat[in_], kind="stable")]
    pos = np.full(flat.shape, -1)
    pos[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[in_], minlength=E))])
    return offsets, pos.reshape(ids.shape), order


SORTS = [   # T, k, E, H, dtype, share without an expert, columns between rows
    (1, 8, 256, 4096, BF16, 0.0, 0), (1, 1, 1, 1, F32, 0.0, 0), (2, 3, 5, 7, F16, 0.3, 0), (64, 8, 256, 512, BF16, 0.05, 0),
    (63, 5, 9, 1001, F32, 0.2, 7), (17, 2, 2048, 64, BF16, 0.0, 64), (300, 8, 128, 130, F16, 0.5, 2),
    (255, 8, 256, 72, BF16, 0.0, 7), (257, 8, 256, 72, BF16, 0.1, 8), (1024, 4, 2048, 33, F32, 0.1, 0),
    (5000, 8, 1025, 16, BF16, 0.1, 0), (40000, 6, 300, 8, F16, 0.0, 0), (7, 64, 64, 24, BF16, 0.5, 0),
    (9000, 1, 3, 40, F32, 0.02, 0), (50, 4, 1024, 20, F32, 1.0, 0)]


@pytest.mark.parametrize("T,k,E,H,dtype,out,wide", SORTS)
def test_sort_rows(T, k, E, H, dtype, out, wide):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(T * k + H)
    x, ids = normal(g, T, H, dtype=dtype, wide=wide), routing(g, T, k, E, out)
    rows = normal(g, T * k, H, dtype=dtype, wide=wide)
    before = rows.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, offsets, pos = M.moe_sort_rows(x, ids, E, rows=rows, d_error=err)
    assert got is rows and int(err) == 0
    off, want, order = sorted_on_host(ids.cpu().numpy(), E)
    assert (offsets.cpu().numpy() == off).all() and (pos.cpu().numpy() == want).all()
    n = int(off[-1])
    assert torch.equal(rows[:n], x[torch.from_numpy(order // k).cuda()])
    assert torch.equal(rows[n:], before[n:])                      # as they were
    # without buffers of the caller's
    rows2, offsets2, pos2 = M.moe_sort_rows(x, ids, E)
    assert torch.equal(rows2[:n], rows[:n]) and torch.equal(offsets2, offsets) and torch.equal(pos2, pos)


def test_sort_rows_agrees_with_group_pairs_and_keeps_bits():
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = routing(g, 700, 6, 256, 0.1)
    x = torch.randint(0, 65536, (700, 64), device="cuda", generator=g).to(torch.int32).to(torch.int16).view(BF16)   # NaN too
    rows, offsets, pos = M.moe_sort_rows(x, ids, 256)
    off, perm, _ = M.moe_group_pairs(ids, 256)
    n = int(off[-1])
    assert torch.equal(off, offsets)
    assert torch.equal(pos.flatten()[perm[:n].long()], torch.arange(n, device="cuda", dtype=torch.int32))
    assert torch.equal(rows[:n].view(torch.int16), x.view(torch.int16)[perm[:n].long() // 6])


@pytest.mark.parametrize("T", [3, 4000])
def test_sort_rows_reports_ids_out_of_range_and_leaves_them_out(T):
    M = load_lib()
    ids = torch.tensor([[1, 9], [2 ** 31 - 1, 0], [-2 ** 31, 4]], dtype=torch.int32, device="cuda").repeat((T + 2) // 3, 1)[:T]
    x = torch.randn(T, 16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, offsets, pos = M.moe_sort_rows(x, ids, 5, d_error=err)
    off, want, _ = sorted_on_host(ids.cpu().numpy(), 5)
    assert int(err) == M.MOE_ERR_INVALID
    assert (offsets.cpu().numpy() == off).all() and (pos.cpu().numpy() == want).all()
    M.moe_sort_rows(x, ids, 5)                                    # without an error word


@pytest.mark.parametrize("T", [40, 3000])
def test_sort_rows_of_one_expert_for_all_and_of_the_same_one_twice(T):
    M = load_lib()
    ids = torch.full((T, 3), 6, dtype=torch.int32, device="cuda")
    ids[::7, 1] = 2
    x = torch.randn(T, 5, device="cuda")
    rows, offsets, pos = M.moe_sort_rows(x, ids, 8)
    off, want, order = sorted_on_host(ids.cpu().numpy(), 8)
    assert (offsets.cpu().numpy() == off).all() and (pos.cpu().numpy() == want).all()
    assert torch.equal(rows, x[torch.from_numpy(order // 3).cuda()])


def test_no_tokens():
    M = load_lib()
    x, ids = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 8, dtype=torch.int32, device="cuda")
    offsets = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    rows, off, pos = M.moe_sort_rows(x, ids, 8, offsets=offsets)
    assert off is offsets and not offsets.any() and rows.shape == (0, 64) and pos.shape == (0, 8)
    assert M.moe_combine_rows(rows, pos).shape == (0, 64)
    assert M.moe_sort_rows_backward(rows, pos).shape == (0, 64)
    d_rows, d_w = M.moe_combine_rows_backward(x, rows, pos)
    assert d_rows.shape == (0, 64) and d_w.shape == (0, 8)


COMBINES = [   # T, k, H, share without an expert, weights, base, columns between rows
    (1, 8, 4096, 0.0, True, True, 0), (64, 8, 512, 0.1, True, False, 0), (33, 5, 1001, 0.2, True, True, 7),
    (20, 6, 130, 0.0, False, False, 2), (3, 1, 1, 0.0, True, True, 0), (7, 17, 72, 0.3, True, True, 8),
    (500, 3, 64, 0.6, False, True, 64), (50, 64, 40, 0.5, True, False, 0), (9, 4, 24, 1.0, True, True, 0),
    (11, 2, 20, 0.0, True, False, 0)]


@pytest.mark.parametrize("rd,yd", TYPES)
@pytest.mark.parametrize("T,k,H,out,weights,base,wide", COMBINES)
def test_combine_rows(T, k, H, out, weights, base, wide, rd, yd):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(T * k + H)
    ids = routing(g, T, k, 64, out).cpu().numpy()
    off, pos, _ = sorted_on_host(ids, 64)
    rows = normal(g, T * k, H, dtype=rd, wide=wide)
    rows[int(off[-1]):] = float("nan")                            # rows that no pair names
    w = normal(g, T, k) if weights else None
    b = normal(g, T, H, dtype=yd, wide=wide) if base else None
    p = torch.from_numpy(pos).to(torch.int32).cuda()
    y = M.moe_combine_rows(rows, p, w, b, out_dtype=yd)
    assert y.dtype is yd
    ref, size = R.combine_rows(f64(rows), pos, None if w is None else f64(w), None if b is None else f64(b))
    tol = (k + 1) * 2.0 ** -24 * size + half(yd) * (np.abs(ref) + (k + 1) * 2.0 ** -24 * size) + tiny(yd)
    assert (np.abs(f64(y) - ref) <= tol).all()
    assert torch.equal(M.moe_combine_rows(rows, p, w, b, out_dtype=yd), y)
    if base:                                                      # in place
        M.moe_combine_rows(rows, p, w, b, y=b)
        assert torch.equal(b, y)
    if rd is yd and not weights and not base:
        assert torch.equal(M.moe_sort_rows_backward(rows, p), y)


@pytest.mark.parametrize("rd,yd", TYPES)
@pytest.mark.parametrize("T,k,H,out,weights,base,wide", COMBINES)
def test_combine_rows_backward(T, k, H, out, weights, base, wide, rd, yd):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(T + k + H)
    ids = routing(g, T, k, 64, out).cpu().numpy()
    off, pos, _ = sorted_on_host(ids, 64)
    n = int(off[-1])
    rows, dy = normal(g, T * k, H, dtype=rd, wide=wide), normal(g, T, H, dtype=yd, wide=wide)
    rows[n:] = float("nan")
    w = normal(g, T, k) if weights else None
    p = torch.from_numpy(pos).to(torch.int32).cuda()
    d_rows = torch.full((T * k, H), 3.0, dtype=rd, device="cuda")
    got, d_w = M.moe_combine_rows_backward(dy, rows, p, w, d_rows=d_rows)
    assert got is d_rows and (d_rows[n:] == 3).all()
    want, want_w, size = R.combine_rows_backward(f64(dy), f64(rows), pos, None if w is None else f64(w))
    ref = np.zeros((n, H))
    for r, v in want.items():
        ref[r] = v
    tol = (half(rd) + 2.0 ** -24) * (1 + 2.0 ** -20) * np.abs(ref) + tiny(rd)
    assert (np.abs(f64(d_rows)[:n] - ref) <= tol).all()
    # a thread's share of a row one after the other, then the threads' sums: at most H / 32 + 8 + 16 additions deep
    assert (np.abs(f64(d_w) - want_w) <= (H / 32 + 24) * 2.0 ** -24 * size).all()
    d2, none = M.moe_combine_rows_backward(dy, rows, p, w, d_rows=torch.full_like(d_rows, 3.0), want_d_w=False)
    assert none is None and torch.equal(d2, d_rows)
    _, d_w2 = M.moe_combine_rows_backward(dy, rows, p, w, d_rows=rows)          # in place
    assert torch.equal(rows[:n], d_rows[:n]) and torch.equal(d_w2, d_w)


def test_gradients_against_differences():
    """The gradient of <c, combine(sort(x) + a)> with respect to x, a and w, against differences in 64 bits of the
    oracle at the kernels' own inputs."""
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(5)
    T, k, E, H = 6, 2, 4, 10
    x, ids, w, c = normal(g, T, H), routing(g, T, k, E, 0.2), normal(g, T, k), normal(g, T, H)
    rows, offsets, pos = M.moe_sort_rows(x, ids, E)
    n = int(offsets[-1])
    d_rows, d_w = M.moe_combine_rows_backward(c, rows, pos, w)
    d_x = M.moe_sort_rows_backward(d_rows, pos)

    def value(xv, wv):
        r, _, p = R.sort_rows(xv, ids.cpu().numpy(), E)
        return (R.combine_rows(r, p, wv)[0] * f64(c)).sum()
    h, x0, w0 = 1e-5, f64(x), f64(w)
    for t, i in [(0, 0), (1, 3), (3, 9), (5, 4)]:
        e = np.zeros_like(x0)
        e[t, i] = h
        assert abs((value(x0 + e, w0) - value(x0 - e, w0)) / (2 * h) - float(d_x[t, i])) < 1e-6
    for t in range(T):
        for j in range(k):
            e = np.zeros_like(w0)
            e[t, j] = h
            assert abs((value(x0, w0 + e) - value(x0, w0 - e)) / (2 * h) - float(d_w[t, j])) < 1e-5
    assert n == int((ids >= 0).sum())


def test_places_out_of_range_are_not_read_or_written():
    M = load_lib()
    pos = torch.tensor([[0, 2 ** 31 - 1], [-2 ** 31, 1], [3, -7]], dtype=torch.int32, device="cuda")
    rows = torch.arange(6.0, device="cuda").view(3, 2)
    y = M.moe_combine_rows(rows, pos)
    assert y.tolist() == [[0, 1], [2, 3], [0, 0]]
    d_rows = torch.full((3, 2), 9.0, device="cuda")
    _, d_w = M.moe_combine_rows_backward(torch.ones(3, 2, device="cuda"), rows, pos, d_rows=d_rows)
    assert d_rows.tolist() == [[1, 1], [1, 1], [9, 9]] and d_w.tolist() == [[1, 0], [0, 5], [0, 0]]


def test_infinities_and_nan_stay_with_their_token():
    M = load_lib()
    rows = torch.tensor([[1.0, 2.0], [float("inf"), float("nan")], [3.0, 4.0]], device="cuda").to(BF16)
    pos = torch.tensor([[0, 2], [1, -1], [-1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [0.5, float("nan")], [float("inf"), 3.0]], device="cuda")   # of pairs without a row: not used
    y = M.moe_combine_rows(rows, pos, w).float()
    assert y[0].tolist() == [7, 10] and y[2].tolist() == [3, 6]
    assert torch.isinf(y[1, 0]) and torch.isnan(y[1, 1])
    _, d_w = M.moe_combine_rows_backward(torch.ones(3, 2, device="cuda", dtype=BF16), rows, pos, w)
    assert d_w[0].tolist() == [3, 7] and d_w[2].tolist() == [0, 3] and torch.isnan(d_w[1, 0]) and d_w[1, 1] == 0


def test_offsets_past_32_bits():
    """Rows whose bytes and elements pass 2^31: the last ones are found."""
    M = load_lib()
    T, k, H = 40000, 2, 65536
    rows = torch.empty(T * k, H // 2, dtype=BF16, device="cuda")                      # 80000 x 32768: 5.2 GB
    pos = torch.full((3, k), -1, dtype=torch.int32, device="cuda")
    pos[1, 0], pos[2, 1] = T * k - 1, 70000
    rows[T * k - 1], rows[70000] = 3, 5
    y = M.moe_combine_rows(rows, pos)
    assert not y[0].any() and (y[1] == 3).all() and (y[2] == 5).all()
    M.moe_combine_rows_backward(torch.full_like(y, 7), rows, pos, d_rows=rows)
    assert (rows[T * k - 1] == 7).all() and (rows[70000] == 7).all()
    tokens = torch.empty(T, H, dtype=BF16, device="cuda")                              # 5.2 GB
    tokens[T - 1], tokens[0] = 2, 4
    ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    ids[T - 1], ids[0] = 0, 1
    out, offsets, place = M.moe_sort_rows(tokens, ids, 2, rows=rows.view(T, H))
    assert (out[0] == 2).all() and (out[1] == 4).all() and offsets.tolist() == [0, 1, 2]
    assert int(place[T - 1]) == 0 and int(place[0]) == 1


def test_other_stream_graph_and_repeats():
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(1)
    T, k, E, H = 512, 4, 64, 256
    x, ids, w = normal(g, T, H, dtype=BF16), routing(g, T, k, E, 0.1), normal(g, T, k)
    bufs = {}

    def step():
        rows, off, pos = M.moe_sort_rows(x, ids, E, rows=bufs.get("rows"), offsets=bufs.get("off"), pos=bufs.get("pos"))
        y = M.moe_combine_rows(rows, pos, w, x, y=bufs.get("y"))
        d_rows, d_w = M.moe_combine_rows_backward(y, rows, pos, w, d_rows=bufs.get("d_rows"), d_w=bufs.get("d_w"))
        d_x = M.moe_sort_rows_backward(d_rows, pos, d_x=bufs.get("d_x"))
        return dict(rows=rows, off=off, pos=pos, y=y, d_rows=d_rows, d_w=d_w, d_x=d_x)
    want = {n: t.clone() for n, t in step().items()}
    n = int(want["off"][-1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    bufs.update({m: torch.zeros_like(t) for m, t in want.items()})
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2 = normal(g, T, H, dtype=BF16)
    x.copy_(x2), ids.copy_(routing(g, T, k, E, 0.3))
    graph.replay()
    torch.cuda.synchronize()
    replayed = {m: t.clone() for m, t in bufs.items()}
    bufs.clear()
    eager = step()
    n2 = int(eager["off"][-1])
    for m in want:
        rows = slice(0, n) if m in ("rows", "d_rows") else slice(None)
        assert torch.equal(got[m][rows], want[m][rows]), m
        rows = slice(0, n2) if m in ("rows", "d_rows") else slice(None)
        assert torch.equal(replayed[m][rows], eager[m][rows]), m
