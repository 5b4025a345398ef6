"""Routing, rows by expert, the products of 4-bit experts and the way back, run together as a layer runs them, and the
gradients from its output to the router's logits; and products whose depth several blocks share.

Tolerances: products by 4-bit weights as in test_gpu_w4_linear. In the layer each operator gets the GPU's results of the
one before, so its own tolerance is all that counts."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from tests.helpers import load_lib
from tests.test_gpu_w4_linear import check, normal, weights

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return t.double().cpu().numpy()


SHARED = [   # P, N, K, group, dtype, out, zeros, swiglu: few tiles, so that clusters of blocks share a row's groups
    (3, 300, 2208, 32, BF16, F32, True, False), (5, 130, 4128, 32, F16, F16, True, True), (8, 256, 1088, 64, BF16, BF16, False, False),
    (7, 64, 640, 128, BF16, F32, True, True), (4, 1, 512, 64, F16, F32, True, False),
    (10, 130, 1056, 32, BF16, F32, True, True), (33, 70, 1184, 32, F16, F16, False, False), (57, 600, 2048, 64, F16, F32, True, False),
    (70, 400, 640, 128, BF16, BF16, True, True), (130, 512, 1152, 64, BF16, F32, True, False), (16, 2, 4096, 128, BF16, BF16, False, True),
    (250, 258, 1152, 128, F16, F32, True, True), (100, 1000, 544, 32, BF16, BF16, True, False)]


@pytest.mark.parametrize("P,N,K,group,dtype,out,zeros,swiglu", SHARED)
def test_blocks_that_share_the_depth(P, N, K, group, dtype, out, zeros, swiglu):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(P * N + K)
    x = normal(g, P, K, dtype)
    codes, scales, z = (t if t is None else t[0] for t in weights(g, 1, N, K, group, dtype, zeros))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out, d_error=err)
    check(got, x, codes, scales, z, None, swiglu)
    for _ in range(20):   # back to back: a launch starts while the one before it ends
        again = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out)
    assert torch.equal(again, got) and int(err) == 0
    x[P // 2] = float("nan")   # stays in its row
    marked = M.moe_w4_linear(x, codes, scales, z, swiglu=swiglu, out_dtype=out)
    keep = [r for r in range(P) if r != P // 2]
    assert torch.isnan(marked[P // 2]).all() and torch.equal(marked[keep], got[keep])


@pytest.mark.parametrize("counts,N,K,group,swiglu", [
    ([3, 17, 0, 8], 200, 1056, 32, False), ([0, 30, 1, 0], 66, 2048, 128, True),      # few rows, experts with more than eight
    ([20, 0, 13, 40], 256, 1056, 32, True), ([64, 1], 500, 1024, 64, False), ([0, 0, 40], 130, 512, 128, False)])
def test_experts_that_share_the_depth(counts, N, K, group, swiglu):
    M = load_lib()
    E, P = len(counts), sum(counts) + 3
    g = torch.Generator(device="cuda").manual_seed(K)
    x = normal(g, P, K, BF16)
    x[P - 3:] = float("nan")
    codes, scales, z = weights(g, E, N, K, group, BF16)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    got = torch.full((P, N // 2 if swiglu else N), 7.0, dtype=F32, device="cuda")
    M.moe_w4_linear(x, codes, scales, z, offsets, swiglu=swiglu, out=got)
    check(got, x, codes, scales, z, offsets, swiglu)
    assert (got[P - 3:] == 7).all()


def test_products_on_two_streams_at_once():
    """Nothing is shared between calls: small and large ones in turn on two streams give what they give alone."""
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(2)
    sets = []
    for P, N, K in ((57, 600, 2048), (5, 512, 4096), (300, 1024, 1024), (1, 512, 4096)):
        x = normal(g, P, K, BF16)
        codes, scales, z = (t[0] for t in weights(g, 1, N, K, 64, BF16))
        sets.append((x, codes, scales, z))
    want = [M.moe_w4_linear(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = [M.moe_w4_linear(*s) for s in sets]
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))


def layer(M, h, router, w13, w2, E, k, dtype, shared, bufs=None):
    """A routed layer of int4 experts, its shared part added: logits, choice, rows, products, sum."""
    b = bufs or {}
    logits = M.moe_adapter_linear(h, router, out_dtype=F32) if "logits" not in b else M.moe_adapter_linear(h, router, out=b["logits"])
    ids, w = M.moe_route(logits, k, topk_ids=b.get("ids"), topk_w=b.get("w"))
    rows, offsets, pos = M.moe_sort_rows(h, ids, E, rows=b.get("rows"), offsets=b.get("offsets"), pos=b.get("pos"))
    mid = M.moe_w4_linear(rows, *w13, offsets=offsets, swiglu=True, out=b.get("mid"))
    down = M.moe_w4_linear(mid, *w2, offsets=offsets, out=b.get("down"), out_dtype=None if "down" in b else F32)
    y = M.moe_combine_rows(down, pos, w, shared, y=b.get("y"))
    return dict(logits=logits, w=w, ids=ids, rows=rows, offsets=offsets, pos=pos, mid=mid, down=down, y=y)


@pytest.mark.parametrize("T,k,E,H,I,dtype", [(1, 4, 32, 256, 128, BF16), (16, 2, 8, 512, 256, F16), (96, 4, 16, 256, 384, BF16)])
def test_a_layer_and_its_gradients(T, k, E, H, I, dtype):
    M = load_lib()
    g = torch.Generator(device="cuda").manual_seed(T)
    h, shared = normal(g, T, H, dtype), normal(g, T, H, dtype)
    router = (torch.randn(E, H, device="cuda", generator=g) * H ** -0.5).to(dtype)
    w13, w2 = weights(g, E, 2 * I, H, 64, dtype), weights(g, E, H, I, 64, dtype, zeros=False)
    r = layer(M, h, router, w13, w2, E, k, dtype, shared)
    n = T * k
    # each operator of what the one before it gave
    rows, offsets, pos = R.sort_rows(f64(h), r["ids"].cpu().numpy(), E)
    assert np.array_equal(f64(r["rows"]), rows)
    assert np.array_equal(r["offsets"].cpu().numpy(), offsets) and np.array_equal(r["pos"].cpu().numpy(), pos)
    check(r["mid"], r["rows"], *w13, r["offsets"], True)
    check(r["down"], r["mid"], *w2, r["offsets"], False)
    y, size = R.combine_rows(f64(r["down"]), pos, f64(r["w"]), f64(shared))
    u = torch.finfo(dtype).eps / 2
    err = (k + 1) * 2.0 ** -24 * size
    assert (np.abs(f64(r["y"]) - y) <= err + u * (np.abs(y) + err)).all()
    # back to the experts' rows and the router's logits
    dy = normal(g, T, H, dtype)
    d_rows, d_w = M.moe_combine_rows_backward(dy, r["down"], r["pos"], r["w"])
    want, want_w, size = R.combine_rows_backward(f64(dy), f64(r["down"]), pos, f64(r["w"]))
    got = f64(d_rows)
    for p in range(n):
        assert (np.abs(got[p] - want[p]) <= 2.0 ** -24 * np.abs(want[p])).all()
    assert (np.abs(f64(d_w) - want_w) <= H * 2.0 ** -24 * size + 2.0 ** -149).all()
    d_logits = f64(M.moe_route_backward(r["logits"], r["ids"], d_w))
    # softmax over all, the k chosen weights divided by their sum: a softmax over the chosen ones alone
    L, ids = f64(r["logits"]), r["ids"].cpu().numpy()
    d = f64(d_w)
    for t in range(T):
        a = np.exp(L[t, ids[t]] - L[t, ids[t]].max())
        a /= a.sum()
        ref = np.zeros(E)
        ref[ids[t]] = a * (d[t] - (a * d[t]).sum())
        # a chain of some 16 operations and expf's 2 units, each off by 2^-24 or a few of what they carry
        assert (np.abs(d_logits[t] - ref) <= 64 * 2.0 ** -24 * (np.abs(d[t]).max() + np.abs(ref))).all()
    # the whole of it captured, then replayed on other tokens
    bufs = {name: torch.zeros_like(t) for name, t in r.items()}
    graph = torch.cuda.CUDAGraph()
    layer(M, h, router, w13, w2, E, k, dtype, shared, bufs)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer(M, h, router, w13, w2, E, k, dtype, shared, bufs)
    h.copy_(normal(g, T, H, dtype))
    graph.replay()
    torch.cuda.synchronize()
    eager = layer(M, h, router, w13, w2, E, k, dtype, shared)
    for name in eager:
        assert torch.equal(bufs[name], eager[name]), name


@pytest.mark.parametrize("group,swiglu", [(128, False), (64, True), (32, False)])
def test_a_batch_that_goes_to_few_of_many_experts(group, swiglu):
    """Some experts have many rows, most none: both ways are taken side by side."""
    M = load_lib()
    counts = [0] * 64
    for e, n in ((0, 24), (1, 25), (2, 1), (7, 300), (30, 8), (31, 9), (62, 64), (63, 26)):
        counts[e] = n
    E, P, N, K = 64, sum(counts) + 2, 192, 640
    g = torch.Generator(device="cuda").manual_seed(group)
    x = normal(g, P, K, BF16)
    x[P - 2:] = float("nan")
    codes, scales, z = weights(g, E, N, K, group, BF16)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    got = torch.full((P, N // 2 if swiglu else N), 7.0, dtype=F32, device="cuda")
    M.moe_w4_linear(x, codes, scales, z, offsets, swiglu=swiglu, out=got)
    check(got, x, codes, scales, z, offsets, swiglu)
    assert (got[P - 2:] == 7).all()
    again = torch.full_like(got, 7.0)
    for _ in range(10):
        M.moe_w4_linear(x, codes, scales, z, offsets, swiglu=swiglu, out=again)
    assert torch.equal(again, got)
