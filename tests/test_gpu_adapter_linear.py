"""moe_adapter_linear against the fp64 oracle.

Tolerances: products of two 16-bit numbers are exact in fp32; a sum of H of them
is added up in steps of 8 or more, each step off by at most 2^-23 of what has
been summed (a tensor-core step may truncate), so (H / 8 + 64) 2^-23 of the sum
of the products' magnitudes bounds it.  The adapter's term adds the same for its
two sums (R <= 128 terms in the second).  Then one rounding to out's type."""
import numpy as np
import pytest
import torch

from oracle import block as O
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _data(seed, T, H, N, R, n, dtype, ids, pad=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(DT[dtype])
    d = dict(x=normal(T, H + pad + offset)[:, offset:offset + H], W=normal(N, H, by=H ** -0.5))
    if n:
        d.update(A=normal(n, R, H, by=H ** -0.5), B=normal(n, N, R, by=R ** -0.5),
                 c=0.5 + torch.rand(n, device="cuda", generator=g))
        rng = np.random.default_rng(seed)
        if ids == "mixed":
            a = rng.integers(-1, n, T)
        elif ids == "runs":
            a = np.sort(rng.integers(-1, n, T))
        elif ids == "none":
            a = np.full(T, -1)
        else:
            a = np.full(T, ids)
        d["ids"] = torch.from_numpy(a.astype(np.int32)).cuda()
    return d


def _check(M, d, dtype, out_dtype, rows=None, **kw):
    out = M.moe_adapter_linear(d["x"], d["W"], d.get("A"), d.get("B"), d.get("ids"), d.get("c"),
                               out_dtype=DT[out_dtype], **kw)
    T = d["x"].shape[0]
    rows = np.arange(T) if rows is None or rows >= T else np.unique(np.linspace(0, T - 1, rows).astype(int))
    pick = torch.from_numpy(rows).cuda()

    def f(t):
        return t.double().cpu().numpy()
    n = d["A"].shape[0] if "A" in d else 0
    ref, size, low = O.adapter_linear(f(d["x"][pick]), f(d["W"]), f(d["A"]) if n else None, f(d["B"]) if n else None,
                                      f(d["ids"][pick]) if n else None, f(d["c"]) if n else None)
    H = d["x"].shape[1]
    tol = (H / 8 + 64) * 2.0 ** -23 * (size + low) + ULP[out_dtype] * np.abs(ref)
    if out_dtype == "f16":
        tol = tol + 2.0 ** -25
    got = f(out[pick])
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
    return out


SHAPES = [(1, 4096, 256, 16, 4), (16, 4096, 256, 16, 8), (64, 4096, 2048, 16, 32), (3, 8, 1, 8, 2), (5, 24, 7, 8, 3),
          (33, 264, 129, 24, 5), (65, 512, 300, 40, 3), (127, 1000, 257, 64, 6), (129, 136, 640, 128, 2),
          (300, 2048, 1000, 8, 40), (1000, 512, 4096, 32, 7), (2, 8192, 33, 56, 1), (700, 1544, 384, 72, 9)]


@pytest.mark.parametrize("T,H,N,R,n", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_matches_oracle(T, H, N, R, n, dtype, out, ids):
    M = load_lib()
    _check(M, _data(T + N, T, H, N, R, n, dtype, ids), dtype, out, rows=150)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 48, 63, 64, 66, 96, 128, 160, 192, 255, 256, 257, 384, 511,
                               513, 640, 1025])
@pytest.mark.parametrize("N", [256, 2048])
def test_adapter_linear_token_counts(T, N):
    M = load_lib()
    _check(M, _data(T, T, 1024, N, 16, 12, "bf16", "mixed"), "bf16", "f32", rows=64)


@pytest.mark.parametrize("T,N", [(4001, 4096), (8192, 256), (2048, 2048)])
def test_adapter_linear_prompts(T, N):
    M = load_lib()
    d = _data(1, T, 4096, N, 32, 8, "bf16", "runs")
    a = _check(M, d, "bf16", "bf16", rows=70)
    b = _check(M, d, "bf16", "bf16", rows=2)
    assert torch.equal(a, b)


# more than 16 x 7 tiles of 128 x 128: the persistent kernel, with ragged H, N and T, ranks past one
# and two 64-wide steps, fp32 results in one sum (H <= 512) and in several
LARGE = [(1300, 1032, 2048, 40, 5), (1030, 136, 2304, 128, 2), (1100, 200, 2200, 72, 3), (16400, 64, 100, 8, 9),
         (1999, 520, 2049, 16, 30), (1024, 4096, 2048, 64, 1)]


@pytest.mark.parametrize("T,H,N,R,n", LARGE)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("ids", ["mixed", "runs", 0])
def test_adapter_linear_large_batches(T, H, N, R, n, dtype, out, ids):
    M = load_lib()
    _check(M, _data(T + N, T, H, N, R, n, dtype, ids), dtype, out, rows=200)


def test_adapter_linear_without_adapters_large():
    M = load_lib()
    for T, H, N in ((1300, 1032, 2048), (16400, 64, 100), (1999, 520, 2049)):
        d = _data(T, T, H, N, 8, 0, "bf16", "none")
        for out in ("bf16", "f32"):
            _check(M, d, "bf16", out, rows=100)


@pytest.mark.parametrize("T", [40, 1300])
def test_adapter_linear_f16_past_its_range(T):
    # A x past fp16's largest value, brought back by B: nothing may be carried in fp16 then
    M = load_lib()
    d = _data(11, T, 256, 2048, 16, 3, "f16", "runs")
    d["A"] = (d["A"].float() * 3e4).to(torch.float16)
    d["B"] = (d["B"].float() * 1e-4).to(torch.float16)
    _check(M, d, "f16", "f32", rows=150)


@pytest.mark.parametrize("T", [5, 700])
@pytest.mark.parametrize("ids", ["none", 0, 2, "mixed"])
def test_adapter_linear_uses_of_adapters(T, ids):
    M = load_lib()
    d = _data(3, T, 512, 384, 16, 3, "bf16", ids)
    out = _check(M, d, "bf16", "f32")
    plain = _check(M, {m: d[m] for m in ("x", "W")}, "bf16", "f32")
    off = d["ids"] < 0
    assert torch.equal(out[off], plain[off])
    # what an unused adapter holds does not matter
    used = set(d["ids"].tolist())
    for a in range(3):
        if a not in used:
            d["A"][a] = float("nan")
            d["B"][a] = float("inf")
    assert torch.equal(_check(M, d, "bf16", "f32"), out)
    one = dict(d, c=torch.ones(3, device="cuda"))
    a = M.moe_adapter_linear(one["x"], one["W"], one["A"], one["B"], one["ids"], one["c"])
    b = M.moe_adapter_linear(one["x"], one["W"], one["A"], one["B"], one["ids"])
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [6, 300, 1300])
def test_adapter_linear_nan_stays_with_its_adapter(T):
    # an adapter of NaN reaches the tokens that use it and no other, whoever shares their tile
    M = load_lib()
    d = _data(4, T, 256, 512, 16, 4, "bf16", "mixed")
    want = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"])
    d["A"][1] = float("nan")
    d["B"][2] = float("inf")
    got = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"])
    ok = (d["ids"] != 1) & (d["ids"] != 2)
    assert torch.equal(got[ok], want[ok]) and torch.isnan(got[d["ids"] == 1]).all()


@pytest.mark.parametrize("T", [4, 70, 900])
@pytest.mark.parametrize("offset,pad", [(0, 8), (8, 16)])
def test_adapter_linear_strides(T, offset, pad):
    M = load_lib()
    d = _data(5, T, 320, 200, 16, 3, "bf16", "mixed", pad, offset)
    want = _check(M, dict(d, x=d["x"].contiguous()), "bf16", "bf16")
    assert torch.equal(_check(M, d, "bf16", "bf16"), want)
    wide_w = torch.zeros(200, 352, dtype=torch.bfloat16, device="cuda")
    wide_w[:, 16:336] = d["W"]
    wide = torch.full((T, 211), 3.0, dtype=torch.bfloat16, device="cuda")
    M.moe_adapter_linear(d["x"], wide_w[:, 16:336], d["A"], d["B"], d["ids"], d["c"], out=wide[:, 7:207])
    assert torch.equal(wide[:, 7:207], want)
    assert (wide[:, :7] == 3).all() and (wide[:, 207:] == 3).all()


@pytest.mark.parametrize("T", [9, 600])
def test_adapter_linear_reports_an_id_out_of_range(T):
    M = load_lib()
    d = _data(6, T, 256, 320, 8, 3, "bf16", "mixed")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ok = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"], d_error=err)
    assert int(err) == M.MOE_OK
    bad = d["ids"].clone()
    bad[T // 2] = 3
    got = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], bad, d["c"], d_error=err)
    assert int(err) == M.MOE_ERR_INVALID
    none = bad.clone()
    none[T // 2] = -1
    want = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], none, d["c"])
    assert torch.equal(got, want)
    assert torch.equal(got[d["ids"] == bad], ok[d["ids"] == bad])


@pytest.mark.parametrize("T", [8, 640])
def test_adapter_linear_on_another_stream_and_repeats(T):
    M = load_lib()
    d = _data(7, T, 1024, 768, 16, 5, "bf16", "mixed")
    args = (d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"])
    want = M.moe_adapter_linear(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((max(16, M.moe_adapter_linear_workspace(T, 1024, 768, 5, 16)),), 255, dtype=torch.uint8,
                    device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for w in (None, ws, ws):
        got = M.moe_adapter_linear(*args, workspace=w, stream=s)
        s.synchronize()
        assert torch.equal(got, want)


def test_adapter_linear_after_the_kernel_that_writes_x():
    # x and the ids are written by kernels right before, on the same stream
    M = load_lib()
    for T in (16, 700):
        d = _data(8, T, 4096, 256, 16, 8, "bf16", "mixed")
        want = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"], out_dtype=torch.float32)
        w1 = torch.ones(4096, device="cuda")
        for _ in range(20):
            x = torch.zeros_like(d["x"])
            ids = torch.full_like(d["ids"], -1)
            out = torch.zeros_like(want)
            torch.cuda._sleep(20000)
            ids.copy_(d["ids"])
            x.copy_(d["x"])
            M.moe_adapter_linear(x, d["W"], d["A"], d["B"], ids, d["c"], out=out)
            x.zero_()
            ids.fill_(-1)
            assert torch.equal(out, want)
        h = M.moe_block_norm(d["x"], next_weight=w1)[1]
        assert torch.isfinite(M.moe_adapter_linear(h, d["W"], d["A"], d["B"], d["ids"], d["c"])).all()


def test_adapter_linear_empty_batch():
    M = load_lib()
    d = _data(9, 2, 64, 48, 8, 2, "bf16", "mixed")
    assert M.moe_adapter_linear(d["x"][:0], d["W"], d["A"], d["B"], d["ids"][:0], d["c"]).shape == (0, 48)


# small batches' tiles of tokens that share an adapter: an adapter a token, a few tokens of each, all of
# one; ranks of one and four 32-wide steps; H small enough that no cluster splits it, and in a cluster
@pytest.mark.parametrize("T,H,N,R,n", [(128, 64, 130, 128, 200), (128, 2048, 256, 104, 16), (97, 128, 1000, 8, 13),
                                       (24, 1024, 96, 32, 2), (520, 256, 1100, 56, 5)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("ids", ["mixed", "runs", 0])
def test_adapter_linear_tiles_of_an_adapter(T, H, N, R, n, dtype, out, ids):
    M = load_lib()
    _check(M, _data(T + R, T, H, N, R, n, dtype, ids), dtype, out, rows=130)


def test_adapter_linear_results_do_not_depend_on_the_neighbours():
    # a token's result is that of its own adapter, in whatever order the batch names them
    M = load_lib()
    d = _data(9, 100, 512, 300, 24, 6, "bf16", "mixed")
    a = M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"])
    order = torch.randperm(100, device="cuda")
    b = M.moe_adapter_linear(d["x"][order].contiguous(), d["W"], d["A"], d["B"], d["ids"][order].contiguous(), d["c"])
    assert torch.equal(b, a[order])
