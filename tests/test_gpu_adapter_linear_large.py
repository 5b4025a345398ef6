"""moe_adapter_linear's large batches (the persistent kernel) for what the small ones are tested for, and the
accuracy of what an adapter adds.

Tolerances of single elements are those of test_gpu_adapter_linear.py.  In the 2-norm, for fp32 results of normal
data: a tensor-core step of 16 products cuts the accumulator's sum off at 24 bits, by 2^-24 of it on average and
always towards zero.  Over the 32 steps of 512 products, the sum growing as their root, that is at most 2/3 x 32 x
2^-24 = 1.3e-6 of an accumulator's sum, and of the whole as much (the accumulators are added in fp32).  What an
adapter adds takes that from A x, and 2^-22 from A x's terms and the few steps of the second product: 1.6e-6."""
import pytest
import torch

from tests.helpers import load_lib
from tests.test_gpu_adapter_linear import DT, _check, _data

pytestmark = pytest.mark.gpu

# 11 x 16 tiles of 128 x 128: past the SMs, so the persistent kernel for results of either kind
T, N = 1300, 2048


def _call(M, d, kind, **kw):
    return M.moe_adapter_linear(d["x"], d["W"], d["A"], d["B"], d["ids"], d["c"], out_dtype=DT[kind], **kw)


@pytest.mark.parametrize("T", [40, 1300])
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("ids", ["runs", 0])
@pytest.mark.parametrize("by", [1e-2, 1e-3, 1e-5])
def test_adapter_linear_f16_below_its_range(T, out, ids, by):
    # A x near and below fp16's smallest steps, brought back by B
    M = load_lib()
    d = _data(12, T, 256, N, 16, 3, "f16", ids)
    d["A"] = (d["A"].float() * by).to(torch.float16)
    d["B"] = (d["B"].float() * min(1 / by, 1e4)).to(torch.float16)
    _check(M, d, "f16", out, rows=150)


def test_adapter_linear_f16_small_and_ordinary_tokens_side_by_side():
    # one group of 16 holds a token of tiny A x, one of none (x = 0) and ordinary ones
    M = load_lib()
    d = _data(13, T, 256, N, 16, 3, "f16", 0)
    d["B"] = (d["B"].float() * 1e3).to(torch.float16)
    d["x"][5::16] *= 2.0 ** -12
    d["x"][6::16] = 0
    _check(M, d, "f16", "f32", rows=400)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_nan_stays_with_its_adapter_large(out, ids):
    M = load_lib()
    d = _data(4, T, 256, N, 16, 4, "bf16", ids)
    want = _call(M, d, out)
    d["A"][1] = float("nan")
    d["B"][2] = float("inf")
    got = _call(M, d, out)
    ok = (d["ids"] != 1) & (d["ids"] != 2)
    assert torch.equal(got[ok], want[ok]) and torch.isnan(got[d["ids"] == 1]).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_reports_an_id_out_of_range_large(out, ids):
    M = load_lib()
    d = _data(6, T, 256, N, 8, 3, "bf16", ids)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = _call(M, d, out, d_error=err)
    assert int(err) == M.MOE_OK
    bad = d["ids"].clone()
    bad[T // 2] = 3
    got = _call(M, dict(d, ids=bad), out, d_error=err)
    assert int(err) == M.MOE_ERR_INVALID
    none = bad.clone()
    none[T // 2] = -1
    assert torch.equal(got, _call(M, dict(d, ids=none), out))
    away = torch.arange(T, device="cuda") // 16 != T // 2 // 16   # its group is taken in another way
    assert torch.equal(got[away], good[away])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_strides_large(out, ids):
    M = load_lib()
    d = _data(5, T, 320, N, 16, 3, "bf16", ids, 16, 8)
    want = _check(M, dict(d, x=d["x"].contiguous()), "bf16", out, rows=40)
    wide_w = torch.zeros(N, 352, dtype=torch.bfloat16, device="cuda")
    wide_w[:, 16:336] = d["W"]
    wide = torch.full((T, N + 11), 3.0, dtype=DT[out], device="cuda")
    M.moe_adapter_linear(d["x"], wide_w[:, 16:336], d["A"], d["B"], d["ids"], d["c"], out=wide[:, 7:N + 7])
    assert torch.equal(wide[:, 7:N + 7], want)
    assert (wide[:, :7] == 3).all() and (wide[:, N + 7:] == 3).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_on_another_stream_and_repeats_large(out, ids):
    M = load_lib()
    d = _data(7, T, 1024, N, 16, 5, "bf16", ids)
    want = _call(M, d, out)
    s = torch.cuda.Stream()
    ws = torch.full((M.moe_adapter_linear_workspace(T, 1024, N, 5, 16),), 255, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for w in (ws, ws):
        got = torch.full_like(want, float("nan"))
        s.wait_stream(torch.cuda.current_stream())
        _call(M, d, out, out=got, workspace=w, stream=s)
        s.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_adapter_linear_after_the_kernel_that_writes_x_large(out):
    M = load_lib()
    for ids in ("mixed", "runs"):
        d = _data(8, T, 1024, N, 16, 8, "bf16", ids)
        want = _call(M, d, out)
        for _ in range(5):
            late = dict(d, x=torch.zeros_like(d["x"]), ids=torch.full_like(d["ids"], -1))
            got = torch.zeros_like(want)
            torch.cuda._sleep(20000)
            late["ids"].copy_(d["ids"])
            late["x"].copy_(d["x"])
            _call(M, late, out, out=got)
            late["x"].zero_()
            late["ids"].fill_(-1)
            assert torch.equal(got, want)


def _norms(M, d, out):
    """(error of the whole result, error of what the adapters add) in the 2-norm, against 64 bits."""
    f = torch.float64
    x, W = d["x"].to(f), d["W"].to(f)
    low = torch.zeros(x.shape[0], W.shape[0], dtype=f, device="cuda")
    for a in range(d["A"].shape[0]):
        at = d["ids"] == a
        low[at] = float(d["c"][a]) * ((x[at] @ d["A"][a].to(f).T) @ d["B"][a].to(f).T)
    whole = x @ W.T + low
    err = (_call(M, d, out).to(f) - whole).norm()
    return float(err / whole.norm()), float(err / low.norm())


@pytest.mark.parametrize("T,N", [(16, 256), (100, 640), (300, 640), (1300, 640), (1300, 2048), (16400, 100)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_accuracy_in_fp32(T, N, dtype, ids):
    M = load_lib()
    d = _data(T, T, 4096, N, 16, 4, dtype, ids)
    assert _norms(M, d, "f32")[0] <= 1.6e-6
    # what the adapters add by itself: no other term hides its error
    d["W"].zero_()
    assert _norms(M, d, "f32")[1] <= 1.6e-6


@pytest.mark.parametrize("T", [5, 100, 1300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_adapter_linear_bits_of_a_x(T, dtype, ids):
    """A picks single elements of x and B single ranks, by 1: a result is c x[j], whose product is rounded to fp32
    (2^-24), cut to the terms' bits (none of bf16's 24; of f16's two 2^-22 of the token's largest) and added up from
    them (2^-23)."""
    M = load_lib()
    d = _data(T, T, 256, N, 16, 4, dtype, ids)
    for m in ("W", "A", "B"):
        d[m].zero_()
    pick = torch.randint(0, 256, (4, 16), device="cuda")
    d["A"].scatter_(2, pick[..., None], 1.0)
    rank = torch.arange(N, device="cuda") % 16
    d["B"][:, torch.arange(N, device="cuda"), rank] = 1.0
    got = _call(M, d, "f32").double()
    a = d["ids"].long().clamp(min=0)
    ref = torch.where(d["ids"][:, None] >= 0, d["c"].double()[a][:, None] * d["x"].double().gather(1, pick[a])[:, rank], 0.0)
    tol = 2.0 ** -22 * ref.abs()
    if dtype == "f16":
        tol = tol + 2.0 ** -22 * ref.abs().amax(1, keepdim=True)
    assert torch.all((got - ref).abs() <= tol)
