"""moe_block_norm and its gradient against the fp64 oracle.

Tolerances: an output is rounded once to its type (half an ulp: 2^-8 of the
value for bf16, 2^-11 for f16, 2^-24 for fp32).  Before that fp32 carries a sum
of H squares in parallel partial sums (at most 16 terms a thread, then a tree:
below 40 roundings of 2^-24), a root, a division and a few products: 2^-18 of
the magnitudes of the terms that the value is the sum of (the oracle gives
them; a norm's gradient cancels) and of the row's mean bounds it.  Sums over T
tokens add T such terms in fp32: (T + 64) 2^-24 more of their magnitudes."""
import numpy as np
import pytest
import torch

from oracle import block as O
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
F32 = 2.0 ** -18


def _close(got, ref, dtype, what, size=None):
    g = got.double().cpu().numpy()
    size = np.abs(ref) if size is None else size
    scale = np.sqrt((size ** 2).mean(axis=-1, keepdims=True)) + size
    tol = ULP[dtype] * np.abs(ref) + F32 * scale + (2.0 ** -25 if dtype == "f16" else 0)
    assert np.isfinite(g).all(), what
    assert np.all(np.abs(g - ref) <= tol), (what, np.max(np.abs(g - ref) / tol))


def _rand(rng, shape, dtype, by=1.0, pad=0, offset=0):
    full = (rng.standard_normal(shape[:-1] + (shape[-1] + pad + offset,)) * by).astype(np.float32)
    return torch.from_numpy(full).cuda().to(DT[dtype])[..., offset:offset + shape[-1]]


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(rng, T, H, x, y, w, post, gate, nxt, pad=0, offset=0):
    p = dict(x=_rand(rng, (T, H), x, 2.0, pad, offset), y=_rand(rng, (T, H), y, 0.3, pad, offset))
    p["post"] = (1 + _rand(rng, (H,), "f32", 0.1)).to(DT[w]) if post else None
    p["gate"] = {None: None, "channel": _rand(rng, (H,), w, 0.5), "token": _rand(rng, (T, 1), w, 0.5)}[gate]
    p["nxt"] = (1 + _rand(rng, (H,), "f32", 0.1)).to(DT[w]) if nxt else None
    p["du"] = _rand(rng, (T, H), x, 0.02, pad, offset)
    p["dh"] = _rand(rng, (T, H), y, 0.02, pad, offset) if nxt else None
    return p


def _both(M, p, x, y, alpha=1.0, eps=1e-6, du=True):
    xo, h = M.moe_block_norm(p["x"], p["y"], p["post"], p["gate"], alpha, p["nxt"], eps)
    ru, rh = O.block_norm(_np(p["x"]), _np(p["y"]), _np(p["post"]), _np(p["gate"]), alpha, _np(p["nxt"]), eps)
    _close(xo, ru, x, "x_out")
    if rh is not None:
        _close(h, rh, y, "h")
    d_u = p["du"] if du else None
    dx, dy, dp, dg, dn = M.moe_block_norm_backward(p["x"], p["y"], d_u, p["dh"], p["post"], p["gate"], alpha,
                                                   p["nxt"], eps)
    ref, mag = O.block_norm_backward(_np(p["x"]), _np(p["y"]), _np(d_u), _np(p["dh"]), _np(p["post"]),
                                     _np(p["gate"]), alpha, _np(p["nxt"]), eps)
    _close(dx, ref["x"], x, "d_x", mag["x"])
    _close(dy, ref["y"], y, "d_y", mag["y"])
    T = p["x"].shape[0]
    for got, name in ((dp, "post"), (dg, "gate"), (dn, "next")):
        assert (got is None) == (name not in ref), name
        if got is not None:
            n = T if got.dim() == 1 else p["x"].shape[1] // 32
            tol = ((n + 64) * 2.0 ** -24 + F32) * mag[name] + 1e-30
            assert np.all(np.abs(_np(got) - ref[name]) <= tol), (name, np.max(np.abs(_np(got) - ref[name]) / tol))
    return xo, h, dx, dy, dp, dg, dn


@pytest.mark.parametrize("T,H", [(1, 4096), (16, 4096), (333, 4096), (5, 8), (3, 1), (7, 33), (40, 256), (700, 128),
                                 (9, 264), (21, 1001), (4, 1025), (6, 2048), (11, 7168), (2, 8200), (3, 16384),
                                 (2, 16383), (17, 520)])
@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f16"), ("f32", "f16")])
def test_block_norm_matches_oracle(T, H, x, y):
    M = load_lib()
    p = _inputs(np.random.default_rng(T + H), T, H, x, y, "f32", True, "channel", True)
    _both(M, p, x, y, 0.5)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("nxt", [True, False])
@pytest.mark.parametrize("H", [512, 1003])
def test_block_norm_parts(post, gate, nxt, H):
    M = load_lib()
    for w in ("f32", "bf16", "f16"):
        p = _inputs(np.random.default_rng(H), 45, H, "bf16", "bf16", w, post, gate, nxt)
        _both(M, p, "bf16", "bf16", 0.7)
        if nxt:
            _both(M, p, "bf16", "bf16", 1.0, du=False)


@pytest.mark.parametrize("offset,pad", [(0, 8), (8, 8), (1, 0), (0, 3), (4, 4)])
def test_block_norm_strides_and_alignment(offset, pad):
    M = load_lib()
    for x, y in (("bf16", "bf16"), ("f32", "bf16")):
        p = _inputs(np.random.default_rng(9), 19, 640, x, y, "f32", True, "channel", True, pad, offset)
        _both(M, p, x, y)
        dense = {m: None if v is None else v.contiguous() for m, v in p.items()}
        _both(M, dense, x, y)
        # into strided outputs: only the row's own elements are written
        wide = torch.full((19, 640 + 16), 3.0, device="cuda", dtype=DT[x])
        hide = torch.full((19, 640 + 5), 3.0, device="cuda", dtype=DT[y])
        xo, h = M.moe_block_norm(p["x"], p["y"], p["post"], p["gate"], 1.0, p["nxt"], x_out=wide[:, 8:648],
                                 h=hide[:, 2:642])
        ru, rh = O.block_norm(*[_np(p[m]) for m in ("x", "y", "post", "gate")], 1.0, _np(p["nxt"]))
        _close(xo, ru, x, "strided x_out")
        _close(h, rh, y, "strided h")
        assert (wide[:, :8] == 3).all() and (wide[:, 648:] == 3).all()
        assert (hide[:, :2] == 3).all() and (hide[:, 642:] == 3).all()


def test_block_norm_in_place():
    M = load_lib()
    p = _inputs(np.random.default_rng(10), 50, 4096, "bf16", "bf16", "f32", True, "channel", True)
    xo, h, dx, dy, *_ = _both(M, p, "bf16", "bf16")
    x = p["x"].clone()
    got = M.moe_block_norm(x, p["y"], p["post"], p["gate"], 1.0, p["nxt"], x_out=x)
    assert got[0] is x and torch.equal(x, xo) and torch.equal(got[1], h)
    du, dh = p["du"].clone(), p["dh"].clone()
    M.moe_block_norm_backward(p["x"], p["y"], du, dh, p["post"], p["gate"], 1.0, p["nxt"], d_x=du, d_y=dh)
    assert torch.equal(du, dx) and torch.equal(dh, dy)


@pytest.mark.parametrize("H", [4096, 77])
def test_block_norm_before_a_first_block(H):
    M = load_lib()
    rng = np.random.default_rng(11)
    x, w = _rand(rng, (30, H), "f32", 3.0), 1 + _rand(rng, (H,), "f32", 0.1)
    xo, h = M.moe_block_norm(x, next_weight=w)
    assert xo is None
    _close(h, O.block_norm(_np(x), nxt=_np(w))[1], "f32", "h")
    h16 = torch.empty(30, H, dtype=torch.bfloat16, device="cuda")
    M.moe_block_norm(x, next_weight=w, h=h16)
    _close(h16, O.block_norm(_np(x), nxt=_np(w))[1], "bf16", "h")
    dh = _rand(rng, (30, H), "f32")
    dx, dy, dp, dg, dn = M.moe_block_norm_backward(x, None, None, dh, next_weight=w)
    ref, mag = O.block_norm_backward(_np(x), None, None, _np(dh), nxt=_np(w))
    assert dy is None and dp is None and dg is None
    _close(dx, ref["x"], "f32", "d_x", mag["x"])
    assert np.all(np.abs(_np(dn) - ref["next"]) <= (94 * 2.0 ** -24 + F32) * mag["next"])


def test_block_norm_rows_of_zeros_and_extremes():
    # zeros: n(0) = 0; values near the ends of the types' ranges that fp32 squares can hold
    M = load_lib()
    x = torch.zeros(4, 512, device="cuda")
    y = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    y[1] = 1e-18
    y[2] = 1e17
    x[3], y[3] = 1e15, -1e12
    one = torch.ones(512, device="cuda")
    p = dict(x=x, y=y, post=one, gate=None, nxt=one, du=torch.ones_like(x), dh=torch.ones_like(y))
    xo, h, dx, dy, dp, _, dn = _both(M, p, "f32", "bf16")
    assert (xo[0] == 0).all() and (h[0] == 0).all()


def test_block_norm_nan_stays_in_its_row():
    M = load_lib()
    p = _inputs(np.random.default_rng(12), 9, 1024, "bf16", "bf16", "f32", True, "channel", True)
    want = M.moe_block_norm(p["x"], p["y"], p["post"], p["gate"], 1.0, p["nxt"])
    p["y"][4, 100] = float("nan")
    p["x"][5, 7] = float("inf")
    got = M.moe_block_norm(p["x"], p["y"], p["post"], p["gate"], 1.0, p["nxt"])
    rest = [0, 1, 2, 3, 6, 7, 8]
    for a, b in zip(want, got):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(got[1][4]).all()


def test_block_norm_gradient_repeats_and_takes_a_workspace():
    M = load_lib()
    p = _inputs(np.random.default_rng(13), 3000, 1032, "bf16", "bf16", "f32", True, "channel", True)
    args = (p["x"], p["y"], p["du"], p["dh"], p["post"], p["gate"], 0.5, p["nxt"])
    a = M.moe_block_norm_backward(*args)
    ws = torch.full((M.moe_block_norm_backward_workspace(3000, 1032),), 255, dtype=torch.uint8, device="cuda")
    b = M.moe_block_norm_backward(*args, workspace=ws)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    with pytest.raises(M.MoeError) as e:
        M.moe_block_norm_backward(*args, workspace=ws[:64])
    assert e.value.status == M.MOE_ERR_INVALID


def test_block_norm_on_another_stream():
    M = load_lib()
    p = _inputs(np.random.default_rng(14), 200, 4096, "bf16", "bf16", "f32", True, "channel", True)
    args = (p["x"], p["y"], p["du"], p["dh"], p["post"], p["gate"], 0.5, p["nxt"])
    want = M.moe_block_norm_backward(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [M.moe_block_norm_backward(*args, stream=s) for _ in range(3)][-1]
    s.synchronize()
    for u, v in zip(want, got):
        assert torch.equal(u, v)


def test_block_norm_long_stream_offsets():
    # 2.2e9 elements between the first row and the last: offsets past 32 bits
    M = load_lib()
    T, H, ld = 70000, 64, 1 << 15
    x = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")[:, :H]
    probe = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    x.copy_(probe)
    w = torch.ones(H, device="cuda")
    _, h = M.moe_block_norm(x, probe, w, None, 1.0, w)
    _, ref = M.moe_block_norm(probe, probe, w, None, 1.0, w)
    assert torch.equal(h, ref)
    dx = M.moe_block_norm_backward(x, probe, x, probe, w, None, 1.0, w)[0]
    assert torch.equal(dx, M.moe_block_norm_backward(probe, probe, probe, probe, w, None, 1.0, w)[0])


def test_block_norm_empty_batch():
    M = load_lib()
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    xo, h = M.moe_block_norm(x, x, w, w, 1.0, w)
    assert xo.shape == (0, 64) and h.shape == (0, 64)
    sums = M.moe_block_norm_backward(x, x, x, x, w, w, 1.0, w)[2:]
    for s in sums:      # sums over no tokens
        assert torch.equal(s, torch.zeros(64, device="cuda"))
