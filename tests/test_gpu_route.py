"""moe_route and its gradient against the fp64 oracle.

Ids are compared bit for bit on the rows whose choice fp32 can settle: a key is
off by at most 4 roundings of a value below 2 plus the 2 ulp of expf, so rows
where two unequal values that the choice hangs on lie within 4e-6 are left out
(and are few).  Weights and gradients: the exponent's argument is rounded
(|z - max| < 32: 2^-20 of the value), expf is off by 2 ulp, sums of up to 32
terms and the divisions by a few more: 4e-6 of the value bounds them, and a
gradient's difference g_j - sum q g carries that of its terms."""
import numpy as np
import pytest
import torch

from oracle import block as O
from tests.helpers import load_lib

pytestmark = pytest.mark.gpu

GAP, REL = 4e-6, 4e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _codes(M, score, group="top2"):
    return (M.MOE_SCORE_SIGMOID if score == "sigmoid" else M.MOE_SCORE_SOFTMAX,
            M.MOE_GROUP_TOP2 if group == "top2" else M.MOE_GROUP_MAX)


def _check(M, lg, k, score="softmax", bias=None, G=1, tg=1, group="top2", renorm=True, scale=1.0, mask=None,
           load=False, settled=True):
    """lg: a CUDA tensor [T, E] of any type, rows strided or not."""
    T, E = lg.shape
    sc, gr = _codes(M, score, group)
    cnt = torch.zeros(E, dtype=torch.int32, device="cuda") if load else None
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    m = None if mask is None else torch.from_numpy(mask).cuda()
    ids, w = M.moe_route(lg, k, sc, b, G, tg, gr, renorm, scale, m, load=cnt)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    rid, rw, margin = O.route(lg.double().cpu().numpy(), k, score, None if bias is None else bias.astype(np.float32),
                              G, tg, group, renorm, scale, mask)
    ok = margin > GAP
    assert not settled or (~ok).sum() <= max(1, T // 50)
    assert np.array_equal(ids[ok], rid[ok])
    assert np.all(np.abs(w[ok] - rw[ok]) <= REL * np.abs(rw[ok]) + 1e-30)
    assert np.all(w[ids < 0] == 0)
    if load:
        assert np.array_equal(cnt.cpu().numpy(), np.bincount(ids[ids >= 0], minlength=E))
    return ids, w


@pytest.mark.parametrize("T,E,k,G,tg", [(1, 256, 8, 8, 4), (64, 256, 8, 8, 4), (257, 256, 6, 1, 1), (33, 160, 6, 8, 3),
                                        (5, 8, 2, 4, 2), (9, 1, 1, 1, 1), (7, 24, 5, 3, 2), (130, 300, 7, 10, 5),
                                        (3, 2048, 32, 32, 7), (40, 1024, 8, 16, 2), (11, 61, 4, 1, 1),
                                        (19, 64, 3, 32, 3), (6, 512, 12, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_matches_oracle(T, E, k, G, tg, score, biased):
    M = load_lib()
    rng = np.random.default_rng(T * 31 + E + G + biased)
    lg = torch.from_numpy((rng.standard_normal((T, E)) * 1.5).astype(np.float32)).cuda()
    bias = np.round(rng.standard_normal(E) * 40) * 1e-3 if biased else None
    k = min(k, tg * (E // G))
    for group in ("max", "top2"):
        for renorm in (True, False):
            _check(M, lg, k, score, bias, G, tg, group, renorm, 2.5, load=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 3), (8, 8), (4, 0)])
def test_route_types_strides_and_alignment(dtype, offset, pad):
    M = load_lib()
    rng = np.random.default_rng(5)
    T, E = 37, 96
    wide = torch.from_numpy(rng.standard_normal((T, E + offset + pad)).astype(np.float32)).cuda().to(DT[dtype])
    lg = wide[:, offset:offset + E]
    _check(M, lg, 6, "sigmoid", np.round(rng.standard_normal(E) * 40) * 1e-3, 6, 3)
    _check(M, lg, 6, "softmax", None, 4, 2)
    sc, _ = _codes(M, "softmax")
    bits = wide.view(torch.int16)[:, offset:offset + E] if dtype == "bf16" else lg   # bf16 bits
    assert torch.equal(M.moe_route(bits, 6, sc)[0], M.moe_route(lg, 6, sc)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_id(score):
    M = load_lib()
    rng = np.random.default_rng(6)
    lg = torch.from_numpy(rng.integers(-2, 3, size=(200, 64)).astype(np.float32)).cuda()
    _check(M, lg, 8, score)
    _check(M, lg, 8, score, np.zeros(64), 8, 4)
    _check(M, lg, 8, score, None, 8, 4, "max")
    _check(M, torch.zeros(5, 100, device="cuda"), 9, score, None, 10, 3)
    z = torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda")
    assert _check(M, z, 3, score)[0].tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks_infinities_and_nan(score, renorm):
    M = load_lib()
    inf, nan, low = np.inf, np.nan, float(np.finfo(np.float32).min)
    rows = np.random.default_rng(7).standard_normal((12, 40)).astype(np.float32)
    rows[0] = -inf                       # nothing is left
    rows[1] = nan
    rows[2] = -inf
    rows[2, 17] = 0.25                   # one expert is left
    rows[3, :30] = low                   # the type's lowest value: eligible, score 0
    rows[4] = low
    rows[5, ::2] = nan
    rows[6, 3] = rows[6, 30] = inf       # +inf: both equal, above all others
    rows[7, :38] = -inf                  # fewer than k
    rows[8] = 200.0                      # the sigmoid saturates
    rows[9] = -200.0                     # the sigmoid underflows
    rows[10] = nan
    mask = np.ones(12, dtype=np.uint8)
    mask[10] = mask[11] = 0
    lg = torch.from_numpy(rows).cuda()
    b = np.round(np.random.default_rng(8).standard_normal(40) * 40) * 1e-3
    for bias, G, tg in ((None, 1, 1), (b, 1, 1), (b, 8, 3), (None, 8, 3)):
        for group in ("max", "top2"):
            ids, w = _check(M, lg, 5, score, bias, G, tg, group, renorm, mask=mask, load=True, settled=False)
            assert np.isfinite(w).all() and (ids[[0, 1, 10, 11]] == -1).all()
            assert ids[2].tolist() == [17, -1, -1, -1, -1]


def test_route_repeats_and_counts_over_calls():
    M = load_lib()
    lg = torch.randn(5000, 256, device="cuda")
    cnt = torch.zeros(256, dtype=torch.int32, device="cuda")
    a, wa = M.moe_route(lg, 8, load=cnt)
    b, wb = M.moe_route(lg, 8, load=cnt)
    assert torch.equal(a, b) and torch.equal(wa, wb)
    assert torch.equal(cnt.cpu(), 2 * torch.bincount(a.flatten().cpu(), minlength=256).to(torch.int32))
    old = M.moe_router_topk(lg, 8)
    assert torch.equal(a, old[0]) and (wa - old[1]).abs().max() <= 1e-6


def test_route_on_another_stream():
    M = load_lib()
    s = torch.cuda.Stream()
    lg = torch.randn(300, 256, device="cuda")
    ref = M.moe_route(lg, 8, M.MOE_SCORE_SIGMOID)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = lg * 1.0
    got = M.moe_route(late, 8, M.MOE_SCORE_SIGMOID, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_route_long_batch_offsets():
    # 8.4 M rows of 256 bf16 logits in a 300-wide buffer: offsets past 32 bits, every tile of the grid used
    M = load_lib()
    T, E = (1 << 23) + 5, 256
    wide = torch.empty(T, 300, dtype=torch.bfloat16, device="cuda")
    probe = torch.randn(64, E, device="cuda").to(torch.bfloat16)
    wide[:, :E] = probe.repeat((T + 63) // 64, 1)[:T]
    ids, w = M.moe_route(wide[:, :E], 4)
    rid, rw = M.moe_route(probe, 4)
    assert torch.equal(ids[-64:], rid.roll(-(T % 64), 0)) and torch.equal(ids[:64], rid)
    assert torch.equal(w[-64:], rw.roll(-(T % 64), 0))


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (65, 256, 6), (9, 300, 7), (3, 2048, 32), (31, 61, 4), (4, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_gradient_matches_oracle(T, E, k, score, renorm, dtype):
    M = load_lib()
    rng = np.random.default_rng(T + E + k)
    lg = torch.from_numpy((rng.standard_normal((T, E + 8)) * 1.5).astype(np.float32)).cuda().to(DT[dtype])[:, :E]
    if T > 2 and E > 8:
        lg[1, 5] = -np.inf
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    mask = np.ones(T, np.uint8)
    if T > 3:
        ids[2, k // 2:] = -1
        mask[3] = 0
    dw = rng.standard_normal((T, k)).astype(np.float32)
    sc, _ = _codes(M, score)
    d = M.moe_route_backward(lg, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), sc, renorm, 2.5,
                             torch.from_numpy(mask).cuda())
    assert d.dtype == lg.dtype
    ref = O.route_backward(lg.double().cpu().numpy(), ids, dw, score, renorm, 2.5, mask)
    # each value is scale * (at most 1) * a difference of terms of the size of the largest |dw|
    tol = 8 * REL * 2.5 * np.abs(dw).max(1, keepdims=True) + ULP[dtype] * np.abs(ref)
    if dtype == "f16":
        tol = tol + 2.0 ** -25      # half of fp16's smallest step
    assert np.all(np.abs(d.double().cpu().numpy() - ref) <= tol)
    assert np.all(d.double().cpu().numpy()[mask == 0] == 0)


def test_route_gradient_rows_without_experts():
    M = load_lib()
    lg = torch.full((3, 16), -float("inf"), device="cuda")
    lg[2] = float("nan")
    ids = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    ids[1] = torch.tensor([3, 99, -7, 4])      # names no eligible expert
    dw = torch.full((3, 4), float("nan"), device="cuda")
    for sc in (M.MOE_SCORE_SOFTMAX, M.MOE_SCORE_SIGMOID):
        for renorm in (True, False):
            d = M.moe_route_backward(lg, ids, dw, sc, renorm)
            assert torch.equal(d, torch.zeros_like(d))


def test_route_gradient_strided_and_of_the_routes_own_choice():
    M = load_lib()
    lg = torch.randn(70, 256, device="cuda")
    ids, w = M.moe_route(lg, 8, M.MOE_SCORE_SIGMOID, scale=2.5)
    dw = torch.randn(70, 8, device="cuda")
    d = M.moe_route_backward(lg, ids, dw, M.MOE_SCORE_SIGMOID, scale=2.5)
    wide = torch.full((70, 300), 7.0, device="cuda")
    M.moe_route_backward(lg, ids, dw, M.MOE_SCORE_SIGMOID, scale=2.5, d_logits=wide[:, 5:261])
    assert torch.equal(wide[:, 5:261], d) and (wide[:, :5] == 7).all() and (wide[:, 261:] == 7).all()
    # renormalised weights sum to the scale whatever the logits' common factor: sum d * 0 moves nothing,
    # and moving along d raises sum dw w by |d|^2
    step = 1e-3
    up = M.moe_route(lg + step * d, 8, M.MOE_SCORE_SIGMOID, scale=2.5)
    same = (up[0] == ids).all(1)
    gain = ((up[1] - w) * dw)[same].double().sum()
    want = step * d[same].double().square().sum()
    assert same.float().mean() > 0.9 and abs(gain - want) <= 0.05 * want


def test_route_empty_batch():
    M = load_lib()
    lg = torch.empty(0, 16, device="cuda")
    ids, w = M.moe_route(lg, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert M.moe_route_backward(lg, ids, w).shape == (0, 16)


@pytest.mark.parametrize("E", [33, 700, 1003, 2047])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_gradient_of_plain_softmax_whatever_the_rows_start(E, dtype):
    # rows that start anywhere take another order of the experts than those on 16-byte boundaries
    M = load_lib()
    rng = np.random.default_rng(E)
    T, k = 21, 5
    wide = torch.from_numpy((rng.standard_normal((T, E + 4)) * 1.5).astype(np.float32)).cuda().to(DT[dtype])
    lg = wide[:, 3:E + 3]
    lg[4, 1:] = -np.inf
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[4] = [0, -1, -1, -1, -1]
    dw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.full((T, E + 6), 7.0, dtype=DT[dtype], device="cuda")
    M.moe_route_backward(lg, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), M.MOE_SCORE_SOFTMAX, False, 2.5,
                         d_logits=out[:, 5:E + 5])
    assert (out[:, :5] == 7).all() and (out[:, E + 5:] == 7).all()
    ref = O.route_backward(lg.double().cpu().numpy(), ids, dw, "softmax", False, 2.5)
    tol = 8 * REL * 2.5 * np.abs(dw).max(1, keepdims=True) + ULP[dtype] * np.abs(ref)
    if dtype == "f16":
        tol = tol + 2.0 ** -25
    assert np.all(np.abs(out[:, 5:E + 5].double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("E,G,tg", [(764, 1, 1), (1003, 1, 1), (2046, 6, 2), (700, 7, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_many_experts_with_bias(E, G, tg, score):
    M = load_lib()
    rng = np.random.default_rng(E)
    wide = torch.from_numpy((rng.standard_normal((23, E + 1)) * 1.5).astype(np.float32)).cuda()
    bias = np.round(rng.standard_normal(E) * 40) * 1e-3
    for lg in (wide[:, :E], wide[:, 1:], wide[:, :E].contiguous()):
        lg = lg.clone() if lg.is_contiguous() else lg
        for load in (True, False):
            _check(M, lg, 9, score, bias, G, tg, load=load)
