"""The layer runner with a Routing."""
import numpy as np
import pytest
import torch

from oracle import block as O
from oracle import formats as F
from oracle.mlp import moe_layer
from synth import configs, gen
from tests.helpers import load_lib, pinned_fp4_bank

pytestmark = pytest.mark.gpu

TOL = 2e-2   # of a row's root mean square, as for the layer


def _runner(M, wl, routing, **kw):
    bank, B = pinned_fp4_bank(wl, (0,))
    slots = torch.empty(wl.S * B, dtype=torch.uint8, device="cuda")
    cache = M.moe_cache(wl.S, 1, wl.E, B, slots, bank)
    views = M.make_views(wl.H, wl.I, slots, wl.S)
    runner = M.DecodeLayerRunner(cache, views, wl.E, wl.k, wl.T, routing=routing, **kw)

    def expert(e, tag):
        return F.decode_fp4_expert(bank.numpy()[e * B:(e + 1) * B], wl.H, wl.I)
    return cache, slots, runner, expert


def _run(runner, wl, lg, x):
    y = torch.empty((wl.T, wl.H), dtype=torch.int16, device="cuda")
    runner.run(0, torch.from_numpy(lg).cuda(), torch.from_numpy(x.view(np.int16)).cuda(), y)
    runner.synchronize()
    return F.bf16_to_f64(y.cpu().numpy().view(np.uint16))


def _off(got, ref):
    rms = np.sqrt((ref ** 2).mean(1, keepdims=True))
    return np.max(np.abs(got - ref) / np.where(rms == 0, 1, rms))


@pytest.mark.parametrize("kw", [dict(copy="engine"), dict(copy="device"), dict(copy="device", graph=True),
                                dict(copy="device", overlap=True)])
@pytest.mark.parametrize("T", [1, 5])
def test_tokens_with_fewer_experts_than_k(kw, T):
    # ids of -1 take part in nothing, whatever the slots that the places of these ids had in the call before
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=16, k=4, S=20, T=T)
    cache, slots, runner, expert = _runner(M, wl, M.Routing(), **kw)
    for step in range(4):
        lg, x = gen.router_logits(wl, 0, step), gen.activations(wl, 0, step)
        if step % 2:
            for t in range(T):
                lg[t, np.argsort(-lg[t], kind="stable")[1 + t % 2:]] = -np.inf   # one or two experts left
            if T > 2:
                lg[2] = np.nan                      # and none
            # what no expert of this step is copied to holds codes that decode to NaN
            cache.reset()
            slots.fill_(255)
        got = _run(runner, wl, lg, x)
        ids, w, _ = O.route(lg, 4, "sigmoid")
        assert (ids < 0).any() == bool(step % 2)
        assert np.isfinite(got).all()
        assert _off(got, moe_layer(x, ids, w, expert)) <= TOL
    cache.close()


def _ladder(M, wl, routing, copy):
    bank4, B4 = pinned_fp4_bank(wl, (0,))
    B2 = M.moe_int2_expert_bytes(wl.H, wl.I)
    bank2 = torch.empty(wl.E * B2, dtype=torch.uint8, pin_memory=True)
    for e in range(wl.E):
        bank2[e * B2:(e + 1) * B2] = torch.from_numpy(gen.int2_expert(wl, 0, e))
    s4 = torch.empty(wl.S * B4, dtype=torch.uint8, device="cuda")
    s2 = torch.empty(wl.S2 * B2, dtype=torch.uint8, device="cuda")
    c4, c2 = M.moe_cache(wl.S, 1, wl.E, B4, s4, bank4), M.moe_cache(wl.S2, 1, wl.E, B2, s2, bank2)
    views = M.make_views(wl.H, wl.I, s4, wl.S, s2, wl.S2, None)
    runner = M.DecodeLayerRunner(c4, views, wl.E, wl.k, wl.T, int2_cache=c2, ladder=wl.ladder, copy=copy,
                                 routing=routing)
    return runner, (c4, c2)


@pytest.mark.parametrize("copy,S", [("engine", 20), ("engine", 6), ("device", 20)])
def test_ladder_keeps_the_routings_scale(copy, S):
    # the survivors' weights sum to the scale, as the chosen experts' do without a ladder
    M = load_lib()
    wl = configs.scaled(configs.LADDER, H=256, I=128, T=8, S=S, S2=30)
    out = []
    for scale in (1.0, 2.5):
        runner, caches = _ladder(M, wl, M.Routing(scale=scale), copy)
        out.append([_run(runner, wl, gen.router_logits(wl, 0, step), gen.activations(wl, 0, step))
                    for step in range(3)])
        for c in caches:
            c.close()
    for one, more in zip(*out):
        # two roundings to bf16, of values 2.5 apart
        assert np.abs(one).max() > 0 and np.all(np.abs(more - 2.5 * one) <= 2.0 ** -8 * (np.abs(more) + 2.5 * np.abs(one)))


def test_ladder_refuses_weights_that_are_not_renormalised():
    M = load_lib()
    wl = configs.scaled(configs.LADDER, H=256, I=128, T=8, S=20, S2=30)
    with pytest.raises(ValueError, match="renorm"):
        _ladder(M, wl, M.Routing(renorm=False), "device")
    runner, caches = _ladder(M, wl, None, "device")
    with pytest.raises(ValueError, match="renorm"):
        runner.routing = M.Routing(renorm=False)
    for c in caches:
        c.close()


def test_ladder_of_weights_that_are_all_zero():
    # sigmoids that all underflow weigh nothing; a row's weights are then 0 and not 0 / 0
    M = load_lib()
    wl = configs.scaled(configs.LADDER, H=256, I=128, T=8, S=20, S2=30)
    runner, caches = _ladder(M, wl, M.Routing(), "device")
    lg = gen.router_logits(wl, 0, 0)
    lg[3] -= 200
    got = _run(runner, wl, lg, gen.activations(wl, 0, 0))
    assert np.isfinite(got).all() and (got[3] == 0).all() and (got[[0, 1, 2, 4, 5, 6, 7]] != 0).any(1).all()
    for c in caches:
        c.close()


@pytest.mark.parametrize("graph", [False, True])
def test_routing_that_changes_between_calls(graph):
    # a bias moved in place, a bias put in another's place, another count, another routing
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=16, k=4, S=20, T=5)
    rng = np.random.default_rng(0)

    def bias():
        return torch.from_numpy(np.round(rng.standard_normal(16) * 400).astype(np.float32) * 1e-3).cuda()
    biases = [bias()]
    load = torch.zeros(1, 16, dtype=torch.int32, device="cuda")
    cache, _, runner, expert = _runner(M, wl, M.Routing(bias=biases, scale=1.5, load=load), copy="device", graph=graph)
    lg, x = gen.router_logits(wl, 0, 0), gen.activations(wl, 0, 0)
    old, counted, steps = [], 0, []

    def step(score="sigmoid", b=None, scale=1.5):
        got = _run(runner, wl, lg, x)
        ids, w, margin = O.route(lg, 4, score, b, 1, 1, "top2", True, scale)
        assert margin.min() > 4e-6
        steps.append((np.array_equal(runner.ids.cpu().numpy(), ids), _off(got, moe_layer(x, ids, w, expert)) <= TOL))
    for i in range(3):
        step(b=biases[0].cpu().numpy())
    biases[0].copy_(bias())
    step(b=biases[0].cpu().numpy())
    old.append(biases[0])            # held here: what is replaced is not freed in this test
    biases[0] = bias()
    step(b=biases[0].cpu().numpy())
    step(b=biases[0].cpu().numpy())
    counts = int(load.sum())
    runner.routing = M.Routing(score=M.MOE_SCORE_SOFTMAX)
    step("softmax", None, 1.0)
    step("softmax", None, 1.0)
    assert all(a and b for a, b in steps), steps
    assert counts == 6 * 5 * 4 and int(load.sum()) == counts
    assert len(runner.graphs) == int(graph)
    cache.close()


def test_streamed_prefill_of_tokens_with_fewer_experts_than_k():
    # padding is masked by logits of NaN or -inf: such a token takes part in nothing and its output is 0
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=8, k=3, T=40, H=512, I=512)   # the grouped GEMM takes multiples of 512
    bank, B = pinned_fp4_bank(wl, (0,))
    ps = M.PrefillStreamer(bank, 1, 8, wl.H, wl.I, 3, 40, routing=M.Routing(scale=2.5))
    ps.begin()
    lg, x = gen.router_logits(wl, 0, 0, 40), gen.activations(wl, 0, 0, 40)
    lg[::3] = np.nan
    lg[1::6, 1:] = -np.inf
    y = torch.full((40, wl.H), -1, dtype=torch.int16, device="cuda")
    ps.run_layer(0, torch.from_numpy(lg).cuda(), torch.from_numpy(x.view(np.int16)).cuda(), y)
    ps.synchronize()
    ids, w, _ = O.route(lg, 3, "sigmoid", scale=2.5)
    ref = moe_layer(x, ids, w, lambda e, tag: F.decode_fp4_expert(bank.numpy()[e * B:(e + 1) * B], wl.H, wl.I))
    got = F.bf16_to_f64(y.cpu().numpy().view(np.uint16))
    assert (got[::3] == 0).all() and _off(got, ref) <= TOL
