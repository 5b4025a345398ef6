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
