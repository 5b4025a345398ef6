"""RoutedBlocks: norms, router projection with adapters, routing, experts and residual run
together, against the fp64 oracle; and the runners with a Routing."""
import numpy as np
import pytest
import torch

from oracle import block as O
from oracle import formats as F
from oracle.mlp import moe_layer
from synth import configs, gen
from tests.helpers import load_lib, pinned_fp4_bank

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _stack(M, wl, layers, copy="device", **routing):
    bank, B = pinned_fp4_bank(wl, range(layers))
    slots = torch.empty(wl.S * B, dtype=torch.uint8, device="cuda")
    cache = M.moe_cache(wl.S, layers, wl.E, B, slots, bank)
    views = M.make_views(wl.H, wl.I, slots, wl.S)
    r = M.Routing(**routing) if routing else None
    return bank, B, cache, M.DecodeLayerRunner(cache, views, wl.E, wl.k, wl.T, copy=copy, routing=r)


@pytest.mark.parametrize("copy", ["engine", "device"])
def test_runner_routing_is_the_oracles(copy):
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=16, k=4, S=20, T=5)
    bias = torch.from_numpy(np.round(np.random.default_rng(0).standard_normal(16) * 40).astype(np.float32) * 1e-3)
    load = torch.zeros(2, 16, dtype=torch.int32, device="cuda")
    bank, B, cache, runner = _stack(M, wl, 2, copy, score=M.MOE_SCORE_SIGMOID, bias=[bias.cuda(), None], n_group=4,
                                    topk_group=2, scale=1.5, load=load)
    for step in range(3):
        for layer in range(2):
            lg, x = gen.router_logits(wl, layer, step), gen.activations(wl, layer, step)
            y = torch.empty((wl.T, wl.H), dtype=torch.int16, device="cuda")
            runner.run(layer, torch.from_numpy(lg).cuda(), torch.from_numpy(x.view(np.int16)).cuda(), y)
            runner.synchronize()
            ids, w, margin = O.route(lg, 4, "sigmoid", bias.numpy() if layer == 0 else None, 4, 2, "top2", True, 1.5)
            assert margin.min() > 4e-6
            ref = moe_layer(x, ids, w, lambda e, tag: F.decode_fp4_expert(
                bank.numpy()[(layer * 16 + e) * B:(layer * 16 + e + 1) * B], wl.H, wl.I))
            got = F.bf16_to_f64(y.cpu().numpy().view(np.uint16))
            assert np.max(np.abs(got - ref) / np.sqrt((ref ** 2).mean(1, keepdims=True))) <= 2e-2
    assert load.sum(1).tolist() == [3 * 5 * 4] * 2
    cache.close()


def test_prefill_streamer_routing_runs_the_choice_it_is_given():
    # with the default's own parameters spelled out, the same bits as the default
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=8, k=2, T=9, H=512, I=512)   # the grouped GEMM takes multiples of 512
    bank, B = pinned_fp4_bank(wl, range(2))
    out = []
    for routing in (None, M.Routing(score=M.MOE_SCORE_SOFTMAX)):
        ps = M.PrefillStreamer(bank, 2, 8, wl.H, wl.I, 2, 9, routing=routing)
        ps.begin()
        for layer in range(2):
            x = torch.from_numpy(gen.activations(wl, layer, 0, 9).view(np.int16)).cuda()
            y = torch.empty((9, wl.H), dtype=torch.int16, device="cuda")
            ps.run_layer(layer, torch.from_numpy(gen.router_logits(wl, layer, 0, 9)).cuda(), x, y)
            ps.synchronize()
            out.append((ps.ids[:9].clone(), y.view(torch.bfloat16).float()))
    for (ia, ya), (ib, yb) in zip(out[:2], out[2:]):
        # the weights may differ by an ulp of fp32, the outputs by one of bf16
        assert torch.equal(ia, ib) and (ya - yb).abs().max() <= 2.0 ** -7 * ya.abs().max()


@pytest.mark.parametrize("stream_type", [torch.float32, torch.bfloat16])
def test_blocks_match_oracle_step_by_step(stream_type):
    """Each block from the GPU's own stream before it (rounding and routing are not carried
    along): the choice, then x within the experts' tolerance of 2e-2 of y's scale."""
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=16, k=4, S=32, T=6)
    layers = 2
    bank, B, cache, runner = _stack(M, wl, layers, score=M.MOE_SCORE_SIGMOID, n_group=4, topk_group=2, scale=1.5)
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*s, by=1.0):
        return torch.randn(*s, device="cuda", generator=g) * by
    H, E = wl.H, wl.E
    blocks = [M.BlockWeights(router=normal(E, H, by=H ** -0.5).bfloat16(), pre=1 + normal(H, by=0.1),
                             post=1 + normal(H, by=0.1), gate=normal(H, by=0.5),
                             lora_a=normal(3, 8, H, by=H ** -0.5).bfloat16(), lora_b=normal(3, E, 8, by=0.3).bfloat16(),
                             lora_scale=0.5 + torch.rand(3, device="cuda", generator=g)) for _ in range(layers)]
    ids = torch.tensor([0, 1, 2, -1, 0, 2], dtype=torch.int32, device="cuda")
    x0 = normal(6, H).to(stream_type)
    x = x0.clone()
    M.RoutedBlocks(runner, blocks, 0.8).run(x, ids)
    ref = _np(x0)
    for i, b in enumerate(blocks):
        one = M.RoutedBlocks(runner, blocks[:i + 1], 0.8)     # the stack up to here, again, for the GPU's stream
        at = x0.clone()
        M.RoutedBlocks(runner, blocks[:i], 0.8).run(at, ids) if i else None
        before = _np(at)
        got = x0.clone()
        one.run(got, ids)
        one.synchronize()
        h = O.block_norm(before, nxt=_np(b.pre))[1]
        h = torch.from_numpy(h).to(torch.bfloat16)            # the experts' input is bf16
        lg, _, _ = O.adapter_linear(_np(h), _np(b.router), _np(b.lora_a), _np(b.lora_b), ids.cpu().numpy(),
                                    _np(b.lora_scale))
        sel, w, margin = O.route(lg, 4, "sigmoid", None, 4, 2, "top2", True, 1.5)
        # h is one bf16 rounding of a value that may lie an ulp off: logits within 2^-8 of their scale
        sure = margin > 2.0 ** -8
        bits = h.view(torch.int16).numpy().view(np.uint16)
        y = moe_layer(bits, sel, w, lambda e, tag: F.decode_fp4_expert(
            bank.numpy()[(i * E + e) * B:(i * E + e + 1) * B], H, wl.I))
        ref, _ = O.block_norm(before, y, _np(b.post), _np(b.gate), 0.8)
        y_scale = np.abs(_np(b.gate) * _np(b.post)) * 3       # n(y) is of unit scale, 3 covers its largest values
        tol = 2e-2 * y_scale + 2.0 ** -7 * np.abs(ref) + 2e-2
        assert sure.sum() >= 2
        assert np.all(np.abs(_np(got) - ref)[sure] <= np.broadcast_to(tol, ref.shape)[sure])
    assert torch.equal(got, x)
    cache.close()


def test_blocks_refusals_and_reports():
    M = load_lib()
    wl = configs.scaled(configs.TINY, E=16, k=4, S=32, T=6)
    bank, B, cache, runner = _stack(M, wl, 1)
    good = torch.zeros(16, wl.H, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(wl.H, device="cuda")
    with pytest.raises(ValueError, match="router"):
        M.RoutedBlocks(runner, [M.BlockWeights(router=good[:8], pre=ones)])
    with pytest.raises(ValueError, match="router"):
        M.RoutedBlocks(runner, [M.BlockWeights(router=good.float(), pre=ones)])
    st = M.RoutedBlocks(runner, [M.BlockWeights(router=good, pre=ones, lora_a=good[None, :8],
                                                lora_b=good[None, :, :8].contiguous())])
    with pytest.raises(ValueError, match="tokens"):
        st.run(torch.zeros(7, wl.H, device="cuda"))
    x = torch.randn(6, wl.H, device="cuda")
    st.run(x, torch.tensor([0, -1, 0, -1, 0, 1], dtype=torch.int32, device="cuda"))   # adapter 1 of 1
    with pytest.raises(M.MoeError) as e:
        st.synchronize()
    assert e.value.status == M.MOE_ERR_INVALID
    st.run(x, torch.tensor([0, -1, 0, -1, 0, 0], dtype=torch.int32, device="cuda"))
    st.synchronize()
    assert torch.isfinite(x).all()
    cache.close()


def test_example_runs():
    load_lib()
    import importlib.util
    import os

    from tests.helpers import ROOT
    spec = importlib.util.spec_from_file_location("decode_blocks", os.path.join(ROOT, "examples", "decode_blocks.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    a, b = m.main(steps=2), m.main(steps=2)
    assert torch.isfinite(a).all() and torch.equal(a, b)
