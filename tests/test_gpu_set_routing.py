"""A handle's forward under a routing rule (moe_set_routing), at every path of
the forward: its choice is moe_route_select's on the forward's own logits, its
output the weighted sum of the chosen experts, and without a rule nothing
changes."""

import dataclasses

import numpy as np
import pytest
import torch

import synthetic
from oracle import block as ob
from oracle import moe as omoe
from oracle import nvfp4 as onv
from tests import parity
from tests.parity import built, gpu, needs_gpu, to_dev

pytestmark = [gpu, needs_gpu]

SHAPE = dataclasses.replace(synthetic.CONFIGS["c0_tiny"], name="rule", H=256, E=16, K=3, I=128, T=200,
                            max_num_tokens=200)
RULES = [dict(score="sigmoid", num_groups=4, top_groups=2, group_score="top2", scale=2.5),
         dict(score="softmax", renormalize=False),
         dict(score="sigmoid", renormalize=False, num_groups=8, top_groups=5)]


@pytest.fixture(scope="module")
def setup():
    built()
    wl = synthetic.make_workload(SHAPE)
    return wl, to_dev(wl), parity.quantize_experts(wl.w13, range(SHAPE.E)), parity.quantize_experts(wl.w2, range(SHAPE.E))


def _bias(seed=0):
    return (torch.randn(SHAPE.E, generator=torch.Generator().manual_seed(seed)) * 0.2).cuda()


def _layer(d, deterministic=True, shape=SHAPE):
    from nvfp4_token_quantized_gb300 import MoE

    layer = MoE.from_shape(shape, deterministic=deterministic)
    layer.load_weights(d["w13"], d["w2"])
    return layer


@pytest.mark.parametrize("deterministic", [True, False])
@pytest.mark.parametrize("rule", range(len(RULES)))
@pytest.mark.parametrize("T", [1, 7, 33, 64, 65, 200])
def test_forward_under_a_rule(setup, T, rule, deterministic):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    wl, d, q13, q2 = setup
    r = ExpertRouter(SHAPE.E, SHAPE.K, **RULES[rule])
    layer = _layer(d, deterministic)
    for bias in (None, _bias()):
        layer.set_routing(r, bias)
        out = layer.forward(d["x"][:T], d["gate_w"])
        rt = layer.debug_routing()
        ids, w = r.select(layer.debug_logits(), bias=bias)
        assert torch.equal(rt["topk_ids"], ids) and torch.equal(rt["topk_w"], w)
        idn = ids.cpu().numpy()
        off, src, _ = omoe.permute(idn, SHAPE.E)
        assert np.array_equal(rt["src_of_row"].cpu().numpy(), src)
        assert np.array_equal(rt["expert_offsets"].cpu().numpy(), off)
        # the experts' second product on the GPU's own intermediate
        hc, hs, hg = (t.cpu().numpy() for t in layer.debug_intermediate())
        hc = onv.unpack_e2m1(hc)
        xc, xs, xg = onv.quantize_rows(omoe.as_f32(wl.x)[:T])
        y = np.zeros((T, SHAPE.K, SHAPE.H), np.float32)
        for e in np.unique(idn):
            t, j = np.nonzero(idn == e)
            s = t * SHAPE.K + j
            y[t, j] = omoe.expert_w2(hc[s], hs[s], hg[s], q2, e)
            full = omoe.expert_rows(xc[t], xs[t], xg[t], q13, q2, e)
            assert np.allclose(full["h_gs"], hg[s], rtol=1e-2)
        ref = onv.bf16_to_f32(onv.bf16_round(omoe.finalize(y, w.cpu().numpy())))
        parity.assert_close(omoe.as_f32(out), ref)


def test_widest_rules():
    # 256 experts, group counts that leave a lane up to 16 of them
    from nvfp4_token_quantized_gb300 import ExpertRouter

    shape = dataclasses.replace(SHAPE, E=240, K=16, I=128, T=70, max_num_tokens=70)
    wl = synthetic.make_workload(shape)
    d = to_dev(wl)
    layer = _layer(d, shape=shape)
    bias = (torch.randn(240, generator=torch.Generator().manual_seed(3)) * 0.1).cuda()
    for groups, top in ((1, 1), (20, 6), (8, 3), (30, 30), (16, 4)):
        r = ExpertRouter(240, 16, score="sigmoid", num_groups=groups, top_groups=top, group_score="top2")
        layer.set_routing(r, bias)
        for T in (3, 64, 70):
            layer.forward(d["x"][:T], d["gate_w"])
            rt = layer.debug_routing()
            logits = layer.debug_logits()
            ids, w = r.select(logits, bias=bias)
            assert torch.equal(rt["topk_ids"], ids) and torch.equal(rt["topk_w"], w)
            ref, _ = ob.route(logits.cpu().numpy().astype(np.float64), 16, "sigmoid",
                              bias.cpu().numpy().astype(np.float64), groups, top, "top2")
            assert (ids.cpu().numpy() == ref).mean() > 0.99


def test_without_a_rule_nothing_changes(setup):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    _, d, _, _ = setup
    fresh, layer = _layer(d), _layer(d)
    r = ExpertRouter(SHAPE.E, SHAPE.K, **RULES[0])
    for T in (5, 40, 150):
        ref = fresh.forward(d["x"][:T], d["gate_w"])
        layer.set_routing(r, _bias())
        assert not torch.equal(layer.forward(d["x"][:T], d["gate_w"]), ref)
        layer.set_routing(None)
        assert torch.equal(layer.forward(d["x"][:T], d["gate_w"]), ref)


@pytest.mark.parametrize("T", [40, 150])
def test_captured_forward_takes_a_new_bias(setup, T):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    _, d, _, _ = setup
    layer = _layer(d)
    r = ExpertRouter(SHAPE.E, SHAPE.K, **RULES[0])
    layer.set_routing(r, _bias(1))
    x, out = d["x"][:T].contiguous(), torch.empty_like(d["x"][:T])
    layer.forward(x, d["gate_w"], out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, d["gate_w"], out)
    g.replay()
    torch.cuda.synchronize()
    before = out.clone()
    layer.set_routing(r, _bias(2))
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert not torch.equal(replayed, before)
    assert torch.equal(replayed, layer.forward(x, d["gate_w"]))


def test_refusals(setup):
    from nvfp4_token_quantized_gb300 import ExpertRouter, MoEError

    _, d, _, _ = setup
    layer = _layer(d)
    for r in (ExpertRouter(SHAPE.E, SHAPE.K + 1), ExpertRouter(SHAPE.E * 2, SHAPE.K)):
        with pytest.raises(MoEError) as e:
            layer.set_routing(r)
        assert e.value.status == 1
    r = ExpertRouter(SHAPE.E, SHAPE.K)
    for bias in (torch.zeros(SHAPE.E), torch.zeros(SHAPE.E + 1, device="cuda"),
                 torch.zeros(SHAPE.E, dtype=torch.float64, device="cuda")):
        with pytest.raises(ValueError):
            layer.set_routing(r, bias)
    ref = _layer(d).forward(d["x"], d["gate_w"])
    assert torch.equal(layer.forward(d["x"], d["gate_w"]), ref)   # a refusal leaves the rule as it was


def test_example_runs_them_together():
    from examples import sparse_block as ex

    stack = ex.SparseStack(ex.SHAPE, 2)
    for T in (48, 200):
        x = synthetic.make_activations(ex.SHAPE, T=T).cuda()
        h, trace = stack.forward(x)
        eps = float(np.float32(1e-6))
        for i, s in enumerate(trace):
            nxt = trace[i + 1]["residual"] if i + 1 < len(trace) else None
            (ref, _), (refh, _) = ob.block_norm(omoe.as_f32(s["residual"]).astype(np.float64), omoe.as_f32(s["y"]),
                                                wp=omoe.as_f32(stack.post[i]), wn=omoe.as_f32(stack.pre[i + 1]),
                                                eps=eps)
            if nxt is not None:
                parity.assert_close(omoe.as_f32(nxt), ref)
            got = trace[i + 1]["h"] if i + 1 < len(trace) else h
            parity.assert_close(omoe.as_f32(got), refh)
    target = torch.full_like(trace[0]["topk_w"], 2.5 / ex.SHAPE.K)
    losses = []
    for _ in range(3):
        losses.append(stack.router_step({"layer": 0, **trace[0]}, target, lr=20.0).item())
        _, trace = stack.forward(x)
    assert losses[2] < losses[0]


def test_state_set_on_one_stream_is_seen_on_another(setup):
    # weights, then a bias, set behind a long kernel of their stream: forwards
    # on other streams wait for them
    from nvfp4_token_quantized_gb300 import ExpertRouter, MoE

    _, d, _, _ = setup
    r = ExpertRouter(SHAPE.E, SHAPE.K, **RULES[0])
    ref = _layer(d)
    ref.set_routing(r, _bias(5))
    want = {T: ref.forward(d["x"][:T], d["gate_w"]) for T in (40, 150)}
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for T in (40, 150):
        a, b, c = (torch.cuda.Stream() for _ in range(3))
        layer = MoE.from_shape(SHAPE, deterministic=True)
        with torch.cuda.stream(a):
            for _ in range(20):
                big.add_(1)
            layer.load_weights(d["w13"], d["w2"])
        with torch.cuda.stream(b):
            layer.set_routing(r, _bias(5))
            got_b = layer.forward(d["x"][:T], d["gate_w"])
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            for _ in range(20):
                big.add_(1)
            layer.set_routing(r, _bias(6))
            layer.set_routing(r, _bias(5))
        with torch.cuda.stream(c):
            got_c = layer.forward(d["x"][:T], d["gate_w"])
        torch.cuda.synchronize()
        assert torch.equal(got_b, want[T]) and torch.equal(got_c, want[T])
