"""A handle whose state is set on one stream and used on another: forwards
wait for the state they follow and setters for the forwards they follow,
whatever the streams' handles are.

Every case holds one stream back behind long kernels and checks that they were
still running when the other stream had its work.
"""

import dataclasses
import threading

import pytest
import torch

import synthetic
from tests.parity import built, gpu, needs_gpu, to_dev

pytestmark = [gpu, needs_gpu]

SHAPE = dataclasses.replace(synthetic.CONFIGS["c0_tiny"], name="streams", H=256, E=16, K=3, I=128, T=200,
                            max_num_tokens=200)
PER_THREAD = 2  # cudaStreamPerThread: one value, a stream a thread


@pytest.fixture(scope="module")
def setup():
    from nvfp4_token_quantized_gb300 import ExpertRouter

    built()
    d = to_dev(synthetic.make_workload(SHAPE))
    r = ExpertRouter(SHAPE.E, SHAPE.K, score="sigmoid", num_groups=4, top_groups=2, group_score="top2", scale=2.5)
    g = torch.Generator().manual_seed(5)
    biases = [(torch.randn(SHAPE.E, generator=g) * 0.2).cuda() for _ in range(2)]
    return d, r, biases, torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")


def _layer(d, **kw):
    from nvfp4_token_quantized_gb300 import MoE

    layer = MoE(SHAPE.H, SHAPE.I, SHAPE.E, SHAPE.K, SHAPE.max_num_tokens, deterministic=True, **kw)
    layer.load_weights(d["w13"], d["w2"])
    return layer


def _hold(big, stream):
    """Keeps `stream` busy for some 20 ms; the event after."""
    with torch.cuda.stream(stream):
        for _ in range(60):
            big.add_(1)
        done = torch.cuda.Event()
        done.record(stream)
    return done


def _both(layer, r, biases, d, T):
    """The outputs of T tokens under either bias; the handle keeps the second."""
    out = []
    for b in biases:
        layer.set_routing(r, b)
        out.append(layer.forward(d["x"][:T], d["gate_w"]))
    torch.cuda.synchronize()
    assert not torch.equal(*out)
    return out


@pytest.mark.parametrize("T", [40, 150])
def test_a_forward_waits_for_a_bias_set_on_another_stream(setup, T):
    d, r, biases, big = setup
    layer = _layer(d)
    want, _ = _both(layer, r, biases, d, T)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    done = _hold(big, a)
    layer.set_routing(r, biases[0], stream=a)
    got = layer.forward(d["x"][:T], d["gate_w"], stream=b)
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [40, 150])
def test_a_forward_waits_for_weights_loaded_on_another_stream(setup, T):
    d, r, biases, big = setup
    layer = _layer(d)
    w13, w2 = -d["w13"], -d["w2"]
    outs = []
    for pair in ((d["w13"], d["w2"]), (w13, w2)):
        layer.load_weights(*pair)
        outs.append(layer.forward(d["x"][:T], d["gate_w"]))
    torch.cuda.synchronize()
    assert not torch.equal(*outs)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    done = _hold(big, a)
    layer.load_weights(d["w13"], d["w2"], stream=a)
    got = layer.forward(d["x"][:T], d["gate_w"], stream=b)
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(got, outs[0])


@pytest.mark.parametrize("T", [40, 150])
def test_a_bias_set_on_another_stream_waits_for_the_forward(setup, T):
    d, r, biases, big = setup
    layer = _layer(d)
    other, kept = _both(layer, r, biases, d, T)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    done = _hold(big, a)
    got = layer.forward(d["x"][:T], d["gate_w"], stream=a)
    layer.set_routing(r, biases[0], stream=b)
    after = layer.forward(d["x"][:T], d["gate_w"], stream=b)
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(got, kept) and torch.equal(after, other)


@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("setter", ["load", "refresh", "shared", "scales"])
def test_state_set_on_another_stream_waits_for_the_forward(setup, setter, T):
    d, _, _, big = setup
    layer = _layer(d, static_scales=setter == "scales", shared_inter=128 if setter == "shared" else 0)
    w13s, w2s = (t.cuda() for t in synthetic.make_shared_weights(SHAPE, 128, seed=2))
    scales = [(torch.full((1,), v, device="cuda"), torch.full((SHAPE.E,), v, device="cuda")) for v in (300.0, 40.0)]
    states = {"load": ((d["w13"], d["w2"]), (-d["w13"], -d["w2"])),
              "refresh": ((d["w13"], d["w2"]), (-d["w13"], -d["w2"])),
              "shared": ((w13s, w2s), (-w13s, -w2s)), "scales": scales}[setter]
    put = {"load": layer.load_weights, "refresh": layer.refresh_scales_inplace, "shared": layer.load_shared_weights,
           "scales": layer.set_static_scales}[setter]
    outs = []
    for s in (states[1], states[0]):
        put(*s)
        outs.append(layer.forward(d["x"][:T], d["gate_w"]))
    torch.cuda.synchronize()
    assert not torch.equal(*outs)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    done = _hold(big, a)
    got = layer.forward(d["x"][:T], d["gate_w"], stream=a)
    put(*states[1], stream=b)
    after = layer.forward(d["x"][:T], d["gate_w"], stream=b)
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(got, outs[1]) and torch.equal(after, outs[0])


@pytest.mark.parametrize("T", [40, 150])
def test_the_per_thread_streams_of_two_threads_are_two_streams(setup, T):
    d, r, biases, big = setup
    layer = _layer(d)
    want, _ = _both(layer, r, biases, d, T)
    queued, leave, seen = threading.Event(), threading.Event(), []

    def other():
        try:
            seen.append(_hold(big, torch.cuda.ExternalStream(PER_THREAD)))
            layer.set_routing(r, biases[0], stream=PER_THREAD)
        finally:
            queued.set()
        leave.wait(60)

    t = threading.Thread(target=other)
    t.start()
    assert queued.wait(60)
    x, out = d["x"][:T].contiguous(), torch.empty(T, SHAPE.H, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, d["gate_w"], out, stream=PER_THREAD)
    still = not seen[0].query()
    leave.set()
    t.join()
    torch.cuda.synchronize()
    assert still and torch.equal(out, want)


@pytest.mark.parametrize("beside_on", ["own", "legacy", "per thread"])
def test_state_set_and_used_beside_a_capture(setup, beside_on):
    # a capture on one stream goes on while the handle works on another
    d, r, biases, _ = setup
    layer = _layer(d)
    want = _both(layer, r, biases, d, 40)
    x = d["x"][:40].contiguous()
    out, beside = torch.empty_like(x), torch.empty_like(x)
    a = torch.cuda.Stream()
    b = {"own": torch.cuda.Stream(), "legacy": 0, "per thread": PER_THREAD}[beside_on]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=a):
        layer.forward(x, d["gate_w"], out)
        layer.set_routing(r, biases[0], stream=b)
        layer.forward(x, d["gate_w"], beside, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(beside, want[0])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
