"""The differentiable layers inside stream captures while eager graphs of the same leaves, or holders of their gradient
accumulators, are alive."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import gen, randn
from kimi_delta_attention_16_gb300 import synth
from test_gpu_block_layers import leaf, pair

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


class Layer:
    """kda_layer on two sequences; its q, conv_w and initial state as leaves (their gradients are the same bits every
    time, or compared by norm)."""

    def __init__(self, saved):
        inp = synth.make_prefill("layer_8k", seed=33, device=DEV, lengths=[70, 58], H=2, s0_std=0.02)
        self.q, self.state = inp.q.detach().clone().requires_grad_(), inp.initial_state.detach().clone().requires_grad_()
        self.inp, self.saved, self.cu = inp, saved, pair([70, 58])
        self.dy = randn(gen(34), 128, 2, 128, dtype=BF).to(DEV)
        self.leaves = [self.q, self.state]

    def out(self):
        i = self.inp
        return kda.kda_layer(self.q, i.k, i.v, i.conv_w, i.g, i.beta, self.cu, gate=i.gate, rms_w=i.rms_w,
                             initial_state=self.state, saved=self.saved)[0]

    def grads(self):
        return torch.autograd.grad(self.out(), self.leaves, self.dy)


def side_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    return s


def capture(side, step):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    return graph, out


@pytest.mark.parametrize("saved", ["io", "e4m3"])
def test_forward_is_captured_while_an_eager_graph_lives(saved):
    """A captured forward pass with gradients enabled waits on no accumulator; the eager graph still differentiates."""
    m = Layer(saved)
    ref = m.grads()
    alive = m.out()
    graph, out = capture(side_stream(), m.out)
    with torch.no_grad():
        m.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = m.out()
    assert torch.equal(out, want) and not torch.equal(out, alive)
    with torch.no_grad():
        m.q.mul_(2.0)  # exact: what the eager graph saved ("io") is the old q again
    assert all(torch.equal(a, b) for a, b in zip(ref, m.grads()))


@pytest.mark.parametrize("saved", ["io", "e4m3"])
def test_captured_backward_is_refused_while_an_accumulator_of_the_default_stream_lives(saved):
    """The refusal comes before the engine reaches the accumulator; with it gone the same step is captured."""
    m = Layer(saved)
    side = side_stream()
    holder = [torch.autograd.graph.get_gradient_edge(t).node for t in m.leaves]  # outlives the eager graph
    ref = m.grads()
    with pytest.raises(RuntimeError, match="accumulator"):
        capture(side, m.grads)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, m.grads()))
    del holder
    with torch.cuda.stream(side):
        m.grads()
    torch.cuda.synchronize()
    graph, got = capture(side, m.grads)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("saved", ["io", "e4m3"])
def test_step_is_captured_while_an_eager_graph_of_another_side_stream_lives(saved):
    """That stream joins the capture: kda_layer and a layer of the block, gradients returned and accumulated."""
    m = Layer(saved)
    ref = m.grads()
    other, side = side_stream(), side_stream()
    x, w = leaf(randn(gen(35), 64, 320, dtype=BF)), leaf(randn(gen(36), 320))
    dx = randn(gen(37), 64, 320, dtype=BF).to(DEV)
    nref = torch.autograd.grad(kda.kda_norm_layer(x, w, saved=saved), [x, w], dx)

    def step():
        kda.kda_norm_layer(x, w, saved=saved).backward(dx)
        return m.grads()
    with torch.cuda.stream(other):
        alive = [m.out(), kda.kda_norm_layer(x, w, saved=saved)]
        x.grad, w.grad = torch.zeros_like(x), torch.zeros_like(w)
    torch.cuda.synchronize()
    graph, got = capture(side, step)
    x.grad.zero_()
    w.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and len(alive) == 2
    assert torch.equal(x.grad, nref[0]) and torch.equal(w.grad, nref[1])
