"""One training step of the token embedding (embed, norm, its gradient, the
tables' gradient, AdamW) captured in a graph, on a stream of its own, and as
the example runs it."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


class Step:
    """Buffers and calls of one step; run() changes the parameters."""

    def __init__(self, rvq, dev, T=1500, L=4, K=100, V=60, D=192, bits=8, seed=1):
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.rvq, self.K, self.V = rvq, K, V
        self.level, self.text, self.weight = r(L, K, D), r(V, D), torch.ones(D, device=dev)
        self.ids = torch.randint(0, min(K, V), (T, L), generator=g, device=dev).int()
        self.ids[:900] = 7                                  # a row longer than a segment of the list
        self.vis = (torch.rand(T, generator=g, device=dev) < 0.8).to(torch.uint8)
        self.dy = r(T, D).to(BF16)
        self.state = rvq.rvq_adamw_init([self.level, self.text, self.weight], bits, 0.01)

    def run(self):
        rvq = self.rvq
        x = rvq.rvq_embed_tokens(self.ids, self.level, self.vis, self.text, out_dtype=BF16)
        y = rvq.rvq_rms_norm(x, self.weight, residual=x, need_rstd=True)
        dx, dw = rvq.rvq_rms_norm_backward(self.dy, y.sum, y.rstd, self.weight, dsum=y.y)
        gl, gt = rvq.rvq_embed_tokens_backward(dx, self.ids, self.K, self.vis, self.V)
        norm = rvq.rvq_adamw_step(self.state, [gl, gt, dw], 5, 1e-2, max_norm=1.0, seed=3)
        return [x, y.y, y.sum, y.rstd, dx, dw, gl, gt, norm]

    def tensors(self):
        s = self.state
        return s.params + s.m + s.v + (s.m_scale or ()) + (s.v_scale or ())


def _bytes(ts):
    return [t.contiguous().view(-1).view(torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("bits", [8, 32])
def test_step_replays_from_a_graph(rvq, dev, bits):
    s = Step(rvq, dev, bits=bits)
    start = [t.clone() for t in s.tensors()]
    want = []
    for _ in range(4):                                      # four eager steps, one after the other
        out = s.run()
        torch.cuda.synchronize()
        want.append(_bytes(out + list(s.tensors())))

    def restore():
        for t, a in zip(s.tensors(), start):
            t.copy_(a)
    restore()
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    restore()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.run()
    restore()
    other = Step(rvq, dev, seed=2)
    for rep in range(4):
        other.run()                                         # eager work between the replays
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(_bytes(out + list(s.tensors())), want[rep])):
            assert torch.equal(a, b), f"replay {rep}: tensor {i}"


def test_step_on_another_stream(rvq, dev):
    a, b = Step(rvq, dev), Step(rvq, dev)
    want = _bytes(a.run() + list(a.tensors()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=dev)
    big = torch.randn(4096, 4096, device=dev)
    ids, dy = b.ids.clone(), b.dy.clone()
    b.ids.zero_()
    b.dy.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):                                 # the inputs arrive late, on the same stream
            big = big @ big * 1e-3
        b.ids.copy_(ids)
        b.dy.copy_(dy)
        out = b.run()
    side.synchronize()
    for i, (x, y) in enumerate(zip(_bytes(out + list(b.tensors())), want)):
        assert torch.equal(x, y), i


def test_example_learns(rvq, dev):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import learn_token_embedding as example
    for bits in (32, 8):
        first, last = example.train(steps=60, state_bits=bits)
        # the loss starts at 2 (two unrelated unit vectors) and has to lose most of it
        assert first > 1.5 and last < 0.5 * first, (bits, first, last)
