"""The calls of a model's head together: one training step from rows to the
gradients of the rows and of the head's weight, eager, captured in a graph and
on a stream of its own, against 64 bits; and one step of serving."""
import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


class Step:
    """Rows -> layer norm -> 8-bit product -> logits -> cross entropy, entropy bonus and
    distillation -> gradients of the logits, the weight, the rows, the norm; AdamW."""

    def __init__(self, rvq, dev, n=150, d=264, V=1000, seed=1):
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.rvq, self.n = rvq, n
        self.x, self.res = r(n, d).to(BF16), r(n, d).to(BF16)
        self.gain, self.bias, self.head = 1 + 0.1 * r(d), 0.1 * r(d), 0.1 * r(V, d)
        self.ids = torch.randint(0, V, (n,), generator=g, device=dev).int()
        self.ids[3] = -1
        self.tids = torch.argsort(r(n, V), dim=1)[:, :16].int().contiguous()
        self.t = 2 * r(n, 16)
        self.dlp = torch.full((n,), -1.0 / n, device=dev)
        self.dent = torch.full((n,), 0.01 / n, device=dev)
        self.dloss = torch.full((n,), 1.0 / n, device=dev)
        self.state = rvq.rvq_adamw_init([self.head, self.gain, self.bias], 32, 0.01)

    def run(self):
        rvq = self.rvq
        y = rvq.rvq_layer_norm(self.x, self.gain, self.bias, residual=self.res, need_stats=True)
        qy, sy = rvq.rvq_quantize_f8(y.y)
        qw, sw = rvq.rvq_quantize_f8(self.head, 128)
        logits = rvq.rvq_matmul_f8(qy, sy, qw, sw)
        lp = rvq.rvq_token_logprobs(logits, self.ids, 0.9, top=4)
        kl = rvq.rvq_distill_loss(logits, self.tids, self.t, 2.0)
        d1 = rvq.rvq_token_logprobs_backward(logits, self.ids, lp.stats, self.dlp, lp.entropy, self.dent, 0.9)
        d2 = rvq.rvq_distill_loss_backward(logits, self.tids, self.t, kl.stats, self.dloss, 2.0)
        dlogits = d1 + d2
        qd, sd = rvq.rvq_quantize_f8(dlogits)
        qwt, swt = rvq.rvq_quantize_f8(self.head, 128, transpose=True)
        dy = rvq.rvq_matmul_f8(qd, sd, qwt, swt)
        qdt, sdt = rvq.rvq_quantize_f8(dlogits, transpose=True)
        qyt, syt = rvq.rvq_quantize_f8(y.y, transpose=True)
        dhead = rvq.rvq_matmul_f8(qdt, sdt, qyt, syt, out_dtype=F32)
        dx, dgain, dbias = rvq.rvq_layer_norm_backward(dy, y.sum, y.mean, y.rstd, self.gain, dsum=self.res)
        norm = rvq.rvq_adamw_step(self.state, [dhead, dgain, dbias], 3, 1e-3, max_norm=1.0)
        return [y.y, y.sum, logits, lp.logprob, lp.entropy, lp.top_logprob, lp.top_ids, kl.loss, dlogits, dy, dhead, dx, dgain,
                dbias, norm]

    def tensors(self):
        s = self.state
        return s.params + s.m + s.v


def _bytes(ts):
    return [t.contiguous().view(-1).view(torch.uint8).clone() for t in ts]


def test_step_against_64_bits(rvq, dev):
    s = Step(rvq, dev)
    head = s.head.clone()
    gain, bias = s.gain.clone(), s.bias.clone()
    y, h, logits, lp, ent, _, _, kl, dlogits, dy, dhead, dx, dgain, dbias, _ = s.run()
    # each call against its definition on the inputs that it was given
    h64, mean, rstd, y64 = ref.layer_norm(s.x, s.res, gain, bias, 1e-6)
    assert float((y.double() - y64).abs().max()) <= 0.02 * float(y64.abs().max())
    want, size = ref.matmul(*rvq.rvq_quantize_f8(y), *rvq.rvq_quantize_f8(head, 128))
    assert torch.all((logits.double() - want).abs() <= ref.BF16_ROUND * want.abs() + ref.matmul_bound(size, 264, True) * (1 + 2 ** -8))
    z = torch.log_softmax(logits.double() / 0.9, 1)
    at = s.ids.clamp(min=0).long()
    want = torch.where(s.ids >= 0, z[torch.arange(s.n, device=dev), at], 0.0)
    assert torch.all((lp.double() - want).abs() <= 1e-4)
    # the whole step's loss moves as its gradient says: along dhead (8-bit operands: a few percent)
    assert torch.isfinite(dhead).all() and torch.isfinite(dx.float()).all()
    full = (dlogits.double().t().contiguous() @ y.double())
    assert float((dhead.double() - full).norm()) <= 0.06 * float(full.norm())
    full = dlogits.double() @ head.double()
    assert float((dy.double() - full).norm()) <= 0.06 * float(full.norm())
    g = dy.double() * gain.double()
    u = (h.double() - h.double().mean(1, keepdim=True))
    u = u / (u.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert float((dgain.double() - (dy.double() * u).sum(0)).abs().max()) <= 1e-2 * float((dy.double() * u).abs().sum(0).max())
    assert float((dbias.double() - dy.double().sum(0)).abs().max()) <= 1e-4 * float(dy.double().abs().sum(0).max())
    assert g.shape == dx.shape


def test_step_replays_from_a_graph(rvq, dev):
    s = Step(rvq, dev)
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
    x, ids = b.x.clone(), b.ids.clone()
    b.x.zero_()
    b.ids.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):                                 # the inputs arrive late, on the same stream
            big = big @ big * 1e-3
        b.x.copy_(x)
        b.ids.copy_(ids)
        out = b.run()
    side.synchronize()
    for i, (x, y) in enumerate(zip(_bytes(out + list(b.tensors())), want)):
        assert torch.equal(x, y), i


def test_serving_step_from_a_graph_beside_another(rvq, dev):
    # two captured steps of single tokens with rows split over workgroups, replayed on two streams at once
    V, d = 40000, 512
    g = torch.Generator(device=dev).manual_seed(9)
    table = 0.1 * torch.randn((V, d), generator=g, device=dev)
    qw, sw = rvq.rvq_quantize_f8(table, 128)
    gain = torch.ones(d, device=dev)

    def step(x, ids):
        y = rvq.rvq_layer_norm(x, gain, out_dtype=F8)
        logits = rvq.rvq_matmul_f8(y.y, y.scale, qw, sw, out_dtype=F32)
        r = rvq.rvq_token_logprobs(logits, ids, 0.8, top=20)
        return [logits, r.logprob, r.entropy, r.top_logprob, r.top_ids]
    runs = []
    for n in (1, 3):
        x = torch.randn((n, d), generator=g, device=dev).to(BF16)
        ids = torch.randint(0, V, (n,), generator=g, device=dev).int()
        want = _bytes(step(x, ids))
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            step(x, ids)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = step(x, ids)
        runs.append((graph, side, out, want, x, ids))
    for rep in range(5):
        for graph, side, out, *_ in runs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for graph, side, *_ in runs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, out, want, *_ in runs:
            for i, (a, b) in enumerate(zip(_bytes(out), want)):
                assert torch.equal(a, b), (rep, i)
