"""rvq_distill_loss and its gradient against their definitions in 64 bits."""
import math

import pytest
import torch

import head_ref as ref
import learn_ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = math.inf


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def _chain(V):
    # as for the log probabilities, and the teacher's own entries beside them
    return max(V / 1024, 64) + 80


def _case(n, V, k, dtype, T, tail, seed, dev):
    """Logits, and a teacher like them: its k best tokens of each row."""
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((n, V), generator=g, device=dev) * 2.5
    t = x + torch.randn((n, V), generator=g, device=dev)
    if tail:
        t = torch.log_softmax(t.double() / T, 1).float()
    v, j = torch.topk(t, k, dim=1)
    mix = torch.argsort(torch.rand((n, k), generator=g, device=dev), dim=1)     # in any order
    return x.to(dtype), j.gather(1, mix).int().contiguous(), v.gather(1, mix).contiguous(), g


def _check(rvq, x, ids, t, T, tail, dloss=None):
    n, V = x.shape
    got = rvq.rvq_distill_loss(x, ids, t, T, tail)
    loss, b_loss, dx, b_dx = ref.distill(x, ids, t, T, tail, _chain(V))
    fine = torch.isfinite(loss)
    assert torch.equal(got.loss[~fine].double(), loss[~fine])
    learn_ref.close(got.loss[fine], loss[fine], b_loss[fine], "loss")
    w = torch.linspace(-1.0, 2.0, n, device=x.device) if dloss is None else dloss
    for place in ("new", "logits"):
        y = x.clone()
        d = rvq.rvq_distill_loss_backward(y, ids, t, got.stats, w, T, tail, out=y if place == "logits" else None)
        want = dx * w.double()[:, None]
        bound = b_dx * w.double().abs()[:, None] + 2 * ref.U * want.abs() + 2.0 ** -125
        if x.dtype == BF16:
            bound = bound + ref.BF16_ROUND * want.abs() + 2.0 ** -134
        learn_ref.close(d, want, bound, f"dlogits {place}")
    return got


SHAPES = [(1, 1, 1), (3, 2, 2), (50, 7, 3), (33, 256, 8), (20, 2048, 64), (12, 2049, 5), (9, 300, 100), (9, 4096, 256),
          (6, 16384, 1), (6, 16385, 64), (3, 65536, 64), (2, 65537, 200), (2, 300001, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_distill(rvq, dev, shape, tail):
    for dtype, T in ((F32, 1.0), (BF16, 2.0), (F32, 0.5)):
        x, ids, t, _ = _case(*shape, dtype, T, tail, sum(shape), dev)
        _check(rvq, x, ids, t, T, tail)


@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_entries_that_repeat_or_do_not_count(rvq, dev, V, tail):
    x, ids, t, g = _case(12, V, 12, F32, 1.0, tail, V, dev)
    t = t - 0.7 if tail else t                       # some weight for the rest
    ids[0, 3:6] = ids[0, 2]                          # repeated: the first counts
    ids[1, ::2] = -1
    ids[2, 4] = V
    ids[2, 5] = -7
    ids[3] = -1                                      # none at all
    ids[4, 1:] = ids[4, 0]
    t[5, 2] = -INF                                   # no weight
    t[6, 1:] = -INF
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    got = _check(rvq, x, ids, t, 1.0, tail)
    again = rvq.rvq_distill_loss(x, ids, t, 1.0, tail, bad_ids=bad)
    assert bad.item() == 2 and torch.equal(again.loss, got.loss) and got.loss[3].item() == 0.0
    if not tail:
        t[7] = -INF                                  # a teacher that says nothing
        assert _check(rvq, x, ids, t, 1.0, tail).loss[7].item() == 0.0


@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_masks_nan_and_rows_of_no_weight(rvq, dev, V):
    for tail in (False, True):
        x, ids, t, _ = _case(10, V, 6, F32, 1.0, tail, V, dev)
        t = t - 0.3 if tail else t
        clean = rvq.rvq_distill_loss(x, ids, t, 1.0, tail)
        w = torch.ones(10, device=dev)
        dclean = rvq.rvq_distill_loss_backward(x, ids, t, clean.stats, w, 1.0, tail)
        x[0, ids[0, 2].long()] = -INF                # weight on a masked token
        others = torch.ones(V, dtype=torch.bool, device=dev)
        others[ids[1].long()] = False
        x[1, others] = -INF                          # nothing but the teacher's tokens
        x[2] = -INF
        x[3, V // 2] = float("nan")
        x[4, ids[4, 0].long()] = INF
        t[5, 1] = float("nan")
        got = rvq.rvq_distill_loss(x, ids, t, 1.0, tail)
        d = rvq.rvq_distill_loss_backward(x, ids, t, got.stats, w, 1.0, tail)
        assert got.loss[0].item() == INF and got.loss[2].item() == INF
        assert (got.loss[1].item() == INF) == tail and torch.all(d[1, others] == 0) and torch.isfinite(d[:2]).all()
        assert torch.all(d[2] == 0)
        for i in (3, 4, 5):
            assert math.isnan(got.loss[i])
        assert torch.isnan(d[3]).all() and torch.isnan(d[4]).all()
        assert torch.equal(got.loss[6:], clean.loss[6:]) and torch.equal(d[6:], dclean[6:])
        w[3:6] = 0
        d = rvq.rvq_distill_loss_backward(x, ids, t, got.stats, w, 1.0, tail)
        assert torch.all(d[3:6] == 0)


def test_a_tail_far_below(rvq, dev):
    # the student's others hold 1e-13, then 1e-45 of the weight, the teacher's a tenth: what is left is
    # told by their own largest value
    for gap in (40.0, 115.0):
        for V in (200, 9000, 70000):
            x, ids, t, _ = _case(4, V, 5, F32, 1.0, True, V, dev)
            x = x.clamp(-3, 3)
            x.scatter_(1, ids.long(), gap)
            t = torch.full_like(t, math.log(0.18))
            _check(rvq, x, ids, t, 1.0, True)


def test_teacher_equals_student(rvq, dev):
    # the teacher's own log probabilities, from the library: no loss, no gradient
    x, _, _, _ = _case(40, 3000, 4, F32, 1.0, True, 3, dev)
    s = rvq.rvq_token_logprobs(x, None, 1.5, top=32)
    got = rvq.rvq_distill_loss(x, s.top_ids, s.top_logprob, 1.5, tail=True)
    r = ref.Logits(x, 1.5, _chain(3000))
    assert torch.all(got.loss.abs().double() <= 4 * r.b_logp.amax(1) + r.b_logS[:, 0] + 300 * ref.U)
    d = rvq.rvq_distill_loss_backward(x, s.top_ids, s.top_logprob, got.stats, torch.ones(40, device=dev), 1.5, tail=True)
    assert float(d.abs().max()) <= 1e-4


def test_gradient_against_differences(rvq, dev):
    n, V, s = 2, 23, 1e-5
    for tail, T in ((False, 2.0), (True, 0.9)):
        x, ids, t, _ = _case(n, V, 6, F32, T, tail, 1, dev)
        w = torch.tensor([0.7, -1.3], device=dev)
        st = rvq.rvq_distill_loss(x, ids, t, T, tail)
        d = rvq.rvq_distill_loss_backward(x, ids, t, st.stats, w, T, tail)

        def loss(x):
            return float((ref.distill(x, ids, t, T, tail, 1)[0] * w.double()).sum())
        for i in range(n):
            for j in range(0, V, 2):
                e = torch.zeros((n, V), dtype=torch.float64, device=dev)
                e[i, j] = s
                num = (loss(x.double() + e) - loss(x.double() - e)) / (2 * s)
                assert abs(num - d[i, j].item()) <= 1e-4, (tail, i, j)


def test_refusals(rvq, dev):
    x, ids, t, _ = _case(4, 32, 3, F32, 1.0, False, 1, dev)
    one = torch.ones(4, device=dev)
    st = rvq.rvq_distill_loss(x, ids, t)
    ok = dict(logits=x, teacher_ids=ids, teacher=t)
    for bad in (dict(teacher_ids=ids.long()), dict(teacher_ids=ids[:3]), dict(teacher_ids=ids[0]), dict(teacher=t.double()),
                dict(teacher=t[:, :2]), dict(teacher=t.cpu()), dict(logits=x.double()), dict(logits=x.t()), dict(bad_ids=ids),
                dict(teacher=t.clone().requires_grad_()), dict(logits=x.clone().requires_grad_())):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_distill_loss(**{**ok, **bad})
    for bad in (dict(temperature=0.0), dict(temperature=float("inf")), dict(teacher_ids=ids[:, :0].contiguous(), teacher=t[:, :0].contiguous()),
                dict(teacher_ids=ids[:, :1].expand(4, 257).contiguous(), teacher=t[:, :1].expand(4, 257).contiguous())):
        with pytest.raises(rvq.RVQError):
            rvq.rvq_distill_loss(**{**ok, **bad})
    ok = dict(ok, stats=st.stats, dloss=one)
    for bad in (dict(stats=st.stats[:, :2]), dict(dloss=one[:3]), dict(dloss=one.double()), dict(out=x[:2]), dict(out=x.bfloat16()),
                dict(dloss=one.clone().requires_grad_())):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_distill_loss_backward(**{**ok, **bad})
    e = rvq.rvq_distill_loss(x[:0], ids[:0], t[:0])
    assert e.loss.shape == (0,) and rvq.rvq_distill_loss_backward(x[:0], ids[:0], t[:0], e.stats, one[:0]).shape == (0, 32)


@pytest.mark.parametrize("V", [17, 300, 5000, 70000])
@pytest.mark.parametrize("tail", [False, True], ids=["top", "tail"])
def test_certain_rows_keep_their_small_numbers(rvq, dev, V, tail):
    """Student and teacher put all but 10^-3 to 10^-9 of their weight on one token: loss and
    gradient are differences of such numbers, and as exact as these."""
    g = torch.Generator(device=dev).manual_seed(V)
    n, k = 24, min(9, V - 3)
    x = torch.randn((n, V), generator=g, device=dev)
    x[:, 3] = torch.linspace(16.0, 30.0, n, device=dev)
    t = x + torch.randn((n, V), generator=g, device=dev)
    z = t.double() if not tail else torch.log_softmax(t.double(), 1)
    if tail:
        # log q of the token itself, as log1p of what the others have
        e = torch.exp(t.double() - t.double()[:, 3:4])
        e[:, 3] = 0
        z[:, 3] = -torch.log1p(e.sum(1))
    _, ids = torch.topk(t, k, dim=1)
    v = z.gather(1, ids).float()
    # 64 bits have numbers just below 1 in steps of 2^-53: p and q of token 3 and 1 - sum q
    # (k + 2 roundings) are off by that on either side, whatever is left of them.
    last = 2 * (k + 2) * 2.0 ** -53
    if tail:
        assert torch.all(1 - v.double().exp().sum(1) > 8 * last)
    ids = ids.int()
    w = torch.rand(n, generator=g, device=dev) + 0.5
    got = rvq.rvq_distill_loss(x, ids, v, 1.0, tail)
    d = rvq.rvq_distill_loss_backward(x, ids, v, got.stats, w, 1.0, tail)

    at = ids.long()
    y = x.double() - x.double()[:, 3:4]
    e = torch.exp(y)
    e[:, 3] = 0
    others = e.sum(1)                                      # of weight 1 for token 3
    logp = y - torch.log1p(others)[:, None]
    p = logp.exp()
    if tail:
        logq = v.double()
        rest = 1 - logq.exp().sum(1)
        left = e.scatter(1, at, 0.0).sum(1)
        p_rest = left / (1 + others)
    else:
        u = v.double() - v.double()[:, :1]
        eu = torch.exp(u)
        logq = u - torch.log1p(eu[:, 1:].sum(1))[:, None]
    q = logq.exp()
    mine = logp.gather(1, at)
    loss = (q * (logq - mine)).sum(1)
    grad = p.clone() if not tail else p * (1 - rest / p_rest)[:, None]
    grad.scatter_(1, at, p.gather(1, at) - q)
    if tail:
        loss = loss + rest * (rest.log() - p_rest.log())
    # What token 3 does not have: sums over it are off by 160 roundings (chains, trees) and a
    # term's exponent below 40 by 3 each; a float32 log q or log p of it carries one more.
    small = 1 - p[:, 3] + (1 - q[:, 0]) + 2.0 ** -52
    tol = (160 + 3 * 40 + 8) * ref.U
    off = 40 * (tol * small + last)                         # logarithms' factors: below 40
    assert torch.all((got.loss.double() - loss).abs() <= off + ref.U * loss.abs())
    want = grad * w.double()[:, None]
    bound = w.double()[:, None] * (tol * (p + torch.zeros_like(p).scatter(1, at, q))) + 2 * ref.U * want.abs()
    bound[:, 3] = w.double() * (tol * small + last) + 2 * ref.U * want[:, 3].abs()
    if tail:
        bound = bound + w.double()[:, None] * p * ((tol * rest + last) / p_rest)[:, None]
    assert torch.all((d.double() - want).abs() <= bound)


def test_entries_that_name_all_there_is(rvq, dev):
    """The teacher's logarithms are rounded, so that its weights do not add up to 1 exactly:
    with no other token to take the rest the loss stays finite."""
    g = torch.Generator(device=dev).manual_seed(11)
    for n, V, k in ((5000, 38, 38), (300, 256, 256), (40, 5000, 20)):
        x = torch.randn((n, V), generator=g, device=dev) * 3
        ids = torch.stack([torch.randperm(V, generator=g, device=dev)[:k] for _ in range(n)]).int()
        if k < V:       # the others are masked
            x = torch.full_like(x, -INF).scatter(1, ids.long(), x.gather(1, ids.long()))
        t = torch.log_softmax(x.gather(1, ids.long()) + torch.randn((n, k), generator=g, device=dev), 1)
        got = rvq.rvq_distill_loss(x, ids, t, 1.0, True)
        logp = torch.log_softmax(x.double(), 1).gather(1, ids.long())
        q = t.double().exp()
        want = (q * (t.double() - logp)).sum(1)
        # the teacher's logarithms as given; log p within 160 roundings and 3 of d < 40
        assert torch.all((got.loss.double() - want).abs() <= (160 + 120) * ref.U + ref.U * want.abs())
        one = torch.ones(n, device=dev)
        d = rvq.rvq_distill_loss_backward(x, ids, t, got.stats, one, 1.0, True)
        p = logp.exp()
        grad = torch.zeros(n, V, device=dev, dtype=torch.float64).scatter(1, ids.long(), p - q)
        assert torch.all((d.double() - grad).abs() <= (160 + 120) * ref.U * (p.amax(1, keepdim=True) + 1))
        t = t - 0.01                                     # and with a rest that is one, it does not
        assert torch.all(torch.isinf(rvq.rvq_distill_loss(x, ids, t, 1.0, True).loss))
