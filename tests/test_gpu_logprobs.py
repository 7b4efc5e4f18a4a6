"""rvq_token_logprobs and its gradient against their definitions in 64 bits."""
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
    # a thread of 64 (rows up to 2048) or more adds 1/4 of 32 values at once, then piece after
    # piece; trees over lanes and waves, and the slices of a split row
    return max(V / 1024, 64) + 80


def _logits(n, V, dtype, seed, dev, std=3.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((n, V), generator=g, device=dev) * std
    if V > 4:
        at = torch.randint(0, V, (n, 1), generator=g, device=dev)
        x.scatter_add_(1, at, 20.0 * torch.rand((n, 1), generator=g, device=dev))
    ids = torch.randint(0, V, (n,), generator=g, device=dev).int()
    return x.to(dtype), ids


def _check(rvq, x, ids, T=1.0, top=0, **kw):
    n, V = x.shape
    got = rvq.rvq_token_logprobs(x, ids, T, top=top, **kw)
    torch.cuda.synchronize()
    r = ref.Logits(x, T, _chain(V))
    rows = torch.arange(n, device=x.device)
    if ids is not None:
        ok = (ids >= 0) & (ids < V)
        at = ids.clamp(0, V - 1).long()
        want = torch.where(ok, r.logp[rows, at], 0.0)
        want = torch.where(want < -torch.finfo(F32).max, -INF, want)     # below fp32: its -inf
        fine = torch.isfinite(want)
        assert torch.equal(got.logprob[~fine].double(), want[~fine])
        learn_ref.close(got.logprob[fine], want[fine], (r.b_logp[rows, at] + ref.U * want.abs())[fine], "logprob")
    assert torch.equal(got.stats[:, 0], x.float().amax(1))
    learn_ref.close(got.stats[:, 1], r.logS[:, 0], (r.b_logS + ref.U * r.logS)[:, 0], "log S")
    if got.entropy is not None:
        learn_ref.close(got.entropy, r.H[:, 0], (r.b_H + 2 * ref.U * r.H)[:, 0], "entropy")
    if top:
        k = min(top, V)
        order = torch.argsort(x.float() + 0.0, dim=1, descending=True, stable=True)[:, :k]
        lp = r.logp.gather(1, order)
        there = x.float().gather(1, order) > -INF
        lp = torch.where(lp < -torch.finfo(F32).max, -INF, lp)
        assert torch.equal(got.top_ids[:, :k], torch.where(there, order, -1).int())
        assert torch.all(got.top_ids[:, k:] == -1) and torch.all(got.top_logprob[:, k:] == -INF)
        b = r.b_logp.gather(1, order) + ref.U * lp.abs()
        there = lp > -INF
        assert torch.all(got.top_logprob[:, :k][~there] == -INF)
        learn_ref.close(got.top_logprob[:, :k][there], lp[there], b[there], "top")
    return got, r


# a wave, 256 and 1024 threads a row, and rows split over workgroups
SHAPES = [(1, 1), (3, 2), (1, 255), (1000, 7), (300, 64), (77, 256), (33, 2048), (33, 2049), (300, 4096), (260, 8192), (1, 8192),
          (5, 8191), (300, 16385), (1, 65536), (9, 65537), (257, 65536), (2, 200001), (256, 131072 + 5), (300, 70000)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logprobs(rvq, dev, shape, dtype):
    x, ids = _logits(*shape, dtype, sum(shape), dev)
    for T, top in ((1.0, 0), (0.7, 5), (2.0, 64), (1.0, 1)):
        _check(rvq, x, ids, T, top)
    a = rvq.rvq_token_logprobs(x, ids, top=20)
    b = rvq.rvq_token_logprobs(x, None, top=20, need_entropy=False)
    assert b.logprob is None and b.entropy is None
    assert torch.equal(a.stats, b.stats) and torch.equal(a.top_ids, b.top_ids)
    # the same bits with and without alternatives, and each row whatever stands beside it
    c = rvq.rvq_token_logprobs(x, ids, top=20)
    for u, v in zip(a, c):
        assert torch.equal(u.view(torch.int32), v.view(torch.int32))


@pytest.mark.parametrize("V", [50, 1000, 9001, 65536, 100000])
def test_masked_rows(rvq, dev, V):
    lowest = torch.finfo(F32).min
    for n in (12, 400):
        x, ids = _logits(n, V, F32, V, dev)
        x[0, 1:] = -INF                              # one token left
        x[1, :] = -INF
        x[1, V // 2:V // 2 + 3] = torch.tensor([2.0, 2.0, 1.0], device=dev)
        x[2, ::2] = -INF
        x[3, :] = lowest                             # masked with the type's lowest value, but for three
        x[3, [5, 7, V - 1]] = torch.tensor([1.0, 3.0, 1.0], device=dev)
        x[4, :] = lowest                             # and all of it: uniform
        x[5, :] = 0.0
        x[5, ::3] = -0.0                             # one value, whatever its sign
        x[6, :] = 7.0
        x[7, :] = torch.arange(V, device=dev).float()  # the best in one place
        ids[0], ids[1], ids[2] = 0, V // 2 + 1, 4
        _check(rvq, x, ids, 1.0, 20)
        _check(rvq, x, ids, 0.5, 64)
        got = rvq.rvq_token_logprobs(x, ids, top=4)
        assert got.logprob[0].item() == 0.0 and got.entropy[0].item() == 0.0
        assert got.top_ids[0].tolist() == [0, -1, -1, -1]
        assert got.top_ids[5].tolist() == [0, 1, 2, 3] and got.top_ids[4].tolist() == [0, 1, 2, 3]
        ids[2] = 2                                   # a masked token
        assert rvq.rvq_token_logprobs(x, ids).logprob[2].item() == -INF


@pytest.mark.parametrize("V", [50, 3000, 65536])
def test_rows_without_a_token_or_with_nan_stay_alone(rvq, dev, V):
    for n in (9, 300):
        x, ids = _logits(n, V, F32, V + 1, dev)
        clean = rvq.rvq_token_logprobs(x, ids, top=6)
        ids2 = ids.clone()
        x[2] = -INF
        x[3, V // 3] = float("nan")
        x[4] = float("nan")
        x[5, V - 1] = INF
        ids2[6], ids2[7] = -1, V
        bad = torch.zeros(1, dtype=torch.int32, device=dev)
        got = rvq.rvq_token_logprobs(x, ids2, top=6, bad_ids=bad)
        keep = torch.tensor([i for i in range(n) if i not in (2, 3, 4, 5, 6, 7)], device=dev)
        for u, v in zip(clean, got):
            assert torch.equal(u[keep].view(torch.int32), v[keep].view(torch.int32))
        assert bad.item() == 1 and got.logprob[6].item() == 0.0 and got.logprob[7].item() == 0.0
        assert torch.equal(got.entropy[6:8], clean.entropy[6:8]) and torch.equal(got.top_ids[6:8], clean.top_ids[6:8])
        assert got.logprob[2].item() == -INF and got.entropy[2].item() == 0.0 and got.stats[2].tolist() == [-INF, 0.0]
        assert torch.all(got.top_ids[2] == -1) and torch.all(got.top_logprob[2] == -INF)
        for i in (3, 4, 5):
            assert math.isnan(got.logprob[i]) and math.isnan(got.entropy[i]) and math.isnan(got.stats[i, 1])
            assert torch.all(got.top_ids[i] == -1) and torch.isnan(got.top_logprob[i]).all()
        # the gradient: zeros without a token or a weight, NaN beside NaN, nothing elsewhere
        g, gh = torch.full((n,), 0.5, device=dev), torch.full((n,), 0.25, device=dev)
        d = rvq.rvq_token_logprobs_backward(x, ids2, got.stats, g, got.entropy, gh)
        assert torch.all(d[2] == 0) and torch.isfinite(d[keep]).all()
        assert torch.isnan(d[3]).all() and torch.isnan(d[4]).all() and torch.isnan(d[5]).all()
        g[3:6] = 0
        gh[3:6] = 0
        d = rvq.rvq_token_logprobs_backward(x, ids2, got.stats, g, got.entropy, gh)
        assert torch.all(d[3:6] == 0)
        d = rvq.rvq_token_logprobs_backward(x, ids2, got.stats, g)
        assert torch.all(d[6:8] == 0)


def test_certain_rows_keep_their_small_numbers(rvq, dev):
    # one logit 15 to 60 above the others: 1 - p from 1e-2 down to 1e-22
    for V, n in ((100, 5), (8192, 300), (65536, 3), (65536, 300)):
        x = torch.zeros((n, V), device=dev)
        gap = torch.linspace(15.0, 60.0, n, device=dev)
        ids = (torch.arange(n, device=dev) * 7919 % V).int()
        x[torch.arange(n, device=dev), ids.long()] = gap
        got, r = _check(rvq, x, ids, 1.0, 2)
        # the log probability itself, relative: rest is exact but for its sum's rounding
        want = r.logp[torch.arange(n, device=dev), ids.long()]
        assert torch.all((got.logprob.double() - want).abs() <= 1e-5 * want.abs())
        g = torch.ones(n, device=dev)
        d = rvq.rvq_token_logprobs_backward(x, ids, got.stats, g)
        one = -torch.expm1(want)
        at = d[torch.arange(n, device=dev), ids.long()].double()
        assert torch.all((at - one).abs() <= 2e-5 * one)


def test_far_logits(rvq, dev):
    # what all logits share does not count, however large
    x, ids = _logits(5, 1000, F32, 4, dev)
    x = (x * 64).round() / 64
    a = rvq.rvq_token_logprobs(x, ids, top=4)
    b = rvq.rvq_token_logprobs(x + 4096.0, ids, top=4)
    for i in (0, 1, 3, 4):
        assert torch.equal(a[i], b[i])
    x = torch.tensor([[3e38, -3e38, 0.0], [1e38, 1e38, -INF]], device=dev)
    got = rvq.rvq_token_logprobs(x, torch.tensor([0, 1], device=dev).int(), 1e-4, top=3)
    assert got.logprob[0].item() == 0.0 and got.logprob[1].item() == pytest.approx(-math.log(2), rel=1e-6)
    assert got.top_ids.tolist() == [[0, 2, 1], [0, 1, -1]]


GRAD_SHAPES = [(1, 1), (3, 2), (1000, 7), (77, 256), (33, 2048), (40, 2049), (5, 8191), (1, 65536), (3, 65537), (1100, 3001)]


@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_gradient(rvq, dev, shape, dtype):
    n, V = shape
    x, ids = _logits(n, V, dtype, n + V, dev)
    if n > 2:
        x[1, ::2] = -INF
        ids[2] = -1
    g = torch.Generator(device=dev).manual_seed(5)
    dl, dh = (torch.randn(n, generator=g, device=dev) for _ in range(2))
    for T in (1.0, 0.6):
        s = rvq.rvq_token_logprobs(x, ids, T)
        r = ref.Logits(x, T, _chain(V))
        for a, b in ((dl, None), (None, dh), (dl, dh)):
            for place in ("new", "logits"):
                y = x.clone()
                d = rvq.rvq_token_logprobs_backward(y, ids, s.stats, a, None if b is None else s.entropy, b, T,
                                                    out=y if place == "logits" else None)
                want, bound = ref.logprob_grad(r, ids, a, b, T)
                bound = bound + (ref.BF16_ROUND * want.abs() + 2.0 ** -134 if dtype == BF16 else 2 * ref.U * want.abs() + 2.0 ** -125)
                learn_ref.close(d, want, bound, f"dlogits {place}")


def test_gradient_against_differences(rvq, dev):
    # the loss sum(dl logprob + dh H) in 64 bits, moved by 1e-5 either way
    n, V, T, s = 3, 37, 0.8, 1e-5
    x, ids = _logits(n, V, F32, 1, dev, std=1.0)
    g = torch.Generator(device=dev).manual_seed(5)
    dl, dh = (torch.randn(n, generator=g, device=dev) for _ in range(2))
    st = rvq.rvq_token_logprobs(x, ids, T)
    d = rvq.rvq_token_logprobs_backward(x, ids, st.stats, dl, st.entropy, dh, T)

    def loss(x):
        lp = torch.log_softmax(x / T, 1)
        return float((dl.double() * lp[torch.arange(n, device=dev), ids.long()]).sum() - (dh.double() * (lp.exp() * lp).sum(1)).sum())
    for i in range(n):
        for j in range(0, V, 3):
            e = torch.zeros((n, V), dtype=torch.float64, device=dev)
            e[i, j] = s
            num = (loss(x.double() + e) - loss(x.double() - e)) / (2 * s)
            assert abs(num - d[i, j].item()) <= 1e-4, (i, j)


def test_ties_at_the_last_alternative(rvq, dev):
    # bf16 logits of few values: many equal ones around the last place
    g = torch.Generator(device=dev).manual_seed(3)
    for n, V in ((4, 1000), (300, 5000), (2, 65536), (300, 65536)):
        x = (torch.randn((n, V), generator=g, device=dev) * 4).round().to(BF16)
        ids = torch.zeros(n, dtype=torch.int32, device=dev)
        for top in (1, 7, 64):
            _check(rvq, x, ids, 1.0, top)


def test_offsets_past_32_bits(rvq, dev):
    # 2^32 + elements: the last rows lie beyond a 32-bit element offset
    n, V = 66000, 65536
    x = torch.zeros((n, V), dtype=BF16, device=dev)
    tail, _ = _logits(3, V, BF16, 7, dev)
    x[-3:] = tail
    ids = torch.zeros(n, dtype=torch.int32, device=dev)
    ids[-3:] = torch.tensor([V - 1, 17, 0], device=dev).int()
    got = rvq.rvq_token_logprobs(x, ids, top=3)
    want = rvq.rvq_token_logprobs(torch.cat([x[:300], tail]), torch.cat([ids[:300], ids[-3:]]), top=3)
    for a, b in zip(got, want):
        assert torch.equal(a[-3:].view(torch.int32), b[-3:].view(torch.int32))
    assert got.top_ids[5].tolist() == [0, 1, 2]
    g = torch.zeros(n, device=dev)
    g[-2] = 1.0
    d = rvq.rvq_token_logprobs_backward(x, ids, got.stats, g, out=x)
    e = rvq.rvq_token_logprobs_backward(tail, ids[-3:], got.stats[-3:].contiguous(), g[-3:])
    assert torch.equal(d[-3:], e) and float(d[:-3:997].float().abs().sum()) == 0.0


def test_refusals(rvq, dev):
    x, ids = _logits(4, 32, F32, 1, dev)
    s = rvq.rvq_token_logprobs(x, ids)
    one = torch.ones(4, device=dev)
    for bad in (dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.cpu()), dict(bad_ids=ids)):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_token_logprobs(x, **{**dict(ids=ids), **bad})
    for bad in (x.cpu(), x[0], x.double(), x[:, ::2], x.t(), x.clone().requires_grad_()):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_token_logprobs(bad)
    for bad in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")), dict(top=65), dict(top=-1)):
        with pytest.raises(rvq.RVQError):
            rvq.rvq_token_logprobs(x, ids, **bad)
    ok = dict(logits=x, ids=ids, stats=s.stats, dlogprob=one)
    for bad in (dict(stats=s.stats[:3]), dict(stats=s.stats.double()), dict(dlogprob=None), dict(dlogprob=one[:3]), dict(ids=None),
                dict(dentropy=one), dict(out=x[:3]), dict(out=x.bfloat16()), dict(logits=x.bfloat16()[0]),
                dict(dlogprob=one.clone().requires_grad_()), dict(entropy=one[:2], dentropy=one)):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_token_logprobs_backward(**{**ok, **bad})
    buf = torch.zeros(4 * 32 + 8, device=dev)
    with pytest.raises(rvq.RVQError):                # an overlap that is not in place
        rvq.rvq_token_logprobs_backward(buf[:128].view(4, 32), ids, s.stats, one, out=buf[8:136].view(4, 32))
    e = rvq.rvq_token_logprobs(x[:0], ids[:0], top=3)
    assert e.logprob.shape == (0,) and e.top_ids.shape == (0, 3)
    assert rvq.rvq_token_logprobs_backward(x[:0], ids[:0], e.stats, one[:0]).shape == (0, 32)


def _top_of(x, k):
    order = torch.argsort(x.float() + 0.0, dim=1, descending=True, stable=True)[:, :k]
    return order, x.float().gather(1, order)


@pytest.mark.parametrize("shape", [(5, 2500), (3, 65536), (260, 33000), (170, 65536), (300, 9001)], ids=lambda s: "x".join(map(str, s)))
def test_alternatives_among_equal_and_near_values(rvq, dev, shape):
    """More than 1024 values reach the bound of the first search: masks of the type's lowest
    value that leave fewer tokens than are asked for, rows of equal values, and fp32 values
    whose upper halves are the same."""
    n, V = shape
    g = torch.Generator(device=dev).manual_seed(V)
    for dtype in (F32, BF16):
        low = torch.finfo(dtype).min
        x = torch.full((n, V), low, device=dev, dtype=dtype)
        x[0] = 0.5                                                  # all equal
        x[1, :] = -INF
        x[1, V // 2:V // 2 + 1500] = low                            # some of them, behind a middle
        for r in range(2, n):                                       # 0 to 14 tokens are left
            x[r, torch.randint(0, V, (r % 15,), generator=g, device=dev)] = torch.randn(r % 15, generator=g, device=dev).to(dtype)
        x[2, ::3] = -0.0
        x[2, 1::3] = 0.0
        for k in (1, 5, 20, 64):
            got = rvq.rvq_token_logprobs(x, torch.zeros(n, dtype=torch.int32, device=dev), top=k)
            ids, values = _top_of(x, k)
            assert torch.equal(got.top_ids, torch.where(values > -INF, ids, -1).int()), (dtype, k)
    # 1 to 1 + 2^-9 in steps of 2^-23: no two values alike in the first 2^14 columns
    x = 1 + torch.randperm(V, generator=g, device=dev).expand(n, V).contiguous() % 2 ** 14 * 2.0 ** -23
    for k in (3, 64):
        got = rvq.rvq_token_logprobs(x, top=k)
        assert torch.equal(got.top_ids, _top_of(x, k)[0].int()), k


def test_alternatives_where_one_thread_holds_the_largest(rvq, dev):
    # 4 columns of each 1024 hold all of the largest values: more than 1024 above the bound
    n, V = 260, 300000
    x = torch.rand(V, device=dev).expand(n, V).contiguous()
    x[:, (torch.arange(V, device=dev) // 4) % 256 == 77] += 5
    got = rvq.rvq_token_logprobs(x, top=3)
    assert torch.equal(got.top_ids, _top_of(x, 3)[0].int())
