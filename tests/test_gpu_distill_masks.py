"""rvq_distill_loss with the rest as one outcome, where the other tokens are masked: by -inf or by
a large negative value alike."""
import math

import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
MASKS = [-math.inf, torch.finfo(F32).min, torch.finfo(BF16).min, -1e30, -1e9, -65504.0, -1e4, -400.0]


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def _case(n, V, k, mask, dtype, dev):
    """k tokens a row that are not masked, all of them the teacher's, whose logarithms are rounded:
    its weights add up to 1 but for that."""
    g = torch.Generator(device=dev).manual_seed(V + k)
    x = (torch.randn((n, V), generator=g, device=dev) * 3).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=g, device=dev)[:k] for _ in range(n)])
    mine = x.gather(1, ids)
    x = torch.full_like(x, mask).scatter(1, ids, mine)
    t = torch.log_softmax(mine.float() + torch.randn((n, k), generator=g, device=dev), 1)
    logp = torch.log_softmax(x.double(), 1)
    return x, ids.int().contiguous(), t.contiguous(), logp.gather(1, ids)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,V,k", [(2000, 300, 40), (300, 256, 250), (100, 5000, 20), (40, 70000, 64)])
def test_masked_others_take_no_rest(rvq, dev, n, V, k, dtype):
    one = torch.ones(n, device=dev)
    for mask in MASKS:
        if dtype == BF16 and mask == torch.finfo(F32).min:
            continue                                # rounds to -inf
        x, ids, t, logp = _case(n, V, k, mask, dtype, dev)
        q, p = t.double().exp(), logp.exp()
        assert bool((1 - q.sum(1) > 0).any())       # some rows have a rest by rounding
        want = (q * (t.double() - logp)).sum(1)
        got = rvq.rvq_distill_loss(x, ids, t, 1.0, True)
        # log p within 160 roundings (chains, trees) and 3 of d < 40
        assert torch.all((got.loss.double() - want).abs() <= (160 + 120) * ref.U + ref.U * want.abs()), mask
        for place in (None, x.clone()):
            d = rvq.rvq_distill_loss_backward(x if place is None else place, ids, t, got.stats, one, 1.0, True, out=place)
            grad = torch.zeros((n, V), device=dev, dtype=torch.float64).scatter(1, ids.long(), p - q)
            bound = (160 + 120) * ref.U * (p.amax(1, keepdim=True) + 1)
            if dtype == BF16:
                bound = bound + ref.BF16_ROUND * grad.abs()
            assert torch.all((d.double() - grad).abs() <= bound), mask
            others = torch.ones((n, V), dtype=torch.bool, device=dev).scatter(1, ids.long(), False)
            assert torch.all(d[others] == 0), mask


@pytest.mark.parametrize("V", [300, 5000, 70000])
def test_a_rest_that_is_weight_meets_the_mask(rvq, dev, V):
    """A hundredth of the teacher's weight on masked tokens: infinite with -inf, else by the formula."""
    for mask in MASKS:
        x, ids, t, logp = _case(20, V, 30, mask, F32, dev)
        t = t - 0.01
        got = rvq.rvq_distill_loss(x, ids, t, 1.0, True).loss
        if mask == -math.inf:
            assert torch.all(torch.isinf(got))
            continue
        q = t.double().exp()
        rest = 1 - q.sum(1)
        log_left = torch.logsumexp(torch.log_softmax(x.double(), 1).scatter(1, ids.long(), -math.inf), 1)
        want = (q * (t.double() - logp)).sum(1) + rest * (rest.log() - log_left)
        assert torch.all((got.double() - want).abs() <= (160 + 120 + 8) * ref.U * (1 + want.abs())), mask
