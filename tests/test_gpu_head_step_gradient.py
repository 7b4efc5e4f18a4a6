"""The gradients of the training step around a model's head (test_gpu_head_step.Step): what arrives
at the logits and at the rows, and the losses, each against 64 bits on the step's own tensors."""
import pytest
import torch

import head_ref as ref
import learn_ref
from test_gpu_head_step import Step

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def test_losses_and_gradients_of_the_step():
    import residual_vector_quantization_rvq_amd as rvq
    dev = torch.device("cuda:0")
    s = Step(rvq, dev)
    gain, bias = s.gain.clone(), s.bias.clone()         # the step updates its parameters
    _, h, logits, lp, ent, _, _, kl, dlogits, dy, _, dx, dgain, dbias, _ = s.run()
    n, V = logits.shape
    d = h.shape[1]
    chain = max(V / 64, 64) + 32
    r = ref.Logits(logits, 0.9, chain)
    learn_ref.close(ent, r.H[:, 0], (r.b_H + 2 * ref.U * r.H)[:, 0], "entropy")
    has = (s.ids >= 0)
    at = s.ids.clamp(min=0).long()[:, None]
    want = r.logp.gather(1, at)[:, 0]
    learn_ref.close(lp[has], want[has], (r.b_logp.gather(1, at)[:, 0] + ref.U * want.abs())[has], "logprob")
    assert torch.all(lp[~has] == 0)
    loss, b_loss, d2, b2 = ref.distill(logits, s.tids, s.t, 2.0, False, chain)
    learn_ref.close(kl, loss, b_loss, "distillation loss")
    # the logits' gradient: two results rounded to bf16, and their sum
    d1, b1 = ref.logprob_grad(r, s.ids, s.dlp, s.dent, 0.9)
    d2, b2 = d2 * s.dloss.double()[:, None], b2 * s.dloss.double()[:, None] + 2 * ref.U * d2.abs() * s.dloss.double()[:, None]
    bound = b1 + 2 * ref.U * d1.abs() + b2 + 2.0 ** -124 + ref.BF16_ROUND * (d1.abs() + d2.abs())
    bound = bound + ref.BF16_ROUND * ((d1 + d2).abs() + bound) + 2.0 ** -132
    learn_ref.close(dlogits, d1 + d2, bound, "dlogits")
    # the rows' gradient from the tensors that the step gave the call; the same call gives the same statistics
    st = rvq.rvq_layer_norm(s.x, gain, bias, residual=s.res, need_stats=True)
    assert torch.equal(st.sum.view(torch.int16), h.view(torch.int16))
    want, size, dw, dwsize, db, dbsize = ref.layer_norm_grad(dy, h, st.mean, st.rstd, gain, s.res)
    learn_ref.close(dx, want, (max(d / 64, 64) + 24) * ref.U * size + ref.BF16_ROUND * want.abs(), "dx")
    b = (min(n, n / 256 + 512) + 16) * ref.U
    learn_ref.close(dgain, dw, b * dwsize, "dgain")
    learn_ref.close(dbias, db, b * dbsize, "dbias")
