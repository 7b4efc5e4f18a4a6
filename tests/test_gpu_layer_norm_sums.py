"""How the sums over rows of rvq_layer_norm_backward are joined."""
import pytest
import torch

import head_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 300, 1024, 1030])
def test_parts_are_joined_without_a_rounding_each(n):
    """Up to 1536 rows of 1152 fp32 values go to workgroups that sum two rows each: one addition,
    off by U of its part at most, and the joined sum is rounded once: 2 U of the sum of magnitudes
    (and 2^-40 of it for the join's own 64 bits)."""
    import residual_vector_quantization_rvq_amd as rvq
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(n)
    dy = 1 + torch.rand((n, 1152), generator=g, device=dev)
    h = torch.randn((n, 1152), generator=g, device=dev)
    st = rvq.rvq_layer_norm(h, need_stats=True)
    _, dw, db = rvq.rvq_layer_norm_backward(dy, h, st.mean, st.rstd)
    want = dy.double().sum(0)
    assert torch.all((db.double() - want).abs() <= (2 * ref.U + 2.0 ** -40) * want)
    # a term of dweight is rounded three times (the difference, u, and with the sum)
    term = dy.double() * (h.double() - st.mean.double()[:, None]) * st.rstd.double()[:, None]
    assert torch.all((dw.double() - term.sum(0)).abs() <= (6 * ref.U + 2.0 ** -40) * term.abs().sum(0))
