"""The calls that train the token embedding at the edges of their types."""

import pytest
import torch

import learn_ref as ref
import test_gpu_adamw as adamw_tests
import test_gpu_embed_grad as embed_tests
import test_gpu_norm as norm_tests

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")
MAX = 3.4028234663852886e38


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


# a part of a wave, a wave, a workgroup per row; rows that are read again
@pytest.mark.parametrize("dtype,d", [(F32, 7), (F32, 40), (F32, 700), (F32, 3000), (F32, 9000),
                                     (BF16, 40), (BF16, 4096), (BF16, 20001)])
def test_norm_8_bit_rows_show_a_weight_that_is_not_finite(rvq, dev, dtype, d):
    x = norm_tests._rows(5, d, dtype, d, dev)
    x[3] = 0.0                                  # 0 * NaN and 0 * infinity are NaN too
    for bad in (NAN, INF, -INF):
        for at in (0, d // 2, d - 1):
            w = torch.ones(d, device=dev)
            w[at] = bad
            out = rvq.rvq_rms_norm(x, w, out_dtype=F8)
            plain = rvq.rvq_rms_norm(x, w)
            assert not torch.isfinite(plain.y[:, at]).any()
            assert torch.isnan(out.scale).all(), (bad, at)
            assert torch.isnan(out.y.float() * out.scale[:, None])[:, at].all()
    # finite weights: the scale is the row's
    assert torch.isfinite(rvq.rvq_rms_norm(x, torch.ones(d, device=dev), out_dtype=F8).scale).all()


@pytest.mark.parametrize("dtype,n,d", [(F32, 20000, 64), (F32, 6000, 1152), (F32, 300, 20001), (BF16, 3000, 4096),
                                       (BF16, 300, 30000)])
def test_norm_8_bit_values_are_those_of_the_quotient(rvq, dev, dtype, n, d):
    # y in fp32 is what the 8-bit rows are made of: their bytes have to be the
    # quotients' (in fp32, correctly rounded, as the CPU divides) to the bit
    x = norm_tests._rows(n, d, dtype, d, dev)
    w = 1 + 0.2 * norm_tests._rows(1, d, F32, 5, dev, False)[0]
    y = rvq.rvq_rms_norm(x, w, out_dtype=F32).y.cpu()
    out = rvq.rvq_rms_norm(x, w, out_dtype=F8)
    scale = out.scale.cpu()
    top = y.abs().amax(1)
    assert torch.all((scale.double() - top.double() / 448).abs() <= 2 * ref.U * scale.double())
    want = (y / scale[:, None]).clamp(-448, 448).to(F8).view(torch.uint8)
    off = int((want != out.y.cpu().view(torch.uint8)).sum())
    assert off == 0, f"{off} of {n * d} bytes"
