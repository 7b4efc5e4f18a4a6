"""rvq_layer_norm_backward at the ends of fp32's range."""
import pytest
import torch

import head_ref as ref
import learn_ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def _chain(d):
    # additions that one lane makes one after the other, the tree over lanes, the roundings of a term
    return max(d / 64, 64) + 24


def _randn(shape, seed, dev, dtype=F32):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(dtype)


def _check(rvq, h, dy, eps, dsum=None):
    """The whole call on rows h with the forward call's own statistics, against 64 bits."""
    n, d = h.shape
    w = 1 + 0.2 * _randn((d,), 5, h.device)
    st = rvq.rvq_layer_norm(h, w, None, eps, need_stats=True)
    mean = h.double().mean(1)
    learn_ref.close(st.mean, mean, 2 * ref.U * mean.abs() + _chain(d) * ref.U * (h.double() - mean[:, None]).abs().mean(1), "mean")
    dx, size, dw, dwsize, db, dbsize = ref.layer_norm_grad(dy, h, st.mean, st.rstd, w, dsum)
    got, gotw, gotb = rvq.rvq_layer_norm_backward(dy, h, st.mean, st.rstd, w, dsum=dsum)
    # beside the bound of ordinary rows: results below fp32's (bf16's) normal numbers have a fixed step
    bound = _chain(d) * ref.U * size + 2.0 ** -147
    if h.dtype == BF16:
        bound = bound + ref.BF16_ROUND * dx.abs() + 2.0 ** -134
    learn_ref.close(got, dx, bound, "dx")
    b = (min(n, n / 256 + 512) + 16) * ref.U
    learn_ref.close(gotw, dw, b * dwsize, "dweight")
    learn_ref.close(gotb, db, b * dbsize, "dbias")


# widths that end inside a 16-byte piece (4 fp32, 8 bf16), and some that do not; rows too wide for registers
WIDTHS = [1, 3, 8, 41, 63, 255, 1001, 1152, 1155, 2050, 5001, 9001, 20001]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_of_one_large_value(rvq, dev, d, dtype):
    """Equal values have u = 0 whatever their size; mean times rstd may be beyond fp32, also
    for the places behind a row's end."""
    for eps, values in ((1e-6, (4e35, -3e38)), (1e-30, (1e24, -1e36))):
        h = _randn((9, d), d, dev)
        h[2], h[5] = values[0], values[1]
        for dsum in (None, _randn((9, d), d + 1, dev, dtype)):
            _check(rvq, h.to(dtype), _randn((9, d), d + 2, dev, dtype), eps, dsum)


@pytest.mark.parametrize("d", [3, 9, 41, 255, 1001, 1152, 5001, 9001, 20001])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_differences_beyond_the_range(rvq, dev, d, dtype):
    """A third of a row at 3.3e38 and the rest at -3e38: the values are within fp32, their
    distances from the mean (4.2e38) are not."""
    g = torch.Generator(device=dev).manual_seed(d)
    h = _randn((7, d), d, dev)
    at = torch.arange(d, device=dev)
    sign = torch.where(at % 3 == 0, 3.3e38, -3e38)
    h[1] = sign * (1 - 0.01 * torch.rand(d, generator=g, device=dev))
    h[4] = -sign * (1 - 0.01 * torch.rand(d, generator=g, device=dev))
    for dsum in (None, _randn((7, d), d + 1, dev, dtype)):
        _check(rvq, h.to(dtype), _randn((7, d), d + 2, dev, dtype), 1e-6, dsum)
