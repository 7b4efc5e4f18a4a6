"""The sums of rvq_matmul_f8: fp32 whatever the result's type and the number of rows."""
import pytest
import torch

import head_ref as ref
import learn_ref

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


def _operand(rvq, rows, k, kind, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((rows, k), generator=g, device=dev) * torch.exp(torch.randn((rows, 1), generator=g, device=dev))
    if kind == "row":
        scale = (x.abs().amax(1) / ref.F8_MAX).clamp(min=1e-30)
        return (x / scale[:, None]).clamp(-448, 448).to(F8), scale
    return rvq.rvq_quantize_f8(x, 128 if kind == "block" else 1)


# straight from memory and in tiles: tiles that share k, of 128 x 128 and larger, whole and broken
SHAPES = [(1, 300, 1000), (1, 4096, 4096), (12, 513, 640), (17, 40000, 128), (33, 257, 640), (300, 500, 129), (512, 640, 100),
          (700, 513, 5000), (1100, 4100, 400), (2560, 4200, 384), (4100, 5001, 273), (4096, 8192, 256)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", ["block", "line", "row"])
def test_a_bf16_result_is_the_fp32_result_rounded_once(rvq, dev, shape, kind):
    m, n, k = shape
    a, sa = _operand(rvq, m, k, "line", 1, dev)
    b, sb = _operand(rvq, n, k, kind, 2, dev)
    want = rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=F32)
    got = rvq.rvq_matmul_f8(a, sa, b, sb)
    assert got.dtype == BF16 and torch.equal(got.view(torch.int16), want.to(BF16).view(torch.int16))
    apart = []
    for t in (a, b):        # rows at any byte, 0x7f (NaN) between them
        buf = torch.full((t.shape[0], k + 3), 0x7f, dtype=torch.uint8, device=dev).view(F8)
        buf[:, :k] = t
        apart.append(buf[:, :k])
    assert torch.equal(rvq.rvq_matmul_f8(apart[0], sa, apart[1], sb).float(),
                       rvq.rvq_matmul_f8(apart[0], sa, apart[1], sb, out_dtype=F32).to(BF16).float())


@pytest.mark.parametrize("m,n,k", [(5, 700, 1024), (300, 700, 1024), (1100, 4100, 640), (2560, 4200, 384)])
@pytest.mark.parametrize("kind", ["block", "line", "row"])
def test_sums_that_cancel(rvq, dev, m, n, k, kind):
    """Each large product is beside its negative, and a small product is left: bf16 results are
    within a rounding and fp32's bound of it."""
    g = torch.Generator(device=dev).manual_seed(k)
    a = torch.randn((m, k), generator=g, device=dev)
    b = torch.randn((n, k), generator=g, device=dev)
    a[:, 1::4], b[:, 1::4] = -a[:, 0::4], b[:, 0::4]
    a[:, 2::4] *= 2.0 ** -6
    a[:, 3::4] *= 2.0 ** -6
    a, sa = rvq.rvq_quantize_f8(a)
    if kind == "row":
        scale = (b.abs().amax(1) / ref.F8_MAX)
        b, sb = (b / scale[:, None]).clamp(-448, 448).to(F8), scale
    else:
        b, sb = rvq.rvq_quantize_f8(b, 128 if kind == "block" else 1)
    want, size = ref.matmul(a, sa, b, sb)
    bound = ref.matmul_bound(size, k)
    assert float(want.abs().median()) < 0.02 * float(size.median())
    learn_ref.close(rvq.rvq_matmul_f8(a, sa, b, sb), want, bound * (1 + 2 ** -8) + ref.BF16_ROUND * want.abs(), "bf16")
    learn_ref.close(rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=F32), want, bound + ref.U * want.abs(), "fp32")
