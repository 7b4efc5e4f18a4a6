"""The 8-bit quantiser and the product of 8-bit operands against 64 bits."""
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


def _rows(n, d, dtype, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((n, d), generator=g, device=dev)
    x *= torch.exp(3.0 * torch.randn((n, 1), generator=g, device=dev))     # rows of unlike sizes
    x[:, ::max(1, d // 3)] *= 30.0
    return x.to(dtype)


def _check_quantised(rvq, x, block_rows, transpose):
    q, scale = rvq.rvq_quantize_f8(x, block_rows, transpose)
    y = x.t().contiguous() if transpose else x
    assert q.shape == y.shape and q.dtype == F8 and scale.dtype == F32
    want = ref.block_scale(y, block_rows)
    assert torch.equal(scale, want.float())          # the nearest fp32 quotient
    s = ref.spread(scale, y.shape)
    v = y.double() / s
    near = torch.clamp(v, -ref.F8_MAX, ref.F8_MAX)
    # half a step, and the quotient's own rounding to fp32 before it
    learn_ref.close(q.float(), near, learn_ref.f8_step(v) * 0.5 + 2 * ref.U * v.abs(), "q")
    return q, scale


@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 7), (5, 127), (130, 129), (128, 128), (1, 4096), (300, 1155),
                                   (257, 640), (1000, 16), (17, 5000)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_quantise(rvq, dev, shape, dtype):
    x = _rows(*shape, dtype, sum(shape), dev)
    for block_rows in (1, 128):
        for transpose in (False, True):
            _check_quantised(rvq, x, block_rows, transpose)


def test_quantise_edges(rvq, dev):
    x = _rows(200, 300, F32, 1, dev)
    x[3] = 0.0                                       # a block of zeros: the smallest scale
    x[5, :128] = 1e-38
    for block_rows in (1, 128):
        for transpose in (False, True):
            _check_quantised(rvq, x, block_rows, transpose)
    q, scale = rvq.rvq_quantize_f8(x)
    assert torch.all(scale[3] == 2.0 ** -100) and torch.all(q[3].float() == 0)
    # a value that is not finite shows in its block's scale and in no other
    bad = x.clone()
    bad[7, 130] = float("nan")
    bad[9, 299] = float("inf")
    q2, s2 = rvq.rvq_quantize_f8(bad)
    hit = torch.zeros_like(scale, dtype=torch.bool)
    hit[7, 1] = hit[9, 2] = True
    assert torch.isnan(s2[hit]).all() and torch.equal(s2[~hit], scale[~hit])
    _, s3 = rvq.rvq_quantize_f8(bad, transpose=True)
    assert int(torch.isnan(s3).sum()) == 2 and torch.isnan(s3[130, 0]) and torch.isnan(s3[299, 0])
    _, s4 = rvq.rvq_quantize_f8(bad, 128, transpose=True)
    assert int(torch.isnan(s4).sum()) == 2 and torch.isnan(s4[1, 0]) and torch.isnan(s4[2, 0])
    # rows that begin at any element; empty ones
    y = torch.empty(200 * 300 + 1, device=dev)[1:].view(200, 300).copy_(x)
    for a, b in zip(rvq.rvq_quantize_f8(y), rvq.rvq_quantize_f8(x)):
        assert torch.equal(a.float(), b.float())
    for n, d in ((0, 5), (5, 0)):
        q, s = rvq.rvq_quantize_f8(torch.empty((n, d), device=dev))
        assert q.shape == (n, d) and s.shape == (n, -(-d // 128))


def test_quantise_leaves_what_is_between_rows(rvq, dev):
    x = _rows(40, 37, BF16, 2, dev)
    for transpose, r, c in ((False, 40, 37), (True, 37, 40)):
        buf = torch.full((r, 64), 0x55, dtype=torch.uint8, device=dev)
        scale = torch.empty((r, 1), device=dev)
        st = rvq.raw_library().rvq_quantize_f8(x.data_ptr(), 1, 40, 37, 1, int(transpose), buf.data_ptr(), 64,
                                               scale.data_ptr(), None)
        torch.cuda.synchronize()
        assert st == 0 and torch.all(buf[:, c:] == 0x55)
        q, s = rvq.rvq_quantize_f8(x, transpose=transpose)
        assert torch.equal(buf[:, :c], q.contiguous().view(torch.uint8)) and torch.equal(s, scale)


def _operand(rvq, rows, k, kind, seed, dev):
    x = _rows(rows, k, F32, seed, dev)
    if kind == "row":
        scale = (x.abs().amax(1) / ref.F8_MAX).clamp(min=1e-30)
        return (x / scale[:, None]).clamp(-448, 448).to(F8), scale
    return rvq.rvq_quantize_f8(x, 128 if kind == "block" else 1)


def _check_product(rvq, a, sa, b, sb, odt, **kw):
    got = rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=odt, **kw)
    assert got.shape == (a.shape[0], b.shape[0]) and got.dtype == odt
    want, size = ref.matmul(a, sa, b, sb)
    bound = ref.matmul_bound(size, a.shape[1], odt == BF16)
    bound = bound * (1 + (2 ** -8 if odt == BF16 else 0)) + (ref.BF16_ROUND if odt == BF16 else ref.U) * want.abs()
    learn_ref.close(got, want, bound, f"product {tuple(a.shape)} x {tuple(b.shape)}")
    return got


# one row, few rows, tiles and what is left of them, contractions within, at and past a block
SHAPES = [(1, 1, 1), (1, 16, 128), (1, 1000, 4096), (2, 17, 31), (5, 300, 129), (16, 64, 256), (17, 65, 384), (33, 257, 640),
          (64, 64, 16), (64, 1152, 1152), (65, 100, 1155), (100, 129, 112), (128, 128, 128), (129, 256, 1000), (200, 700, 2048),
          (256, 256, 1024), (257, 511, 4096), (300, 1000, 1280), (512, 640, 100), (1000, 1024, 256), (700, 513, 5000),
          # few rows beside many, on either side; tiles of each size, whole and broken
          (1, 50000, 260), (16, 40001, 1000), (17, 33000, 128), (32, 30000, 129), (30000, 16, 200), (40000, 31, 1155), (40000, 20, 256),
          (900, 1300, 300), (1300, 1400, 1155), (2560, 4200, 384), (4100, 5001, 273), (4096, 8192, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product(rvq, dev, shape):
    m, n, k = shape
    for i, (ka, kb) in enumerate((("row", "block"), ("line", "block"), ("line", "line"), ("block", "row"), ("row", "row"))):
        a, sa = _operand(rvq, m, k, ka, i, dev)
        b, sb = _operand(rvq, n, k, kb, i + 10, dev)
        _check_product(rvq, a, sa, b, sb, (F32, BF16)[i & 1])


def test_product_of_small_whole_numbers_is_exact(rvq, dev):
    g = torch.Generator(device=dev).manual_seed(3)
    for m, n, k in ((1, 333, 1000), (7, 128, 2048), (100, 300, 999), (256, 512, 1024), (515, 700, 640), (1024, 2048, 4096),
                    (9, 44000, 500), (31, 34000, 300), (2700, 4300, 999)):
        a = torch.randint(-4, 5, (m, k), generator=g, device=dev).to(F8)
        b = torch.randint(-4, 5, (n, k), generator=g, device=dev).to(F8)
        kb = -(-k // 128)
        sa = torch.pow(2.0, torch.randint(-1, 2, (m, kb), generator=g, device=dev).float())
        sb = torch.pow(2.0, torch.randint(-1, 2, (n, kb), generator=g, device=dev).float())
        sblock = torch.pow(2.0, torch.randint(-1, 2, (-(-n // 128), kb), generator=g, device=dev).float())
        for s in (sb, sblock, sb[:, 0].contiguous()):
            want, _ = ref.matmul(a, sa, b, s)
            # terms are multiples of 1/4 and their sums below 2^18
            assert torch.equal(rvq.rvq_matmul_f8(a, sa, b, s, out_dtype=F32).double(), want), (m, n, k, tuple(s.shape))


def test_product_of_rows_that_are_apart(rvq, dev):
    # padding between rows (NaN bytes in it), slices of columns, rows at any byte
    # (few rows of one operand, and tiles, for which both ways are the same sums in the same order)
    for m, n, k in ((3, 200, 300), (70, 130, 777), (300, 260, 1000), (260, 513, 130), (1100, 1000, 300), (1000, 2100, 130)):
        a, sa = _operand(rvq, m, k, "line", 1, dev)
        b, sb = _operand(rvq, n, k, "block", 2, dev)
        want = rvq.rvq_matmul_f8(a.contiguous(), sa, b.contiguous(), sb, out_dtype=F32)
        for stride in (k + 1, k + -k % 16 + 16, k + -k % 128 + 128):
            wide = []
            for t in (a, b):
                buf = torch.full((t.shape[0], stride), 0x7f, dtype=torch.uint8, device=dev).view(F8)
                buf[:, :k] = t
                wide.append(buf[:, :k])
            assert torch.equal(rvq.rvq_matmul_f8(wide[0], sa, wide[1], sb, out_dtype=F32), want), (m, n, k, stride)
        bytes_a = torch.empty(m * k + 1, dtype=torch.uint8, device=dev)[1:].view(F8).view(m, k)
        bytes_a.copy_(a)
        _check_product(rvq, bytes_a, sa, b, sb, F32)


def test_product_empty_and_nan(rvq, dev):
    a, sa = _operand(rvq, 40, 300, "line", 1, dev)
    b, sb = _operand(rvq, 200, 300, "block", 2, dev)
    want = rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=F32)
    e = lambda r, k: torch.empty((r, k), device=dev).to(F8)  # noqa: E731
    assert rvq.rvq_matmul_f8(e(0, 300), torch.empty((0, 3), device=dev), b, sb).shape == (0, 200)
    assert rvq.rvq_matmul_f8(a, sa, e(0, 300), torch.empty((0, 3), device=dev)).shape == (40, 0)
    z = rvq.rvq_matmul_f8(e(4, 0), torch.ones(4, device=dev), e(5, 0), torch.ones(5, device=dev), out_dtype=F32)
    assert z.shape == (4, 5) and torch.all(z == 0)
    # a NaN scale or byte reaches its rows' results and no others
    s2 = sa.clone()
    s2[7, 2] = float("nan")
    got = rvq.rvq_matmul_f8(a, s2, b, sb, out_dtype=F32)
    keep = torch.arange(40, device=dev) != 7
    assert torch.isnan(got[7]).all() and torch.equal(got[keep], want[keep])
    b2 = b.contiguous().clone()
    b2.view(torch.uint8)[11, 299] = 0x7f
    got = rvq.rvq_matmul_f8(a, sa, b2, sb, out_dtype=F32)
    keep = torch.arange(200, device=dev) != 11
    assert torch.isnan(got[:, 11]).all() and torch.equal(got[:, keep], want[:, keep])


def test_product_repeats_and_rows_do_not_depend_on_others(rvq, dev):
    for m, n, k in ((5, 900, 4096), (300, 700, 2000), (1000, 513, 1024)):
        a, sa = _operand(rvq, m, k, "line", 1, dev)
        b, sb = _operand(rvq, n, k, "block", 2, dev)
        x = rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=F32)
        y = torch.full((m, n), float("nan"), device=dev)
        assert rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=F32, out=y) is y
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))


def test_both_gradients_of_a_linear_layer(rvq, dev):
    # y = x w^T: dx = dy w, dw = dy^T x with transposed operands
    T, K, N = 333, 260, 391
    x, w, dy = _rows(T, K, BF16, 1, dev), _rows(N, K, BF16, 2, dev), _rows(T, N, BF16, 3, dev)
    qd, sd = rvq.rvq_quantize_f8(dy)
    qw, sw = rvq.rvq_quantize_f8(w, 128, transpose=True)
    # 128 x 128 blocks turn with the matrix
    q0, s0 = rvq.rvq_quantize_f8(w, 128)
    assert torch.equal(qw.float(), q0.float().t()) and torch.equal(sw, s0.t())
    dx = _check_product(rvq, qd, sd, qw, sw, F32)
    qa, sa = rvq.rvq_quantize_f8(dy, transpose=True)
    qx, sx = rvq.rvq_quantize_f8(x, transpose=True)
    dw = _check_product(rvq, qa, sa, qx, sx, F32)
    # against the exact gradients: an operand's value is off by half a step of its grid at most, 2^-4 of
    # itself (or 2^-10 scales where it is far below its block's largest), so a product by (2 2^-4 + 2^-8) of
    # the sum of magnitudes, plus what small values lose
    for got, (p, sp, fp), (q, sq, fq) in ((dx, (qd, sd, dy), (qw, sw, w.t())), (dw, (qa, sa, dy.t()), (qx, sx, x.t()))):
        p0, q0 = fp.double(), fq.double()
        ep = p0.abs() * 2 ** -4 + ref.spread(sp, p0.shape) * 2 ** -10
        eq = q0.abs() * 2 ** -4 + ref.spread(sq, q0.shape) * 2 ** -10
        bound = ep @ q0.abs().t().contiguous() + p0.abs() @ eq.t().contiguous() + ep @ eq.t().contiguous()
        learn_ref.close(got, p0 @ q0.t().contiguous(), bound * (1 + 1e-3), "gradient")


def test_norm_rows_are_operands(rvq, dev):
    x = _rows(50, 1155, BF16, 4, dev)
    b, sb = _operand(rvq, 300, 1155, "block", 5, dev)
    for norm in (rvq.rvq_rms_norm, rvq.rvq_layer_norm):
        r = norm(x, out_dtype=F8)
        _check_product(rvq, r.y, r.scale, b, sb, F32)


def test_product_refusals(rvq, dev):
    a, sa = _operand(rvq, 40, 300, "line", 1, dev)
    b, sb = _operand(rvq, 200, 300, "block", 2, dev)
    c = a.contiguous()
    for bad in (dict(a=c.float()), dict(a=c[0]), dict(a=c.cpu()), dict(a=c[:, :299]), dict(a=c.t()), dict(a=c[:1].expand(40, 300)),
                dict(a_scale=sa.double()), dict(a_scale=sa[:39]), dict(a_scale=sa.cpu()), dict(a_scale=sa[:, :2]),
                dict(a_scale=sa.t().contiguous().t()), dict(b_scale=sb.t()), dict(b=c), dict(out=torch.empty(40, 199, device=dev)),
                dict(out_dtype=torch.float16), dict(out=torch.empty(40, 200, device=dev)),
                dict(a_scale=sa.clone().requires_grad_())):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_matmul_f8(**{**dict(a=a, a_scale=sa, b=b, b_scale=sb), **bad})
    # a last row whose memory ends before the others' padding
    buf = torch.zeros(40 * 304 - 4, dtype=torch.uint8, device=dev).view(F8)
    short = buf.as_strided((40, 300), (304, 1))
    with pytest.raises(ValueError):
        rvq.rvq_matmul_f8(short, sa, b, sb)
    x = _rows(4, 32, F32, 1, dev)
    for bad in (x.cpu(), x[0], x.double(), x[:, ::2], x.clone().requires_grad_()):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_quantize_f8(bad)
    with pytest.raises(ValueError):
        rvq.rvq_quantize_f8(x, 64)


@pytest.mark.parametrize("shape", [(1100, 4100, 400), (1700, 2600, 1155), (2050, 4097, 128), (130, 140, 100), (300, 500, 129), (900, 1000, 257)],
                         ids=lambda s: "x".join(map(str, s)))
def test_tiles_that_share_k_and_tiles_that_do_not(rvq, dev, shape):
    """More tiles of 128 than a device has CUs, and fewer (then two groups of waves share k, one of
    them without a block where k is a block or less): every layout, result and alignment."""
    m, n, k = shape
    a, sa = _operand(rvq, m, k, "line", 1, dev)
    for kind in ("block", "line", "row"):
        b, sb = _operand(rvq, n, k, kind, 2, dev)
        for odt in (F32, BF16):
            want = _check_product(rvq, a, sa, b, sb, odt)
            apart = []
            for t in (a, b):        # rows at any byte, 0x7f (NaN) between them
                buf = torch.full((t.shape[0], k + 3), 0x7f, dtype=torch.uint8, device=dev).view(F8)
                buf[:, :k] = t
                apart.append(buf[:, :k])
            assert torch.equal(rvq.rvq_matmul_f8(apart[0], sa, apart[1], sb, out_dtype=odt), want)
            again = rvq.rvq_matmul_f8(a, sa, b, sb, out_dtype=odt)
            assert torch.equal(again, want)
