"""rvq_layer_norm and its gradient against their definitions in 64 bits."""
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


def _chain(d):
    # a row's terms that one lane adds one after the other (at most d / 64, or 64
    # where fewer lanes share a narrow row), the tree over 256 lanes, and the
    # roundings of the mean, the root and the products
    return max(d / 64, 64) + 24


def _rows(n, d, dtype, seed, dev, spread=True, offset=0.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((n, d), generator=g, device=dev)
    if spread:
        x[:, ::max(1, d // 3)] *= 30.0
    return (x + offset).to(dtype)


def _param(d, dtype, seed, dev, mid=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (mid + 0.2 * torch.randn(d, generator=g, device=dev)).to(dtype)


def _check(rvq, x, res, w, b, odt, eps=1e-5, **kw):
    n, d = x.shape
    x0, r0 = x.clone(), None if res is None else res.clone()
    out = rvq.rvq_layer_norm(x, w, b, eps, residual=res, out_dtype=odt, need_stats=True, **kw)
    torch.cuda.synchronize()
    h, mean, rstd, y = ref.layer_norm(x0, r0, w, b, eps)
    bm, br, by = ref.layer_norm_bounds(h, mean, rstd, w, b, _chain(d), res is not None)
    learn_ref.close(out.mean, mean, bm, "mean")
    learn_ref.close(out.rstd, rstd, br + 4 * ref.U * rstd, "rstd")
    if res is not None:
        learn_ref.close(out.sum, h, h.abs() * (ref.U if x.dtype == F32 else ref.BF16_ROUND), "sum")
    assert out.y.dtype == odt and out.y.shape == (n, d)
    if odt == F8:
        top = y.abs().amax(1) / ref.F8_MAX
        worst = by.amax(1) / ref.F8_MAX + 2 * ref.U * top
        learn_ref.close(out.scale, top.clamp(min=ref.SCALE_MIN), worst, "scale")
        v = y / out.scale.double()[:, None]
        near = torch.clamp(v, -ref.F8_MAX, ref.F8_MAX)
        learn_ref.close(out.y.float(), near, learn_ref.f8_step(v) * 0.5 * (1 + 2 ** -8) + by / out.scale.double()[:, None],
                        "y (e4m3)")
    else:
        assert out.scale is None
        learn_ref.close(out.y, y, by + (ref.BF16_ROUND if odt == BF16 else ref.U) * y.abs(), "y")
    return out


# every width class (a few lanes, a wave, a workgroup per row; rows that stay in
# registers or are read again), whole and broken 16-byte pieces
WIDTHS = [1, 2, 7, 8, 24, 63, 64, 65, 128, 200, 256, 257, 500, 512, 1000, 1024, 1152, 1155, 2048,
          2050, 4096, 4100, 5001, 8192, 8193, 12288, 20001]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_layer_norm(rvq, dev, d, dtype):
    for n, odt, with_res, wdt, bdt in ((1, dtype, True, F32, F32), (37, F8, True, BF16, BF16), (300, dtype, False, None, None),
                                       (5, BF16 if dtype == F32 else F32, True, F32, None), (64, F8, False, None, F32)):
        x = _rows(n, d, dtype, d + n, dev)
        res = _rows(n, d, dtype, d + n + 1, dev) if with_res else None
        w = None if wdt is None else _param(d, wdt, 5, dev)
        b = None if bdt is None else _param(d, bdt, 6, dev, 0.0)
        _check(rvq, x, res, w, b, odt)


@pytest.mark.parametrize("offset", [100.0, 1e4, -3e6])
def test_layer_norm_far_from_zero(rvq, dev, offset):
    # the mean is up to 2^21 times the spread: what fp32 still holds of it counts
    for d in (48, 1152, 4096, 9000):
        x = _rows(23, d, F32, d, dev, False, offset)
        _check(rvq, x, None, _param(d, F32, 5, dev), None, F32)
    x = torch.full((3, 1000), offset, device=dev)
    out = rvq.rvq_layer_norm(x, None, None, need_stats=True)
    assert torch.all(out.y == 0) and torch.all(out.mean == x[:, 0])
    assert out.rstd.tolist() == pytest.approx([1e3] * 3, rel=1e-6)


def test_layer_norm_squares_that_leave_fp32(rvq, dev):
    for d in (40, 1000, 9000):
        for big in (1e17, 1e25, 1e37):
            x = _rows(5, d, F32, d, dev, False) * big
            _check(rvq, x, None, None, None, F32)
            _check(rvq, x, None, None, None, F8)
        same = torch.full((2, d), 2.0 ** 100, device=dev)       # equal values: no variance, whatever their size
        out = rvq.rvq_layer_norm(same, None, _param(d, F32, 6, dev, 0.0), need_stats=True)
        assert torch.equal(out.y, _param(d, F32, 6, dev, 0.0).expand(2, d)) and torch.all(out.mean == 2.0 ** 100)
        assert out.rstd.tolist() == pytest.approx([1e3] * 2, rel=1e-6)
        small = _rows(5, d, F32, d, dev, False) * 1e-20         # squares below fp32, with an eps as small
        _check(rvq, small, None, None, None, F32, eps=1e-38)


def test_layer_norm_many_rows(rvq, dev):
    for n, d in ((100003, 8), (70001, 64), (20011, 512)):
        _check(rvq, _rows(n, d, BF16, n, dev), _rows(n, d, BF16, n + 1, dev), None, _param(d, F32, 3, dev, 0.0), BF16)


def test_layer_norm_in_place_and_unaligned(rvq, dev):
    for dtype in (F32, BF16):
        for d in (100, 1155, 4096, 20001):
            w, b = _param(d, F32, 3, dev), _param(d, F32, 4, dev, 0.0)
            for which in ("x", "residual"):
                x, res = _rows(9, d, dtype, d, dev), _rows(9, d, dtype, d + 1, dev)
                _check(rvq, x, res, w, b, dtype, sum_out=x if which == "x" else res)
            x, res = _rows(9, d, dtype, d, dev), _rows(9, d, dtype, d + 1, dev)
            _check(rvq, x, res, w, b, dtype, out=x)
            # rows, weights and outputs that begin one element into a buffer
            buf = _rows(1, 20 * d + 2, dtype, d + 2, dev)[0]
            x, res = buf[1:1 + 9 * d].view(9, d), buf[10 * d + 1:19 * d + 1].view(9, d)
            w1, b1 = _param(d + 1, F32, 3, dev)[1:], _param(d + 1, F32, 4, dev)[1:]
            o = torch.empty(9 * d + 1, dtype=dtype, device=dev)[1:].view(9, d)
            _check(rvq, x, res, w1, b1, dtype, out=o)
            q = torch.empty(9 * d + 1, dtype=F8, device=dev)[1:].view(9, d)
            _check(rvq, x, res, w1, b1, F8, out=q)


def test_layer_norm_rows_with_nan_or_infinity_stay_alone(rvq, dev):
    for d in (40, 3000, 9000):
        x = _rows(8, d, F32, d, dev)
        clean = rvq.rvq_layer_norm(x, out_dtype=F8)
        x[1, d // 2] = float("nan")
        x[5, 0] = float("inf")
        out = rvq.rvq_layer_norm(x, out_dtype=F8, need_stats=True)
        plain = rvq.rvq_layer_norm(x)
        keep = torch.tensor([0, 2, 3, 4, 6, 7], device=dev)
        assert torch.equal(out.y[keep].view(torch.uint8), clean.y[keep].view(torch.uint8))
        assert torch.equal(out.scale[keep], clean.scale[keep])
        for i in (1, 5):
            assert torch.isnan(out.scale[i]) and torch.isnan(plain.y[i]).all() and torch.isnan(out.rstd[i])
        e = rvq.rvq_layer_norm(x[:0], need_stats=True, out_dtype=F8)
        assert e.y.shape == (0, d) and e.mean.shape == (0,) and e.scale.shape == (0,)


def _check_grad(rvq, n, d, dtype, wdt, with_sum, dev, in_place=None):
    h, dy = _rows(n, d, dtype, n + d, dev, offset=0.5), _rows(n, d, dtype, n + d + 1, dev, False)
    ds = _rows(n, d, dtype, n + d + 2, dev, False) if with_sum else None
    w = None if wdt is None else _param(d, wdt, 5, dev)
    mean = h.double().mean(1)
    rstd = ((h.double() - mean[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    mean = mean.float()
    dx, size, dw, dwsize, db, dbsize = ref.layer_norm_grad(dy, h, mean, rstd, w, ds)
    out = {None: None, "dy": dy, "dsum": ds}[in_place]
    got, gotw, gotb = rvq.rvq_layer_norm_backward(dy, h, mean, rstd, w, dsum=ds, out=out)
    torch.cuda.synchronize()
    learn_ref.close(got, dx, _chain(d) * ref.U * size + (0.0 if dtype == F32 else ref.BF16_ROUND * dx.abs()), "dx")
    # at most n / 256 + 512 additions in a row, and four roundings of each term
    b = (min(n, n / 256 + 512) + 16) * ref.U
    learn_ref.close(gotw, dw, b * dwsize, "dweight")
    learn_ref.close(gotb, db, b * dbsize, "dbias")
    return got, gotw, gotb


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_layer_norm_grad(rvq, dev, d, dtype):
    for n, wdt, with_sum in ((1, F32, False), (41, BF16, True), (300, None, True), (1030, F32, False)):
        _check_grad(rvq, n, d, dtype, wdt, with_sum, dev)


def test_layer_norm_grad_many_rows_and_in_place(rvq, dev):
    for n, d in ((100003, 8), (30011, 200), (20011, 1024)):
        _check_grad(rvq, n, d, BF16, F32, True, dev)
    for d in (100, 4096, 9000, 20001):
        for which in ("dy", "dsum"):
            _check_grad(rvq, 700, d, BF16, F32, True, dev, which)


def test_layer_norm_grad_repeats_and_options(rvq, dev):
    h, dy = _rows(5000, 1152, BF16, 1, dev), _rows(5000, 1152, BF16, 2, dev)
    s = rvq.rvq_layer_norm(h, need_stats=True)
    args = (dy, h, s.mean, s.rstd)
    a, aw, ab = rvq.rvq_layer_norm_backward(*args)
    b, bw, bb = rvq.rvq_layer_norm_backward(*args)
    c, none, none2 = rvq.rvq_layer_norm_backward(*args, need_dweight=False, need_dbias=False)
    d, none3, db = rvq.rvq_layer_norm_backward(*args, need_dweight=False)
    e, dw, none4 = rvq.rvq_layer_norm_backward(*args, need_dbias=False)
    assert none is None and none2 is None and none3 is None and none4 is None
    for x in (b, c, d, e):
        assert torch.equal(a.view(torch.int16), x.view(torch.int16))
    for x, y in ((aw, bw), (aw, dw), (ab, bb), (ab, db)):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    dx, dw, db = rvq.rvq_layer_norm_backward(dy[:0], h[:0], s.mean[:0], s.rstd[:0])
    assert dx.shape == (0, 1152) and torch.all(dw == 0) and torch.all(db == 0)


def test_layer_norm_grad_against_differences(rvq, dev):
    # the loss sum(dy y + dsum h) of the forward definition in 64 bits, moved by 1e-5
    # either way: the difference is off by about 1e-10 (third order) and 1e-11
    # (cancellation), the kernel by its fp32 bound
    n, d, eps, s = 3, 37, 1e-5, 1e-5
    h, dy, ds = (_rows(n, d, F32, k, dev, False) for k in (1, 2, 3))
    w, b = _param(d, F32, 4, dev), _param(d, F32, 5, dev, 0.0)
    st = rvq.rvq_layer_norm(h, w, b, eps, need_stats=True)
    dx, dw, db = rvq.rvq_layer_norm_backward(dy, h, st.mean, st.rstd, w, dsum=ds)

    def loss(h, w, b):
        return float((dy.double() * ref.layer_norm(h, None, w, b, eps)[3]).sum() + (ds.double() * h).sum())
    for i in range(n):
        for j in range(0, d, 5):
            e = torch.zeros((n, d), dtype=torch.float64, device=dev)
            e[i, j] = s
            num = (loss(h.double() + e, w, b) - loss(h.double() - e, w, b)) / (2 * s)
            assert abs(num - dx[i, j].item()) <= 1e-4, (i, j)
    for j in range(0, d, 4):
        e = torch.zeros(d, dtype=torch.float64, device=dev)
        e[j] = s
        num = (loss(h.double(), w.double() + e, b) - loss(h.double(), w.double() - e, b)) / (2 * s)
        assert abs(num - dw[j].item()) <= 1e-4, j
        num = (loss(h.double(), w, b.double() + e) - loss(h.double(), w, b.double() - e)) / (2 * s)
        assert abs(num - db[j].item()) <= 1e-4, j


def test_layer_norm_refusals(rvq, dev):
    x = _rows(4, 32, F32, 1, dev)
    one = torch.ones(4, device=dev)
    for bad in (dict(residual=x[:3]), dict(residual=x.bfloat16()), dict(weight=torch.ones(31, device=dev)),
                dict(weight=torch.ones(32, device=dev, dtype=torch.float64)), dict(out=x.bfloat16()),
                dict(sum_out=x[:, :16]), dict(weight=torch.ones(32)), dict(residual=x.t().contiguous().t()),
                dict(bias=torch.ones(31, device=dev)), dict(bias=torch.ones(32)),
                dict(weight=torch.ones(32, device=dev), bias=torch.ones(32, device=dev, dtype=BF16)),
                dict(bias=torch.ones(32, device=dev, requires_grad=True))):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_layer_norm(x, **bad)
    for bad in (x.cpu(), x[0], x.double(), x[:, ::2], x.clone().requires_grad_()):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_layer_norm(bad)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(rvq.RVQError):
            rvq.rvq_layer_norm(x, eps=eps)
    with pytest.raises(rvq.RVQError):
        rvq.rvq_layer_norm(x, residual=x, out=x, sum_out=x)
    for bad in (dict(h=x[:3]), dict(h=x.bfloat16()), dict(rstd=one[:3]), dict(mean=one.double()), dict(mean=one[:3]),
                dict(dsum=x.bfloat16()), dict(out=x[:2]), dict(weight=one)):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_layer_norm_backward(**{**dict(dy=x, h=x, mean=one, rstd=one), **bad})
