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


@pytest.mark.parametrize("dtype,d", [(F32, 5), (F32, 64), (F32, 500), (F32, 1155), (F32, 4096), (F32, 9000),
                                     (BF16, 40), (BF16, 1152), (BF16, 4096), (BF16, 20001)])
def test_norm_rows_whose_squares_leave_fp32(rvq, dev, dtype, d):
    w = 1 + 0.2 * norm_tests._rows(1, d, F32, 5, dev, False)[0]
    x = norm_tests._rows(12, d, F32, d, dev)
    size = torch.tensor([1.0, 1e18, 3e19, 1e25, 1e30, 1e36, 1.0, 2e19, 1e35, 1e20, 1e19, 1e-3], device=dev)
    x = (x * size[:, None]).to(dtype)
    assert torch.isfinite(x).all()
    for odt in (F32, BF16, F8):
        norm_tests._check_norm(rvq, x, None, w, odt)
    # with a residual, whose sum the norm takes
    norm_tests._check_norm(rvq, x, (x.float() * 0.5).to(dtype), w, dtype)
    # the largest values there are; in rows of their own, beside NaN and infinity
    x = torch.full((4, d), MAX if dtype == F32 else 3.3895313892515355e38, device=dev).to(dtype)
    x[1, 0], x[2, d - 1] = NAN, -INF
    out = rvq.rvq_rms_norm(x, out_dtype=F32, need_rstd=True)
    one = torch.ones(d, device=dev)
    for row in (0, 3):
        # 1 / sqrt(mean) is below fp32's normal values: a unit there is 2^-149
        assert torch.all((out.y[row] - one).abs() <= 1e-6)
        assert abs(out.rstd[row].item() * x[row, 0].item() - 1) <= 2.0 ** -21
    assert torch.isnan(out.y[1]).all() and torch.isnan(out.y[2, d - 1])


@pytest.mark.parametrize("d", [5, 300, 4096, 9000])
def test_norm_rows_whose_squares_are_below_fp32(rvq, dev, d):
    # an eps of fp32's smallest value and rows whose squares are about as large
    x = norm_tests._rows(6, d, F32, d, dev, False)
    x = x * torch.tensor([1.0, 1e-15, 1e-19, 1e-22, 1e-25, 0.0], device=dev)[:, None]
    for odt in (F32, F8):
        norm_tests._check_norm(rvq, x, None, None, odt, eps=2.0 ** -149)


def _state8(st, i=0):
    n = st.m[i].numel()
    rep = lambda s: s.double().repeat_interleave(256)[:n]  # noqa: E731
    return st.m[i].double() * rep(st.m_scale[i]), st.v[i].double() * rep(st.v_scale[i])


def test_adamw_keeps_nan_in_8_bit_roots(rvq, dev):
    for gdt in (F32, BF16):
        for seed in (None, 3):
            p, g = torch.ones(1000, device=dev), torch.ones(1000, device=dev, dtype=gdt)
            g[300] = NAN
            st = rvq.rvq_adamw_init([p], 8, 0.0)
            rvq.rvq_adamw_step(st, [g], 1, 0.1, seed=seed)
            m, r = _state8(st)
            for x in (p, m, r):
                bad = torch.isnan(x)
                assert bad[300] and int(bad.sum()) == 1
            rvq.rvq_adamw_step(st, [torch.ones_like(g)], 2, 0.1, seed=seed)
            m, r = _state8(st)
            assert torch.isnan(p[300]) and torch.isnan(m[300]) and torch.isnan(r[300])
            assert int(torch.isnan(p).sum()) == 1


def test_adamw_stores_small_8_bit_roots(rvq, dev):
    # v = 1e-3 * 4^-k in fp32 (a unit is 2^-149 from k = 59 on)
    for k in (40, 58, 60, 62, 64, 66):
        g = torch.full((256,), 2.0 ** -k, device=dev)
        st = rvq.rvq_adamw_init([torch.zeros(256, device=dev)], 8)
        rvq.rvq_adamw_step(st, [g], 1, 0.1)
        _, r = _state8(st)
        want = (1.0 - 0.999) ** 0.5 * 2.0 ** -k
        # the moment is off by a unit or two of 2^-149 and 4 U, its root by half as much
        assert torch.all((r - want).abs() <= want * (2.0 ** -149 / want ** 2 + 6 * ref.U)), k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(F32, F32), (F32, BF16), (BF16, BF16)], ids=["ff", "fb", "bb"])
def test_adamw_gradients_whose_squares_leave_fp32(rvq, dev, bits, pdt, gdt):
    # without a norm: the definition is finite, and so has every element to be
    for seed in (None, 5):
        for top in (1e18, 3e19, 6e20, 1e25, 1e32, 3e38):
            t = adamw_tests._tensors([3000, 5, 2048], pdt, gdt, bits, dev, seed=11, copies=True)
            for g in t["g"]:
                g[::7] = (g[::7].double() * (top / 0.6)).clamp(-3.3e38, 3.3e38).to(gdt)
                g[4] = top
                assert torch.isfinite(g).all()
            _check_saturating(rvq, t, bits, pdt, seed)
    # the state itself past that range, and no gradient
    t = adamw_tests._tensors([1000], pdt, gdt, bits, dev, seed=12)
    t["g"][0].zero_()
    if bits == 8:
        t["vs"][0][1], t["ms"][0][1] = 1e34, 1e33
    else:
        t["v"][0][300:500], t["m"][0][300:500] = 3e38, 1e18
    _check_saturating(rvq, t, bits, pdt, None)


def _check_saturating(rvq, t, bits, pdt, seed):
    """_check of the step's own tests with v held at fp32's largest value at most."""
    before = [(p.clone(), *adamw_tests._moments(t, bits, i)) for i, p in enumerate(t["p"])]
    st = rvq.rvq_adamw_init(t["p"], bits, adamw_tests.DECAY, t["copies"], t["m"], t["v"], t["ms"], t["vs"])
    rvq.rvq_adamw_step(st, t["g"], 3, adamw_tests.LR, adamw_tests.BETAS, adamw_tests.EPS, seed=seed)
    torch.cuda.synchronize()
    for i, (p0, m0, v0) in enumerate(before):
        p, m, v, upd = ref.adamw(p0, t["g"][i], m0, v0, 3, adamw_tests.LR, adamw_tests.BETAS, adamw_tests.EPS,
                                 adamw_tests.DECAY)
        pb = 4 * ref.U * p0.double().abs() + 24 * ref.U * upd.abs()
        if pdt == BF16:
            pb = pb + (1 if seed is None else 2) * ref.BF16_HALF * (1 + 2 ** -7) * p.abs()
        ref.close(t["p"][i], p, pb, f"p[{i}]")
        if t["copies"]:
            assert torch.equal(t["copies"][i], t["p"][i].to(BF16)), f"copy[{i}]"
        mb = 4 * ref.U * (m0.abs() + t["g"][i].double().abs())
        if bits == 32:
            ref.close(t["m"][i], m, mb, f"m[{i}]")
            ref.close(t["v"][i], v.clamp(max=MAX), 6 * ref.U * v.clamp(max=MAX), f"v[{i}]")
            continue
        for q, scale, x, xb in ((t["m"][i], t["ms"][i], m, mb),
                                (t["v"][i], t["vs"][i], v.sqrt(), 6 * ref.U * v.sqrt())):
            peak = ref.blocks(x).abs().amax(1) / 448
            ref.close(scale, peak.clamp(min=ref.SCALE_MIN), ref.blocks(xb).amax(1) / 448 + 4 * ref.U * peak,
                      f"scale[{i}]")
            per = scale.double().repeat_interleave(256)[:x.numel()]
            y = (x / per).clamp(-448, 448)
            # up to a whole step of the grid: a root beside an m that is not zero is not stored as zero
            ref.close(q.float(), y, ref.f8_step(y) * (1 + 2 ** -8) + xb / per + 4 * ref.U * y.abs(), f"state[{i}]")


def test_adamw_infinite_gradient_stays_alone(rvq, dev):
    for bits in (32, 8):
        for seed in (None, 3):
            p, g = torch.ones(600, device=dev), torch.ones(600, device=dev)
            g[300], g[400] = INF, -INF
            st = rvq.rvq_adamw_init([p], bits, 0.0)
            rvq.rvq_adamw_step(st, [g], 1, 0.1, seed=seed)
            rvq.rvq_adamw_step(st, [torch.ones_like(g)], 2, 0.1, seed=seed)
            bad = torch.isnan(p)
            assert bad[300] and bad[400] and int(bad.sum()) == 2, (bits, seed)
            assert torch.allclose(p[~bad], torch.full_like(p[~bad], 0.8), rtol=0.02)


def test_adamw_infinite_32_bit_v_leaves_the_decay(rvq, dev):
    # a state from elsewhere: m / infinity is 0
    for pdt in (F32, BF16):
        p, v = torch.ones(300, device=dev, dtype=pdt), torch.ones(300, device=dev)
        v[100] = INF
        st = rvq.rvq_adamw_init([p], 32, 0.5, m=[torch.zeros(300, device=dev)], v=[v])
        for g in (1.0, 1e30):
            p.fill_(1.0)
            rvq.rvq_adamw_step(st, [torch.full((300,), g, device=dev)], 2, 0.5)
            assert p[100].item() == 0.75 and st.v[0][100].item() == INF
            assert torch.isfinite(p).all() and torch.all(p[:100].float() < 0.75)


@pytest.mark.parametrize("gdt", [F32, BF16], ids=["f", "b"])
def test_adamw_norm_of_gradients_whose_squares_leave_fp32(rvq, dev, gdt):
    for size in (1e-35, 1e-30, 1e-24, 1e-20, 1.0, 1e19, 1e25, 1e36):
        g = (torch.randn(70001, generator=torch.Generator(device=dev).manual_seed(1), device=dev) * size).to(gdt)
        want = float(g.double().square().sum().sqrt())
        p = torch.zeros(70001, device=dev)
        st = rvq.rvq_adamw_init([p], 32)
        norm = rvq.rvq_adamw_step(st, [g], 1, 0.1, eps=1e-12, max_norm=1.0)
        if want > 3.4e38:
            assert float(norm) == INF and torch.all(p == 0)
            continue
        # fp32's own unit where the norm is below 2^-126
        assert abs(float(norm) - want) <= 16 * ref.U * want + 2.0 ** -149, size
        f = min(1.0, 1.0 / (want + 1e-6))
        want_m = 0.1 * g.double() * f
        # f is below fp32's normal values from a norm of 2^126 on
        ref.close(st.m[0], want_m, (16 * ref.U + 2.0 ** -149 / f) * want_m.abs() + 2.0 ** -148, f"m {size}")


def test_adamw_rounds_nan_to_nan(rvq, dev):
    # NaN with every bit of the significand set (memory that was filled with
    # ones), which random bits added to it would carry out of
    words = torch.tensor([0x7fffffff, -1, 0x7fc00000, 0x7f800001, -0x800000 + 1, 0x7fff8000], dtype=torch.int32)
    nans = words.view(F32).to(dev)
    assert torch.isnan(nans).all()
    n = 64 * nans.numel()
    for bits in (32, 8):
        for seed in (1, 2):
            p = torch.ones(2 * n, dtype=BF16, device=dev)
            g = torch.ones(2 * n, device=dev)
            g[:n] = nans.repeat(64)
            st = rvq.rvq_adamw_init([p], bits, 0.0)
            rvq.rvq_adamw_step(st, [g], 1, 0.1, seed=seed)
            assert torch.isnan(p[:n]).all() and torch.isfinite(p[n:]).all(), bits
            # and of a parameter
            p = torch.full((n,), -1, dtype=torch.int16, device=dev).view(BF16)
            st = rvq.rvq_adamw_init([p], bits, 0.0)
            rvq.rvq_adamw_step(st, [torch.ones(n, device=dev)], 1, 0.1, seed=seed)
            assert torch.isnan(p).all()
            # and of a state
            if bits == 32:
                continue
            code = torch.tensor([0x7f, 0xff], dtype=torch.uint8).view(F8).to(dev)
            for mv, scale in ((code, 1.0), (torch.ones(2, device=dev).to(F8), nans[1])):
                p = torch.ones(512, dtype=BF16, device=dev)
                one = lambda: torch.ones(2, device=dev)  # noqa: E731
                m = mv.view(torch.uint8).repeat(256).view(F8)
                v = torch.ones(512, device=dev).to(F8)
                st = rvq.rvq_adamw_init([p], 8, 0.0, m=[m], v=[v], m_scale=[one() * scale], v_scale=[one()])
                rvq.rvq_adamw_step(st, [torch.ones(512, device=dev)], 2, 0.1, seed=seed)
                assert torch.isnan(p).all()


@pytest.mark.parametrize("seed", [7, None], ids=["random", "nearest"])
@pytest.mark.parametrize("small,gone", [(1e-4, 0.99), (1e-5, 0.0), (1e-5, 0.5), (1e-6, 0.0), (1e-8, 0.5)])
def test_adamw_8_bit_steps_are_bounded_in_blocks_of_unlike_magnitudes(rvq, dev, seed, small, gone):
    # One element a block has gradients of standard deviation 1, the others of
    # `small`; a share `gone` of the steps has none.  With exact moments and as
    # many steps behind it, |m| / sqrt(v) is at most (Cauchy-Schwarz)
    # sqrt(0.1^2 / 0.001 / (1 - 0.81 / 0.999)) = 7.27.  Storing may add one
    # step of m's grid, and leaves the root at least the smallest step of its
    # own where m is not zero: at most 7.27 times the ratio of the two scales,
    # itself at most 7.27, more; and either grid's rounding is 1/8 of a value.
    blocks, steps = 64, 300
    g0 = torch.Generator(device=dev).manual_seed(3)
    std = torch.full((blocks, 256), small, device=dev)
    std[:, 0] = 1.0
    p = torch.zeros(blocks * 256, device=dev)
    st = rvq.rvq_adamw_init([p], 8, 0.0)
    worst = torch.zeros((), device=dev)
    for t in range(1, steps + 1):
        g = torch.randn((blocks, 256), generator=g0, device=dev) * std
        g *= torch.rand((blocks, 1), generator=g0, device=dev) >= gone
        old = p.clone()
        rvq.rvq_adamw_step(st, [g.view(-1)], t, 1.0, eps=1e-12, seed=None if seed is None else seed + t)
        # the bias corrections' quotient is at most its limit, 1, from the first step on
        worst = torch.maximum(worst, (p - old).abs().max())
    assert float(worst) <= 2 * 7.27 * 1.125 ** 2, float(worst)
    m, r = st.m[0].float(), st.v[0].float()
    assert torch.all(r[m != 0] > 0)


def test_adamw_8_bit_roots_stay_above_zero_beside_m(rvq, dev):
    # The first element of a block grows: the others' roots come to 2.7e-4 of the
    # new scale, under half the smallest e4m3 value, their m to many steps.  In the
    # second block m is zero: the same roots may become 0.  In the third they
    # are 0 already, by no rounding of the step's, and stay so (small gradients give
    # half of them roots of 2e-4 of the scale; which is the formula alone).
    m, v = torch.zeros(768, device=dev), torch.full((768,), 2.0 ** -9, device=dev)
    m[:256], m[512:], v[512:] = 1.0, 1.0, 0.0
    m[::256], v[::256] = 448.0, 448.0
    for seed in (None, 1, 2):
        p = torch.zeros(768, device=dev)
        g = torch.zeros(768, device=dev)
        g[::256] = 1e5
        g[640:] = 0.05
        one = lambda: torch.ones(3, device=dev)  # noqa: E731
        st = rvq.rvq_adamw_init([p], 8, 0.0, m=[m.to(F8)], v=[v.to(F8)], m_scale=[one()], v_scale=[one()])
        rvq.rvq_adamw_step(st, [g], 5, 0.0, seed=seed)
        root = st.v[0].float()
        assert torch.all(st.m[0].float()[1:256] > 0)
        assert torch.all(root[1:256] == 2.0 ** -9)
        assert torch.all(root[513:640] == 0)
        if seed is None:
            assert torch.all(root[257:512] == 0) and torch.all(root[640:] == 0)
        else:  # 0.140 of them go up
            assert abs(float((root[257:512] > 0).double().mean()) - 0.140) <= 6 * 0.0217


def test_adamw_norm_over_several_launches(rvq, dev):
    # more tensors than a launch of the norm takes, more workgroups' sums than a step adds itself
    g0 = torch.Generator().manual_seed(8)
    for count, top in ((400, 60), (500, 9000), (161, 40000)):
        sizes = [int(x) for x in torch.randint(0, top, (count,), generator=g0)]
        sizes[7] = 5000000
        g = [torch.full((n,), 0.5, device=dev) for n in sizes]
        p = [torch.zeros(n, device=dev) for n in sizes]
        st = rvq.rvq_adamw_init(p)
        norm = rvq.rvq_adamw_step(st, g, 1, 0.1, max_norm=1e9)
        want = 0.5 * sum(sizes) ** 0.5
        assert abs(float(norm) - want) <= 16 * ref.U * want
        for x in st.m:
            assert torch.all((x - 0.05).abs() <= 1e-8)


def test_adamw_state_holds_no_buffer_of_its_own(rvq, dev):
    # what a step works in belongs to the step's stream: a buffer that the state
    # had made on its own stream would be given away when the state is dropped,
    # whatever still ran elsewhere
    p = [torch.zeros(300, device=dev)]
    st = rvq.rvq_adamw_init(p, 8)
    known = {t.data_ptr() for ts in (st.params, st.m, st.v, st.m_scale, st.v_scale) for t in ts}
    held = [t for x in vars(st).values() for t in (x if isinstance(x, (tuple, list)) else [x])
            if isinstance(t, torch.Tensor)]
    assert {t.data_ptr() for t in held} <= known
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        norm = rvq.rvq_adamw_step(st, [torch.ones(300, device=dev)], 1, 0.1, max_norm=1.0)
    side.synchronize()
    assert abs(float(norm) - 300 ** 0.5) <= 1e-4


def test_embed_grad_bits_do_not_depend_on_which_tables_are_asked_for(rvq, dev):
    # rows longer than a segment of the list, in both tables, with random values
    for T, L, K, V, D, dtype, gdt in ((3000, 3, 7, 5, 72, BF16, F32), (9001, 5, 40, 11, 40, F32, F32),
                                      (60000, 8, 9, 3, 16, F32, F32), (5000, 2, 6, 4, 264, BF16, BF16)):
        dout, ids, vis = embed_tests._problem(T, L, K, V, D, dtype, dev, text=0.5, hot=0.3, whole=False)
        level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt)
        only, _ = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt, need_text=False)
        _, alone = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt, need_level=False)
        none, _ = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, 0, gdt)
        raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(raw(only), raw(level)) and torch.equal(raw(none), raw(level)), (T, "level")
        assert torch.equal(raw(alone), raw(text)), (T, "text")
        if gdt == F32:
            wl, wt, al, at, _ = ref.embed_grad(dout, ids, vis, L, K, V)
            ref.close(level, wl, T * ref.U * al, "level")
            ref.close(text, wt, T * ref.U * at, "text")


def test_learning_calls_refuse_sizes_past_32_bits(rvq, dev):
    wide = torch.empty((0, 2 ** 32 + 8), device=dev)
    rstd, ids = torch.empty(0, device=dev), torch.empty((0, 2), dtype=torch.int32, device=dev)
    dout = torch.empty((0, 8), device=dev)
    for call in (lambda: rvq.rvq_rms_norm(wide), lambda: rvq.rvq_rms_norm_backward(wide, wide, rstd),
                 lambda: rvq.rvq_rms_norm_backward(wide, wide, rstd, need_dweight=False),
                 lambda: rvq.rvq_embed_tokens_backward(wide, ids, 3, V=4, need_level=False),
                 lambda: rvq.rvq_embed_tokens_backward(dout, ids, 2 ** 32 + 5, V=4, need_level=False),
                 lambda: rvq.rvq_embed_tokens_backward(dout, ids, -2 ** 32 + 5, V=4, need_level=False),
                 lambda: rvq.rvq_embed_tokens_backward(dout, ids, 5, V=2 ** 64 + 4, need_level=False)):
        with pytest.raises((ValueError, rvq.RVQError)):
            call()


def test_adamw_options_outside_fp32(rvq, dev):
    p, g = torch.ones(10, device=dev), torch.ones(10, device=dev)
    st = rvq.rvq_adamw_init([p], 32, 0.0)
    for bad in (dict(grad_scale=1e39), dict(lr=1e38, betas=(0.9999, 0.999)), dict(lr=1e40)):
        with pytest.raises(rvq.RVQError) as e:
            rvq.rvq_adamw_step(st, [g], **{**dict(step=1, lr=0.1), **bad})
        assert e.value.status == 1
    # a positive max_norm below fp32's smallest value clips all the same
    rvq.rvq_adamw_step(st, [g], 1, 0.1, max_norm=1e-60)
    assert float(st.m[0].abs().max()) <= 1e-44


def test_learning_calls_refuse_tensors_that_want_a_gradient(rvq, dev):
    x, rstd = torch.ones((4, 32), device=dev), torch.ones(4, device=dev)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    want = lambda t: t.clone().requires_grad_()  # noqa: E731
    w = torch.ones(32, device=dev)
    calls = (lambda: rvq.rvq_rms_norm(want(x)), lambda: rvq.rvq_rms_norm(x, want(w)),
             lambda: rvq.rvq_rms_norm(x, residual=want(x)), lambda: rvq.rvq_rms_norm_backward(want(x), x, rstd),
             lambda: rvq.rvq_rms_norm_backward(x, want(x), rstd, w), lambda: rvq.rvq_rms_norm_backward(x, x, rstd, want(w)),
             lambda: rvq.rvq_rms_norm_backward(x, x, rstd, dsum=want(x)),
             lambda: rvq.rvq_embed_tokens_backward(want(x), ids, 3))
    for call in calls:
        with pytest.raises(ValueError):
            call()
    with torch.no_grad():
        for call in calls:
            call()
    rvq.rvq_rms_norm(want(x).detach())
    # parameters of an optimizer want gradients as a matter of course
    p = torch.nn.Parameter(torch.ones(8, device=dev))
    rvq.rvq_adamw_step(rvq.rvq_adamw_init([p]), [torch.ones(8, device=dev)], 1, 0.1)


# launch forms that the other cases do not reach
FORMS = [
    # more than 512 index workgroups: of four waves with the IDs read in place and laid out by table, of sixteen
    (3000, 16, 16384, 1001, 8), (5003, 16, 16384, 1001, 8), (8192, 16, 16384, 40, 4), (2049, 1, 300000, 7, 12),
    # several rows in turn for a part of a wave (W < 64), rows longer than a segment among them
    (1000, 2, 70000, 9, 8), (3000, 4, 40000, 1000, 24), (900, 1, 140000, 11, 128), (1500, 8, 20000, 100, 200),
    # more than four rows a wave
    (900, 3, 200000, 5, 520),
    # three slabs of columns in panels of two and one, and five in panels
    (41000, 1, 50, 3, 1300), (50000, 2, 30, 40, 2500),
]


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "T%d_L%d_K%d_V%d_D%d" % c)
def test_embed_grad_launch_forms(rvq, dev, case):
    T, L, K, V, D = case
    for dtype, gdt in ((BF16, F32), (F32, BF16)):
        dout, ids, vis = embed_tests._problem(T, L, K, V, D, dtype, dev)
        # hot rows: a table's first, one in the middle of a group of rows, and two next to each other
        hot = torch.rand(T, generator=torch.Generator(device=dev).manual_seed(2), device=dev)
        for k, at in enumerate((0, K // 2 + 1, K // 2 + 2, min(5, K - 1))):
            ids[(hot >= 0.12 * k) & (hot < 0.12 * (k + 1))] = at
        if V:
            ids[vis == 0, 0] = (ids[vis == 0, 0] % V).int()
        embed_tests._check_exact(rvq, dout, ids, vis, K, V, gdt)
        # added to what is there
        wl, wt, _, _, _ = ref.embed_grad(dout, ids, vis, L, K, V)
        l0, t0 = torch.full((L, K, D), 2.0, device=dev, dtype=gdt), torch.full((V, D), -1.0, device=dev, dtype=gdt)
        level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt, level_grad=l0, text_grad=t0,
                                                    accumulate=True)
        assert torch.equal(level, (wl + 2.0).to(gdt)) and torch.equal(text, (wt - 1.0).to(gdt))
        del wl, wt, l0, t0, level, text


def test_adamw_large_gradients_of_a_slow_v(rvq, dev):
    # with beta2 = 1 - 1e-7 the first v is 10^-7 of the square: not lost beside an
    # element of the block that is 10^20 times larger
    betas = (0.9, 1.0 - 1e-7)
    for bits in (32, 8):
        for size in (1e3, 3e9, 1e11, 1e14, 1e17, 1e20, 1e24, 1e28):
            p = torch.ones(256, device=dev)
            g = torch.full((256,), size, device=dev)
            g[0] = 1e30
            st = rvq.rvq_adamw_init([p], bits, 0.0)
            rvq.rvq_adamw_step(st, [g], 1, 0.25, betas)
            want, _, _, upd = ref.adamw(torch.ones(256, device=dev), g, torch.zeros_like(g), torch.zeros_like(g), 1, 0.25,
                                        betas, 1e-8, 0.0)
            ref.close(p, want, 4 * ref.U + 24 * ref.U * upd.abs(), f"{bits} {size}")


def test_adamw_refuses_tensors_that_share_memory(rvq, dev):
    buf = torch.zeros(1000, device=dev)
    f = lambda n: torch.zeros(n, device=dev)  # noqa: E731
    for bits in (32, 8):
        for params in ([buf, buf], [f(10), buf, f(10), buf[:10]], [buf[:600], buf[599:]], [buf.view(10, 100), buf[500:501]]):
            with pytest.raises(ValueError):
                rvq.rvq_adamw_init(params, bits)
        rvq.rvq_adamw_init([buf[:600], buf[600:], buf[:0], buf[5:5]], bits)   # next to each other, and nothing at all
    a, b = f(300), f(300)
    for kw in (dict(m=[buf[:300]], v=[f(300)]), dict(m=[a], v=[a]), dict(m=[a], v=[b], copies=[buf[:150].view(BF16)]),
               dict(copies=[a.view(BF16)[:300]], m=[b], v=[a])):
        with pytest.raises(ValueError):
            rvq.rvq_adamw_init([buf[:300]], 32, **kw)
    rvq.rvq_adamw_init([buf[:300]], 32, m=[a], v=[b], copies=[buf[300:450].view(BF16)])
    q = f(600).view(torch.uint8).view(F8)
    s = f(8)
    with pytest.raises(ValueError):
        rvq.rvq_adamw_init([a], 8, m=[q[:300]], v=[q[300:600]], m_scale=[s[:2]], v_scale=[s[1:3]])
    rvq.rvq_adamw_init([a], 8, m=[q[:300]], v=[q[300:600]], m_scale=[s[:2]], v_scale=[s[2:4]])
