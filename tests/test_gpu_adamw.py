"""rvq_adamw_step against its definition in 64 bits."""
import pytest
import torch

import learn_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
BETAS, EPS, LR, DECAY = (0.9, 0.999), 1e-8, 1e-2, 0.1


@pytest.fixture(scope="module")
def rvq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import residual_vector_quantization_rvq_amd as m
    return m


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


SIZES = [1, 2, 255, 256, 257, 1000, 2047, 2048, 2049, 0, 4099, 70001]


def _tensors(sizes, pdt, gdt, bits, dev, seed=0, shift=0, copies=False):
    g = torch.Generator(device=dev).manual_seed(seed + 1)

    def place(x):
        buf = torch.empty(x.numel() + shift, dtype=x.dtype, device=dev)
        buf[shift:] = x
        return buf[shift:]
    rand = lambda n: torch.randn(n, generator=g, device=dev)  # noqa: E731
    p = [place(rand(n).to(pdt)) for n in sizes]
    grads = [place((rand(n) * 0.1).to(gdt)) for n in sizes]
    m, v = [place(rand(n) * 0.01) for n in sizes], [place((rand(n) * 0.1).square()) for n in sizes]
    for x in m + v + grads:       # rows that nothing touched
        x[:x.numel() // 3] = 0
    out = dict(p=p, g=grads, ms=None, vs=None, copies=[place(x.to(BF16)) for x in p] if copies else None)
    if bits == 8:
        out["ms"], out["vs"] = [], []
        for xs, scales, root in ((m, out["ms"], False), (v, out["vs"], True)):
            for i, x in enumerate(xs):
                x = x.sqrt() if root else x
                s = (ref.blocks(x).abs().amax(1) / 448).clamp(min=ref.SCALE_MIN) if x.numel() else x[:0].clone()
                q = (x / s.repeat_interleave(256)[:x.numel()]).clamp(-448, 448)
                xs[i] = place(q.to(F8).view(torch.uint8)).view(F8)
                scales.append(s)
    out["m"], out["v"] = m, v
    return out


def _moments(t, bits, i):
    m, v = t["m"][i], t["v"][i]
    if bits == 32:
        return m.double(), v.double()
    n = m.numel()
    return (m.double() * t["ms"][i].double().repeat_interleave(256)[:n],
            (v.double() * t["vs"][i].double().repeat_interleave(256)[:n]).square())


def _check(rvq, t, bits, pdt, step=3, factor=1.0, stochastic=False, **kw):
    dev = t["p"][0].device
    before = [(p.clone(), *_moments(t, bits, i)) for i, p in enumerate(t["p"])]
    st = rvq.rvq_adamw_init(t["p"], bits, DECAY, t["copies"], t["m"], t["v"], t["ms"], t["vs"])
    norm = rvq.rvq_adamw_step(st, t["g"], step, LR, BETAS, EPS, **kw)
    torch.cuda.synchronize()
    for i, (p0, m0, v0) in enumerate(before):
        p, m, v, upd = ref.adamw(p0, t["g"][i], m0, v0, step, LR, BETAS, EPS, DECAY, factor)
        # p: the decayed value, the quotient (three operations on the root's
        # side, two on m's, the moments' own roundings) and the difference
        pb = 4 * ref.U * p0.double().abs() + 24 * ref.U * upd.abs()
        if pdt == BF16:
            pb = pb + (2 if stochastic else 1) * ref.BF16_HALF * (1 + 2 ** -7) * p.abs()
        ref.close(t["p"][i], p, pb, f"p[{i}]")
        if t["copies"]:
            assert torch.equal(t["copies"][i], t["p"][i].to(BF16)), f"copy[{i}]"
        gf = (t["g"][i].double() * factor).abs()
        mb = 4 * ref.U * (m0.abs() + gf)
        vb = 6 * ref.U * v
        if bits == 32:
            ref.close(t["m"][i], m, mb, f"m[{i}]")
            ref.close(t["v"][i], v, vb, f"v[{i}]")
            continue
        if not m.numel():
            continue
        for q, scale, x, xb in ((t["m"][i], t["ms"][i], m, mb), (t["v"][i], t["vs"][i], v.sqrt(), 6 * ref.U * v.sqrt())):
            top = ref.blocks(x).abs().amax(1) / 448
            ref.close(scale, top.clamp(min=ref.SCALE_MIN), ref.blocks(xb).amax(1) / 448 + 4 * ref.U * top, f"scale[{i}]")
            per = scale.double().repeat_interleave(256)[:x.numel()]
            y = (x / per).clamp(-448, 448)
            half = 1.0 if stochastic else 0.5
            # a step above: a value may round up to where the grid is twice as wide
            ref.close(q.float(), y, half * ref.f8_step(y) * (1 + 2 ** -8) + xb / per + 4 * ref.U * y.abs(), f"8-bit state [{i}]")
    return norm


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)], ids=["ff", "fb", "bb", "bf"])
def test_adamw(rvq, dev, bits, pdt, gdt):
    for shift, seed, copies in ((0, None, False), (1, None, True), (0, 77, True), (3, 78, False)):
        t = _tensors(SIZES, pdt, gdt, bits, dev, seed=shift, shift=shift, copies=copies)
        _check(rvq, t, bits, pdt, seed=seed, stochastic=seed is not None)


def test_adamw_first_step_from_zero_states(rvq, dev):
    for bits in (32, 8):
        p = [torch.ones(1000, device=dev), torch.zeros(3, 100, device=dev)]
        g = [torch.zeros(1000, device=dev), torch.ones(3, 100, device=dev)]
        st = rvq.rvq_adamw_init(p, bits, [0.5, 0.0])
        rvq.rvq_adamw_step(st, g, 1, 0.1)
        # no gradient: decay alone; a first step moves by lr against the sign
        assert torch.allclose(p[0], torch.full_like(p[0], 0.95), rtol=1e-6, atol=0)
        assert torch.allclose(p[1], torch.full_like(p[1], -0.1), rtol=1e-6, atol=0)


def test_adamw_many_tensors(rvq, dev):
    g = torch.Generator().manual_seed(4)
    sizes = [int(x) for x in torch.randint(0, 900, (133,), generator=g)]
    for bits in (32, 8):
        t = _tensors(sizes, F32, F32, bits, dev, copies=True)
        _check(rvq, t, bits, F32)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_clips(rvq, dev, bits):
    sizes = [5000, 1, 257, 300000] + [37] * 60
    for max_norm, scale in ((0.5, 1.0), (1e6, 1.0), (0.5, 0.125)):
        t = _tensors(sizes, F32, BF16, bits, dev)
        norm64 = torch.sqrt(sum(x.double().square().sum() for x in t["g"])) * scale
        factor = scale * min(1.0, max_norm / (float(norm64) + 1e-6))
        norm = _check(rvq, t, bits, F32, factor=factor, max_norm=max_norm, grad_scale=scale)
        # eight squares to a lane's fp32 sum, the rest in fp64
        assert abs(float(norm) - float(norm64)) <= 16 * ref.U * float(norm64)
    t = _tensors(sizes, F32, BF16, bits, dev)
    assert _check(rvq, t, bits, F32) is None
    norm = _check(rvq, t, bits, F32, need_norm=True)
    assert abs(float(norm) - float(norm64) * 8) <= 16 * ref.U * float(norm64) * 8


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_where_the_norm_is_not_finite(rvq, dev, bits):
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        t = _tensors([300, 5000], F32, F32, bits, dev, copies=True)
        t["g"][1][4321] = bad
        if bad == 3e38:
            t["g"][1][4320] = bad   # finite values whose squares' sum is not finite in fp32
        raw = lambda: [x.view(torch.uint8).clone() for k in ("p", "m", "v", "ms", "vs", "copies") if t[k] for x in t[k]]  # noqa: E731
        before = raw()
        st = rvq.rvq_adamw_init(t["p"], bits, DECAY, t["copies"], t["m"], t["v"], t["ms"], t["vs"])
        norm = rvq.rvq_adamw_step(st, t["g"], 1, LR, max_norm=1.0)
        assert not torch.isfinite(norm).any()
        for a, b in zip(before, raw()):
            assert torch.equal(a, b)


def test_adamw_rounding_at_random(rvq, dev):
    # one value for a whole tensor: the share of elements that round up has to
    # be the remainder's, within 6 standard deviations, and another seed,
    # step or tensor gives other choices
    n = 1 << 18
    p0 = 1.0 + 2.0 ** -8 * 0.3            # between two bf16 values, 0.3 / 2 of the way up
    outs = []
    for seed, step in ((1, 1), (2, 1), (1, 2)):
        p = [torch.full((n,), 1.0, dtype=BF16, device=dev) for _ in range(2)]
        g = [torch.zeros(n, device=dev) for _ in range(2)]
        st = rvq.rvq_adamw_init(p, 32, weight_decay=-(p0 - 1.0))
        rvq.rvq_adamw_step(st, g, step, 1.0, seed=seed)
        for x in p:
            up = (x.float() > 1.0).double().mean().item()
            assert set(x.float().unique().tolist()) <= {1.0, 1.0 + 2.0 ** -7}
            assert abs(up - 0.15) <= 6 * (0.15 * 0.85 / n) ** 0.5 + 2.0 ** -11
            outs.append(x.clone())
    for i in range(len(outs)):
        for j in range(i):
            same = (outs[i] == outs[j]).double().mean().item()
            assert abs(same - (0.15 ** 2 + 0.85 ** 2)) <= 0.01, (i, j)
    # the 8-bit moments: one large element a block fixes the scale at 1
    for target in (0.3, 5.3, 0.0101, 0.0011, -77.0, -0.003):
        m = torch.full((n,), 0.0, device=dev)
        g = torch.full((n,), target * 10, device=dev)
        g.view(-1, 256)[:, 0] = 4480.0
        st = rvq.rvq_adamw_init([torch.zeros(n, device=dev)], 8)
        rvq.rvq_adamw_step(st, [g], 1, 0.0, seed=9)
        m = (st.m[0].float() * st.m_scale[0].repeat_interleave(256)).view(-1, 256)[:, 1:].double()
        step = float(ref.f8_step(torch.tensor(target, dtype=torch.float64)))
        assert (m - target).abs().max().item() <= step * (1 + 1e-5)
        assert abs(m.mean().item() - target) <= 6 * step / 2 / m.numel() ** 0.5 + step * 2 ** -10 + 1e-6 * abs(target)
        r = (st.v[0].float() * st.v_scale[0].repeat_interleave(256)).view(-1, 256)[:, 1:].double()
        root = abs(target * 10) * 0.001 ** 0.5
        unit = float(st.v_scale[0][0])
        step = unit * float(ref.f8_step(torch.tensor(root / unit, dtype=torch.float64)))
        assert abs(r.mean().item() - root) <= 6 * step / 2 / r.numel() ** 0.5 + step * 2 ** -11 + 1e-5 * root


def test_adamw_rounding_bits_depend_on_seed_step_place_and_element_alone(rvq, dev):
    # the same tensor at place 70 of a call, among small and among large ones
    # (other launches, other workgroups), and on a second run
    g0 = torch.Generator(device=dev).manual_seed(1)
    p0, g = torch.randn(5000, generator=g0, device=dev), torch.randn(5000, generator=g0, device=dev)
    outs = []
    for others in (1, 3000, 0, 3000):
        p = [torch.zeros(others, device=dev) for _ in range(70)] + [p0.to(BF16).float()] + [torch.zeros(9, device=dev)]
        st = rvq.rvq_adamw_init(p, 8)
        rvq.rvq_adamw_step(st, [torch.zeros_like(x) for x in p[:70]] + [g, torch.zeros(9, device=dev)], 7, 0.1, seed=5)
        outs.append([x.view(torch.uint8).clone() for x in (st.m[70], st.v[70], st.m_scale[70], p[70])])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_adamw_norm_of_few_and_of_many_workgroups(rvq, dev):
    # up to 1024 workgroups' sums are added in the step itself, more by a launch
    # of their own; empty tensors first, and a call of nothing but empty ones
    for n in (1, 2048 * 1024 - 5, 2048 * 1024 + 1, 5000000):
        for bits in (32, 8):
            p = [torch.zeros(0, device=dev), torch.zeros(n, device=dev)]
            g = [torch.zeros(0, device=dev), torch.full((n,), 0.5, device=dev)]
            st = rvq.rvq_adamw_init(p, bits)
            norm = rvq.rvq_adamw_step(st, g, 1, 0.1, max_norm=0.25 * n ** 0.5)
            assert abs(float(norm) - 0.5 * n ** 0.5) <= 16 * ref.U * 0.5 * n ** 0.5
            m = st.m[1].double() if bits == 32 else st.m[1].double() * float(st.m_scale[1][0])
            # the factor is 1/2 (1e-6 less the smaller the norm): m = 0.1 * 0.25
            assert torch.all((m - 0.025).abs() <= 0.025 * (1e-5 + 1e-5 / n ** 0.5)), (n, bits)
    st = rvq.rvq_adamw_init([torch.zeros(0, device=dev)])
    assert float(rvq.rvq_adamw_step(st, [torch.zeros(0, device=dev)], 1, 0.1, max_norm=1.0)) == 0.0


def test_adamw_8_bit_states_follow_32_bit_ones(rvq, dev):
    # a noisy quadratic: 300 steps of both; the 8-bit run has to end about as
    # near the minimum (within twice the 32-bit run's distance)
    n, steps = 20000, 300
    g0 = torch.Generator(device=dev).manual_seed(5)
    target = torch.randn(n, generator=g0, device=dev)
    curve = torch.logspace(-2, 1, n, device=dev)
    ends = {}
    for bits in (32, 8):
        g = torch.Generator(device=dev).manual_seed(6)
        p = torch.zeros(n, device=dev)
        st = rvq.rvq_adamw_init([p], bits, 0.0)
        for t in range(1, steps + 1):
            noise = 0.1 * torch.randn(n, generator=g, device=dev)
            rvq.rvq_adamw_step(st, [curve * (p - target) + noise * curve.sqrt()], t, 0.02, seed=11)
        ends[bits] = float((p - target).norm() / target.norm())
    assert ends[32] < 0.5 and ends[8] < 2 * ends[32], ends


def test_adamw_offsets_past_32_bits(rvq, dev):
    n = (1 << 32) + 1000
    p = torch.zeros(n, dtype=BF16, device=dev)
    g = torch.zeros(n, dtype=BF16, device=dev)
    p[-700:], g[-300:], p[:5] = 1.0, 1.0, 2.0
    st = rvq.rvq_adamw_init([p], 8, 0.5)
    norm = rvq.rvq_adamw_step(st, [g], 1, 0.25, max_norm=1e9)
    assert abs(float(norm) - 300 ** 0.5) <= 1e-5
    assert torch.all(p[:5] == 2.0 * 0.875) and torch.all(p[-700:-300] == 0.875) and torch.all(p[-300:] == 0.625)
    assert torch.all(p[5:1 << 20] == 0) and torch.all(p[1 << 32:(1 << 32) + 300] == 0)


def test_adamw_refusals(rvq, dev):
    p = [torch.zeros(100, device=dev), torch.zeros(50, device=dev)]
    g = [torch.zeros(100, device=dev), torch.zeros(50, device=dev)]
    st = rvq.rvq_adamw_init(p)
    for bad in ([g[0]], [g[0], g[1][:49]], [g[0], g[1].bfloat16()], [g[0], g[1].cpu()],
                [g[0], torch.zeros(100, device=dev)[::2]], [g[0].double(), g[1].double()]):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_adamw_step(st, bad, 1, 0.1)
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(eps=0.0),
                dict(grad_scale=float("inf"))):
        with pytest.raises(rvq.RVQError) as e:
            rvq.rvq_adamw_step(st, g, **{**dict(step=1, lr=0.1), **bad})
        assert e.value.status == 1
    with pytest.raises(ValueError):
        rvq.rvq_adamw_step(st, g, 1, 0.1, max_norm=0.0)
    f = torch.zeros
    for args, kw in (([[]], {}), ([[p[0], p[1].bfloat16()]], {}), ([[p[0].cpu()]], {}), ([p, 16], {}),
                     ([p], dict(m=[f(100, device=dev)])), ([p], dict(weight_decay=[0.1])),
                     ([p], dict(m=[f(100, device=dev), f(49, device=dev)], v=g)), ([p], dict(m_scale=g)),
                     ([p, 8], dict(m=g, v=g)), ([p], dict(copies=p))):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_adamw_init(*args, **kw)
    assert all(torch.all(x == 0) for x in p)
    # memory that was replaced after init
    p[0].data = torch.ones(100, device=dev)
    with pytest.raises(ValueError):
        rvq.rvq_adamw_step(st, g, 1, 0.1)
    assert torch.all(p[0] == 1)


def test_adamw_nan_and_infinity_stay_in_their_places(rvq, dev):
    # without a norm nothing is skipped: the elements become NaN, and those of
    # other blocks are untouched by it
    for bits, seed in ((32, None), (8, None), (8, 3)):
        p, g = torch.ones(1024, device=dev), torch.ones(1024, device=dev)
        g[300], g[700] = float("nan"), float("inf")
        st = rvq.rvq_adamw_init([p], bits, 0.0)
        rvq.rvq_adamw_step(st, [g], 1, 0.1, seed=seed)
        bad = torch.isnan(p)
        assert bad[300] and bad[700] and int(bad.sum()) == 2
        assert torch.allclose(p[~bad], torch.full_like(p[~bad], 0.9), rtol=1e-5)
        if bits == 8:
            m = st.m[0].float() * st.m_scale[0].repeat_interleave(256)
            assert torch.isnan(m[300]) and torch.isnan(m[700])
            assert torch.isfinite(m[:256]).all() and torch.isfinite(m[768:]).all()
