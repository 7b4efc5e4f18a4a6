"""rvq_embed_tokens_backward against its definition: whole-number gradients,
whose sums fp32 holds exactly, have to come out exactly."""
import pytest
import torch

import learn_ref as ref

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


def _problem(T, L, K, V, D, dtype, dev, text=0.3, hot=0.0, bad=0.0, seed=0, whole=True):
    g = torch.Generator(device=dev).manual_seed(T + 31 * L + K + seed)
    rand = lambda *s: torch.rand(s, generator=g, device=dev)  # noqa: E731
    ids = (rand(T, L) * K).int().clamp_(max=K - 1)
    ids[rand(T) < hot] = K - 1
    vis = rand(T) >= text if V else torch.ones(T, dtype=torch.bool, device=dev)
    if V:
        ids[:, 0] = torch.where(vis, ids[:, 0], (rand(T) ** 2 * V).int().clamp_(max=V - 1))
    off = rand(T, L)
    ids[off < bad] = -2
    ids[off > 1 - bad] = max(K, V) + 5
    dout = (rand(T, D) * 7 - 3).floor_() if whole else torch.randn((T, D), generator=g, device=dev)
    return dout.to(dtype), ids.contiguous(), vis.to(torch.uint8)


def _check_exact(rvq, dout, ids, vis, K, V, gdt, **kw):
    L = ids.shape[1]
    bad = torch.zeros(1, dtype=torch.int32, device=dout.device)
    level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt, bad_ids=bad, **kw)
    torch.cuda.synchronize()
    wl, wt, _, _, wb = ref.embed_grad(dout, ids, vis, L, K, V)
    assert torch.equal(level, wl.to(gdt)), "level tables"
    if V:
        assert torch.equal(text, wt.to(gdt)), "text table"
    else:
        assert text is None
    if V:
        assert int(bad) == wb
    return level, text


# T, L, K, V, D: one token; fewer rows than a range; ranges and pieces that
# end unevenly; rows longer than a segment of the list; every level count
CASES = [(1, 1, 1, 0, 1), (1, 8, 300, 20, 64), (2, 3, 5, 2, 7), (63, 2, 128, 129, 8), (64, 4, 129, 1, 24),
         (65, 16, 50, 300, 40), (1000, 8, 257, 1000, 100), (1025, 64, 3, 5, 16), (3000, 2, 2, 3, 96),
         (5000, 1, 1, 1, 33), (4099, 4, 700, 3000, 260), (20000, 2, 1000, 40, 128), (257, 8, 8192, 65, 512),
         (700, 3, 40, 10, 2100), (900, 2, 11, 7, 4096)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_L%d_K%d_V%d_D%d" % c)
def test_embed_grad(rvq, dev, case):
    T, L, K, V, D = case
    for dtype, gdt, hot, bad in ((BF16, F32, 0.0, 0.0), (F32, F32, 0.3, 0.05), (BF16, BF16, 0.6, 0.02),
                                 (F32, BF16, 0.0, 0.1)):
        dout, ids, vis = _problem(T, L, K, V, D, dtype, dev, hot=hot, bad=bad)
        _check_exact(rvq, dout, ids, vis, K, V, gdt)


def test_embed_grad_one_kind_of_token(rvq, dev):
    T, L, K, V, D = 2000, 4, 90, 70, 72
    dout, ids, vis = _problem(T, L, K, V, D, BF16, dev)
    ids.clamp_(max=69)
    for flags in (None, torch.ones_like(vis), torch.zeros_like(vis), vis.bool()):
        _check_exact(rvq, dout, ids, flags, K, V, F32)
    # all tokens on one row
    _check_exact(rvq, dout, torch.zeros_like(ids), vis, K, V, F32)
    # no tokens: zeros
    level, text = rvq.rvq_embed_tokens_backward(dout[:0], ids[:0], K, None, V)
    assert torch.all(level == 0) and torch.all(text == 0)


def test_embed_grad_counts_every_out_of_range_id(rvq, dev):
    for T in (40, 5000):                      # IDs read in place, and laid out by table first
        ids = torch.zeros((T, 3), dtype=torch.int32, device=dev)
        odd = [-1, -2 ** 31, 2 ** 31 - 1, 7, -2 ** 31 + 1]
        for i, v in enumerate(odd):
            ids[3 * i, i % 3] = v
        vis = torch.ones(T, dtype=torch.uint8, device=dev)
        vis[30:36] = 0
        ids[30:32, 0] = torch.tensor([-2 ** 31, 4], dtype=torch.int32, device=dev)
        ids[32:36, 0] = 3
        ids[30:36, 1:] = -5                   # not read: text tokens have one ID
        bad = torch.zeros(1, dtype=torch.int32, device=dev)
        dout = torch.ones((T, 8), device=dev)
        level, text = rvq.rvq_embed_tokens_backward(dout, ids, 7, vis, 4, bad_ids=bad)
        assert int(bad) == len(odd) + 2
        assert torch.all(level.sum((1, 2)) == 8 * (T - 6) - 8 * torch.tensor([2, 2, 1], device=dev))
        assert torch.all(text[3] == 4) and torch.all(text[:3] == 0)


def test_embed_grad_accumulates(rvq, dev):
    for gdt, T in ((F32, 3000), (BF16, 200), (F32, 0)):
        L, K, V, D = 3, 25, 400, 50
        dout, ids, vis = _problem(T, L, K, V, D, BF16, dev, hot=0.4)
        wl, wt, _, _, _ = ref.embed_grad(dout, ids, vis, L, K, V)
        l0, t0 = torch.full((L, K, D), 5.0, device=dev, dtype=gdt), torch.full((V, D), -3.0, device=dev, dtype=gdt)
        level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, gdt, level_grad=l0, text_grad=t0,
                                                    accumulate=True)
        assert level.data_ptr() == l0.data_ptr() and text.data_ptr() == t0.data_ptr()
        assert torch.equal(level, (wl + 5.0).to(gdt)) and torch.equal(text, (wt - 3.0).to(gdt))


def test_embed_grad_frozen_tables(rvq, dev):
    T, L, K, V, D = 3000, 4, 30, 50, 64
    dout, ids, vis = _problem(T, L, K, V, D, BF16, dev, hot=0.3)
    both = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V)
    level, none = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, need_text=False)
    assert none is None and torch.equal(level, both[0])
    none, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, need_level=False)
    assert none is None and torch.equal(text, both[1])


def test_embed_grad_unaligned(rvq, dev):
    for dtype, gdt in ((BF16, F32), (F32, BF16), (F32, F32), (BF16, BF16)):
        for D in (64, 77, 520):
            T, L, K, V = 500, 2, 40, 30
            dout, ids, vis = _problem(T, L, K, V, D, dtype, dev)
            buf = torch.empty(T * D + 1, dtype=dtype, device=dev)
            buf[1:] = dout.view(-1)
            lg = torch.full((L * K * D + 2,), 9.0, dtype=gdt, device=dev)
            tg = torch.full((V * D + 2,), 9.0, dtype=gdt, device=dev)
            _check_exact(rvq, buf[1:].view(T, D), ids, vis, K, V, gdt, level_grad=lg[1:-1].view(L, K, D),
                         text_grad=tg[1:-1].view(V, D))
            assert lg[0] == 9 and lg[-1] == 9 and tg[0] == 9 and tg[-1] == 9


def test_embed_grad_rounding_and_repeats(rvq, dev):
    T, L, K, V, D = 6000, 8, 500, 300, 320
    dout, ids, vis = _problem(T, L, K, V, D, BF16, dev, hot=0.2, whole=False)
    wl, wt, al, at, _ = ref.embed_grad(dout, ids, vis, L, K, V)
    level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V)
    # a row of c tokens is c - 1 additions, in pieces of at most T
    ref.close(level, wl, T * ref.U * al, "level")
    ref.close(text, wt, T * ref.U * at, "text")
    for _ in range(3):
        again = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V)
        assert torch.equal(again[0].view(torch.int32), level.view(torch.int32))
        assert torch.equal(again[1].view(torch.int32), text.view(torch.int32))
    lb, tb = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V, BF16)
    assert torch.equal(lb, level.to(BF16)) and torch.equal(tb, text.to(BF16))


def test_embed_grad_is_the_transpose_of_the_embedding(rvq, dev):
    # <embed(tables), dout> = <tables, grad>; and the difference of the loss
    # along a direction of the tables, which is linear, is the gradient's
    T, L, K, V, D = 300, 4, 40, 25, 48
    dout, ids, vis = _problem(T, L, K, V, D, F32, dev, whole=False)
    g = torch.Generator(device=dev).manual_seed(3)
    lt, tt = (torch.randn(s, generator=g, device=dev) for s in ((L, K, D), (V, D)))
    level, text = rvq.rvq_embed_tokens_backward(dout, ids, K, vis, V)
    out = rvq.rvq_embed_tokens(ids, lt, vis, tt)
    a = (out.double() * dout.double()).sum()
    b = (level.double() * lt.double()).sum() + (text.double() * tt.double()).sum()
    size = (out.double() * dout.double()).abs().sum()
    assert abs(float(a - b)) <= (L + T) * ref.U * float(size)


def test_embed_grad_offsets_past_32_bits(rvq, dev):
    D = 65536
    # gradient rows of dout beyond 2^32 elements
    T = 66000
    dout = torch.zeros((T, D), dtype=BF16, device=dev)
    dout[-1], dout[0] = 3.0, 1.0
    ids = torch.zeros((T, 1), dtype=torch.int32, device=dev)
    ids[-1] = 2
    level, _ = rvq.rvq_embed_tokens_backward(dout, ids, 3, grad_dtype=BF16)
    assert torch.all(level[0, 0] == 1) and torch.all(level[0, 1] == 0) and torch.all(level[0, 2] == 3)
    del dout
    # table rows beyond 2^32 elements
    K = 66000
    dout = torch.full((3, D), 2.0, dtype=BF16, device=dev)
    ids = torch.tensor([[K - 1], [1], [K - 1]], dtype=torch.int32, device=dev)
    level, _ = rvq.rvq_embed_tokens_backward(dout, ids, K, grad_dtype=BF16)
    assert torch.all(level[0, -1] == 4) and torch.all(level[0, 1] == 2) and torch.all(level[0, 0] == 0)
    assert torch.all(level[0, 65535:-1] == 0)


def test_embed_grad_refusals(rvq, dev):
    dout, ids, vis = _problem(20, 2, 9, 4, 16, F32, dev)
    ok = dict(dout=dout, ids=ids, K=9, is_visual=vis, V=4)
    f = torch.empty
    for bad in (dict(ids=ids.long()), dict(ids=ids[:19]), dict(ids=ids.cpu()), dict(dout=dout.double()),
                dict(dout=dout[:, ::2]), dict(is_visual=vis[:19]), dict(is_visual=vis.int()),
                dict(level_grad=f((2, 9, 15), device=dev)), dict(text_grad=f((4, 16), device=dev, dtype=BF16)),
                dict(accumulate=True), dict(need_level=False, need_text=False), dict(need_level=False, V=0),
                dict(grad_dtype=torch.float16), dict(bad_ids=f(2, device=dev, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            rvq.rvq_embed_tokens_backward(**{**ok, **bad})
    for bad in (dict(K=0), dict(V=-1)):
        with pytest.raises(rvq.RVQError) as e:
            rvq.rvq_embed_tokens_backward(**{**ok, **bad})
        assert e.value.status == 1
