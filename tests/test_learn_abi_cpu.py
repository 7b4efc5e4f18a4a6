"""Host-side checks of the calls that train the token embedding: sizes and
bad arguments, which return a status before any HIP call (no GPU needed).
Addresses are fakes that nothing reads."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "residual_vector_quantization_rvq_amd", "librvq.so")
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def rvq():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__._builder().build()
    import residual_vector_quantization_rvq_amd as m
    return m


def _caller(fn, names, ok):
    def call(**kw):
        a = {**ok, **kw}
        return fn(*[a[n] for n in names])
    return call


def test_exports_the_learning_calls(rvq):
    names = set(rvq.exported_symbols())
    assert {"rvq_rms_norm", "rvq_rms_norm_backward", "rvq_rms_norm_backward_workspace_size",
            "rvq_embed_tokens_backward", "rvq_embed_tokens_backward_workspace_size", "rvq_adamw_step",
            "rvq_adamw_workspace_size"} <= names


def test_norm_arguments(rvq):
    names = "x res xdt n d w wdt eps sum y ydt scale rstd stream".split()
    ok = dict(x=256, res=256, xdt=0, n=4, d=8, w=256, wdt=0, eps=1e-6, sum=256, y=256, ydt=0, scale=None, rstd=256,
              stream=None)
    call = _caller(rvq.raw_library().rvq_rms_norm, names, ok)
    for bad in (dict(n=-1), dict(d=0), dict(xdt=2), dict(xdt=7), dict(ydt=3), dict(wdt=2), dict(eps=0.0),
                dict(eps=float("nan")), dict(x=None), dict(x=258), dict(res=257), dict(y=None), dict(y=2),
                dict(w=2), dict(sum=2), dict(rstd=2), dict(ydt=2), dict(ydt=2, scale=2)):
        assert call(**bad) == 1, bad
    assert call(n=(1 << 25) + 1) == 2 and call(d=(1 << 20) + 1) == 2
    assert call(n=0, x=None, y=None) == 0


def test_norm_gradient_arguments(rvq):
    names = "dy h dt n d rstd w wdt dsum dx dw ws bytes stream".split()
    ok = dict(dy=256, h=256, dt=1, n=4, d=8, rstd=256, w=256, wdt=1, dsum=None, dx=256, dw=256, ws=256,
              bytes=1 << 30, stream=None)
    call = _caller(rvq.raw_library().rvq_rms_norm_backward, names, ok)
    for bad in (dict(n=-1), dict(d=0), dict(dt=2), dict(wdt=5), dict(dy=None), dict(h=None), dict(rstd=None),
                dict(dx=None), dict(dy=257), dict(dsum=257), dict(dw=2), dict(ws=None), dict(ws=128)):
        assert call(**bad) == 1, bad
    assert call(bytes=16) == 3
    assert call(n=(1 << 25) + 1) == 2
    assert call(n=0, dw=None, dy=None, h=None, rstd=None, dx=None, ws=None) == 0
    size = rvq.rvq_rms_norm_backward_workspace_size
    assert size(0, 8) >= 32 and size(100000, 4096) % 256 == 0 and size(1, 1) > 0


def test_embedding_gradient_arguments(rvq):
    names = "dout dt ids vis T L K V D dl dtx gdt acc bad ws bytes stream".split()
    ok = dict(dout=256, dt=0, ids=256, vis=None, T=4, L=2, K=3, V=5, D=8, dl=256, dtx=256, gdt=0, acc=0, bad=None,
              ws=256, bytes=1 << 30, stream=None)
    call = _caller(rvq.raw_library().rvq_embed_tokens_backward, names, ok)
    for bad in (dict(T=-1), dict(L=0), dict(K=0), dict(D=0), dict(V=-1), dict(dt=2), dict(gdt=2), dict(dout=None),
                dict(ids=None), dict(ids=2), dict(dout=2), dict(dl=2), dict(dtx=2), dict(bad=2), dict(ws=None),
                dict(ws=128), dict(dl=None, dtx=None)):
        assert call(**bad) == 1, bad
    assert call(bytes=16) == 3
    assert call(L=65) == 2 and call(T=1 << 25, L=64) == 2 and call(V=(1 << 28)) == 2 and call(K=1 << 28) == 2
    size = rvq.rvq_embed_tokens_backward_workspace_size
    # a call may leave either table out and use the same workspace
    for T, L, K, V, D in ((100, 2, 3, 5, 8), (70000, 16, 300, 1000, 64), (300000, 8, 8192, 65536, 128), (0, 1, 1, 0, 1)):
        assert size(T, L, K, V, D) >= size(T, L, K, 0, D) > 0


def test_adamw_arguments(rvq):
    lib = rvq.raw_library()
    import residual_vector_quantization_rvq_amd as m
    one = m._AdamWTensor(256, 256, 256, 256, None, None, None, 10, 0.1, 0)

    def call(tensor=None, count=1, pdt=0, gdt=0, bits=32, norm=None, ws=None, nbytes=0, **kw):
        t = m._AdamWTensor.from_buffer_copy(one)
        for k, v in (tensor or {}).items():
            setattr(t, k, v)
        o = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, step=1, grad_scale=1.0, max_norm=0.0, stochastic=0, seed=0)
        o.update(kw)
        opt = m._AdamWOptions(*o.values())
        return lib.rvq_adamw_step(ctypes.byref(t), count, pdt, gdt, bits, ctypes.byref(opt), norm, ws, nbytes, None)
    for bad in (dict(count=-1), dict(pdt=2), dict(gdt=2), dict(bits=16), dict(lr=-1.0), dict(lr=float("inf")),
                dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(step=0), dict(grad_scale=float("nan")),
                dict(max_norm=float("inf")), dict(tensor=dict(param=None)), dict(tensor=dict(grad=None)),
                dict(tensor=dict(m=None)), dict(tensor=dict(v=2)), dict(tensor=dict(param=2)),
                dict(tensor=dict(copy=1)), dict(tensor=dict(numel=-1)), dict(bits=8),
                dict(tensor=dict(weight_decay=float("nan"))), dict(max_norm=1.0), dict(norm=256),
                dict(max_norm=1.0, ws=128, nbytes=1 << 20)):
        assert call(**bad) == 1, bad
    assert call(max_norm=1.0, ws=256, nbytes=8) == 3
    assert call(tensor=dict(numel=(1 << 34) + 1)) == 2
    assert lib.rvq_adamw_step(None, 1, 0, 0, 32, None, None, None, 0, None) == 1
    # empty tensors are left out; nothing to do makes no HIP call
    assert call(tensor=dict(numel=0, param=None, grad=None, m=None, v=None)) == 0
    assert call(count=0) == 0
    assert rvq.rvq_adamw_workspace_size(0) > 0 and rvq.rvq_adamw_workspace_size(1000) >= rvq.rvq_adamw_workspace_size(10)
