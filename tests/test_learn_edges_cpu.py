"""Host-side checks of the calls that train the token embedding, beside those of
test_learn_abi_cpu.py (no GPU needed)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "residual_vector_quantization_rvq_amd", "librvq.so")


@pytest.fixture(scope="module")
def rvq():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__._builder().build()
    import residual_vector_quantization_rvq_amd as m
    return m


def test_adamw_workspace_is_that_of_its_launches(rvq):
    # a launch of the norm takes 160 tensors and leaves 2,048 sums of 8 bytes
    for count in (0, 1, 96, 160, 161, 10000, 1000000):
        launches = max(1, -(-count // 160))
        assert launches * 16384 <= rvq.rvq_adamw_workspace_size(count) <= launches * 16384 + 1024


def test_sizes_past_32_bits_are_refused(rvq):
    # ctypes would hand their low bits to the library
    for call in (lambda: rvq.rvq_rms_norm_backward_workspace_size(4, 2 ** 32 + 8),
                 lambda: rvq.rvq_embed_tokens_backward_workspace_size(4, 2, 2 ** 32 + 3, 0, 8),
                 lambda: rvq.rvq_embed_tokens_backward_workspace_size(4, 2, 3, 0, 2 ** 32 + 8),
                 lambda: rvq.rvq_embed_tokens_backward_workspace_size(4, 2, 3, 2 ** 64 + 4, 8),
                 lambda: rvq.rvq_adamw_workspace_size(2 ** 32 + 1)):
        with pytest.raises((ValueError, rvq.RVQError)):
            call()


def test_adamw_options_outside_fp32(rvq):
    lib = rvq.raw_library()

    def call(**kw):
        o = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, step=1, grad_scale=1.0, max_norm=0.0, stochastic=0, seed=0)
        o.update(kw)
        opt = rvq._AdamWOptions(*o.values())
        return lib.rvq_adamw_step(None, 0, 0, 0, 32, ctypes.byref(opt), None, None, 0, None)
    for bad in (dict(grad_scale=1e39), dict(grad_scale=-1e39), dict(lr=1e39), dict(lr=1e38, beta1=0.9999)):
        assert call(**bad) == 1, bad
    for ok in (dict(grad_scale=3e38), dict(lr=1e37), dict(max_norm=1e-60, lr=0.0)):
        # nothing to do, so nothing is launched (max_norm asks for a workspace first)
        assert call(**ok) == (1 if "max_norm" in ok else 0), ok


def test_norm_refuses_one_place_for_sum_and_y(rvq):
    # x, residual, x_dtype, n, d, weight, weight_dtype, eps, sum_out, y, y_dtype, y_scale, rstd, stream
    args = [256, 256, 0, 4, 8, None, 0, 1e-6, 512, 512, 0, None, None, None]
    assert rvq.raw_library().rvq_rms_norm(*args) == 1
