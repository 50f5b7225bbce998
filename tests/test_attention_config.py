"""What a configuration of the attention operators may hold at its edges. No
GPU."""
import ctypes

import pytest

pytest.importorskip("torch")

from test_attention_host import config, lib  # noqa: F401
from w4a16_routed_expert_gb300 import capi


@pytest.mark.parametrize("factor,m", [(1e-6, 1.0), (0.5, 1.0), (1.0, 1.0), (2.718281828459045, 1.1)])
def test_yarn_grows_cosine_and_sine_only_where_it_stretches(lib, factor, m):  # noqa: F811
    """0.1 ln(factor) + 1 is the published factor for contexts made longer;
    below, it is 1 (the formula would shrink them, and turn them over below
    e^-10)."""
    got = ctypes.c_double()
    c = config(rope_scaling=capi.MOE_ROPE_YARN, rope_factor=factor)
    assert lib.moe_attn_frequencies(ctypes.byref(c), None, ctypes.byref(got)) == capi.MOE_OK
    assert got.value == pytest.approx(m, rel=1e-14)


@pytest.mark.parametrize("scale", [1e-46, 5e-324, 3e38, 1e300])
def test_a_scale_beyond_32_bits_is_refused(lib, scale):  # noqa: F811
    """In the kernels it would be zero or infinity, and every output NaN."""
    h = ctypes.c_void_p(1)
    buf = capi.moe_attn_buffers_t(k_cache=4096, v_cache=8192)
    assert lib.moe_attn_create(ctypes.byref(config(scale=scale)), ctypes.byref(buf), ctypes.byref(h)) == capi.MOE_ERR_INVALID_ARG
    assert h.value is None and "scale" in capi.last_error()
