"""Host side of the attention operators: frequencies against their formulas
and the refusals of create. No GPU."""
import ctypes

import numpy as np
import pytest

pytest.importorskip("torch")

import attention_oracle as AO
from w4a16_routed_expert_gb300 import build as B
from w4a16_routed_expert_gb300 import capi


@pytest.fixture(scope="module")
def lib():
    B.build()
    return capi.lib()


def config(**kw):
    d = dict(dtype=0, num_q_heads=16, num_kv_heads=4, head_dim=128, max_tokens=8, max_seqs=4, rotary_dim=128,
             rope_interleaved=0, rope_scaling=0, rope_original_max_position=4096, rope_theta=10000.0, rope_factor=1.0,
             rope_beta_fast=0.0, rope_beta_slow=0.0, norm_eps=1e-6, scale=0.0, page_size=16, reserved=0, num_pages=8,
             page_stride=16 * 4 * 128, slot_stride=4 * 128, head_stride=128)
    d.update(kw)
    return capi.moe_attn_config_t(**d)


@pytest.mark.parametrize("rotary", [8, 24, 64, 128])
@pytest.mark.parametrize("kind,code,factor", [("none", 0, 1.0), ("linear", 1, 4.0), ("ntk", 2, 8.0), ("yarn", 3, 16.0),
                                              ("yarn", 3, 1.0)])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_frequencies(lib, rotary, kind, code, factor, theta):
    c = config(rotary_dim=rotary, rope_scaling=code, rope_factor=factor, rope_theta=theta)
    f, m = (ctypes.c_double * 64)(), ctypes.c_double()
    assert lib.moe_attn_frequencies(ctypes.byref(c), f, ctypes.byref(m)) == capi.MOE_OK
    want, wm = AO.frequencies(rotary, theta, kind, factor)
    np.testing.assert_allclose(list(f)[:rotary // 2], want, rtol=1e-13)
    assert m.value == pytest.approx(wm, rel=1e-14)
    if kind == "yarn" and factor > 1:  # fast pairs keep their frequency, slow ones are divided
        plain = AO.frequencies(rotary, theta)[0]
        assert f[0] == pytest.approx(plain[0]) and (rotary < 64 or f[rotary // 2 - 1] == pytest.approx(plain[-1] / factor))


def test_frequencies_of_no_rotation_and_null_outputs(lib):
    m = ctypes.c_double()
    assert lib.moe_attn_frequencies(ctypes.byref(config(rotary_dim=0)), None, ctypes.byref(m)) == capi.MOE_OK
    assert m.value == 1.0
    assert lib.moe_attn_frequencies(ctypes.byref(config()), None, None) == capi.MOE_OK
    assert lib.moe_attn_frequencies(None, None, None) == capi.MOE_ERR_INVALID_ARG


INVALID = [dict(dtype=2), dict(num_kv_heads=0), dict(num_kv_heads=3), dict(num_q_heads=2048), dict(rotary_dim=136),
           dict(rotary_dim=-8), dict(rope_interleaved=2), dict(rope_scaling=4), dict(rope_theta=1.0),
           dict(rope_theta=float("nan")), dict(rope_scaling=1, rope_factor=0.0), dict(rope_scaling=2, rope_factor=-1.0),
           dict(rope_scaling=3, rope_factor=2.0, rope_original_max_position=0),
           dict(rope_scaling=3, rope_factor=2.0, rope_beta_fast=-1.0), dict(norm_eps=-1e-6), dict(norm_eps=float("inf")),
           dict(scale=-1.0), dict(scale=float("nan")), dict(reserved=1), dict(max_tokens=0), dict(max_tokens=(1 << 20) + 1),
           dict(max_seqs=0), dict(max_seqs=4097), dict(num_pages=0), dict(num_pages=1 << 28), dict(page_stride=0),
           dict(slot_stride=12), dict(slot_stride=64), dict(head_stride=-128), dict(head_stride=120)]
UNSUPPORTED = [dict(head_dim=136, rotary_dim=0), dict(head_dim=20, rotary_dim=0), dict(head_dim=0, rotary_dim=0),
               dict(rotary_dim=20), dict(page_size=8), dict(page_size=24), dict(page_size=2048)]


@pytest.mark.parametrize("bad,status", [(b, capi.MOE_ERR_INVALID_ARG) for b in INVALID]
                         + [(b, capi.MOE_ERR_UNSUPPORTED) for b in UNSUPPORTED], ids=str)
def test_create_refuses(lib, bad, status):
    h = ctypes.c_void_p(1)
    buf = capi.moe_attn_buffers_t(k_cache=4096, v_cache=8192)
    assert lib.moe_attn_create(ctypes.byref(config(**bad)), ctypes.byref(buf), ctypes.byref(h)) == status
    assert h.value is None and capi.last_error()


def test_create_refuses_pointers(lib):
    h = ctypes.c_void_p()
    for buf in (capi.moe_attn_buffers_t(k_cache=4096), capi.moe_attn_buffers_t(v_cache=4096),
                capi.moe_attn_buffers_t(k_cache=4096, v_cache=8200),
                capi.moe_attn_buffers_t(k_cache=4096, v_cache=8192, q_norm=4100),
                capi.moe_attn_buffers_t(k_norm=4104)):
        assert lib.moe_attn_create(ctypes.byref(config()), ctypes.byref(buf), ctypes.byref(h)) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_attn_create(None, None, ctypes.byref(h)) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_attn_create(ctypes.byref(config()), ctypes.byref(capi.moe_attn_buffers_t()), None) == capi.MOE_ERR_INVALID_ARG
