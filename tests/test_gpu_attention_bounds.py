"""Attention calls whose device-side lengths and offsets contradict what the
host was told."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_attention import F16, _cuda, caches  # noqa: E402,F401
from w4a16_routed_expert_gb300 import capi  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402


@pytest.mark.parametrize("prefix", [0, 40])
def test_sequences_that_overlap_by_more_than_32_bits_of_tiles(prefix):
    """Every second sequence says that all tokens are its own: the key tiles
    of them all pass 2^32. That is reported, and the next call is right."""
    T, H, D, B, page = 8192, 64, 8, 2048, 1024
    kc, vc = caches(3, page, H, D, F16, "slot", fill=0.5)
    a = PagedAttention(num_q_heads=H, num_kv_heads=H, head_dim=D, max_tokens=T, max_seqs=B, k_cache=kc, v_cache=vc)
    q = torch.ones(T, H, D, dtype=F16, device="cuda")
    table = torch.zeros(B, 1024, dtype=torch.int32, device="cuda")
    pages = torch.ones(1, dtype=torch.int32, device="cuda")

    def run(offsets, lens, max_q, max_keys):
        return a.forward(q, q_offsets=offsets.to(torch.int32).cuda(), max_q_len=max_q, max_seq_len=max_keys,
                         seq_lens=torch.full((B,), lens, dtype=torch.int32, device="cuda"), block_table=table,
                         prefix_len=prefix, prefix_pages=pages)

    run(torch.arange(B + 1) % 2 * T, 1 << 20, T, 1 << 20)
    with pytest.raises(capi.MoEError) as e:
        a.sync()
    assert e.value.status == capi.MOE_ERR_INVALID_ARG
    for max_q, max_keys in ((T // B, 64), (T, 1 << 20)):  # the few-row kernel; the tile kernel with the bounds from before
        out = run(torch.arange(B + 1) * (T // B), 37, max_q, max_keys)
        a.sync()
        assert (out == 0.5).all()
