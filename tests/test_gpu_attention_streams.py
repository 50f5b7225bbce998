"""The attention operators on streams beside one another."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_attention import F16, _cuda  # noqa: E402,F401
from w4a16_routed_expert_gb300 import capi  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402


def test_a_report_on_one_stream_leaves_a_forward_on_another_alone():
    """Appends with a bad slot are reported again and again while forwards of
    the same handle run: some words of each stand between its kernels and its
    join at any time, and none of them may go."""
    Hk, D, page, seqs, n = 8, 64, 16, 64, 3000
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-n // page)
    kc, vc = (torch.randn(seqs * pages, page, Hk, D, generator=gen, device="cuda").half() for _ in range(2))
    a = PagedAttention(num_q_heads=Hk, num_kv_heads=Hk, head_dim=D, max_tokens=seqs, max_seqs=seqs, k_cache=kc, v_cache=vc)
    q = torch.randn(seqs, Hk, D, generator=gen, device="cuda").half()
    args = dict(q_offsets=torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), max_q_len=1, max_seq_len=n,
                seq_lens=torch.full((seqs,), n, dtype=torch.int32, device="cuda"),
                block_table=torch.arange(seqs * pages, dtype=torch.int32, device="cuda").view(seqs, pages))
    want = a.forward(q, **args)
    a.sync()
    outs = torch.empty(400, seqs, Hk, D, dtype=F16, device="cuda")
    x = torch.ones(1, Hk, D, dtype=F16, device="cuda")
    zero, beyond = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in (0, kc.shape[0] * page))
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    a.append(None, x, x, zero, beyond)  # its kernel is loaded at its first launch
    with pytest.raises(capi.MoEError):
        a.sync()
    torch.cuda.synchronize()
    end = torch.cuda.Event()
    with torch.cuda.stream(s):
        for o in outs:
            a.forward(q, out=o, **args)
        end.record()
    reports = 0
    with torch.cuda.stream(other):
        while not end.query():
            a.append(None, x, x, zero, beyond)
            with pytest.raises(capi.MoEError) as e:
                a.sync(other)
            assert e.value.status == capi.MOE_ERR_INVALID_ARG
            reports += 1
    torch.cuda.synchronize()
    assert reports > 3
    assert all(torch.equal(o, want) for o in outs)
    a.sync()
    assert float(want.abs().max()) > 0


def test_outputs_of_a_call_on_a_given_stream_have_memory_of_that_stream():
    """Memory that the current stream has freed, but will still write, is not
    handed to a call on another stream."""
    H, D, page = 4, 64, 16
    kc, vc = (torch.zeros(4, page, H, D, device="cuda").half() for _ in range(2))
    a = PagedAttention(num_q_heads=H, num_kv_heads=H, head_dim=D, rotary_dim=D, max_tokens=8, max_seqs=8, k_cache=kc, v_cache=vc)
    x = torch.randn(8, H, D, device="cuda").half()
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    batch = dict(q_offsets=torch.arange(9, dtype=torch.int32, device="cuda"), max_q_len=1, seq_lens=pos, max_seq_len=8,
                 block_table=torch.zeros(8, 1, dtype=torch.int32, device="cuda"))
    s = torch.cuda.Stream()

    def calls(stream):
        q, k = a.rotate(x, x, pos, stream=stream)
        return (q, k, a.append(x, x, x, pos, pos, stream=stream)) + a.forward(x, return_lse=True, stream=stream, **batch)

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        freed = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in freed:
            t.fill_(9)
        del freed, t
        got = calls(s)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    a.sync()


def test_outputs_of_a_layer_call_on_a_given_stream_have_memory_of_that_stream():
    """The same of the routed-expert layer beside these operators."""
    import gpu_harness as GH
    from w4a16_routed_expert_gb300 import synth

    ml = GH.upload(synth.make_layer(synth.TINY, seed=3), max_tokens=16)
    x = torch.from_numpy(synth.make_tokens(synth.TINY.hidden, 16, seed=4)).cuda()
    want = ml.forward(x).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        freed = torch.empty_like(want)
        torch.cuda._sleep(20_000_000)  # about 10 ms
        freed.fill_(9)
        del freed
        got = ml.forward(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    ml.sync()
    ml.close()
