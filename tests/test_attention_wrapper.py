"""The torch-tensor wrapper of the attention operators without a GPU: what it
refuses before the library is called, and on which stream it allocates. The
tensors and the library are stand-ins."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from w4a16_routed_expert_gb300 import attention, capi
from w4a16_routed_expert_gb300.attention import PagedAttention

HQ, HK, D, T, B = 4, 2, 64, 3, 2


class Tensor:
    """A tensor that says it is on the GPU."""

    def __init__(self, *shape, dtype=torch.float16):
        self._on_cpu = torch.empty(shape, dtype=dtype)
        self.is_cuda, self.device = True, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getitem__(self, at):
        return self._on_cpu[at]

    def __getattr__(self, name):
        return getattr(self._on_cpu, name)


def ints(*shape):
    return Tensor(*shape, dtype=torch.int32)


@pytest.fixture
def attn():
    """A wrapper whose library notes each call's name and last argument (the
    stream)."""
    calls = []
    a = PagedAttention.__new__(PagedAttention)
    a.handle, a.dtype, a.num_q_heads, a.num_kv_heads, a.head_dim = None, torch.float16, HQ, HK, D
    a.cfg = capi.moe_attn_config_t(page_size=16)
    a.calls = calls

    def entry(name):
        return lambda *args: calls.append((name, args[-1])) or 0

    a._lib = types.SimpleNamespace(**{n: entry(n) for n in ("moe_attn_rotate", "moe_attn_append", "moe_attn_forward")})
    return a


def forward(a, **kw):
    return a.forward(Tensor(T, HQ, D), q_offsets=ints(B + 1), max_q_len=2, seq_lens=ints(B), max_seq_len=20,
                     block_table=ints(B, 2), out=Tensor(T, HQ, D), **kw)


def test_an_lse_that_is_not_on_the_gpu_is_refused(attn, monkeypatch):
    monkeypatch.setattr(attention, "_raw_stream", lambda index: 7)
    with pytest.raises(ValueError):
        forward(attn, lse=torch.empty(T, HQ))
    assert not attn.calls
    lse = Tensor(T, HQ, dtype=torch.float32)
    assert forward(attn, lse=lse, return_lse=True)[1] is lse
    assert attn.calls == [("moe_attn_forward", 7)]


class Streams:
    """torch.cuda's current stream and torch.empty, which notes the stream."""

    def __init__(self, monkeypatch):
        self.current = types.SimpleNamespace(cuda_stream=7)
        self.allocated, self.recorded = [], []
        monkeypatch.setattr(torch.cuda, "stream", self.use)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: self.current)
        monkeypatch.setattr(attention, "_raw_stream", lambda index: self.current.cuda_stream)
        empty = torch.empty

        def new(*shape, dtype=None, device=None):
            self.allocated.append(self.current)
            t = Tensor.__new__(Tensor)
            t._on_cpu, t.is_cuda, t.device = empty(*shape, dtype=dtype), True, torch.device("cuda", 0)
            t.record_stream = self.recorded.append
            return t

        monkeypatch.setattr(torch, "empty", new)

    @contextlib.contextmanager
    def use(self, stream):
        kept, self.current = self.current, stream
        yield
        self.current = kept


def test_outputs_belong_to_the_stream_that_writes_them(attn, monkeypatch):
    q, k, v, pos, q_out = Tensor(T, HQ, D), Tensor(T, HK, D), Tensor(T, HK, D), ints(T), Tensor(T, HQ, D)
    batch = dict(q_offsets=ints(B + 1), max_q_len=2, seq_lens=ints(B), max_seq_len=20, block_table=ints(B, 2))
    own = types.SimpleNamespace(cuda_stream=9)
    for stream, number in ((None, 7), (own, 9)):
        at = Streams(monkeypatch)
        attn.calls.clear()
        attn.rotate(q, k, pos, stream=stream)
        attn.append(q, k, v, pos, pos, stream=stream)
        attn.forward(q, return_lse=True, stream=stream, **batch)
        attn.append(q, k, v, pos, pos, q_out=q_out, stream=stream)  # nothing to allocate
        assert [s for _, s in attn.calls] == [number] * 4
        assert len(at.allocated) == 5 and all(s.cuda_stream == number for s in at.allocated)
        assert at.recorded == ([] if stream is None else [at.current] * 5)  # a reader on the current stream is waited for
        monkeypatch.undo()
