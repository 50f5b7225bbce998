"""PagedAttention: a torch-tensor convenience wrapper over include/moe_attention.h.

The attention half of a decoder block beside the routed-expert layer: norm
and rotary rotation of query and key heads, the append of keys and values to
a paged cache, and attention over that cache for a batch that may share a
prefix. PyTorch only provides device memory and streams here; the work runs
in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import capi
from .layer import _output, _ptr, _stream_handle

try:  # the handle of a device's current stream without building a Stream object (3 us a call)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

_DTYPES = {torch.float16: capi.MOE_DTYPE_F16, torch.bfloat16: capi.MOE_DTYPE_BF16}
_SCALINGS = {"none": capi.MOE_ROPE_NONE, "linear": capi.MOE_ROPE_LINEAR, "ntk": capi.MOE_ROPE_NTK,
             "yarn": capi.MOE_ROPE_YARN}


class PagedAttention:
    """Attention operators over one paged cache.

    k_cache, v_cache: cuda [num_pages][page_size][num_kv_heads][head_dim], the
    last dimension contiguous, the others in any order of strides (the same
    for both; ``cache.permute(0, 2, 1, 3)`` for pages kept head by head); both
    None for a handle that only rotates. q_norm, k_norm: cuda fp32 [head_dim]
    or None. rope_scaling: None or a dict with "kind" ("linear", "ntk",
    "yarn"), "factor" and for yarn "original_max_position" and optionally
    "beta_fast", "beta_slow". scale: of the logits (None: head_dim ** -0.5).
    The tensors must stay alive and in place while the object is used.

    Calls run on the current stream, or on `stream`, which then has to wait for
    what wrote their inputs (and these must live until it has read them);
    outputs that a call allocates belong to the stream it runs on.
    """

    def __init__(self, *, num_q_heads, num_kv_heads, head_dim, dtype=torch.float16, max_tokens=1, max_seqs=1,
                 k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None, rotary_dim=0,
                 rope_interleaved=False, rope_theta=10000.0, rope_scaling=None, q_norm=None, k_norm=None,
                 norm_eps=1e-6, scale=None):
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype}: float16 or bfloat16")
        scaling = dict(rope_scaling or {})
        kind = scaling.pop("kind", "none")
        if kind not in _SCALINGS:
            raise ValueError(f"rope_scaling kind {kind!r} unknown")
        cfg = capi.moe_attn_config_t(
            dtype=_DTYPES[dtype], num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
            max_tokens=max_tokens, max_seqs=max_seqs, rotary_dim=rotary_dim,
            rope_interleaved=int(bool(rope_interleaved)), rope_scaling=_SCALINGS[kind],
            rope_original_max_position=int(scaling.pop("original_max_position", 0)), rope_theta=rope_theta,
            rope_factor=float(scaling.pop("factor", 1.0)), rope_beta_fast=float(scaling.pop("beta_fast", 0.0)),
            rope_beta_slow=float(scaling.pop("beta_slow", 0.0)), norm_eps=norm_eps,
            scale=0.0 if scale is None else float(scale))
        if scaling:
            raise ValueError(f"rope_scaling: unknown keys {sorted(scaling)}")
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache and v_cache go together")
        if k_cache is not None:
            for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
                if (c.dim() != 4 or c.dtype != dtype or not c.is_cuda or c.shape[2:] != (num_kv_heads, head_dim)
                        or c.stride(3) != 1):
                    raise ValueError(f"{name}: cuda {dtype} [num_pages][page_size][{num_kv_heads}][{head_dim}]")
            if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
                raise ValueError("k_cache and v_cache must have the same shape and strides")
            cfg.num_pages, cfg.page_size = k_cache.shape[:2]
            cfg.page_stride, cfg.slot_stride, cfg.head_stride = k_cache.stride()[:3]
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None and (w.dtype != torch.float32 or not w.is_cuda or w.shape != (head_dim,)
                                  or not w.is_contiguous()):
                raise ValueError(f"{name}: cuda float32 [{head_dim}]")
        self.cfg, self.dtype = cfg, dtype
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        # keep the borrowed buffers alive for the handle's lifetime
        self._keep = (k_cache, v_cache, q_norm, k_norm)
        buf = capi.moe_attn_buffers_t(k_cache=_ptr(k_cache), v_cache=_ptr(v_cache), q_norm=_ptr(q_norm),
                                      k_norm=_ptr(k_norm))
        h = capi._P()
        self._lib = capi.lib()
        capi.check(self._lib.moe_attn_create(ctypes.byref(cfg), ctypes.byref(buf), ctypes.byref(h)),
                   "moe_attn_create")
        self.handle = h.value

    def _rows(self, name, t, T, heads):
        """Pointer and token stride of a [T][heads][head_dim] tensor."""
        if t.dim() != 3 or t.shape != (T, heads, self.head_dim) or t.dtype != self.dtype or not t.is_cuda:
            raise ValueError(f"{name}: cuda {self.dtype} [{T}][{heads}][{self.head_dim}], got {tuple(t.shape)} "
                             f"{t.dtype}")
        if T == 0:
            return None, 0
        st, sh, sd = t.stride()
        if sd != 1 or (heads > 1 and sh != self.head_dim):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        return t.data_ptr(), st if T > 1 else heads * self.head_dim

    def _new_rows(self, like, T, heads, stream):
        """A new [T][heads][head_dim] tensor, its pointer and token stride."""
        t = _output((T, heads, self.head_dim), self.dtype, like.device, stream)
        return t, t.data_ptr(), heads * self.head_dim

    @staticmethod
    def _ints(name, t, n):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() < n:
            raise ValueError(f"{name}: contiguous cuda int32 with at least {n} elements")
        return t.data_ptr()

    @staticmethod
    def _stream(stream, t):
        return stream.cuda_stream if stream is not None else _raw_stream(t.get_device())

    def rotate(self, q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
        """Norm and rotation of q [T][Hq][D] and k [T][Hk][D] (either may be
        None) at int32 positions [T]; returns (q_out, k_out), new tensors
        unless given. An output may be its input."""
        T = positions.shape[0]
        qp = kp = qo = ko = None
        qs = ks = qos = kos = 0
        if q is not None:
            qp, qs = self._rows("q", q, T, self.num_q_heads)
            if q_out is None:
                q_out, qo, qos = self._new_rows(q, T, self.num_q_heads, stream)
            else:
                qo, qos = self._rows("q_out", q_out, T, self.num_q_heads)
        if k is not None:
            kp, ks = self._rows("k", k, T, self.num_kv_heads)
            if k_out is None:
                k_out, ko, kos = self._new_rows(k, T, self.num_kv_heads, stream)
            else:
                ko, kos = self._rows("k_out", k_out, T, self.num_kv_heads)
        st = self._lib.moe_attn_rotate(self.handle, qp, qs, kp, ks, self._ints("positions", positions, T), T, qo, qos,
                                       ko, kos, self._stream(stream, positions))
        if st:
            capi.check(st, "moe_attn_rotate")
        return q_out, k_out

    def append(self, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
               slots: torch.Tensor, q_out: Optional[torch.Tensor] = None, stream=None):
        """rotate, with the rotated keys and the values stored at the cache's
        int32 slots [T] (page * page_size + slot of the page; negative: not
        stored). Returns q_out (None without q)."""
        T = positions.shape[0]
        qp = qo = None
        qs = qos = 0
        if q is not None:
            qp, qs = self._rows("q", q, T, self.num_q_heads)
            if q_out is None:
                q_out, qo, qos = self._new_rows(q, T, self.num_q_heads, stream)
            else:
                qo, qos = self._rows("q_out", q_out, T, self.num_q_heads)
        kp, ks = self._rows("k", k, T, self.num_kv_heads)
        vp, vs = self._rows("v", v, T, self.num_kv_heads)
        st = self._lib.moe_attn_append(self.handle, qp, qs, kp, ks, vp, vs, self._ints("positions", positions, T),
                                       self._ints("slots", slots, T), T, qo, qos, self._stream(stream, positions))
        if st:
            capi.check(st, "moe_attn_append")
        return q_out

    def forward(self, q: torch.Tensor, *, q_offsets: torch.Tensor, max_q_len: int, seq_lens: torch.Tensor,
                max_seq_len: int, block_table: Optional[torch.Tensor] = None, prefix_len: int = 0,
                prefix_pages: Optional[torch.Tensor] = None, causal: bool = True, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, return_lse: bool = False, stream=None):
        """Attention of q [T][Hq][D] over the cache (moe_attn_forward).

        Sequence b's queries are tokens q_offsets[b] .. q_offsets[b + 1]; its
        seq_lens[b] own keys are in the pages of block_table[b], after the
        prefix_len keys in prefix_pages that all sequences share. max_q_len
        and max_seq_len are upper bounds known on the host. Returns out, or
        (out, lse) when return_lse (lse fp32 [T][Hq])."""
        T, B = q.shape[0], seq_lens.shape[0]
        qp, qs = self._rows("q", q, T, self.num_q_heads)
        if out is None:
            out, op, os_ = self._new_rows(q, T, self.num_q_heads, stream)
        else:
            op, os_ = self._rows("out", out, T, self.num_q_heads)
        if lse is None and return_lse:
            lse = _output((T, self.num_q_heads), torch.float32, q.device, stream)
        if lse is not None and (lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous()
                                or lse.shape != (T, self.num_q_heads)):
            raise ValueError(f"lse: contiguous cuda float32 [{T}][{self.num_q_heads}]")
        bt, ts = None, 0
        if block_table is not None and block_table.numel():
            if (block_table.dim() != 2 or block_table.dtype != torch.int32 or not block_table.is_cuda
                    or block_table.shape[0] != B or (block_table.shape[1] > 1 and block_table.stride(1) != 1)):
                raise ValueError(f"block_table: cuda int32 [{B}][pages]")
            bt, ts = block_table.data_ptr(), block_table.stride(0) if B > 1 else block_table.shape[1]
            if max_seq_len > block_table.shape[1] * self.cfg.page_size:
                raise ValueError("max_seq_len is beyond the block table")
        pp = None
        if prefix_len > 0:
            if prefix_pages is None:
                raise ValueError("prefix_len needs prefix_pages")
            pp = self._ints("prefix_pages", prefix_pages, -(-prefix_len // self.cfg.page_size))
        batch = capi.moe_attn_batch_t(T, B, self._ints("q_offsets", q_offsets, B + 1), max_q_len,
                                      self._ints("seq_lens", seq_lens, B), max_seq_len, bt, ts, prefix_len, pp,
                                      int(bool(causal)))
        st = self._lib.moe_attn_forward(self.handle, qp, qs, ctypes.byref(batch), op, os_, _ptr(lse),
                                        self._stream(stream, q))
        if st:
            capi.check(st, "moe_attn_forward")
        return (out, lse) if return_lse else out

    def sync(self, stream=None):
        """Wait for the stream and raise for anything the kernels recorded."""
        capi.check(self._lib.moe_attn_sync(self.handle, _stream_handle(stream)), "moe_attn_sync")

    def close(self):
        if getattr(self, "handle", None):
            self._lib.moe_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
