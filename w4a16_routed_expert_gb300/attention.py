"""PagedAttention: a torch-tensor convenience wrapper over include/moe_attention.h.

The attention half of a decoder block beside the routed-expert layer: norm
and rotary rotation of query and key heads, the append of keys and values to
a paged cache, and attention over that cache for a batch that may share a
prefix and whose new tokens may be trees of drafted ones; around such a step,
the tables that it needs from lengths on the GPU, the branch that the model
confirms and the move of its keys and values. PyTorch only provides device memory and streams here; the work runs
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


def _int32(name, t, *shape):
    """Checks a contiguous cuda int32 tensor (None in the shape: any size)."""
    if (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != len(shape)
            or any(n is not None and n != m for n, m in zip(shape, t.shape))):
        raise ValueError(f"{name}: contiguous cuda int32 {['any' if n is None else n for n in shape]}, got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t


class PagePool:
    """The pages of a cache and the sequences that hold them, on the GPU.

    block_table: int32 [num_seqs][max_pages], row b the pages of sequence b;
    free_pages: int32 ring of as many places as there are pages in use; state:
    int32 [2 + num_seqs], the first free place of the ring, the number of free
    pages behind it, then the pages that each sequence holds.
    """

    def __init__(self, *, block_table: torch.Tensor, free_pages: torch.Tensor, state: torch.Tensor):
        self.block_table = _int32("block_table", block_table, None, None)
        self.free_pages = _int32("free_pages", free_pages, None)
        self.num_seqs = block_table.shape[0]
        self.state = _int32("state", state, 2 + self.num_seqs)
        if block_table.shape[1] < 1 or free_pages.shape[0] < 1:
            raise ValueError("block_table and free_pages must not be empty")

    @classmethod
    def of(cls, pages: torch.Tensor, *, num_seqs: int, max_pages: int) -> "PagePool":
        """A pool in which all of `pages` (cuda int32) are free and no
        sequence holds any."""
        state = torch.zeros(2 + num_seqs, dtype=torch.int32, device=pages.device)
        state[1] = pages.shape[0]
        return cls(block_table=torch.zeros(num_seqs, max_pages, dtype=torch.int32, device=pages.device),
                   free_pages=pages.clone(), state=state)


class StepTables:
    """What PagedAttention.plan fills for a step of up to num_tokens new tokens:
    q_offsets [num_seqs + 1], seq_lens [num_seqs], positions and slots
    [num_tokens], and with max_nodes (most new tokens of a tree) tree
    [num_tokens][words], else None; all int32. Allocated once, filled by every
    step's plan."""

    def __init__(self, *, num_seqs: int, num_tokens: int, max_nodes: int = 0, device="cuda"):
        words = -(-max_nodes // 32)
        self.num_seqs, self.num_tokens, self.max_nodes = num_seqs, num_tokens, max_nodes
        parts, at = [], 0
        for n in (num_seqs + 1, num_seqs, num_tokens, num_tokens, num_tokens * words):
            parts.append((at, n))
            at += -(-n // 4) * 4
        buf = torch.zeros(at, dtype=torch.int32, device=device)
        self.q_offsets, self.seq_lens, self.positions, self.slots, tree = (buf[i:i + n] for i, n in parts)
        self.tree = tree.view(num_tokens, words) if max_nodes else None
        self._plan = capi.moe_attn_plan_t(
            num_seqs=num_seqs, num_tokens=num_tokens, max_nodes=max_nodes, q_offsets=_ptr(self.q_offsets),
            seq_lens=_ptr(self.seq_lens), positions=_ptr(self.positions), slots=_ptr(self.slots), tree=_ptr(self.tree))


class Accepted:
    """What PagedAttention.accept fills: path [num_seqs][max_path], counts,
    next_tokens and context_lens [num_seqs], all int32."""

    def __init__(self, *, num_seqs: int, max_path: int, device="cuda", stream=None):
        self.num_seqs, self.max_path = num_seqs, max_path
        # (one buffer and four views of it take twice as long)
        self.path = _output((num_seqs, max_path), torch.int32, device, stream)
        self.counts, self.next_tokens, self.context_lens = (_output((num_seqs,), torch.int32, device, stream)
                                                            for _ in range(3))


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
                lse: Optional[torch.Tensor] = None, return_lse: bool = False, stream=None,
                tree: Optional[torch.Tensor] = None):
        """Attention of q [T][Hq][D] over the cache (moe_attn_forward, with
        tree moe_attn_forward_tree).

        Sequence b's queries are tokens q_offsets[b] .. q_offsets[b + 1]; its
        seq_lens[b] own keys are in the pages of block_table[b], after the
        prefix_len keys in prefix_pages that all sequences share. max_q_len
        and max_seq_len are upper bounds known on the host. tree: int32
        [T or more][words]; a token then sees, behind its sequence's earlier
        keys, the new tokens whose bits its row has (StepTables.tree), and
        causal is not looked at. Returns out, or (out, lse) when return_lse
        (lse fp32 [T][Hq])."""
        T, B = q.shape[0], seq_lens.shape[0]
        qp, qs = self._rows("q", q, T, self.num_q_heads)
        if out is None:
            out, op, os_ = self._new_rows(q, T, self.num_q_heads, stream)
        else:
            op, os_ = self._rows("out", out, T, self.num_q_heads)
        if lse is None:
            if return_lse:
                lse = _output((T, self.num_q_heads), torch.float32, q.device, stream)
        elif (lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous()
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
        if tree is None:
            st = self._lib.moe_attn_forward(self.handle, qp, qs, ctypes.byref(batch), op, os_, _ptr(lse),
                                            self._stream(stream, q))
        else:
            if (tree.dim() != 2 or tree.dtype != torch.int32 or not tree.is_cuda or tree.shape[0] < T
                    or tree.shape[1] * 32 < max_q_len or (tree.shape[1] > 1 and tree.stride(1) != 1)):
                raise ValueError(f"tree: cuda int32 [{T}][{-(-max_q_len // 32)}]")
            st = self._lib.moe_attn_forward_tree(self.handle, qp, qs, ctypes.byref(batch), tree.data_ptr(),
                                                 tree.stride(0) if T > 1 else tree.shape[1], op, os_, _ptr(lse),
                                                 self._stream(stream, q))
        if st:
            capi.check(st, "moe_attn_forward_tree" if tree is not None else "moe_attn_forward")
        return (out, lse) if return_lse else out

    def plan(self, pool: PagePool, context_lens: torch.Tensor, new_lens: torch.Tensor, tables: StepTables, *,
             parents: Optional[torch.Tensor] = None, prefix_len: int = 0, next_state: Optional[torch.Tensor] = None,
             stream=None) -> StepTables:
        """Fills a step's tables from lengths on the GPU (moe_attn_plan) and
        returns them.

        Sequence b holds context_lens[b] own keys and adds new_lens[b] tokens
        (-1: it ends and gives its pages back; neither may stand in the tables
        themselves, as their seq_lens do: copy those); the pages that they need come
        from the pool in order of sequences, and one whose need it cannot meet
        (nor any later one that needs some) gets seq_lens 0 and slots -1.
        parents (tables with max_nodes): int32, of each new token the new token
        of its sequence that it continues, -1: the context. prefix_len: the
        position of the first own key. The pool's state is updated in place, or
        left and the new one written to next_state."""
        B, T = tables.num_seqs, tables.num_tokens
        if pool.num_seqs != B:
            raise ValueError(f"the pool is of {pool.num_seqs} sequences, the tables of {B}")
        if (parents is not None) != (tables.max_nodes > 0):
            raise ValueError("parents go with tables that have max_nodes")
        c = tables._plan
        c.prefix_len = prefix_len
        c.context_lens = _int32("context_lens", context_lens, B).data_ptr()
        c.new_lens = _int32("new_lens", new_lens, B).data_ptr()
        c.parents = None if parents is None else self._ints("parents", parents, T)
        c.block_table, c.table_stride = pool.block_table.data_ptr(), pool.block_table.shape[1]
        c.free_pages, c.free_capacity = pool.free_pages.data_ptr(), pool.free_pages.shape[0]
        c.state = pool.state.data_ptr()
        c.state_out = c.state if next_state is None else _int32("next_state", next_state, 2 + B).data_ptr()
        st = self._lib.moe_attn_plan(self.handle, ctypes.byref(c), self._stream(stream, context_lens))
        if st:
            capi.check(st, "moe_attn_plan")
        return tables

    def accept(self, tokens: torch.Tensor, targets: torch.Tensor, parents: torch.Tensor, *, q_offsets: torch.Tensor,
               context_lens: torch.Tensor, max_path: Optional[int] = None, seq_lens: Optional[torch.Tensor] = None,
               out: Optional[Accepted] = None, stream=None) -> Accepted:
        """The branch of each sequence's tree that the model confirms
        (moe_attn_accept).

        tokens, parents: what was drafted, int32 [T]; targets: the model's
        choice after each of them. Node 0 of a sequence is accepted; from an
        accepted node the branch goes on to the first later one that continues
        it and holds its target, max_path nodes at most (needed without out).
        seq_lens: a sequence with fewer keys than tokens (not served by plan)
        accepts nothing. Returns the branches' nodes, their counts, the model's
        choice after each branch and context_lens + counts, in `out` if given
        (whose context_lens may be context_lens)."""
        T, B = tokens.shape[0], context_lens.shape[0]
        if out is None:
            if max_path is None or max_path < 1:
                raise ValueError("max_path (at least 1) or out is needed")
            out = Accepted(num_seqs=B, max_path=max_path, device=tokens.device, stream=stream)
        elif out.num_seqs != B or (max_path is not None and max_path != out.max_path):
            raise ValueError(f"out is of {out.num_seqs} sequences and {out.max_path} nodes")
        c = capi.moe_attn_accept_t(
            B, T, out.max_path, 0, self._ints("q_offsets", q_offsets, B + 1), self._ints("parents", parents, T),
            self._ints("tokens", tokens, T), self._ints("targets", targets, T),
            None if seq_lens is None else self._ints("seq_lens", seq_lens, B),
            self._ints("context_lens", context_lens, B), out.path.data_ptr(), out.counts.data_ptr(),
            out.next_tokens.data_ptr(), out.context_lens.data_ptr())
        st = self._lib.moe_attn_accept(self.handle, ctypes.byref(c), self._stream(stream, tokens))
        if st:
            capi.check(st, "moe_attn_accept")
        return out

    def keep(self, path: torch.Tensor, counts: torch.Tensor, *, q_offsets: torch.Tensor, seq_lens: torch.Tensor,
             max_seq_len: int, block_table: torch.Tensor, others=(), stream=None):
        """Moves the keys and values of the first counts[b] nodes of path
        [B][nodes] (int32, ascending) to the end of sequence b's context, in
        this object's cache and those of `others` (the other layers', of the
        same shape and strides) (moe_attn_keep)."""
        B = counts.shape[0]
        for name, t in (("path", path), ("block_table", block_table)):
            if (t.dim() != 2 or t.dtype != torch.int32 or not t.is_cuda or t.shape[0] != B or t.shape[1] < 1
                    or (t.shape[1] > 1 and t.stride(1) != 1)):
                raise ValueError(f"{name}: cuda int32 [{B}][1 or more]")
        if max_seq_len > block_table.shape[1] * self.cfg.page_size:
            raise ValueError("max_seq_len is beyond the block table")
        n, width, stride = 1 + len(others), path.shape[1], path.stride(0) if B > 1 else path.shape[1]
        args = ((capi._P * n)(self.handle, *[a.handle for a in others]), n, B, self._ints("q_offsets", q_offsets, B + 1),
                self._ints("seq_lens", seq_lens, B), max_seq_len, block_table.data_ptr(),
                block_table.stride(0) if B > 1 else block_table.shape[1], path.data_ptr(), stride)
        counts, on = self._ints("counts", counts, B), self._stream(stream, counts)
        st = (self._lib.moe_attn_keep(*args, counts, on) if stride == width
              else self._lib.moe_attn_keep_strided(*args, width, counts, on))
        if st:
            capi.check(st, "moe_attn_keep")

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
