"""The operators around drafted trees without a GPU: what their torch-tensor
wrapper refuses before the library is called, what it hands over, and the plain
definitions that the GPU tests compare with. Tensors and library are stand-ins."""
import ctypes
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import tree_oracle as TO
from test_attention_wrapper import B, D, HK, HQ, T, Tensor, ints
from w4a16_routed_expert_gb300 import attention, capi
from w4a16_routed_expert_gb300.attention import PagedAttention, PagePool

MOE_CALLS = ("moe_attn_forward", "moe_attn_forward_tree", "moe_attn_plan", "moe_attn_accept", "moe_attn_keep")


@pytest.fixture
def attn(monkeypatch):
    monkeypatch.setattr(attention, "_raw_stream", lambda index: 7)
    calls = []
    a = PagedAttention.__new__(PagedAttention)
    a.handle, a.dtype, a.num_q_heads, a.num_kv_heads, a.head_dim = 11, torch.float16, HQ, HK, D
    a.cfg = capi.moe_attn_config_t(page_size=16)
    a.calls = calls
    a.close = lambda: None
    a._lib = types.SimpleNamespace(**{n: (lambda *args, n=n: calls.append((n, args)) or 0) for n in MOE_CALLS})
    return a


def forward(a, **kw):
    return a.forward(Tensor(T, HQ, D), q_offsets=ints(B + 1), max_q_len=2, seq_lens=ints(B), max_seq_len=20, block_table=ints(B, 2),
                     out=Tensor(T, HQ, D), **kw)


def test_a_tree_picks_the_entry_point(attn):
    forward(attn)
    tree = Tensor(T + 2, 1, dtype=torch.int32)
    forward(attn, tree=tree)
    assert [n for n, _ in attn.calls] == ["moe_attn_forward", "moe_attn_forward_tree"]
    args = attn.calls[1][1]
    assert args[4:6] == (tree.data_ptr(), 1) and args[-1] == 7


@pytest.mark.parametrize("tree", [Tensor(T - 1, 1, dtype=torch.int32), Tensor(T, 0, dtype=torch.int32), Tensor(T, 1, dtype=torch.int64),
                                  Tensor(T, dtype=torch.int32), torch.zeros(T, 1, dtype=torch.int32)], ids=str)
def test_trees_that_are_refused(attn, tree):
    with pytest.raises(ValueError):
        forward(attn, tree=tree)
    assert not attn.calls


def pool(seqs=B, width=3, places=5, state=None):
    return PagePool(block_table=ints(seqs, width), free_pages=ints(places), state=ints(2 + seqs) if state is None else state)


def tables(seqs=B, tokens=T, nodes=0):
    return types.SimpleNamespace(num_seqs=seqs, num_tokens=tokens, max_nodes=nodes, _plan=capi.moe_attn_plan_t())


def test_pools_that_are_refused():
    for bad in (dict(width=0), dict(places=0), dict(state=ints(1 + B)), dict(state=ints(2 + B, 1)),
                dict(state=torch.zeros(2 + B, dtype=torch.int32)), dict(state=Tensor(2 + B, dtype=torch.int64))):
        with pytest.raises(ValueError):
            pool(**bad)


def test_plan_hands_over_the_pool_and_refuses_what_does_not_fit(attn):
    p, t = pool(), tables(nodes=2)
    after = ints(2 + B)
    assert attn.plan(p, ints(B), ints(B), t, parents=ints(T + 1), prefix_len=9, next_state=after) is t
    c = t._plan
    assert (c.prefix_len, c.table_stride, c.free_capacity) == (9, 3, 5)
    assert (c.state, c.state_out) == (p.state.data_ptr(), after.data_ptr())
    attn.plan(p, ints(B), ints(B), tables())
    assert len(attn.calls) == 2
    for bad in (dict(t=tables(seqs=B + 1)), dict(ctx=ints(B + 1)), dict(new=Tensor(B, dtype=torch.int64)), dict(parents=ints(T)),
                dict(t=tables(nodes=2)), dict(t=tables(nodes=2), parents=ints(T - 1)), dict(next_state=ints(B))):
        kw = dict(ctx=ints(B), new=ints(B), t=tables())
        kw.update(bad)
        with pytest.raises(ValueError):
            attn.plan(p, kw.pop("ctx"), kw.pop("new"), kw.pop("t"), **kw)
    assert len(attn.calls) == 2


def accepted(seqs=B, path=4):
    return types.SimpleNamespace(num_seqs=seqs, max_path=path, path=ints(seqs, path), counts=ints(seqs), next_tokens=ints(seqs),
                                 context_lens=ints(seqs))


def test_accept_refuses_what_does_not_fit(attn):
    out = accepted()
    ok = dict(q_offsets=ints(B + 1), context_lens=ints(B), out=out)
    assert attn.accept(ints(T), ints(T), ints(T), **ok) is out
    c = ctypes.cast(attn.calls[0][1][1], ctypes.POINTER(capi.moe_attn_accept_t)).contents
    assert (c.num_seqs, c.num_tokens, c.max_path, c.seq_lens) == (B, T, 4, None)
    for bad in (dict(out=None), dict(out=None, max_path=0), dict(out=accepted(seqs=B + 1)), dict(max_path=3), dict(q_offsets=ints(B)),
                dict(seq_lens=ints(B - 1))):
        with pytest.raises(ValueError):
            attn.accept(ints(T), ints(T), ints(T), **{**ok, **bad})
    for bad in ((ints(T), ints(T - 1), ints(T)), (ints(T), ints(T), Tensor(T, dtype=torch.int64)),
                (torch.zeros(T, dtype=torch.int32), ints(T), ints(T))):
        with pytest.raises(ValueError):
            attn.accept(*bad, **ok)
    assert len(attn.calls) == 1


def test_keep_refuses_what_does_not_fit(attn):
    ok = dict(q_offsets=ints(B + 1), seq_lens=ints(B), max_seq_len=32, block_table=ints(B, 2))
    attn.keep(ints(B, 3), ints(B), others=[attn], **ok)
    args = attn.calls[0][1]
    assert list(args[0]) == [11, 11] and args[1:3] == (2, B) and args[8:10] == (attn.calls[0][1][8], 3)
    for bad in (dict(max_seq_len=33), dict(block_table=ints(B + 1, 2)), dict(block_table=ints(B)), dict(seq_lens=ints(B - 1)),
                dict(q_offsets=Tensor(B + 1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            attn.keep(ints(B, 3), ints(B), **{**ok, **bad})
    for path in (ints(B), ints(B + 1, 3), ints(B, 0), Tensor(B, 3, dtype=torch.int64), torch.zeros(B, 3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            attn.keep(path, ints(B), **ok)
    assert len(attn.calls) == 1


# ------------------------------------------------------- the definitions

def test_branches_and_bits():
    rows = TO.branches([-1, 0, 0, 1, 3, 2])
    assert rows.astype(int).tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0], [1, 1, 0, 1, 1, 0],
                                         [1, 0, 1, 0, 0, 1]]
    assert TO.pack(rows, 1)[:, 0].tolist() == [1, 3, 5, 11, 27, 37]
    wide = np.zeros((1, 40), dtype=bool)
    wide[0, [31, 33]] = True
    assert TO.pack(wide, 2).tolist() == [[-2 ** 31, 2]]


def test_a_step_by_hand():
    """Pages of 4: two sequences grow, one ends, and the last finds no page."""
    table, ring = [[5, -1], [6, -1], [7, 8], [-1, -1]], [0, 1, 2, 3, -9, -9, -9, -9, -9]
    got = TO.plan(table, ring, [3, 1, 1, 1, 2, 0], [3, 1, 6, 0], [3, 2, -1, 2], 4, 8, prefix=100, parents=[-1, 0, 0, -1, 0, -1, 0], words=1)
    assert got["q_offsets"] == [0, 3, 5, 5, 7] and got["seq_lens"] == [6, 3, 0, 0]
    assert table[0] == [5, 3]  # the one free page, from the ring's place 3
    assert got["slots"] == [23, 12, 13, 25, 26, -1, -1, -1]
    assert got["positions"] == [103, 104, 104, 101, 102, 100, 101, 0]
    assert got["tree"] == [[1], [3], [5], [1], [3], [1], [3], [0]]
    assert ring[4:6] == [7, 8] and got["state"] == [4, 2, 2, 1, 0, 0]  # pages given back stand behind the free ones


def test_a_branch_by_hand():
    #            0 -> 1, 2 (the same token twice: the first counts), 1 -> 3, 2 -> 4
    parents, tokens, targets = [-1, 0, 0, 1, 2], [9, 5, 5, 7, 8], [5, 8, 8, 1, 2]
    assert TO.accept(tokens, targets, parents, 5) == [0, 1]
    targets[1] = 7
    assert TO.accept(tokens, targets, parents, 5) == [0, 1, 3] and TO.accept(tokens, targets, parents, 2) == [0, 1]
