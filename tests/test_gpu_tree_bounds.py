"""The operators around drafted trees at the edges of what their declarations
allow: lengths far out of range, rows of wider arrays."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import numpy as np  # noqa: E402

import tree_oracle as TO  # noqa: E402
from test_gpu_attention import F16, _cuda, build, caches  # noqa: E402,F401
from w4a16_routed_expert_gb300 import capi  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention, PagePool, StepTables  # noqa: E402


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,B,nodes", [(1 << 22, 1793, 0), (1 << 22, 2048, 64), (1 << 21, 4096, 0), ((1 << 22) - 1, 4096, 32)])
def test_plan_of_lengths_far_out_of_range_stays_in_its_outputs(T, B, nodes):
    """More tokens than room, in every sequence, as memory that was not filled
    may hold: recorded, none served, nothing stored beside the outputs."""
    kc, vc = caches(4, 16, 1, 8, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, k_cache=kc, v_cache=vc)
    words, guard = -(-nodes // 32), 1 << 16
    sizes = dict(q_offsets=B + 1, seq_lens=B, positions=T, slots=T, tree=T * words)
    sizes = {k: n for k, n in sizes.items() if n}
    buf = torch.full((sum(-(-n // 4) * 4 + guard for n in sizes.values()) + guard,), -5, dtype=torch.int32, device="cuda")
    at, out, mine = guard, {}, torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
    for name, n in sizes.items():
        out[name] = buf[at:at + n]
        mine[at:at + n] = True
        at += -(-n // 4) * 4 + guard
    ctx, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    parents = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    table, ring, state = ints([[0, 1]] * B), ints([0, 1, 2, 3]), ints([0, 4] + [0] * B)
    p = capi.moe_attn_plan_t(num_seqs=B, num_tokens=T, max_nodes=nodes, prefix_len=3, context_lens=ctx.data_ptr(), new_lens=new.data_ptr(),
                             parents=parents.data_ptr() if nodes else None, block_table=table.data_ptr(), table_stride=2, free_capacity=4,
                             free_pages=ring.data_ptr(), state=state.data_ptr(), state_out=state.data_ptr(),
                             **{k: t.data_ptr() for k, t in out.items()})
    s = torch.cuda.current_stream().cuda_stream
    assert capi.lib().moe_attn_plan(a.handle, ctypes.byref(p), s) == capi.MOE_OK
    with pytest.raises(capi.MoEError) as e:
        a.sync()
    assert e.value.status == capi.MOE_ERR_INVALID_ARG
    assert out["q_offsets"].tolist() == [min(b * (T + 1), T) for b in range(B + 1)]
    assert (out["seq_lens"] == 0).all() and (out["slots"] == -1).all()
    assert not nodes or (out["tree"] == 0).all()  # a tree of more than max_nodes
    assert (buf[~mine] == -5).all()
    assert state.tolist() == [0, 4] + [0] * B and ring.tolist() == [0, 1, 2, 3] and (table == ints([0, 1])).all()


@pytest.mark.parametrize("D,Hq,nodes,context", [(64, 2, [5, 13], [20, 200]), (128, 2, [31, 17], [400, 3]), (64, 4, [90, 40], [33, 500])])
def test_a_tree_in_the_last_columns_of_a_wider_array(D, Hq, nodes, context):
    """The last token's words are the array's last ones."""
    a, q, _, _, args = build(F16, Hq, 2, D, 16, "slot", nodes, [c + m for c, m in zip(context, nodes)], 0, seed=3)
    words = -(-max(nodes) // 32)
    bits = torch.cat([TO.pack(TO.branches(TO.random_tree(np.random.default_rng(4), m, "bushy")), words) for m in nodes]).cuda()
    wide = torch.full((bits.shape[0], words + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:] = bits
    want = a.forward(q.cuda(), tree=bits, **args)
    assert torch.equal(a.forward(q.cuda(), tree=wide[:, 3:], **args), want)
    a.sync()


def numbered(pages=8, page=16, heads=2, dim=64):
    kc, vc = caches(pages, page, heads, dim, F16, "slot", fill=0.0)
    kc.copy_(torch.arange(pages * page, device="cuda").view(pages, page, 1, 1).expand_as(kc))
    vc.copy_(kc)
    return PagedAttention(num_q_heads=heads, num_kv_heads=heads, head_dim=dim, max_seqs=2, k_cache=kc, v_cache=vc), kc, vc


@pytest.mark.parametrize("width,lo", [(4, 0), (7, 3), (64, 60), (130, 126)])
def test_keep_of_paths_in_columns_of_a_wider_array(width, lo):
    """Two sequences' paths of four nodes: the words beside them are no nodes, and
    a count that passes the four is out of range."""
    table, off, lens = ints([[1, 4], [3, 6]]), ints([0, 9, 18]), ints([20, 25])
    paths, counts = [[0, 2, 3, 8], [0, 4, 5, 7]], [4, 3]
    a, kc, vc = numbered()
    place = lambda b, key: table[b, key // 16].item() * 16 + key % 16  # noqa: E731
    want = list(range(8 * 16))
    for b, start in enumerate((11, 16)):
        for i in range(counts[b]):
            want[place(b, start + i)] = place(b, start + paths[b][i])
    wide = torch.arange(width, dtype=torch.int32, device="cuda").repeat(2, 1)  # (ascending: would pass for nodes)
    wide[:, lo:lo + 4] = ints(paths)
    args = dict(q_offsets=off, seq_lens=lens, max_seq_len=32, block_table=table)
    a.keep(wide[:, lo:lo + 4], ints(counts), **args)
    a.sync()
    assert kc[:, :, 1, 5].flatten().tolist() == want and torch.equal(kc, vc)
    a, kc, vc = numbered()
    a.keep(wide[:, lo:lo + 4], ints([5, 3]), **args)
    with pytest.raises(capi.MoEError) as e:
        a.sync()
    assert e.value.status == capi.MOE_ERR_INVALID_ARG
    got = kc[:, :, 1, 5].flatten().tolist()
    assert [got[place(0, k)] for k in range(20)] == [place(0, k) for k in range(20)]  # its sequence is left alone
    assert [got[place(1, 16 + i)] for i in range(3)] == [place(1, 16 + n) for n in (0, 4, 5)]


def test_keep_strided_refuses_rows_that_overlap():
    a, kc, _ = numbered()
    x = torch.zeros(64, dtype=torch.int32, device="cuda").data_ptr()
    one = (ctypes.c_void_p * 1)(a.handle)
    for stride, width in ((3, 4), (4, 0), (0, 0), (4, -1)):
        assert capi.lib().moe_attn_keep_strided(one, 1, 2, x, x, 16, x, 1, x, stride, width, x, None) == capi.MOE_ERR_INVALID_ARG
    assert capi.lib().moe_attn_keep_strided(one, 1, 0, x, x, 16, x, 1, x, 4, 3, x, None) == capi.MOE_OK


def test_plan_refuses_its_own_lengths():
    """The last step's seq_lens as lengths: refused in the same tables, right in
    others and as a copy."""
    kc, vc = caches(8, 16, 1, 8, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, k_cache=kc, v_cache=vc)
    pool = PagePool.of(torch.arange(8, dtype=torch.int32, device="cuda"), num_seqs=2, max_pages=4)
    t, u = (StepTables(num_seqs=2, num_tokens=20) for _ in range(2))
    new = ints([13, 2])
    a.plan(pool, ints([0, 0]), new, t)
    was = [x.clone() for x in (pool.state, t.seq_lens, t.slots)]
    for lengths in ((t.seq_lens, new), (new, t.seq_lens), (t.q_offsets[:2], new), (t.slots[18:], new)):
        with pytest.raises(capi.MoEError) as e:
            a.plan(pool, *lengths, t)
        assert e.value.status == capi.MOE_ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(was, (pool.state, t.seq_lens, t.slots)))
    held = pool.state.clone()
    a.plan(pool, t.seq_lens, new, u, next_state=torch.empty_like(held))
    want = [x.clone() for x in (u.q_offsets, u.seq_lens, u.positions, u.slots)]
    a.plan(pool, t.seq_lens.clone(), new, t)
    a.sync()
    assert all(torch.equal(x, y) for x, y in zip(want, (t.q_offsets, t.seq_lens, t.positions, t.slots)))
    assert t.seq_lens.tolist() == [26, 4] and t.positions[:15].tolist() == list(range(13, 26)) + [2, 3]
