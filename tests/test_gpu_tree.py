"""Operators around a step over trees of drafted tokens against their plain
definitions: the step's tables, attention over trees, the confirmed branch, its
keys and values; their refusals; and steps that use them together."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_oracle as TO  # noqa: E402
from test_gpu_attention import BF16, F16, _cuda, build, caches, within  # noqa: E402,F401
from w4a16_routed_expert_gb300 import capi  # noqa: E402
from w4a16_routed_expert_gb300.attention import Accepted, PagedAttention, PagePool, StepTables  # noqa: E402


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan

PLAN = {  # page, context, new tokens, trees, free pages, extra pages held, first place of the ring
    "one token": (16, [0], [1], None, 4, 0, 0),
    "a page's last slot": (16, [15, 16, 31], [1, 1, 2], "line", 5, 0, 3),
    "nothing new": (16, [5, 0], [0, 0], "bushy", 3, 0, 1),
    "pages that do not reach": (16, [10, 20, 30, 40], [8, 40, 3, 60], "bushy", 5, 0, 0),
    "none left": (32, [31, 32, 64], [1, 1, 1], "chain", 0, 0, 0),
    "one needs too many": (16, [0, 0, 7, 16], [100, 5, 3, 1], None, 4, 0, 2),
    "some end": (16, [100, 33, 64, 7], [-1, 5, -1, 8], "bushy", 6, 1, 0),
    "all end": (48, [100, 200], [-1, -1], "bushy", 0, 0, 5),
    "prompts": (16, [0] * 7, [1, 500, 33, 16, 17, 999, 64], None, 200, 0, 150),
    "trees of 32 and 33": (64, [3, 5, 1000], [32, 33, 31], "bushy", 20, 2, 0),
    "trees of hundreds": (16, [77, 0, 5], [300, 257, 64], "chain", 80, 0, 11),
    "lines of a thousand": (128, [5, 9], [1024, 1000], "line", 30, 0, 0),
    "the widest tree": (1024, [1], [1024], "bushy", 4, 0, 0),
    "as many sequences as go": (16, [(7 * i) % 100 for i in range(4096)], [(3 * i) % 5 - (i % 11 == 3) for i in range(4096)], "bushy", 3000, 0, 77),
    "three hundred lines": (16, [(13 * i) % 50 for i in range(300)], [(7 * i) % 40 for i in range(300)], None, 900, 1, 700),
}


def plan_case(name, seed=0):
    page, context, new, kind, free, surplus, first = PLAN[name]
    new = [max(n, -1) for n in new]
    rng = np.random.default_rng(seed + len(name))
    held = [-(-c // page) + surplus for c in context]
    width = max(max(held), max(-(-(c + max(n, 0)) // page) for c, n in zip(context, new)), 1) + 1
    pages = sum(held) + free + 2
    order = rng.permutation(pages).tolist()
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-7] * (width - h))
        at += h
    ring = [-9] * pages
    for i in range(free):
        ring[(first + i) % pages] = order[at + i]
    m = [max(n, 0) for n in new]
    parents = [p for n in m for p in TO.random_tree(rng, n, kind)] if kind else None
    return page, context, new, m, parents, pages, table, ring, [first, free] + held


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", PLAN)
def test_plan_matches_the_definition(name, in_place):
    page, context, new, m, parents, pages, table, ring, state = plan_case(name)
    kc, vc = caches(pages, page, 1, 8, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, k_cache=kc, v_cache=vc)
    B, room, nodes = len(new), sum(m) + 5, max(max(m), 1) if parents is not None else 0
    words = -(-nodes // 32)
    pool = PagePool(block_table=ints(table), free_pages=ints(ring), state=ints(state))
    tables = StepTables(num_seqs=B, num_tokens=room, max_nodes=nodes)
    for x in (tables.q_offsets, tables.seq_lens, tables.positions, tables.slots, tables.tree):
        if x is not None:
            x.fill_(-5)  # everything is written
    after = torch.full((2 + B,), -5, dtype=torch.int32, device="cuda")
    par = ints(parents + [0] * 5) if parents is not None else None
    args = dict(parents=par, prefix_len=300)
    for _ in range(1 if in_place else 3):  # with another next_state a step can be planned again
        got = a.plan(pool, ints(context), ints(new), tables, next_state=None if in_place else after, **args)
        assert got is tables
    a.sync()
    want = TO.plan(table, ring, state, context, new, page, room, 300, parents, words)
    assert tables.q_offsets.tolist() == want["q_offsets"]
    assert tables.seq_lens.tolist() == want["seq_lens"]
    assert tables.positions.tolist() == want["positions"]
    assert tables.slots.tolist() == want["slots"]
    assert pool.block_table.tolist() == table and pool.free_pages.tolist() == ring
    assert (pool.state if in_place else after).tolist() == want["state"]
    assert in_place or pool.state.tolist() == state
    if parents is not None:
        assert tables.tree.tolist() == want["tree"]


def test_steps_of_a_pool_take_and_give_back_every_page():
    """Sequences grow, end and start again for many steps, planned in place: at
    every step the pages held and those that are free are all pages, each once."""
    page, B, width, pages = 16, 37, 12, 230
    rng = np.random.default_rng(3)
    kc, vc = caches(pages, page, 1, 8, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, k_cache=kc, v_cache=vc)
    pool = PagePool.of(torch.randperm(pages, device="cuda").to(torch.int32), num_seqs=B, max_pages=width)
    tables = StepTables(num_seqs=B, num_tokens=B * 40)
    table, ring, state = pool.block_table.tolist(), pool.free_pages.tolist(), pool.state.tolist()
    context = [0] * B
    short = 0
    for _ in range(40):
        new = [-1 if rng.random() < 0.1 else int(rng.integers(0, 40)) for _ in range(B)]
        new = [n if n < 0 or c + n <= width * page else -1 for n, c in zip(new, context)]
        a.plan(pool, ints(context), ints(new), tables)
        a.sync()
        want = TO.plan(table, ring, state, context, new, page, B * 40)
        state = want["state"]
        assert pool.state.tolist() == state and pool.block_table.tolist() == table and pool.free_pages.tolist() == ring
        assert tables.slots.tolist() == want["slots"] and tables.seq_lens.tolist() == want["seq_lens"]
        short += sum(n > 0 and s == 0 for n, s in zip(new, want["seq_lens"]))
        context = [0 if n < 0 else s if s else c for n, s, c in zip(new, want["seq_lens"], context)]
        free = [ring[(state[0] + i) % pages] for i in range(state[1])]
        assert sorted(free + [p for b in range(B) for p in table[b][:state[2 + b]]]) == list(range(pages))
    assert short > 10


def test_plan_reports_what_is_out_of_range():
    page, pages = 16, 12
    kc, vc = caches(pages, page, 1, 8, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, k_cache=kc, v_cache=vc)

    def run(context=(3, 20), new=(2, 5), held=(1, 2), table=((0, -1, -1), (1, 2, -1)), ring=(3, 4, 5, 6, 7, 8, 9, 10), first=0, free=6,
            parents=(-1, 0, -1, 0, 1, 1, 3, 0), T=8, nodes=6):
        pool = PagePool(block_table=ints(table), free_pages=ints(ring), state=ints([first, free, *held]))
        tables = StepTables(num_seqs=2, num_tokens=T, max_nodes=nodes)
        a.plan(pool, ints(context), ints(new), tables, parents=ints(parents))
        torch.cuda.synchronize()
        return tables

    good = run()
    a.sync()
    assert good.slots.tolist() == [3, 4, 36, 37, 38, 39, 40, -1]
    for bad, where in ((dict(context=(-1, 20)), 0), (dict(new=(-2, 5)), 0), (dict(held=(4, 2)), 0), (dict(held=(-1, 2)), 0),
                       (dict(context=(3, 47)), 1), (dict(new=(2, 7)), 1), (dict(context=(3, 2 ** 31 - 1)), 1), (dict(context=(3, 2 ** 30)), 1),
                       (dict(table=((12, -1, -1), (1, 2, -1))), 0), (dict(table=((0, 0, 0), (1, -1, -1))), 1),
                       (dict(context=(3, 40), ring=(3, 99, 5, 6, 7, 8, 9, 10), held=(1, 1)), 1), (dict(new=(2, 6), T=7), 1)):
        t = run(**bad)
        with pytest.raises(capi.MoEError) as e:
            a.sync()
        assert e.value.status == capi.MOE_ERR_INVALID_ARG, bad
        off = t.q_offsets.tolist()
        assert all(-1 <= s < pages * page for s in t.slots.tolist()) and 0 <= min(off) and max(off) <= t.num_tokens, bad
        own, other = t.slots[off[where]:off[where + 1]].tolist(), t.slots[off[1 - where]:off[2 - where]].tolist()
        assert -1 in own or not own, bad
        assert -1 not in other, bad
    for bad in (dict(first=8), dict(first=-1), dict(free=9), dict(free=-1), dict(parents=(-1, 1, -1, 0, 1, 1, 3, 0)),
                dict(parents=(-1, 0, -1, -2, 1, 1, 3, 0)), dict(new=(-1, 5), held=(3, 2), free=8)):
        run(**bad)
        with pytest.raises(capi.MoEError):
            a.sync()
    run()
    a.sync()


# --------------------------------------------------------------- attention

TREE = {  # dtype, Hq, Hk, D, page, order, nodes, context, prefix, what a token sees
    "one token": (F16, 1, 1, 128, 16, "slot", [1], [0], 0, "bushy"),
    "eight of one": (F16, 16, 16, 128, 16, "slot", [8], [300], 0, "bushy"),
    "few rows": (BF16, 8, 8, 64, 16, "head", [5, 1, 13, 16], [0, 1, 63, 640], 0, "bushy"),
    "few rows, two tiles": (F16, 4, 2, 64, 32, "slot", [16, 9, 2], [48, 100, 5], 70, "chain"),
    "tiles end within trees": (F16, 2, 2, 128, 16, "slot", [15, 16, 14, 16], [50, 48, 64, 120], 0, "bushy"),
    "words end within tiles": (BF16, 4, 4, 128, 16, "slot", [31, 32, 33, 64, 65], [97, 31, 64, 1, 127], 0, "bushy"),
    "rows that see nothing": (F16, 8, 4, 64, 16, "slot", [9, 20, 3], [0, 0, 0], 0, "random"),
    "few rows that see nothing": (BF16, 4, 4, 128, 16, "head", [7, 16, 1], [0, 3, 0], 0, "random"),
    "no bits": (F16, 4, 2, 128, 32, "slot", [40, 3], [0, 17], 0, "none"),
    "no bits behind a prefix": (F16, 4, 4, 64, 16, "slot", [3, 60], [0, 0], 45, "none"),
    "all bits": (BF16, 8, 2, 128, 64, "head", [33, 70], [0, 130], 65, "all"),
    "later tokens only": (F16, 8, 1, 64, 16, "slot", [40, 17], [100, 0], 0, "later"),
    "grouped heads behind a prefix": (BF16, 32, 8, 64, 32, "head", [13, 1, 7, 10], [0, 300, 77, 700], 1000, "chain"),
    "heads of 96": (F16, 12, 4, 96, 48, "head", [120, 301], [17, 500], 300, "bushy"),
    "heads of 8": (F16, 3, 1, 8, 16, "slot", [5, 40], [9, 100], 70, "bushy"),
    "a long context": (BF16, 64, 8, 128, 64, "slot", [24, 48], [5000, 801], 0, "bushy"),
    "blocks of their own behind a prefix": (F16, 8, 1, 64, 16, "slot", [60, 40], [33, 0], 333, "bushy"),
    "trees of one row block and of two": (BF16, 16, 2, 128, 64, "slot", [64, 20, 40, 1, 33], [3000, 500, 0, 90, 128], 0, "bushy"),
    "the same behind a prefix of their own": (F16, 16, 2, 64, 32, "head", [64, 1, 2, 3, 5, 1, 1, 40], [700, 9, 0, 4000, 90, 130, 1, 64], 500, "chain"),
    "the same read with the prefix": (F16, 24, 2, 128, 16, "slot", [60, 22, 43], [100, 0, 1500], 140, "bushy"),
    "trees of three and four row blocks": (BF16, 8, 1, 96, 48, "head", [128, 97, 80], [0, 1000, 333], 0, "bushy"),
    "two streams of many rows": (BF16, 64, 8, 128, 64, "slot", [12, 16, 10, 9, 15, 16], [5000, 300, 0, 127, 200, 131], 0, "bushy"),
    "two streams of many rows of 64": (F16, 64, 4, 64, 16, "head", [7, 8, 5, 6, 8, 8, 8, 8, 8, 8], [300, 0, 127, 900, 131, 500, 64, 65, 1000, 2], 0, "chain"),
    "a tree wider than a tile": (F16, 4, 2, 64, 16, "slot", [300], [60], 0, "random"),
    "a tree of a thousand": (BF16, 2, 1, 64, 128, "slot", [1000], [130], 0, "bushy"),
    "many": (F16, 4, 4, 64, 16, "slot", [(3 * i) % 8 for i in range(130)], [(37 * i) % 150 for i in range(130)], 200, "bushy"),
    "fewer keys than tokens": (F16, 4, 4, 64, 16, "slot", [6, 20], [-4, -20], 40, "bushy"),
    "few with fewer keys than tokens": (F16, 2, 2, 128, 16, "slot", [6, 9], [-4, -9], 0, "random"),
    "whole groups of two row tiles": (BF16, 32, 8, 64, 32, "head", [20 + (7 * i) % 41 for i in range(20)], [(113 * i) % 700 for i in range(20)], 0, "bushy"),
    "whole groups behind a prefix in front of each": (F16, 32, 8, 128, 48, "head", [33 + (7 * i) % 30 for i in range(20)], [(57 * i) % 300 for i in range(20)], 300, "chain"),
    "whole groups, some of them empty": (F16, 16, 2, 128, 16, "slot", [20, 0, 33, 0, 7, 64], [0, 0, 5, 90, 400, 127], 0, "random"),
    "whole groups of one row tile": (BF16, 32, 4, 128, 16, "slot", [8, 5, 8, 3], [400, 900, 0, 333], 0, "bushy"),
    "whole groups of one row tile and few keys": (F16, 32, 4, 96, 16, "head", [8, 0, 5, 8, 3], [100, 0, 0, 200, 119], 0, "random"),
    "whole groups with fewer keys than tokens": (F16, 16, 4, 64, 16, "slot", [40, 30, 50], [-40, -7, 20], 200, "bushy"),
    "whole groups without keys": (F16, 8, 2, 128, 16, "slot", [40, 30], [-40, -30], 0, "random"),
    "two streams of 64 over many keys": (F16, 64, 4, 64, 16, "slot", [7, 8, 5], [3000, 2100, 900], 0, "chain"),
    "a prefix of many rows beside trees": (BF16, 32, 8, 64, 32, "head", [(3 * i) % 4 for i in range(30)], [(13 * i) % 100 for i in range(30)], 2000, "bushy"),
}


def seen_by(rng, kind, m):
    if kind == "random":
        return rng.random((m, m)) < np.maximum(rng.random((m, 1)) - 0.2, 0)
    if kind == "later":
        return np.triu(np.ones((m, m), dtype=bool), 1)
    if kind in ("none", "all"):
        return np.full((m, m), kind == "all")
    return TO.branches(TO.random_tree(rng, m, kind))


def tree_case(name):
    dtype, Hq, Hk, D, page, order, nodes, context, prefix, kind = TREE[name]
    rng = np.random.default_rng(len(name))
    own = [c + m for c, m in zip(context, nodes)]
    rows = [seen_by(rng, kind, m) for m in nodes]
    # a sequence with fewer keys than tokens: its first tokens have no key
    sees = [np.concatenate([np.ones((m, max(c, 0)), dtype=bool), r[:, max(-c, 0):]], 1) for m, c, r in zip(nodes, context, rows)]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, page, order, nodes, own, prefix, seed=len(name))
    words = -(-max(nodes) // 32)
    bits = torch.cat([TO.pack(r, words, rng) for r in rows]).cuda()
    return a, q, ks, vs, args, nodes, own, prefix, sees, bits, D


@pytest.mark.parametrize("name", TREE)
def test_forward_over_trees_matches_the_definition(name):
    a, q, ks, vs, args, nodes, own, prefix, sees, bits, D = tree_case(name)
    out, lse = a.forward(q.cuda(), tree=bits, return_lse=True, **args)
    a.sync()
    want, wlse, tol, ltol = TO.attend(q, ks, vs, nodes, prefix, own, D ** -0.5, sees)
    within(out, want, tol, "out")
    within(lse, wlse, ltol, "lse")
    # the same bits again, from rows of a wider array
    wide = torch.full((bits.shape[0] + 1, bits.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:-1, :bits.shape[1]] = bits
    assert torch.equal(a.forward(q.cuda(), tree=wide[:-1], **args), out)


@pytest.mark.parametrize("prefix", [0, 30])
@pytest.mark.parametrize("context", [20, 700])
@pytest.mark.parametrize("node", [3, 90])
def test_tokens_behind_the_last_sequence(node, context, prefix):
    """A padded step: the other rows are those of the step without padding."""
    nodes, own = [node, 2, 0], [context + node, 2, 40]
    a, q, _, _, args = build(F16, 4, 2, 64, 16, "slot", nodes, own, prefix, seed=8)
    bits = torch.cat([TO.pack(TO.branches(TO.random_tree(np.random.default_rng(1), m, "bushy")), 4) for m in nodes]).cuda()
    want, wlse = a.forward(q.cuda(), tree=bits, return_lse=True, **args)
    pad = 7
    wide = PagedAttention(num_q_heads=4, num_kv_heads=2, head_dim=64, max_tokens=node + 2 + pad, max_seqs=4, k_cache=a._keep[0],
                          v_cache=a._keep[1])
    qp = torch.cat([q.cuda(), torch.full((pad, 4, 64), float("nan"), dtype=F16, device="cuda")])
    bp = torch.cat([bits, torch.full((pad, 4), -1, dtype=torch.int32, device="cuda")])
    args["max_q_len"] = node + pad
    if prefix:  # (the number of tokens says how the prefix is read)
        args["max_q_len"] = max(args["max_q_len"], (node + 2 + pad + 2) // 3)
    out, lse = torch.full_like(qp, 9.0), torch.full((node + 2 + pad, 4), 9.0, device="cuda")
    wide.forward(qp, tree=bp, out=out, lse=lse, **args)
    wide.sync()
    tol = 2.0 ** -9 * want.double().abs().cpu() + 2.0 ** -9  # (both round the weights and the result: 2^-11 each of values to 4)
    within(out[:node + 2], want.double().cpu(), tol, "out")
    assert ((lse[:node + 2] - wlse).abs() < 1e-4).all()
    if not prefix:  # (a prefix is everybody's)
        assert (out[node + 2:] == 0).all() and (lse[node + 2:] == -float("inf")).all()


@pytest.mark.parametrize("name", ["few rows", "words end within tiles", "grouped heads behind a prefix", "heads of 96"])
def test_a_line_is_a_tree(name):
    """Every token continues the one before: what causal attention gives."""
    dtype, Hq, Hk, D, page, order, nodes, context, prefix, _ = TREE[name]
    own = [c + m for c, m in zip(context, nodes)]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, page, order, nodes, own, prefix, seed=1)
    words = -(-max(nodes) // 32)
    bits = torch.cat([TO.pack(np.tril(np.ones((m, m), dtype=bool)), words) for m in nodes]).cuda()
    got, want = a.forward(q.cuda(), tree=bits, **args), a.forward(q.cuda(), causal=True, **args)
    a.sync()
    # both are within the bound of the same result
    sees = [np.arange(n)[None] <= n - m + np.arange(m)[:, None] for m, n in zip(nodes, own)]
    tol = TO.attend(q, ks, vs, nodes, prefix, own, D ** -0.5, sees)[2]
    within(got, want.double().cpu(), 2 * tol, name)


@pytest.mark.parametrize("D,g", [(64, 1), (128, 1), (64, 8), (128, 4)])
def test_extreme_logits_over_trees(D, g):
    """Masked keys hold the largest logits: they count nothing, whatever tile
    they are in, and rows whose first tiles are all masked start later."""
    nodes, context = [200, 13], [70, 0]
    own = [c + m for c, m in zip(context, nodes)]

    def keys(Hk, n, D, gen):
        return torch.randn(Hk, n, D, generator=gen) * 60

    a, q, ks, vs, args = build(F16, 2 * g, 2, D, 16, "slot", nodes, own, 0, seed=9, sharp=200.0, keys=keys)
    # each token sees itself and the token before alone (and the context)
    rows = [np.eye(m, dtype=bool) | np.eye(m, k=-1, dtype=bool) for m in nodes]
    sees = [np.concatenate([np.ones((m, c), dtype=bool), r], 1) for m, c, r in zip(nodes, context, rows)]
    out, lse = a.forward(q.cuda(), tree=torch.cat([TO.pack(r, 7) for r in rows]).cuda(), return_lse=True, **args)
    a.sync()
    want, wlse, tol, ltol = TO.attend(q, ks, vs, nodes, 0, own, D ** -0.5, sees)
    within(lse, wlse, ltol, "lse")
    within(out, want, tol, "out")


def test_values_that_are_not_finite_stay_in_their_sequence():
    nodes, context = [40, 20], [100, 30]
    own = [c + m for c, m in zip(context, nodes)]
    a, q, ks, vs, args = build(F16, 4, 4, 64, 16, "slot", nodes, own, 0, seed=2)
    bits = torch.cat([TO.pack(TO.branches(TO.random_tree(np.random.default_rng(1), m, "bushy")), 2) for m in nodes]).cuda()
    clean = a.forward(q.cuda(), tree=bits, **args)
    page = int(args["block_table"][0, 0])
    a._keep[1][page, 3] = float("nan")
    out = a.forward(q.cuda(), tree=bits, **args)
    a.sync()
    assert torch.isnan(out[:40]).all() and torch.equal(out[40:], clean[40:])


# ------------------------------------------------------------------ accept

ACCEPT = {  # nodes, kind, vocabulary, longest branch
    "one node each": ([1, 1, 1], "bushy", 5, 3),
    "small": ([3, 8, 5, 0, 7], "bushy", 3, 8),
    "the same token twice": ([30, 32, 33], "bushy", 2, 40),
    "cut": ([64, 20, 9], "chain", 2, 4),
    "a path of one": ([64, 20, 9], "chain", 2, 1),
    "lines": ([200, 129, 128, 127], "line", 1, 300),
    "a thousand nodes": ([1000, 0, 777], "chain", 2, 1000),
    "many": ([(7 * i) % 70 for i in range(999)], "chain", 3, 33),
}


@pytest.mark.parametrize("name", ACCEPT)
def test_accept_matches_the_definition(name):
    nodes, kind, vocab, P = ACCEPT[name]
    rng = np.random.default_rng(len(name))
    trees = [TO.random_tree(rng, m, kind) for m in nodes]
    tok = [rng.integers(0, vocab, m).tolist() for m in nodes]
    tgt = [rng.integers(0, vocab, m).tolist() for m in nodes]
    context = rng.integers(0, 1000, len(nodes)).tolist()
    lens = [c + m for c, m in zip(context, nodes)]
    if len(nodes) > 2:
        lens[1] = max(nodes[1] - 1, 0)  # not served
    flat = lambda x: ints(sum(x, []))  # noqa: E731
    off = ints(np.concatenate([[0], np.cumsum(nodes)]).tolist())
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8)
    ctx = ints(context)
    want = [TO.accept(t, g, p, P) if m and n >= m else [] for t, g, p, m, n in zip(tok, tgt, trees, nodes, lens)]
    got = a.accept(flat(tok), flat(tgt), flat(trees), q_offsets=off, context_lens=ctx, seq_lens=ints(lens), max_path=P)
    a.sync()
    assert got.path.tolist() == [w + [-1] * (P - len(w)) for w in want]
    assert got.counts.tolist() == [len(w) for w in want]
    assert got.next_tokens.tolist() == [g[w[-1]] if w else -1 for g, w in zip(tgt, want)]
    assert got.context_lens.tolist() == [c + len(w) for c, w in zip(context, want)] and ctx.tolist() == context
    # into the same buffers, without seq_lens, the lengths in place
    got.context_lens.copy_(ctx)
    again = a.accept(flat(tok), flat(tgt), flat(trees), q_offsets=off, context_lens=got.context_lens, out=got)
    want = [TO.accept(t, g, p, P) if m else [] for t, g, p, m in zip(tok, tgt, trees, nodes)]
    assert again is got and got.counts.tolist() == [len(w) for w in want]
    assert got.context_lens.tolist() == [c + len(w) for c, w in zip(context, want)]
    assert max(len(w) for w in want) > 1 or P == 1 or max(nodes) < 3


def test_accept_reports_offsets_out_of_order():
    a = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8)
    x = ints([1, 1, 1, 1])
    for off in ([0, 5], [2, 1], [-1, 3]):
        a.accept(x, x, ints([-1, 0, 1, 2]), q_offsets=ints(off), context_lens=ints([0]), max_path=4)
        with pytest.raises(capi.MoEError):
            a.sync()
    assert a.accept(x, x, ints([-1, 0, 1, 2]), q_offsets=ints([0, 4]), context_lens=ints([0]), max_path=4).counts.tolist() == [4]
    a.sync()


# -------------------------------------------------------------------- keep

KEEP = {  # dtype, layers, Hk, D, page, order, nodes, context, paths
    "one": (F16, 1, 1, 8, 16, "slot", [4], [14], [[0, 2, 3]]),
    "nothing moves": (BF16, 2, 4, 64, 16, "head", [5, 3], [0, 7], [[0, 1, 2], []]),
    "some": (BF16, 3, 8, 128, 32, "head", [8, 1, 30, 6], [31, 0, 100, 15], [[0, 5], [0], [0, 3, 4, 9, 29], []]),
    "long branches": (F16, 2, 2, 96, 48, "slot", [300, 200], [5, 60], [list(range(0, 300, 2)), [0] + list(range(60, 200))]),
    "many layers": (F16, 70, 2, 64, 16, "slot", [9, 20], [3, 30], [[0, 4, 8], [0, 1, 19]]),
    "without the first": (F16, 1, 3, 72, 16, "slot", [9], [20], [[3, 4, 8]]),
    "many sequences": (BF16, 2, 16, 128, 16, "slot", [10] * 100, [(7 * i) % 40 for i in range(100)], [[0, 2, 3, 7, 9][:1 + i % 5] for i in range(100)]),
}


@pytest.mark.parametrize("name", KEEP)
def test_keep_moves_the_branch(name):
    dtype, layers, Hk, D, page, order, nodes, context, paths = KEEP[name]
    B, lens = len(nodes), [c + m for c, m in zip(context, nodes)]
    n_pages = [-(-n // page) for n in lens]
    count = sum(n_pages) + 2
    pages = torch.randperm(count, generator=torch.Generator().manual_seed(1)).tolist()
    table, at = [], 0
    for n in n_pages:
        table.append(pages[at:at + n] + [-1] * (max(n_pages) - n))
        at += n
    kv = [caches(count, page, Hk, D, dtype, order, fill=0.0) for _ in range(layers)]
    for k, v in kv:
        k.copy_(torch.randn(k.shape, device="cuda"))
        v.copy_(torch.randn(v.shape, device="cuda"))
    attns = [PagedAttention(num_q_heads=Hk, num_kv_heads=Hk, head_dim=D, dtype=dtype, max_seqs=B, k_cache=k, v_cache=v) for k, v in kv]
    want = [[c.clone() for c in layer] for layer in kv]
    for b, path in enumerate(paths):
        at = lambda node: (table[b][(context[b] + node) // page], (context[b] + node) % page)  # noqa: E731
        for layer, old in zip(want, kv):
            for c, o in zip(layer, old):
                for i, p in enumerate(path):
                    c[at(i)] = o[at(p)]
    P = max(len(p) for p in paths)
    attns[0].keep(ints([p + [-1] * (P - len(p)) for p in paths]), ints([len(p) for p in paths]), max_seq_len=max(lens),
                  q_offsets=ints(np.concatenate([[0], np.cumsum(nodes)]).tolist()), seq_lens=ints(lens), block_table=ints(table),
                  others=attns[1:])
    attns[0].sync()
    for layer, w in zip(kv, want):
        assert torch.equal(layer[0], w[0]) and torch.equal(layer[1], w[1])


def test_keep_of_keys_that_are_the_values():
    """One tensor as both caches is moved once."""
    c = torch.arange(4 * 16, device="cuda").half().view(4, 16, 1, 1).expand(4, 16, 2, 64).contiguous()
    a = PagedAttention(num_q_heads=2, num_kv_heads=2, head_dim=64, k_cache=c, v_cache=c)
    a.keep(ints([[0, 2, 3, 7]]), ints([4]), q_offsets=ints([0, 9]), seq_lens=ints([20]), max_seq_len=32, block_table=ints([[1, 3]]))
    a.sync()
    was = list(range(64))
    want = list(was)
    at = lambda j: (1, 3)[j // 16] * 16 + j % 16  # noqa: E731
    for i, p in enumerate([0, 2, 3, 7]):
        want[at(11 + i)] = was[at(11 + p)]
    assert c[:, :, 1, 5].flatten().tolist() == want


def test_keep_reports_what_is_out_of_range():
    kc, vc = caches(6, 16, 2, 64, F16, "slot")
    kc.copy_(torch.arange(6 * 16, device="cuda").view(6, 16, 1, 1).expand_as(kc))
    vc.copy_(kc)
    first = kc.clone()
    a = PagedAttention(num_q_heads=2, num_kv_heads=2, head_dim=64, max_seqs=2, k_cache=kc, v_cache=vc)

    def run(path=((0, 2, 3),), counts=(3,), off=(0, 5), lens=(20,), table=((1, 4),)):
        kc.copy_(first), vc.copy_(first)
        a.keep(ints(path), ints(counts), q_offsets=ints(off), seq_lens=ints(lens), max_seq_len=32, block_table=ints(table))
        torch.cuda.synchronize()
        return kc[:, :, 0, 0].flatten().tolist()

    was = first[:, :, 0, 0].flatten().tolist()
    good = list(was)
    good[64], good[65] = was[65], was[66]  # keys 15 (of page 1), 16, 17: nodes 0, 2, 3
    assert run() == good
    a.sync()
    for bad in (dict(counts=(4,)), dict(counts=(-1,)), dict(off=(0, 21)), dict(off=(5, 0)), dict(lens=(33,)), dict(lens=(-1,)),
                dict(path=((0, 0, 3),)), dict(path=((0, 5, 6),)), dict(path=((-1, 2, 3),)), dict(table=((1, 6),)), dict(table=((1, -1),))):
        got = run(**bad)
        with pytest.raises(capi.MoEError) as e:
            a.sync()
        assert e.value.status == capi.MOE_ERR_INVALID_ARG, bad
        assert got == was, bad
    part = run(path=((0, 2, 2),))  # what stands before the fault is moved
    with pytest.raises(capi.MoEError):
        a.sync()
    assert part[64] == was[65] and part[65:] == was[65:] and part[:64] == was[:64]


# ---------------------------------------------------------------- refusals

def test_refusals():
    lib, INV = capi.lib(), capi.MOE_ERR_INVALID_ARG
    kc, vc = caches(4, 16, 2, 64, F16, "slot", fill=0.0)
    mk = lambda **kw: PagedAttention(num_q_heads=4, num_kv_heads=2, head_dim=64, max_tokens=4, max_seqs=2, **kw)  # noqa: E731
    a, bare = mk(k_cache=kc, v_cache=vc), mk()
    p = torch.zeros(4096, device="cuda").data_ptr()
    batch = dict(num_tokens=2, num_seqs=2, q_offsets=p, max_q_len=1, seq_lens=p, max_seq_len=16, block_table=p, table_stride=1,
                 prefix_len=0, prefix_pages=None, causal=7)

    def tree(h=a.handle, bits=p, stride=1, **kw):
        return lib.moe_attn_forward_tree(h, p, 256, ctypes.byref(capi.moe_attn_batch_t(**{**batch, **kw})), bits, stride, p + 8192, 256,
                                         None, None)

    for bad in (dict(h=None), dict(h=bare.handle), dict(bits=None), dict(bits=p + 2), dict(stride=0), dict(stride=-1), dict(stride=1 << 30),
                dict(num_tokens=5), dict(max_q_len=3), dict(max_seq_len=17)):
        assert tree(**bad) == INV, bad
        assert capi.last_error()

    def plan(h=a.handle, **kw):
        d = dict(num_seqs=2, num_tokens=4, max_nodes=2, prefix_len=0, context_lens=p, new_lens=p, parents=p, block_table=p, table_stride=1,
                 free_capacity=4, free_pages=p, state=p, state_out=p, q_offsets=p, seq_lens=p, positions=p, slots=p, tree=p)
        d.update(kw)
        return lib.moe_attn_plan(h, ctypes.byref(capi.moe_attn_plan_t(**d)), None)

    for bad in (dict(h=None), dict(h=bare.handle), dict(num_seqs=-1), dict(num_seqs=4097), dict(num_tokens=-1), dict(num_tokens=(1 << 22) + 1),
                dict(max_nodes=1025), dict(max_nodes=-1), dict(prefix_len=-1), dict(table_stride=0), dict(free_capacity=0),
                dict(free_capacity=(1 << 30) + 1), *[{k: None} for k in ("context_lens", "new_lens", "parents", "block_table", "free_pages",
                                                                       "state", "state_out", "q_offsets", "seq_lens", "positions",
                                                                       "slots", "tree")]):
        assert plan(**bad) == INV, bad
    assert lib.moe_attn_plan(a.handle, None, None) == INV

    def accept(h=a.handle, **kw):
        d = dict(num_seqs=2, num_tokens=4, max_path=2, q_offsets=p, parents=p, tokens=p, targets=p, seq_lens=None, context_lens=p, path=p,
                 counts=p, next_tokens=p, context_out=p)
        d.update(kw)
        return lib.moe_attn_accept(h, ctypes.byref(capi.moe_attn_accept_t(**d)), None)

    for bad in (dict(h=None), dict(num_seqs=-1), dict(num_tokens=-1), dict(max_path=0), dict(reserved=1), dict(num_seqs=(1 << 20) + 1),
                *[{k: None} for k in ("q_offsets", "parents", "tokens", "targets", "context_lens", "path", "counts", "next_tokens",
                                      "context_out")]):
        assert accept(**bad) == INV, bad
    assert accept(num_seqs=0) == capi.MOE_OK

    other = mk(k_cache=kc, v_cache=vc)  # the same cache
    kc2, vc2 = caches(4, 16, 2, 64, F16, "head", fill=0.0)
    strides = mk(k_cache=kc2, v_cache=vc2)

    def keep(hs=(a.handle,), n=None, num_seqs=2, off=p, lens=p, max_len=16, table=p, ts=1, path=p, ps=2, counts=p):
        return lib.moe_attn_keep((ctypes.c_void_p * len(hs))(*hs), len(hs) if n is None else n, num_seqs, off, lens, max_len, table, ts,
                                 path, ps, counts, None)

    for bad in (dict(hs=(None,)), dict(hs=(bare.handle,)), dict(n=0), dict(n=1025), dict(hs=(a.handle, other.handle)), dict(hs=(a.handle, a.handle)),
                dict(hs=(a.handle, strides.handle)), dict(num_seqs=-1), dict(num_seqs=4097), dict(max_len=17), dict(max_len=-1), dict(ts=0),
                dict(ps=0), dict(off=None), dict(lens=None), dict(table=None), dict(path=None), dict(counts=None)):
        assert keep(**bad) == INV, bad
    assert lib.moe_attn_keep(None, 1, 2, p, p, 16, p, 1, p, 2, p, None) == INV
    assert keep(num_seqs=0) == capi.MOE_OK
    a.sync()


def test_no_sequences_and_no_tokens_is_no_work():
    kc, vc = caches(2, 16, 2, 64, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=2, num_kv_heads=2, head_dim=64, k_cache=kc, v_cache=vc)
    none = ints([])
    pool = PagePool(block_table=torch.zeros(0, 1, dtype=torch.int32, device="cuda"), free_pages=ints([1]), state=ints([0, 1]))
    t = a.plan(pool, none, none, StepTables(num_seqs=0, num_tokens=0))
    assert t.q_offsets.tolist() == [0] and pool.state.tolist() == [0, 1]
    assert a.accept(none, none, none, q_offsets=ints([0]), context_lens=none, max_path=3).counts.tolist() == []
    got = a.accept(none, none, none, q_offsets=ints([0, 0]), context_lens=ints([7]), max_path=3)
    assert got.counts.tolist() == [0] and got.path.tolist() == [[-1] * 3] and got.context_lens.tolist() == [7]
    e = torch.empty(0, 2, 64, device="cuda", dtype=F16)
    assert a.forward(e, q_offsets=ints([0, 0]), max_q_len=1, seq_lens=ints([0]), max_seq_len=0,
                     tree=torch.zeros(0, 1, dtype=torch.int32, device="cuda")).shape == (0, 2, 64)
    a.sync()
