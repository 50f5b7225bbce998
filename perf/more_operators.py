"""Cases of the operators around a decode step that checks trees of drafted tokens.

The lengths of the sequences stand on the GPU, because how many drafted tokens were right is known
there first. Four operators, in the order a step runs them:

* ``plan``    from the sequences' lengths, the trees' parents and a ring of free pages: offsets,
  positions, cache slots, new entries of the block table, and which tokens of its tree each token sees;
* ``attend``  attention of a ragged batch over the paged cache, where a drafted token sees the shared
  prefix, its sequence's context and its own branch of the tree;
* ``accept``  the branch that the model's own choices confirm;
* ``keep``    that branch's keys and values moved behind the context, in the caches of all layers.

``own`` selects the framework's calls; without it ``run`` computes the same from elementary torch
operations, in 32 bits (whole numbers in 64).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # four conversations, trees of a few tokens: launch latency
        dict(name="plan-small-4", op="plan", seqs=4, ctx_min=1, ctx_max=900, new_min=3, new_max=8, page=16, tree="bushy",
             prefix=0, end_every=0, surplus=1, short=False),
        # a batch in which some conversations end and the pages do not reach for all
        dict(name="plan-trees-50", op="plan", seqs=50, ctx_min=0, ctx_max=6000, new_min=1, new_max=63, page=32, tree="bushy",
             prefix=501, end_every=7, surplus=0, short=True),
        # prompts of 512 new conversations: whole columns of the block table, no trees
        dict(name="plan-prompts-512", op="plan", seqs=512, ctx_min=0, ctx_max=0, new_min=1, new_max=1999, page=16, tree="none",
             prefix=0, end_every=0, surplus=0, short=False),
        # one conversation and a tree of eight tokens: latency
        dict(name="attend-one-8", op="attend", dtype="f16", seqs=1, new_min=8, new_max=8, tree="bushy", q_heads=16, kv_heads=16,
             dim=128, prefix=0, ctx_min=300, ctx_max=300, page=16, order="slot"),
        # a decode batch of 16 behind a common system text, up to 31 drafted tokens each
        dict(name="attend-batch-16", op="attend", dtype="f16", seqs=16, new_min=5, new_max=31, tree="bushy", q_heads=16, kv_heads=16,
             dim=128, prefix=1000, ctx_min=0, ctx_max=2600, page=16, order="slot"),
        # 50 sequences with two or three branches of a few tokens, small grouped heads, pages kept head by head
        dict(name="attend-branches-50", op="attend", dtype="bf16", seqs=50, new_min=1, new_max=13, tree="chain", q_heads=32, kv_heads=8,
             dim=64, prefix=4099, ctx_min=0, ctx_max=700, page=32, order="head"),
        # long conversations with large trees, nothing shared: the cache's bytes and the products
        dict(name="attend-long-8", op="attend", dtype="bf16", seqs=8, new_min=24, new_max=64, tree="bushy", q_heads=64, kv_heads=8,
             dim=128, prefix=0, ctx_min=1000, ctx_max=30000, page=64, order="slot"),
        # few sequences, trees of hundreds: the masked tiles count
        dict(name="attend-wide-3", op="attend", dtype="f16", seqs=3, new_min=301, new_max=500, tree="bushy", q_heads=12, kv_heads=4,
             dim=96, prefix=300, ctx_min=17, ctx_max=800, page=48, order="head"),
        # four trees of a few tokens: launch latency
        dict(name="accept-small-4", op="accept", seqs=4, new_min=3, new_max=8, tree="bushy", vocab=1000, path=5),
        # many sequences, large trees
        dict(name="accept-batch-500", op="accept", seqs=500, new_min=1, new_max=200, tree="chain", vocab=50000, path=24),
        # one layer, a few sequences: launch latency
        dict(name="keep-one-4", op="keep", dtype="f16", layers=1, seqs=4, new_min=3, new_max=8, path=5, kv_heads=8, dim=128,
             ctx_min=0, ctx_max=200, page=16, order="slot"),
        # all layers of a 16-layer model after a step of 64 sequences
        dict(name="keep-layers-64", op="keep", dtype="bf16", layers=16, seqs=64, new_min=9, new_max=40, path=9, kv_heads=16, dim=128,
             ctx_min=0, ctx_max=500, page=16, order="slot"),
    ]


def _log(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["plan", "attend", "attend", "attend", "accept", "keep"])
        tree = rng.choice(["bushy", "chain"])
        if op == "plan":
            c = dict(op=op, seqs=_log(rng, 1, 512), page=rng.choice([16, 32, 48, 64, 128]), prefix=rng.choice([0, _log(rng, 1, 5000)]),
                     end_every=rng.choice([0, 0, 2, 5, 9]), surplus=rng.choice([0, 1, 3]), short=rng.random() < 0.4)
            if rng.random() < 0.3:
                c.update(tree="none", ctx_min=0, ctx_max=_log(rng, 1, 3000), new_min=1, new_max=_log(rng, 1, 1999))
            else:
                hi = _log(rng, 1, 200)
                c.update(tree=tree, ctx_min=0, ctx_max=_log(rng, 1, 20000), new_min=rng.choice([0, 1, hi]), new_max=hi)
        elif op == "attend":
            heads = rng.choice([(16, 16), (32, 8), (32, 4), (64, 8), (8, 1), (12, 4), (40, 40)])
            hi = rng.choice([_log(rng, 1, 16), _log(rng, 8, 64), _log(rng, 40, 500)])
            ctx = _log(rng, 1, 30000)
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), seqs=_log(rng, 1, 100), new_min=rng.choice([1, hi]), new_max=hi,
                     tree=rng.choice(["bushy", "chain", "random"]), q_heads=heads[0], kv_heads=heads[1], dim=rng.choice([64, 96, 128]),
                     prefix=rng.choice([0, 0, _log(rng, 1, 20000)]), ctx_min=rng.choice([0, ctx // 2, ctx]), ctx_max=ctx,
                     page=rng.choice([16, 32, 48, 64, 128]), order=rng.choice(["slot", "head"]))
            # what the plain form holds in 32 bits at once has to stay small beside the card's memory
            rows = c["seqs"] * hi * c["q_heads"]
            if rows * (c["prefix"] + ctx + hi) > 1.2e9 or c["seqs"] * (ctx + hi) * c["kv_heads"] * c["dim"] > 1.2e9:
                continue
        elif op == "accept":
            hi = _log(rng, 1, 200)
            c = dict(op=op, seqs=_log(rng, 1, 500), new_min=rng.choice([0, 1, hi]), new_max=hi, tree=tree,
                     vocab=rng.choice([3, 1000, 50000]), path=rng.choice([min(4, hi), hi]))
        else:
            hi = _log(rng, 1, 64)
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), layers=_log(rng, 1, 20), seqs=_log(rng, 1, 64), new_min=rng.choice([0, 1, hi]),
                     new_max=hi, path=rng.choice([min(5, hi), hi]), kv_heads=rng.choice([1, 4, 8, 16, 40]), dim=rng.choice([64, 96, 128]),
                     ctx_min=0, ctx_max=_log(rng, 1, 500), page=rng.choice([16, 32, 48, 64, 128]), order=rng.choice(["slot", "head"]))
            if c["layers"] * c["seqs"] * (c["ctx_max"] + hi) * c["kv_heads"] * c["dim"] > 1.2e9:
                continue
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------ shapes

def _spread(n, lo, hi, start):
    """n whole numbers from lo to hi, odd ones among them, the same for the same case."""
    return [lo + int((hi - lo + 1) * ((start + 0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _lengths(case):
    """(new tokens, context) of each sequence."""
    B = case["seqs"]
    return _spread(B, case["new_min"], case["new_max"], 0.999), _spread(B, case.get("ctx_min", 0), case.get("ctx_max", 0), 0.3 if B > 1 else 0.999)


def _counts(case):
    """Accepted tokens of each sequence (keep)."""
    return [min(n, m) for n, m in zip(_spread(case["seqs"], 1, case["path"], 0.7), _lengths(case)[0])]


def _plan_lengths(case):
    """(new tokens or -1, context, pages held) of each sequence and the free pages of the ring."""
    new, ctx = _lengths(case)
    p = case["page"]
    held = [-(-c // p) + case["surplus"] for c in ctx]
    need = []
    for b in range(len(new)):
        if case["end_every"] and b % case["end_every"] == case["end_every"] - 1:
            new[b] = -1
        need.append(max(0, -(-(ctx[b] + new[b]) // p) - held[b]) if new[b] >= 0 else 0)
    total = sum(need)
    return new, ctx, held, need, (total * 3 // 5 if case["short"] else total + 5)


def _words(case):
    return 0 if case["tree"] == "none" else -(-case["new_max"] // 32)


def work(case):
    new, ctx = _lengths(case)
    if case["op"] == "plan":
        new, ctx, held, need, free = _plan_lengths(case)
        t, B = sum(max(n, 0) for n in new), len(new)
        given, back, cum = 0, sum(h for h, n in zip(held, new) if n < 0), 0
        for n in need:
            cum += n
            given = cum if cum <= free else given
        parents = 4 * t if case["tree"] != "none" else 0
        # lengths, state and parents read; offsets, lengths, state, positions, slots and masks written; pages moved
        return {"bytes": 4 * (3 * B + 2) + parents + 4 * (3 * B + 3) + 8 * t + 4 * t * _words(case) + 8 * (given + back), "flops": 0}
    if case["op"] == "accept":
        t, B = sum(new), len(new)
        return {"bytes": 12 * t + 4 * (2 * B + 1) + 4 * B * (case["path"] + 3), "flops": 0}
    if case["op"] == "keep":
        # the first token of a branch stands where it is kept
        moved = sum(max(n - 1, 0) for n in _counts(case))
        return {"bytes": 2 * moved * case["layers"] * 2 * case["kv_heads"] * case["dim"] * 2 + 4 * sum(_counts(case)) + 12 * len(new), "flops": 0}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    t, keys = sum(new), sum(new) + sum(ctx)
    kv = (case["prefix"] + keys) * hk * d * 2 * 2
    pages = -(-case["prefix"] // case["page"]) + sum(-(-(n + c) // case["page"]) for n, c in zip(new, ctx))
    # a token of a tree sees its branch: counted as the sixteen tokens that a branch of these trees hardly passes
    seen = sum(n * (case["prefix"] + c + min(n, 16)) for n, c in zip(new, ctx))
    return {"bytes": kv + 2 * t * hq * d * 2 + 4 * t * hq + 4 * pages + 4 * t * _words(case), "flops": 4 * d * hq * seen}


# ------------------------------------------------------------------ inputs

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _tokens(new, dev):
    """(offsets [B + 1], sequence and place in its sequence of each token), 64-bit."""
    counts = torch.tensor([max(n, 0) for n in new], device=dev)
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), counts.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(len(new), device=dev), counts)
    return off, seq, torch.arange(seq.shape[0], device=dev) - off[seq]


def _parents(case, local, gen):
    """Each token's parent in its sequence: -1 for the first, then any earlier token (bushy) or mostly
    the one before (chain)."""
    n = local.shape[0]
    at = (torch.rand(n, generator=gen, device=local.device) * local).floor().long()
    if case["tree"] == "chain":
        at = torch.where(torch.rand(n, generator=gen, device=local.device) < 0.75, local - 1, at)
    return torch.where(local == 0, -1, torch.minimum(at, local - 1))


def _branches(off, seq, parents, nodes):
    """(depth, [T][nodes] which tokens of its sequence each token's branch holds), by doubling."""
    t, dev = seq.shape[0], seq.device
    none = torch.full((1,), t, device=dev)
    jump = torch.cat([torch.where(parents < 0, t, off[seq] + parents), none])
    depth = torch.cat([(parents >= 0).long(), none * 0])
    anc = torch.zeros(t + 1, nodes, dtype=torch.bool, device=dev)
    at = torch.arange(t, device=dev)
    anc[at, at - off[seq]] = True
    for _ in range(max(nodes - 1, 0).bit_length()):
        depth = depth + depth[jump]
        anc |= anc[jump]
        jump = jump[jump]
    return depth[:t], anc[:t]


def _pack(anc, words):
    """Bits of 32-bit words, as signed numbers."""
    t, n = anc.shape
    full = torch.zeros(t, words * 32, dtype=torch.bool, device=anc.device)
    full[:, :n] = anc
    v = (full.view(t, words, 32).long() << torch.arange(32, device=anc.device)).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def _unpack(bits, nodes):
    """[T][nodes] truth values of [T][words] bits."""
    return ((bits.long()[:, :, None] >> torch.arange(32, device=bits.device)) & 1).bool().flatten(1)[:, :nodes]


def _pages(case, count, dtype, dev, layers=None):
    """Keys and values of `count` pages as [page][slot][head][dim] tensors kept slot by slot or head by
    head, behind one another for each layer."""
    p, h, d = case["page"], case["kv_heads"], case["dim"]
    lead = (2,) if layers is None else (layers, 2)
    if case["order"] == "slot":
        return torch.zeros(*lead, count, p, h, d, dtype=dtype, device=dev)
    return torch.zeros(*lead, count, h, p, d, dtype=dtype, device=dev).transpose(-3, -2)


def _table(lens, first, order, page, dev):
    """[B][pages] block table: row b the pages of its lens[b] tokens, in order from order[first] on."""
    used = torch.tensor([-(-n // page) for n in lens], device=dev)
    column = torch.arange(max(int(used.max()), 1), device=dev)
    start = first + used.cumsum(0) - used
    inside = column < used[:, None]
    return torch.where(inside, order[(start[:, None] + column).clamp(max=order.shape[0] - 1)], 0).to(torch.int32), inside


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 11)
    return globals()["_prepare_" + case["op"]](case, dev, gen)


def _prepare_plan(case, dev, gen):
    new, ctx, held, need, free = _plan_lengths(case)
    B, p = case["seqs"], case["page"]
    width = max(h + n for h, n in zip(held, need)) + 1
    pages = sum(held) + max(free, sum(need)) + 3
    order = torch.randperm(pages, generator=gen, device=dev)
    st = {"case": case, "new": _ints(new, dev), "context": _ints(ctx, dev)}
    held_t = torch.tensor(held, device=dev)
    column = torch.arange(width, device=dev)
    start = held_t.cumsum(0) - held_t
    table = torch.where(column < held_t[:, None], order[(start[:, None] + column).clamp(max=pages - 1)], 0).to(torch.int32)
    # the ring's free pages start anywhere and may pass its end
    first = int(torch.randint(0, pages, (1,), generator=gen, device=dev))
    ring = torch.zeros(pages, dtype=torch.int32, device=dev)
    ring[(first + torch.arange(free, device=dev)) % pages] = order[sum(held):sum(held) + free].to(torch.int32)
    state = _ints([first, free] + held, dev)
    off, seq, local = _tokens(new, dev)
    room = off[-1].item() + 3  # a few tokens of padding behind the last sequence
    st["parents"] = None
    if case["tree"] != "none":
        st["parents"] = torch.cat([_parents(case, local, gen), torch.zeros(3, dtype=torch.long, device=dev)]).to(torch.int32)
    st.update(table=table, ring=ring, state=state, next_state=torch.zeros_like(state), room=room)
    if own:
        from w4a16_routed_expert_gb300.attention import PagedAttention, PagePool, StepTables
        cache = torch.zeros(2, pages, p, 1, 8, dtype=torch.float16, device=dev)
        st["attn"] = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8, max_tokens=1, max_seqs=1, k_cache=cache[0], v_cache=cache[1])
        st["pool"] = PagePool(block_table=table, free_pages=ring, state=state)
        st["tables"] = StepTables(num_seqs=B, num_tokens=room, max_nodes=0 if st["parents"] is None else case["new_max"], device=dev)
    return st


def _prepare_attend(case, dev, gen):
    new, ctx = _lengths(case)
    dtype, p, B = DTYPES[case["dtype"]], case["page"], case["seqs"]
    lens = [n + c for n, c in zip(new, ctx)]
    n_prefix = -(-case["prefix"] // p)
    count = n_prefix + sum(-(-n // p) for n in lens) + 2
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    st = {"case": case, "prefix_pages": order[:n_prefix].clone()}
    st["table"], used = _table(lens, n_prefix, order, p, dev)
    # how many slots of each page hold a token; the others hold whatever the memory held: here NaN
    held = torch.zeros(count, dtype=torch.long, device=dev)
    held[st["prefix_pages"].long()] = (case["prefix"] - torch.arange(n_prefix, device=dev) * p).clamp(max=p)
    lens_t = torch.tensor(lens, device=dev)
    held[st["table"].long()[used]] = (lens_t[:, None] - torch.arange(used.shape[1], device=dev) * p).clamp(max=p)[used]
    empty = torch.arange(p, device=dev)[None, :] >= held[:, None]
    kv = _pages(case, count, dtype, dev)
    for c in kv:
        for i in range(0, count, 4096):
            part = torch.randn(min(4096, count - i), p, case["kv_heads"], case["dim"], generator=gen, device=dev)
            part[empty[i:i + 4096]] = float("nan")
            c[i:i + 4096] = part.to(dtype)
    off, seq, local = _tokens(new, dev)
    t, nodes = seq.shape[0], max(new)
    # rotated, normed queries against normed keys, sharp enough that some keys stand out
    st["q"] = (torch.randn(t, case["q_heads"], case["dim"], generator=gen, device=dev) * 2.0).to(dtype)
    if case["tree"] == "random":  # any tokens of the tree, sometimes none
        sees = torch.rand(t, nodes, generator=gen, device=dev) < torch.rand(t, 1, generator=gen, device=dev) - 0.05
    else:
        _, sees = _branches(off, seq, _parents(case, local, gen), nodes)
    st["tree"] = _pack(sees, -(-case["new_max"] // 32))
    st.update(k_cache=kv[0], v_cache=kv[1], seq_lens=_ints(lens, dev), q_offsets=off.to(torch.int32), max_q=nodes, max_own=max(lens))
    if own:
        from w4a16_routed_expert_gb300.attention import PagedAttention
        st["attn"] = PagedAttention(num_q_heads=case["q_heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype=dtype,
                                    max_tokens=t, max_seqs=B, k_cache=kv[0], v_cache=kv[1])
    return st


def _prepare_accept(case, dev, gen):
    new, _ = _lengths(case)
    off, seq, local = _tokens(new, dev)
    t = seq.shape[0]
    parents = _parents(case, local, gen)
    tokens = torch.randint(0, case["vocab"], (t,), generator=gen, device=dev)
    # the model's choice after a token: mostly what one of its drafted children holds
    targets = torch.randint(0, case["vocab"], (t,), generator=gen, device=dev)
    rank = torch.randperm(t, generator=gen, device=dev)
    best = torch.full((t,), -1, device=dev)
    child = torch.nonzero(parents >= 0)[:, 0]
    best = best.scatter_reduce(0, off[seq[child]] + parents[child], rank[child], "amax")
    back = torch.empty_like(rank)
    back[rank] = torch.arange(t, device=dev)
    hit = (best >= 0) & (torch.rand(t, generator=gen, device=dev) < 0.85)
    targets = torch.where(hit, tokens[back[best.clamp(min=0)]], targets) if t else targets
    context = torch.randint(0, 4000, (case["seqs"],), generator=gen, device=dev)
    lens = context + torch.tensor(new, device=dev)
    if case["seqs"] > 3:
        lens[2] = 0  # no pages were left for this one
    st = {"case": case, "parents": parents.to(torch.int32), "tokens": tokens.to(torch.int32), "targets": targets.to(torch.int32),
          "context": context.to(torch.int32), "seq_lens": lens.to(torch.int32), "q_offsets": off.to(torch.int32), "max_q": max(max(new), 1)}
    if own:
        from w4a16_routed_expert_gb300.attention import PagedAttention
        st["attn"] = PagedAttention(num_q_heads=1, num_kv_heads=1, head_dim=8)
    return st


def _prepare_keep(case, dev, gen):
    new, ctx = _lengths(case)
    dtype, p, B, P = DTYPES[case["dtype"]], case["page"], case["seqs"], case["path"]
    lens = [n + c for n, c in zip(new, ctx)]
    count = sum(-(-n // p) for n in lens) + 2
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    st = {"case": case}
    st["table"], _ = _table(lens, 0, order, p, dev)
    kv = _pages(case, count, dtype, dev, case["layers"])
    for layer in kv:
        for c in layer:
            c.copy_(torch.randn(c.shape, generator=gen, device=dev, dtype=dtype))
    # accepted branches: the first token, then any later ones in ascending order
    counts, width = _counts(case), max(max(new), P)
    key = torch.rand(B, width, generator=gen, device=dev) + (torch.arange(width, device=dev) >= torch.tensor(new, device=dev)[:, None]) * 4.0
    key[:, 0] = -1.0
    picked = key.argsort(1)[:, :P]
    kept = torch.arange(P, device=dev) < torch.tensor(counts, device=dev)[:, None]
    path = torch.where(kept, picked, width).sort(1).values
    st["path"] = torch.where(kept, path, -1).to(torch.int32)
    st.update(kv=kv, counts=_ints(counts, dev), seq_lens=_ints(lens, dev), q_offsets=_tokens(new, dev)[0].to(torch.int32), max_own=max(max(lens), 1))
    if own:
        from w4a16_routed_expert_gb300.attention import PagedAttention
        st["attns"] = [PagedAttention(num_q_heads=case["kv_heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype=dtype, max_tokens=1,
                                      max_seqs=B, k_cache=layer[0], v_cache=layer[1]) for layer in kv]
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if not own:
        return globals()["_" + op](st)
    if op == "plan":
        t = st["attn"].plan(st["pool"], st["context"], st["new"], st["tables"], parents=st["parents"], prefix_len=st["case"]["prefix"],
                            next_state=st["next_state"])
        out = [t.q_offsets, t.seq_lens, t.positions, t.slots, st["table"], st["ring"], st["next_state"]]
        return out if st["parents"] is None else out + [t.tree]
    if op == "attend":
        return st["attn"].forward(st["q"], q_offsets=st["q_offsets"], max_q_len=st["max_q"], seq_lens=st["seq_lens"], max_seq_len=st["max_own"],
                                  block_table=st["table"], prefix_len=st["case"]["prefix"], prefix_pages=st["prefix_pages"], tree=st["tree"],
                                  return_lse=True)
    if op == "accept":
        a = st["attn"].accept(st["tokens"], st["targets"], st["parents"], q_offsets=st["q_offsets"], seq_lens=st["seq_lens"],
                              context_lens=st["context"], max_path=st["case"]["path"])
        return a.path, a.counts, a.next_tokens, a.context_lens
    st["attns"][0].keep(st["path"], st["counts"], q_offsets=st["q_offsets"], seq_lens=st["seq_lens"], max_seq_len=st["max_own"],
                        block_table=st["table"], others=st["attns"][1:])
    return st["kv"]


def _plan(st):
    case, table, ring = st["case"], st["table"], st["ring"]
    dev, p, F, T = table.device, case["page"], ring.shape[0], st["room"]
    new, ctx, state = st["new"].long(), st["context"].long(), st["state"].long()
    first, free, held = state[0], state[1], state[2:]
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.clamp(min=0).cumsum(0)])
    need = torch.where(new >= 0, ((ctx + new + p - 1) // p - held).clamp(min=0), 0)
    cum = need.cumsum(0)
    served = (new >= 0) & ((need == 0) | (cum <= free))
    taken = torch.where(cum <= free, cum, 0).amax()
    column = torch.arange(table.shape[1], device=dev)
    # pages given back, to the ring's end in order
    back = torch.where(new < 0, held, 0)
    place = (first + free + (back.cumsum(0) - back)[:, None] + column) % F
    longer = torch.cat([ring, ring[:1]])
    longer[torch.where(column < back[:, None], place, F)] = table
    # pages given out, from its front
    place = (first + (cum - need)[:, None] + column - held[:, None]) % F
    given = served[:, None] & (column >= held[:, None]) & (column < (held + need)[:, None])
    table.copy_(torch.where(given, ring.long()[place], table.long()))
    ring.copy_(longer[:F])
    held = torch.where(new < 0, 0, torch.where(served, held + need, held))
    st["next_state"].copy_(torch.cat([((first + taken) % F)[None], (free - taken + back.sum())[None], held]))
    lens = torch.where(served, ctx + new, 0)
    at = torch.arange(T, device=dev)
    seq = torch.searchsorted(off[1:], at, right=True)
    inside = seq < case["seqs"]
    seq = seq.clamp(max=case["seqs"] - 1)
    local = torch.where(inside, at - off[seq], 0)
    key = ctx[seq] + local
    slot = table.long()[seq, (key // p).clamp(max=table.shape[1] - 1)] * p + key % p
    slots = torch.where(inside & served[seq], slot, -1)
    out = [off.to(torch.int32), lens.to(torch.int32)]
    if st["parents"] is None:
        depth = local
    else:
        nodes = case["new_max"]
        parents = torch.where(inside, st["parents"].long(), -1)
        depth, anc = _branches(torch.where(inside, off[seq], at), at, parents, nodes)
        tree = _pack(anc & inside[:, None], _words(case))
    positions = torch.where(inside, case["prefix"] + ctx[seq] + depth, 0)
    out += [positions.to(torch.int32), slots.to(torch.int32), table, ring, st["next_state"]]
    return out if st["parents"] is None else out + [tree]


def _attend(st):
    case = st["case"]
    hq, hk, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    g, B, P = hq // hk, case["seqs"], case["prefix"]
    dev, t = st["q"].device, st["q"].shape[0]
    off, lens = st["q_offsets"].long(), st["seq_lens"].long()
    q = st["q"].float().view(t, hk, g, d) * d ** -0.5
    counts = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(B, device=dev), counts, output_size=t)
    local = torch.arange(t, device=dev) - off[seq]
    # own keys, gathered to [sequence][place][head][dim], and every token's logits against its sequence's
    L, mq = st["max_own"], st["max_q"]
    pages, place = st["table"].long(), torch.arange(L, device=dev)
    page, slot = pages[:, place // p], place % p
    inside = place[None, :] < lens[:, None]
    # which own keys each token sees: the context, and of the tree what its bits say
    start = (lens - counts)[seq]
    node = (place[None, :] - start[:, None]).clamp(0, mq - 1)
    sees = torch.where(place[None, :] < start[:, None], True, torch.gather(_unpack(st["tree"], mq), 1, node)) & inside[seq]
    k = torch.where(inside[..., None, None], st["k_cache"][page, slot[None, :]].float(), 0.0)
    qb = torch.zeros(B, mq, hk, g, d, device=dev)
    qb[seq, local] = q
    s = torch.matmul(qb.permute(0, 2, 1, 3, 4).reshape(B, hk, mq * g, d), k.permute(0, 2, 3, 1)).view(B, hk, mq, g, L)
    del k, qb
    hidden = torch.ones(B, mq, L, dtype=torch.bool, device=dev)
    hidden[seq, local] = ~sees
    s = s.masked_fill(hidden[:, None, :, None, :], -math.inf)
    m = s.amax(-1).permute(0, 2, 1, 3)[seq, local]
    if P:
        pre = torch.arange(P, device=dev)
        ppage, pslot = st["prefix_pages"].long()[pre // p], pre % p
        kp = st["k_cache"][ppage, pslot].float()
        sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, t * g, d), kp.permute(1, 2, 0))
        del kp
        m = torch.maximum(m, sp.amax(-1).view(hk, t, g).permute(1, 0, 2))
    ref = torch.where(m == -math.inf, 0.0, m)
    rb = torch.zeros(B, mq, hk, g, device=dev)
    rb[seq, local] = ref
    e = torch.exp(s.sub_(rb.permute(0, 2, 1, 3)[..., None]))
    del s
    v = torch.where(inside[..., None, None], st["v_cache"][page, slot[None, :]].float(), 0.0)
    o = torch.matmul(e.view(B, hk, mq * g, L), v.permute(0, 2, 1, 3)).view(B, hk, mq, g, d).permute(0, 2, 1, 3, 4)[seq, local]
    total = e.sum(-1).permute(0, 2, 1, 3)[seq, local]
    del e, v
    if P:
        e = torch.exp(sp.sub_(ref.permute(1, 0, 2).reshape(hk, t * g)[..., None]))
        del sp
        vp = st["v_cache"][ppage, pslot].float()
        o = o + torch.matmul(e, vp.permute(1, 0, 2)).view(hk, t, g, d).permute(1, 0, 2, 3)
        total = total + e.sum(-1).view(hk, t, g).permute(1, 0, 2)
    out = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = torch.where(m == -math.inf, m, m + torch.log(total))
    return out.view(t, hq, d).to(st["q"].dtype), lse.view(t, hq)


def _accept(st):
    case = st["case"]
    B, P = case["seqs"], case["path"]
    tokens, targets, parents, off = (st[k].long() for k in ("tokens", "targets", "parents", "q_offsets"))
    dev, t = tokens.device, tokens.shape[0]
    at = torch.arange(t, device=dev)
    seq = torch.searchsorted(off[1:], at, right=True)
    up = torch.where(parents < 0, t, off[seq] + parents)  # the parent among all tokens, t where there is none
    hit = (parents >= 0) & (tokens == torch.cat([targets, targets[:1]])[up])
    # of a token's children that hold the model's choice, the first
    first = torch.full((t + 1,), t, device=dev).scatter_reduce(0, torch.where(hit, up, t), torch.where(hit, at, t), "amin")
    root = at == off[seq]
    good = torch.cat([root | (hit & (first[up] == at)), torch.zeros(1, dtype=torch.bool, device=dev)])
    depth = torch.cat([(~root).long(), torch.zeros(1, dtype=torch.long, device=dev)])
    jump = torch.cat([torch.where(root, at, up), torch.full((1,), t, device=dev)])
    for _ in range(max(st["max_q"] - 1, 0).bit_length()):  # good: all of the branch up to here
        good = good & good[jump]
        depth = depth + torch.where(jump == torch.arange(t + 1, device=dev), 0, depth[jump])
        jump = jump[jump]
    count = off[1:] - off[:-1]
    alive = st["seq_lens"].long() >= count
    good = good[:t] & alive[seq] & (depth[:t] < P)
    path = torch.full((B * P + 1,), -1, device=dev)
    path[torch.where(good, seq * P + depth[:t], B * P)] = torch.where(good, at - off[seq], -1)
    path = path[:B * P].view(B, P)
    counts = (path >= 0).sum(1)
    last = off[:-1] + path.gather(1, (counts - 1).clamp(min=0)[:, None])[:, 0]
    following = torch.where(counts > 0, targets[last.clamp(0, max(t - 1, 0))], -1) if t else torch.full_like(counts, -1)
    return tuple(x.to(torch.int32) for x in (path, counts, following, st["context"] + counts))


def _keep(st):
    case, kv = st["case"], st["kv"]
    p, P, dev = case["page"], case["path"], kv.device
    off, lens = st["q_offsets"].long(), st["seq_lens"].long()
    start = lens - (off[1:] - off[:-1])
    i = torch.arange(P, device=dev)[None, :]
    kept = i < st["counts"][:, None]
    table = st["table"].long()

    def place(node):
        key = (start[:, None] + node).clamp(0, table.shape[1] * p - 1)
        return torch.gather(table, 1, key // p)[kept], (key % p)[kept]

    page, slot = place(st["path"].long())
    to_page, to_slot = place(i)
    kv[:, :, to_page, to_slot] = kv[:, :, page, slot]
    return kv


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    global own
    if case["op"] in ("plan", "accept") or work(case)["flops"] > 4e12:
        return None
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    new, ctx = _lengths(case)
    p = case["page"]
    if case["op"] == "keep":
        kv = st["kv"].double()
        table, path = st["table"].tolist(), st["path"].tolist()
        for b, n in enumerate(_counts(case)):
            rows = [(table[b][j // p], j % p) for j in range(ctx[b], ctx[b] + new[b])]
            held = [kv[:, :, page, slot].clone() for page, slot in rows]
            for i in range(n):
                kv[:, :, rows[i][0], rows[i][1]] = held[path[b][i]]
        return kv
    dev = st["q"].device
    hq, hk, d, P = case["q_heads"], case["kv_heads"], case["dim"], case["prefix"]
    g = hq // hk

    def keys(cache, pages, n):
        return cache[pages.long()].reshape(-1, hk, d)[:n].double() if n else torch.zeros(0, hk, d, dtype=torch.float64, device=dev)

    kp, vp = keys(st["k_cache"], st["prefix_pages"], P), keys(st["v_cache"], st["prefix_pages"], P)
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((sum(new), hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b in range(case["seqs"]):
        n, c = new[b], ctx[b]
        pages = st["table"][b, :-(-(n + c) // p)]
        k = torch.cat([kp, keys(st["k_cache"], pages, n + c)])
        v = torch.cat([vp, keys(st["v_cache"], pages, n + c)])
        sees = torch.ones(n, P + c + n, dtype=torch.bool, device=dev)
        for j in range(n):
            sees[:, P + c + j] = (st["tree"][at:at + n, j // 32] >> (j % 32)) & 1 == 1
        some = sees.any(1)
        for h in range(hq if n and bool(some.any()) else 0):
            s = st["q"][at:at + n, h].double() @ k[:, h // g].T / math.sqrt(d)
            s[~sees] = -math.inf
            z = torch.logsumexp(s[some], 1)
            lse[at:at + n, h][some] = z
            out[at:at + n, h][some] = torch.exp(s[some] - z[:, None]) @ v[:, h // g]
        at += n
    return out, lse
