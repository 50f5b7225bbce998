"""Steps over trees of drafted tokens, the operators used together: a small
decoder that checks its drafts against its own choices, its steps captured in a
graph, on given streams, and in caches beyond 32-bit offsets."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attention_oracle as AO  # noqa: E402
import tree_oracle as TO  # noqa: E402
from test_gpu_attention import F16, _cuda, build, caches, within  # noqa: E402,F401
from w4a16_routed_expert_gb300.attention import Accepted, PagedAttention, PagePool, StepTables  # noqa: E402

HQ, HK, D, H, VOCAB, LAYERS, PAGE = 4, 2, 64, 128, 80, 2, 16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """Two attention layers over one-hot-like embeddings, greedy."""

    def __init__(self, seed):
        gen = torch.Generator().manual_seed(seed)
        self.emb = torch.randn(VOCAB, H, generator=gen)
        self.w = [(torch.randn(H, (HQ + 2 * HK) * D, generator=gen) * H ** -0.5, torch.randn(HQ * D, H, generator=gen) * (HQ * D) ** -0.5)
                  for _ in range(LAYERS)]
        self.inv = AO.frequencies(D)[0]

    def logits(self, tokens):
        """In 64 bits, rounded where the caches and the kernels' outputs are."""
        x, n = self.emb[tokens].double(), len(tokens)
        pos = torch.arange(n)
        for wi, wo in self.w:
            qkv = (x @ wi.double()).half().view(n, -1, D)
            q, k = (AO.norm_rotate(y, pos, D, self.inv)[0].half().double() for y in (qkv[:, :HQ], qkv[:, HQ:HQ + HK]))
            v = qkv[:, HQ + HK:].double()
            k, v = k.repeat_interleave(HQ // HK, 1), v.repeat_interleave(HQ // HK, 1)
            s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
            s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -np.inf)
            o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).half().double()
            x = x + o.flatten(1) @ wo.double()
        return x @ self.emb.double().T


class Decoder:
    """The same on the GPU, over paged caches."""

    def __init__(self, model, *, pages, seqs, max_pages, prefix, max_tokens, max_nodes):
        self.dev = [(wi.cuda(), wo.cuda()) for wi, wo in model.w]
        self.emb = model.emb.cuda()
        n = -(-len(prefix) // PAGE)
        order = torch.randperm(pages + n, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.prefix_pages, self.prefix_len = order[:n].cuda(), len(prefix)
        self.kv = [caches(pages + n, PAGE, HK, D, F16, "slot") for _ in range(LAYERS)]
        self.attn = [PagedAttention(num_q_heads=HQ, num_kv_heads=HK, head_dim=D, rotary_dim=D, max_tokens=max_tokens, max_seqs=seqs,
                                    k_cache=k, v_cache=v) for k, v in self.kv]
        self.pool = PagePool.of(order[n:].cuda(), num_seqs=seqs, max_pages=max_pages)
        self.tables = StepTables(num_seqs=seqs, num_tokens=max_tokens, max_nodes=max_nodes)
        self.lines = StepTables(num_seqs=seqs, num_tokens=max_tokens)
        self.max_pages = max_pages
        at = torch.arange(len(prefix))
        slots = (self.prefix_pages.cpu()[at // PAGE] * PAGE + at % PAGE).to(torch.int32).cuda()
        ends = ints([0, len(prefix)])
        self.layers(torch.tensor(prefix, device="cuda"), at.to(torch.int32).cuda(), slots, q_offsets=ends, max_q_len=len(prefix),
                    seq_lens=ends[1:], max_seq_len=len(prefix), block_table=self.prefix_pages[None])

    def layers(self, tokens, positions, slots, **batch):
        x = self.emb[tokens.long()]
        for a, (wi, wo) in zip(self.attn, self.dev):
            qkv = (x @ wi).half().view(len(x), -1, D)
            q = a.append(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], positions, slots)
            x = x + a.forward(q, **batch).flatten(1).float() @ wo
        return (x @ self.emb.T).argmax(-1).to(torch.int32)

    def step(self, context, new, tokens, parents=None, max_len=None):
        """Plans and runs a step; returns the model's choices."""
        tables = self.lines if parents is None else self.tables
        t = self.attn[0].plan(self.pool, context, new, tables, parents=parents, prefix_len=self.prefix_len)
        most = self.max_pages * PAGE
        return t, self.layers(tokens, t.positions, t.slots, q_offsets=t.q_offsets, max_q_len=max_len or len(tokens), seq_lens=t.seq_lens,
                              max_seq_len=most, block_table=self.pool.block_table, prefix_len=self.prefix_len,
                              prefix_pages=self.prefix_pages, tree=t.tree)

    def sync(self):
        for a in self.attn:
            a.sync()


def draft(rng, root, future, m):
    """A tree of m nodes whose branches hold some of what comes: (tokens, parents)."""
    parents = TO.random_tree(rng, m, "chain")
    depth = [0] * m
    right, tokens = [True] + [False] * (m - 1), [root]
    for i in range(1, m):
        depth[i] = depth[parents[i]] + 1
        hit = right[parents[i]] and depth[i] <= len(future) and rng.random() < 0.6
        tokens.append(future[depth[i] - 1] if hit else int(rng.integers(0, VOCAB)))
        right[i] = right[parents[i]] and depth[i] <= len(future) and tokens[-1] == future[depth[i] - 1]
    return tokens, parents


def test_decoding_by_trees_gives_what_decoding_token_by_token_gives():
    """Five conversations behind a common text, drafted by trees, in a pool whose
    pages do not always reach for all: every conversation ends with the tokens
    that the model would have chosen one at a time."""
    B, total, most = 5, 40, 23
    rng = np.random.default_rng(5)
    model = Model(3)
    prefix = rng.integers(0, VOCAB, 21).tolist()
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (3, 17, 1, 30, 8)]
    want, margin = [], []
    for p in prompts:
        seq, gap = prefix + p, []
        for _ in range(total + most):
            top = model.logits(torch.tensor(seq))[-1].topk(2)
            seq = seq + [int(top.indices[0])]
            gap.append(float(top.values[0] - top.values[1]))
        want.append(seq[len(prefix) + len(p):])
        margin.append(gap)
    # an output that is off by a few roundings moves a logit by 2^-8 or so; no choice here is that near
    assert min(min(g) for g in margin) > 0.02, min(min(g) for g in margin)

    d = Decoder(model, pages=18, seqs=B, max_pages=8, prefix=prefix, max_tokens=B * 30, max_nodes=most)
    got = [[] for _ in range(B)]
    context = ints([0] * B)
    room = B * 30  # a call takes max_q_len tokens a sequence at most
    flat = sum(prompts, [])
    t, choice = d.step(context, ints([len(p) for p in prompts]), ints(flat + [0] * (room - len(flat))), max_len=30)
    assert t.seq_lens.tolist() == [len(p) for p in prompts]
    last = np.cumsum([len(p) for p in prompts]) - 1
    for b in range(B):
        got[b].append(int(choice[last[b]]))
    context = t.seq_lens.clone()
    out = Accepted(num_seqs=B, max_path=most)
    steps = waited = 0
    over = [False] * B
    while not all(over):
        new, tokens, parents = [], [], []
        for b in range(B):
            if over[b] or len(got[b]) >= total:
                new.append(0 if over[b] else -1)
                over[b] = True
                continue
            m = int(rng.integers(1, most + 1))
            tk, pr = draft(rng, got[b][-1], want[b][len(got[b]):], m)
            new.append(m)
            tokens += tk
            parents += pr
        pad = room - len(tokens)
        tk, pr = ints(tokens + [0] * pad), ints(parents + [0] * pad)
        ctx = torch.where(ints(new) < 0, 0, context)
        t, choice = d.step(context, ints(new), tk, pr, max_len=30)
        a = d.attn[0].accept(tk, choice, pr, q_offsets=t.q_offsets, seq_lens=t.seq_lens, context_lens=ctx, out=out)
        d.attn[0].keep(a.path, a.counts, q_offsets=t.q_offsets, seq_lens=t.seq_lens, max_seq_len=d.max_pages * PAGE,
                       block_table=d.pool.block_table, others=d.attn[1:])
        d.sync()
        off, counts, path, nxt = t.q_offsets.tolist(), a.counts.tolist(), a.path.tolist(), a.next_tokens.tolist()
        for b in range(B):
            if new[b] <= 0:
                assert counts[b] == 0
                continue
            if t.seq_lens[b] == 0:  # no pages were left
                assert counts[b] == 0 and int(a.context_lens[b]) == int(context[b])
                waited += 1
                continue
            assert counts[b] >= 1
            got[b] += [tokens[off[b] + i] for i in path[b][1:counts[b]]] + [nxt[b]]
            assert got[b] == want[b][:len(got[b])], (b, steps)
        context = a.context_lens.clone()
        steps += 1
        assert steps < 100
    assert waited > 0 and steps < 60  # some had to wait, and the trees were worth it
    assert sorted(d.pool.free_pages[(d.pool.state[0] + torch.arange(18, device="cuda")) % 18].tolist()) == \
        sorted(set(range(20)) - set(d.prefix_pages.tolist())) and int(d.pool.state[1]) == 18


def test_a_captured_step_replays_as_the_sequences_grow():
    """plan, append, forward, accept and keep in one graph, lengths in place: as
    the same calls made one by one."""
    B, m, most = 3, 7, 12
    rng = np.random.default_rng(2)
    model = Model(4)
    prefix = rng.integers(0, VOCAB, 5).tolist()
    drafts = [[draft(rng, int(rng.integers(0, VOCAB)), [], m) for _ in range(B)] for _ in range(6)]
    results = []
    for graph in (False, True):
        d = Decoder(model, pages=40, seqs=B, max_pages=most, prefix=prefix, max_tokens=B * m, max_nodes=m)
        context, new = ints([0] * B), ints([m] * B)
        tk, pr = ints([0] * B * m), ints([-1] * B * m)
        out = Accepted(num_seqs=B, max_path=m)
        choices = torch.zeros(B * m, dtype=torch.int32, device="cuda")

        def step():
            t, c = d.step(context, new, tk, pr, max_len=m)
            choices.copy_(c)
            a = d.attn[0].accept(tk, c, pr, q_offsets=t.q_offsets, seq_lens=t.seq_lens, context_lens=context, out=out)
            d.attn[0].keep(a.path, a.counts, q_offsets=t.q_offsets, seq_lens=t.seq_lens, max_seq_len=most * PAGE,
                           block_table=d.pool.block_table, others=d.attn[1:])
            context.copy_(a.context_lens)

        state = [x.clone() for x in (d.pool.state, d.pool.block_table, context)]
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for x, y in zip((d.pool.state, d.pool.block_table, context), state):
                x.copy_(y)
        run = []
        for ds in drafts:
            tk.copy_(ints(sum((t for t, _ in ds), [])))
            pr.copy_(ints(sum((p for _, p in ds), [])))
            g.replay() if graph else step()
            d.sync()
            run.append([x.clone() for x in (d.tables.positions, d.tables.slots, d.tables.tree, out.path, out.counts, choices, context,
                                            d.pool.state)])
        run.append([c[d.pool.block_table[b, j]].clone() for k, v in d.kv for c in (k, v) for b in range(B)
                    for j in range(int(context[b]) // PAGE)])
        results.append(run)
    for a, b in zip(*results):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_on_a_given_stream():
    """The operators on a stream that is not the current one, each waiting for
    what wrote its inputs."""
    nodes, context = [5, 1, 13], [20, 0, 70]
    own = [c + n for c, n in zip(context, nodes)]
    rng = np.random.default_rng(1)
    a, q, ks, vs, args = build(F16, 4, 2, 64, 16, "slot", nodes, own, 33, seed=6)
    trees = [TO.random_tree(rng, n, "bushy") for n in nodes]
    bits = torch.cat([TO.pack(TO.branches(p), 1) for p in trees]).cuda()
    par, tok = ints(sum(trees, [])), ints(rng.integers(0, 2, 19).tolist())
    q = q.cuda()
    free = torch.arange(30, dtype=torch.int32, device="cuda")

    def calls(stream):
        pool = PagePool.of(free, num_seqs=3, max_pages=8)
        tables = StepTables(num_seqs=3, num_tokens=19, max_nodes=13)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            torch.cuda._sleep(20_000_000)  # about 10 ms: what runs on the wrong stream runs too early
            par2, tok2, q2 = par.clone(), tok.clone(), q.clone()
        t = a.plan(pool, ints(context) if stream is None else CTX, ints(nodes) if stream is None else NEW, tables, parents=par2, stream=stream)
        o = a.forward(q2, tree=bits, stream=stream, **args)
        acc = a.accept(tok2, tok2, par2, q_offsets=args["q_offsets"], context_lens=CTX, max_path=4, stream=stream)
        a.keep(acc.path, acc.counts, q_offsets=args["q_offsets"], seq_lens=args["seq_lens"], max_seq_len=args["max_seq_len"],
               block_table=args["block_table"], stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        return [x.clone() for x in (t.slots, t.positions, t.tree, o, acc.path, acc.counts, acc.next_tokens, acc.context_lens,
                                    a._keep[0].nan_to_num(), a._keep[1].nan_to_num())]

    CTX, NEW = ints(context), ints(nodes)
    kept = [c.clone() for c in a._keep[:2]]
    want = calls(None)
    for c, k in zip(a._keep[:2], kept):
        c.copy_(k)
    got = calls(torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    a.sync()


def test_a_cache_whose_offsets_pass_32_bits():
    Hk, dim, page, count = 8, 128, 64, 72000
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    kc = torch.zeros(count, page, Hk, dim, dtype=F16, device="cuda")
    vc = torch.zeros_like(kc)
    a = PagedAttention(num_q_heads=16, num_kv_heads=Hk, head_dim=dim, max_tokens=130, max_seqs=2, k_cache=kc, v_cache=vc)
    gen = torch.Generator().manual_seed(1)
    pages = [count - 1, 3, count - 7, 71000]
    nodes, context = [80], [110]
    k, v = (torch.randn(Hk, 190, dim, generator=gen).half() for _ in range(2))
    flat = [pages[j // page] * page + j % page for j in range(190)]
    assert max(flat) * Hk * dim > 2 ** 32
    at = torch.tensor(flat, device="cuda")
    kc.view(-1, Hk, dim)[at], vc.view(-1, Hk, dim)[at] = k.transpose(0, 1).cuda(), v.transpose(0, 1).cuda()
    table, off, lens = ints([pages]), ints([0, 80]), ints([190])
    for n in (80, 7):  # the tile kernel's rows, the few-row kernel's
        q = torch.randn(n, 16, dim, generator=gen).half()
        rows = TO.branches(TO.random_tree(np.random.default_rng(n), n, "bushy"))
        out = a.forward(q.cuda(), q_offsets=ints([0, n]), max_q_len=n, seq_lens=lens, max_seq_len=190, block_table=table,
                        tree=TO.pack(rows, 3).cuda())
        a.sync()
        sees = [np.concatenate([np.ones((n, 190 - n), dtype=bool), rows], 1)]
        none = torch.zeros(Hk, 0, dim).half()
        want, _, tol, _ = TO.attend(q, [none, k], [none, v], [n], 0, [190], dim ** -0.5, sees)
        within(out, want, tol, str(n))
    path = [0, 30, 50, 79]
    a.keep(ints([path]), ints([4]), q_offsets=off, seq_lens=lens, max_seq_len=190, block_table=table)
    a.sync()
    for i, p in enumerate(path):
        assert torch.equal(kc.view(-1, Hk, dim)[flat[110 + i]].cpu(), k[:, 110 + p])
        assert torch.equal(vc.view(-1, Hk, dim)[flat[110 + i]].cpu(), v[:, 110 + p])
    pool = PagePool(block_table=ints([[0, 0]]), free_pages=ints(pages[:1] + pages[3:]), state=ints([0, 2, 0]))
    t = a.plan(pool, ints([0]), ints([70]), StepTables(num_seqs=1, num_tokens=70))
    assert t.slots.tolist() == [pages[0] * page + j for j in range(64)] + [pages[3] * page + j for j in range(6)]
    a.sync()
