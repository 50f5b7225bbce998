"""Cases of the attention operators that stand beside the routed-expert layer in a decoder block.

Three operators, in the order a decoder runs them:

* ``rotate``  RMS norm of every query and key head, then the rotary position rotation (half or
  interleaved pairs, all or the first part of a head, frequencies scaled for long contexts);
* ``append``  the same pass, with the keys and the values stored into the pages of a cache;
* ``attend``  attention of a ragged batch over that cache: one prefix that all sequences share,
  then each sequence's own pages, causal at the end.

``own`` selects the framework's calls; without it ``run`` computes the same from elementary torch
operations in 32 bits.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
MAX_POS = 131072


def listed():
    return [
        # one token of a 16-head layer on its way through a decode step: launch latency
        dict(name="rotate-decode-1", op="rotate", dtype="f16", tokens=1, q_heads=16, kv_heads=16, dim=128, rotary=128,
             pairs="half", norm=True, scaling="none", factor=1.0, max_pos=4096, fused=True),
        # a ragged chunk of prompt, grouped heads of 96 with a quarter rotated in interleaved pairs, no norm
        dict(name="rotate-partial-777", op="rotate", dtype="bf16", tokens=777, q_heads=32, kv_heads=8, dim=96, rotary=24,
             pairs="interleaved", norm=False, scaling="linear", factor=4.0, max_pos=32768, fused=True),
        # a long prompt at the prefill size of the layer (8192 tokens, hidden 2048), scaled to long contexts
        dict(name="rotate-prompt-8192", op="rotate", dtype="f16", tokens=8192, q_heads=16, kv_heads=16, dim=128, rotary=128,
             pairs="half", norm=True, scaling="yarn", factor=16.0, max_pos=131072, fused=False),
        # a decode step of 16 sequences: 16 tokens into 16 pages
        dict(name="append-decode-16", op="append", dtype="f16", tokens=16, q_heads=16, kv_heads=16, dim=128, rotary=128,
             pairs="half", norm=True, scaling="none", factor=1.0, max_pos=32768, page=16, order="slot", padded=0),
        # a batch of prompts cut into 64-slot pages kept head by head, with padding tokens that go nowhere
        dict(name="append-grouped-1111", op="append", dtype="bf16", tokens=1111, q_heads=64, kv_heads=8, dim=64, rotary=64,
             pairs="half", norm=False, scaling="ntk", factor=8.0, max_pos=65536, page=64, order="head", padded=23),
        # the 8192-token prompt written to 16-slot pages
        dict(name="append-prompt-8192", op="append", dtype="f16", tokens=8192, q_heads=16, kv_heads=16, dim=128, rotary=128,
             pairs="half", norm=True, scaling="none", factor=1.0, max_pos=8192, page=16, order="slot", padded=0),
        # two short conversations behind a short common instruction: latency
        dict(name="attend-short-2", op="attend", dtype="f16", seqs=2, q_min=1, q_max=1, q_heads=16, kv_heads=16, dim=128,
             prefix=500, own_min=1, own_max=64, page=16, order="slot", causal=True),
        # a decode batch of 16 behind a common system text
        dict(name="attend-shared-16", op="attend", dtype="f16", seqs=16, q_min=1, q_max=1, q_heads=16, kv_heads=16, dim=128,
             prefix=4099, own_min=0, own_max=1000, page=16, order="slot", causal=True),
        # 48 sequences checking up to 5 drafted tokens each, small heads, pages kept head by head
        dict(name="attend-drafts-48", op="attend", dtype="bf16", seqs=48, q_min=1, q_max=5, q_heads=32, kv_heads=8, dim=64,
             prefix=10007, own_min=5, own_max=700, page=32, order="head", causal=True),
        # 64 samples of one long document, grouped heads: the prefix's products count
        dict(name="attend-document-64", op="attend", dtype="f16", seqs=64, q_min=1, q_max=1, q_heads=64, kv_heads=8, dim=128,
             prefix=32768, own_min=1, own_max=512, page=64, order="slot", causal=True),
        # chunks of four prompts behind the same examples: rows by the hundred for every sequence
        dict(name="attend-chunks-4", op="attend", dtype="bf16", seqs=4, q_min=301, q_max=1024, q_heads=32, kv_heads=8, dim=128,
             prefix=8200, own_min=301, own_max=2500, page=64, order="slot", causal=True),
        # nothing shared: 32 conversations of very different lengths, the cache's bytes count
        dict(name="attend-ragged-32", op="attend", dtype="bf16", seqs=32, q_min=1, q_max=1, q_heads=32, kv_heads=8, dim=128,
             prefix=0, own_min=0, own_max=24000, page=16, order="head", causal=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v + 1 if v == 3072 else v


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["rotate", "append", "attend", "attend"])
        heads = rng.choice([(16, 16), (32, 8), (32, 4), (64, 8), (8, 1), (12, 4), (40, 40)])
        c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), q_heads=heads[0], kv_heads=heads[1])
        if op != "attend":
            dim = rng.choice([64, 80, 96, 128])
            c.update(tokens=_log(rng, 1, 8192), dim=dim, rotary=rng.choice([dim, dim, dim // 2 // 8 * 8]),
                     pairs=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.7,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([2, 8, 16])),
                     max_pos=_log(rng, 16, MAX_POS))
            if c["scaling"] == "none":
                c["factor"] = 1.0
            if op == "rotate":
                c["fused"] = rng.random() < 0.5
            else:
                c.update(page=rng.choice([16, 32, 48, 64, 128]), order=rng.choice(["slot", "head"]),
                         padded=rng.choice([0, 0, min(c["tokens"] // 4, 31)]))
        else:
            q = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 32, 1024)])
            hi = _log(rng, 1, 24000)
            c.update(seqs=_log(rng, 1, 128), q_min=rng.choice([1, q]), q_max=q, dim=rng.choice([64, 96, 128]),
                     prefix=rng.choice([0, _log(rng, 1, 40000), _log(rng, 1, 40000)]), own_min=rng.choice([0, hi // 2, hi]), own_max=hi,
                     page=rng.choice([16, 32, 48, 64, 128]), order=rng.choice(["slot", "head"]), causal=rng.random() < 0.8)
            # what the plain form holds in 32 bits at once has to stay small beside the card's memory
            rows = c["seqs"] * q * c["q_heads"]
            if rows * (c["prefix"] + c["own_max"]) > 1.5e9 or c["seqs"] * c["own_max"] * c["kv_heads"] * c["dim"] > 1.5e9:
                continue
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------ shapes

def _spread(n, lo, hi, start):
    """n whole numbers from lo to hi, odd ones among them, the same for the same case."""
    return [lo + int((hi - lo + 1) * ((start + 0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _lengths(case):
    """(query tokens, own keys) of each sequence."""
    B = case["seqs"]
    nq, nk = _spread(B, case["q_min"], case["q_max"], 0.999), _spread(B, case["own_min"], case["own_max"], 0.0 if B > 1 else 0.999)
    if case["own_min"]:  # the query tokens' own keys are in the cache; without them, rows that see nothing
        nk = [max(n, m) for n, m in zip(nk, nq)]
    return nq, nk


def _visible(case):
    """Sum over the query tokens of the own keys that each one sees."""
    total = 0
    for nq, nk in zip(*_lengths(case)):
        for i in range(nq):
            total += min(nk, max(0, nk - nq + i + 1)) if case["causal"] else nk
    return total


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        n = case["tokens"] * (hq + hk) * d
        # square, add, two products for the norm; two products and a sum for the rotation
        return {"bytes": 2 * 2 * n + 4 * case["tokens"], "flops": (4 * n if case["norm"] else 0) + 3 * n}
    if case["op"] == "append":
        t = case["tokens"]
        n = t * (hq + hk) * d
        kept = t - case["padded"]
        moved = 2 * (t * hq + kept * 2 * hk) * d * 2
        return {"bytes": moved + 8 * t, "flops": (4 * n if case["norm"] else 0) + 3 * n}
    nq, nk = _lengths(case)
    t = sum(nq)
    kv = (case["prefix"] + sum(nk)) * hk * d * 2 * 2
    pages = -(-case["prefix"] // case["page"]) + sum(-(-n // case["page"]) for n in nk)
    flops = 4 * d * hq * (t * case["prefix"] + _visible(case))
    return {"bytes": kv + 2 * t * hq * d * 2 + 4 * t * hq + 4 * pages, "flops": flops}


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """Radians per position of each pair and the factor on cosine and sine, in 64 bits.

    linear: positions divided by the factor; ntk: the base raised so that the slowest pair slows by
    the factor; yarn: pairs that turn over 32 times within the original context (4096) keep their
    frequency, those under one turn are divided, a ramp between, and cosine and sine grow by
    0.1 ln(factor) + 1."""
    rd, base, f = case["rotary"], 10000.0, case["factor"]
    if case["scaling"] == "ntk" and rd > 2:
        base = base * f ** (rd / (rd - 2))
    i = torch.arange(0, rd, 2, dtype=torch.float64)
    inv = base ** (-i / rd)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "yarn":
        def dim_of(turns):
            return rd * math.log(4096.0 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rd - 1)
        ramp = ((torch.arange(rd // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _scaling_args(case):
    if case["scaling"] == "none":
        return {}
    d = {"kind": case["scaling"], "factor": case["factor"]}
    if case["scaling"] == "yarn":
        d["original_max_position"] = 4096
    return {"rope_scaling": d}


def _pages(case, count, dtype, dev):
    """A cache of `count` pages as a [page][slot][head][dim] tensor kept slot by slot or head by head."""
    p, h, d = case["page"], case["kv_heads"], case["dim"]
    if case["order"] == "slot":
        return torch.zeros(count, p, h, d, dtype=dtype, device=dev)
    return torch.zeros(count, h, p, d, dtype=dtype, device=dev).permute(0, 2, 1, 3)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 11)
    dtype = DTYPES[case["dtype"]]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": case}
    if case["op"] in ("rotate", "append"):
        t = case["tokens"]
        # the rows of a fused projection (queries, keys, values side by side) or separate tensors
        if case["op"] == "append" or case["fused"]:
            qkv = (normal(t, (hq + 2 * hk), d) * 1.5).to(dtype)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            st["q"], st["k"] = (normal(t, hq, d) * 1.5).to(dtype), (normal(t, hk, d) * 1.5).to(dtype)
        start = torch.randint(0, max(case["max_pos"] - t, 0) + 1, (1,), generator=gen, device=dev)
        pos = start + torch.arange(t, device=dev)
        if t <= 64:  # a decode step: every token at a place of its own
            pos = torch.randint(0, case["max_pos"], (t,), generator=gen, device=dev)
        st["positions"] = pos.clamp(max=case["max_pos"] - 1).to(torch.int32)
        st["q_norm"] = 1 + 0.2 * normal(d) if case["norm"] else None
        st["k_norm"] = 1 + 0.2 * normal(d) if case["norm"] else None
        inv, m = _frequencies(case)
        if not own:
            ang = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * inv.to(dev)[None, :]
            st["cos"], st["sin"] = (ang.cos() * m).float(), (ang.sin() * m).float()
            del ang
        if case["op"] == "append":
            count = -(-t // case["page"]) + 3
            st["k_cache"], st["v_cache"] = _pages(case, count, dtype, dev), _pages(case, count, dtype, dev)
            order = torch.randperm(count, generator=gen, device=dev)
            i = torch.arange(t, device=dev)
            slots = order[i // case["page"]] * case["page"] + i % case["page"]
            if t <= 64:  # a decode step: tokens land anywhere
                slots = torch.randperm(count * case["page"], generator=gen, device=dev)[:t]
            if case["padded"]:
                slots[torch.randperm(t, generator=gen, device=dev)[:case["padded"]]] = -1
            st["slots"] = slots.to(torch.int32)
        else:
            st["k_cache"] = st["v_cache"] = None
        if own:
            from w4a16_routed_expert_gb300.attention import PagedAttention
            st["attn"] = PagedAttention(num_q_heads=hq, num_kv_heads=hk, head_dim=d, dtype=dtype, max_tokens=t, max_seqs=1,
                                        k_cache=st["k_cache"], v_cache=st["v_cache"], rotary_dim=case["rotary"],
                                        rope_interleaved=case["pairs"] == "interleaved", rope_theta=10000.0,
                                        q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=EPS, **_scaling_args(case))
        return st

    nq, nk = _lengths(case)
    p = case["page"]
    n_prefix = -(-case["prefix"] // p)
    n_own = [-(-n // p) for n in nk]
    count = n_prefix + sum(n_own) + 2
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    st["prefix_pages"] = order[:n_prefix].clone()
    # row b of the table: the pages of sequence b, in order, then zeros
    n_own_t = torch.tensor(n_own, device=dev)
    column = torch.arange(max(max(n_own), 1), device=dev)[None, :]
    first = n_prefix + torch.cumsum(n_own_t, 0) - n_own_t
    used = column < n_own_t[:, None]
    st["table"] = torch.where(used, order[(first[:, None] + column).clamp(max=count - 1)], 0).to(torch.int32)
    # how many slots of each page hold a token; what none has been written to holds whatever the
    # memory held: here NaN
    held = torch.zeros(count, dtype=torch.long, device=dev)
    held[st["prefix_pages"].long()] = (case["prefix"] - torch.arange(n_prefix, device=dev) * p).clamp(max=p)
    lens = torch.tensor(nk, device=dev)
    held[st["table"].long()[used]] = (lens[:, None] - column * p).clamp(max=p)[used]
    mask = torch.arange(p, device=dev)[None, :] >= held[:, None]
    kc, vc = _pages(case, count, dtype, dev), _pages(case, count, dtype, dev)
    for c in (kc, vc):
        for i in range(0, count, 4096):
            part = normal(min(4096, count - i), p, hk, d)
            part[mask[i:i + 4096]] = float("nan")
            c[i:i + 4096] = part.to(dtype)
    t = sum(nq)
    # rotated, normed queries against normed keys, sharp enough that some keys stand out
    st["q"] = (normal(t, hq, d) * 2.0).to(dtype)
    st["k_cache"], st["v_cache"] = kc, vc
    st["seq_lens"] = torch.tensor(nk, dtype=torch.int32, device=dev)
    off = [0]
    for n in nq:  # tokens of all sequences stand back to back
        off.append(off[-1] + n)
    st["q_offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
    st["max_q"], st["max_own"] = max(nq), max(nk)
    if own:
        from w4a16_routed_expert_gb300.attention import PagedAttention
        st["attn"] = PagedAttention(num_q_heads=hq, num_kv_heads=hk, head_dim=d, dtype=dtype, max_tokens=t,
                                    max_seqs=case["seqs"], k_cache=kc, v_cache=vc)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        a = st["attn"]
        if case["op"] == "rotate":
            return a.rotate(st["q"], st["k"], st["positions"])
        if case["op"] == "append":
            q = a.append(st["q"], st["k"], st["v"], st["positions"], st["slots"])
            return q, st["k_cache"], st["v_cache"]
        return a.forward(st["q"], q_offsets=st["q_offsets"], max_q_len=st["max_q"], seq_lens=st["seq_lens"],
                         max_seq_len=st["max_own"], block_table=st["table"], prefix_len=case["prefix"],
                         prefix_pages=st["prefix_pages"], causal=case["causal"], return_lse=True)
    if case["op"] == "attend":
        return _attend(st)
    q = _norm_rotate(st, st["q"], st["q_norm"])
    k = _norm_rotate(st, st["k"], st["k_norm"])
    if case["op"] == "rotate":
        return q, k
    slots = st["slots"].long()
    keep = slots >= 0
    page, slot = slots[keep] // case["page"], slots[keep] % case["page"]
    st["k_cache"][page, slot] = k[keep]
    st["v_cache"][page, slot] = st["v"][keep]
    return q, st["k_cache"], st["v_cache"]


def _norm_rotate(st, x, w):
    case = st["case"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    rd = case["rotary"]
    pos = st["positions"].long()
    cos, sin = st["cos"][pos][:, None, :], st["sin"][pos][:, None, :]
    out = y.clone()
    if case["pairs"] == "half":
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        out[..., :rd // 2], out[..., rd // 2:rd] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        out[..., 0:rd:2], out[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def _attend(st):
    case = st["case"]
    hq, hk, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    g, B, P = hq // hk, case["seqs"], case["prefix"]
    dev = st["q"].device
    t = st["q"].shape[0]
    off, lens = st["q_offsets"].long(), st["seq_lens"].long()
    q = st["q"].float().view(t, hk, g, d) * d ** -0.5
    counts = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(B, device=dev), counts, output_size=t)
    local = torch.arange(t, device=dev) - off[seq]
    limit = lens[seq]
    if case["causal"]:
        limit = torch.minimum(limit, limit - counts[seq] + local + 1)
    m = torch.full((t, hk, g), -math.inf, device=dev)
    # own keys, gathered to [sequence][place][head][dim] and every token's logits against its sequence's
    L, mq = st["max_own"], st["max_q"]
    if L:
        pages = st["table"].long()
        place = torch.arange(L, device=dev)
        page, slot = pages[:, place // p], place % p
        inside = place[None, :] < lens[:, None]
        k = torch.where(inside[..., None, None], st["k_cache"][page, slot[None, :]].float(), 0.0)
        qb = torch.zeros(B, mq, hk, g, d, device=dev)
        qb[seq, local] = q
        s = torch.matmul(qb.permute(0, 2, 1, 3, 4).reshape(B, hk, mq * g, d), k.permute(0, 2, 3, 1))
        del k, qb
        s = s.view(B, hk, mq, g, L)
        lim = torch.zeros(B, mq, dtype=torch.long, device=dev)
        lim[seq, local] = limit
        s = s.masked_fill(place >= lim[:, None, :, None, None], -math.inf)
        m = torch.maximum(m, s.amax(-1).permute(0, 2, 1, 3)[seq, local])
    if P:
        place = torch.arange(P, device=dev)
        page, slot = st["prefix_pages"].long()[place // p], place % p
        kp = st["k_cache"][page, slot].float()
        sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, t * g, d), kp.permute(1, 2, 0))
        del kp
        m = torch.maximum(m, sp.amax(-1).view(hk, t, g).permute(1, 0, 2))
    ref = torch.where(m == -math.inf, 0.0, m)
    total = torch.zeros(t, hk, g, device=dev)
    o = torch.zeros(t, hk, g, d, device=dev)
    if L:
        rb = torch.zeros(B, mq, hk, g, device=dev)
        rb[seq, local] = ref
        e = torch.exp(s.sub_(rb.permute(0, 2, 1, 3)[..., None]))
        del s
        page = pages[:, torch.arange(L, device=dev) // p]
        slot = torch.arange(L, device=dev) % p
        v = torch.where(inside[..., None, None], st["v_cache"][page, slot[None, :]].float(), 0.0)
        ob = torch.matmul(e.view(B, hk, mq * g, L), v.permute(0, 2, 1, 3)).view(B, hk, mq, g, d)
        total += e.sum(-1).permute(0, 2, 1, 3)[seq, local]
        o += ob.permute(0, 2, 1, 3, 4)[seq, local]
        del e, v, ob
    if P:
        e = torch.exp(sp.sub_(ref.permute(1, 0, 2).reshape(hk, t * g)[..., None]))
        del sp
        page, slot = st["prefix_pages"].long()[torch.arange(P, device=dev) // p], torch.arange(P, device=dev) % p
        vp = st["v_cache"][page, slot].float()
        o += torch.matmul(e, vp.permute(1, 0, 2)).view(hk, t, g, d).permute(1, 0, 2, 3)
        total += e.sum(-1).view(hk, t, g).permute(1, 0, 2)
    out = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = m + torch.log(total)
    lse = torch.where(m == -math.inf, m, lse)
    return out.view(t, hq, d).to(st["q"].dtype), lse.view(t, hq)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    dev = st["q"].device
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    g = hq // hk
    if case["op"] == "attend":
        if work(case)["flops"] > 8e12:
            return None
        nq, nk = _lengths(case)
        p, P = case["page"], case["prefix"]

        def keys(cache, pages, n):
            return cache[pages.long()].reshape(-1, hk, d)[:n].double() if n else torch.zeros(0, hk, d, dtype=torch.float64, device=dev)

        kp, vp = keys(st["k_cache"], st["prefix_pages"], P), keys(st["v_cache"], st["prefix_pages"], P)
        out = torch.zeros(sum(nq), hq, d, dtype=torch.float64, device=dev)
        lse = torch.full((sum(nq), hq), -math.inf, dtype=torch.float64, device=dev)
        at = 0
        for b in range(case["seqs"]):
            own_pages = st["table"][b, :-(-nk[b] // p)]
            k, v = keys(st["k_cache"], own_pages, nk[b]), keys(st["v_cache"], own_pages, nk[b])
            sees = torch.ones(nq[b], P + nk[b], dtype=torch.bool, device=dev)
            if case["causal"]:
                i = torch.arange(nq[b], device=dev)[:, None]
                sees[:, P:] = torch.arange(nk[b], device=dev)[None, :] <= i + (nk[b] - nq[b])
            some = sees.any(1)
            if not bool(some.any()):
                at += nq[b]
                continue
            for h in range(hk):
                kk, vv = torch.cat([kp[:, h], k[:, h]]), torch.cat([vp[:, h], v[:, h]])
                for j in range(h * g, (h + 1) * g):
                    s = st["q"][at:at + nq[b], j].double() @ kk.T / math.sqrt(d)
                    s[~sees] = -math.inf
                    z = torch.logsumexp(s[some], 1)
                    lse[at:at + nq[b], j][some] = z
                    out[at:at + nq[b], j][some] = torch.exp(s[some] - z[:, None]) @ vv
            at += nq[b]
        return out, lse

    inv, m = _frequencies(case)
    angle = st["positions"].double()[:, None, None] * inv.to(dev)
    turn = torch.polar(torch.full_like(angle, m), angle)
    rd = case["rotary"]

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        head, rest = y[..., :rd], y[..., rd:]
        if case["pairs"] == "half":
            z = torch.complex(head[..., :rd // 2].contiguous(), head[..., rd // 2:].contiguous()) * turn
            return torch.cat([z.real, z.imag, rest], -1)
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rd // 2, 2).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)

    q, k = turned(st["q"], st["q_norm"]), turned(st["k"], st["k_norm"])
    if case["op"] == "rotate":
        return q, k
    caches = []
    for cache, new in ((st["k_cache"], k), (st["v_cache"], st["v"].double())):
        c = cache.double().reshape(-1, hk, d)
        for t, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                c[s] = new[t]
        caches.append(c.view(cache.shape))
    return q, caches[0], caches[1]
