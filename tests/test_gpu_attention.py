"""The attention operators (include/moe_attention.h) against their plain
64-bit definitions, at the sizes, masks, strides and values where they can go
wrong; their refusals; and one decoder block that uses them together."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attention_oracle as AO  # noqa: E402
from w4a16_routed_expert_gb300 import capi  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    capi.lib()


def within(got, want, tol, what=""):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), what
    err = (got - want).abs()
    err[inf] = 0
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err / tol)[~inf].max()):.2f} of the bound"


def caches(pages, page, heads, dim, dtype, order, fill=float("nan")):
    shape = (pages, page, heads, dim) if order == "slot" else (pages, heads, page, dim)
    return [(c if order == "slot" else c.permute(0, 2, 1, 3))
            for c in (torch.full(shape, fill, dtype=dtype, device="cuda") for _ in range(2))]


# ------------------------------------------------------------- rotate, append

ROTATE = [  # dtype, Hq, Hk, D, rotary, interleaved, norm, T, scaling
    (F16, 16, 16, 128, 128, False, True, 1, {}),
    (F16, 16, 16, 128, 128, False, True, 300, dict(kind="yarn", factor=16.0)),
    (BF16, 32, 8, 96, 24, True, False, 77, dict(kind="linear", factor=4.0)),
    (BF16, 12, 4, 80, 40, False, True, 33, dict(kind="ntk", factor=8.0)),  # pairs 20 apart: 8-byte words
    (F16, 3, 1, 64, 32, False, False, 5, {}),
    (F16, 7, 7, 8, 8, False, True, 19, {}),  # pairs 4 apart in heads of 8
    (F16, 1, 1, 8, 8, True, True, 2, {}),
    (BF16, 40, 40, 72, 0, False, True, 9, {}),  # norm alone
    (F16, 64, 8, 128, 64, True, True, 1025, {}),
    (BF16, 5, 5, 40, 16, False, False, 3, {}),
]


def _rotation(case):
    _, _, _, _, rotary, _, _, _, scaling = case
    inv, m = AO.frequencies(rotary, **{k if k != "original_max_position" else "original": v for k, v in scaling.items()})
    s = dict(scaling)
    if s.get("kind") == "yarn":
        s["original_max_position"] = 4096
    return inv, m, (s or None)


def _rotate_inputs(case, seed=0):
    dtype, Hq, Hk, D, rotary, inter, norm, T, _ = case
    gen = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=gen) * 2).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[0] = (1 << 30) + 12345  # far beyond what a 32-bit angle can hold
    if T > 2:
        pos[1], pos[2] = 0, -17
    w = [(1 + 0.3 * torch.randn(D, generator=gen)) if norm else None for _ in range(2)]
    return qkv, pos, w


@pytest.mark.parametrize("case", ROTATE, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}r{c[4]}T{c[7]}")
def test_rotate_matches_the_definition(case):
    dtype, Hq, Hk, D, rotary, inter, norm, T, _ = case
    qkv, pos, w = _rotate_inputs(case)
    inv, m, scaling = _rotation(case)
    dev = qkv.cuda()
    wd = [None if x is None else x.cuda() for x in w]
    a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, dtype=dtype, rotary_dim=rotary,
                       rope_interleaved=inter, rope_scaling=scaling, q_norm=wd[0], k_norm=wd[1])
    q, k = a.rotate(dev[:, :Hq], dev[:, Hq:Hq + Hk], pos.cuda())  # slices of a fused projection
    a.sync()
    for got, x, ww, name in ((q, qkv[:, :Hq], w[0], "q"), (k, qkv[:, Hq:Hq + Hk], w[1], "k")):
        want, tol = AO.norm_rotate(x, pos, rotary, inv, m, inter, ww)
        within(got, want, tol, name)
    # one side alone, in place, and again: the same bits
    buf = dev.clone()
    qv, kv = buf[:, :Hq], buf[:, Hq:Hq + Hk]
    a.rotate(qv, None, pos.cuda(), q_out=qv)
    a.rotate(None, kv, pos.cuda(), k_out=kv)
    assert torch.equal(qv, q) and torch.equal(kv, k) and torch.equal(buf[:, Hq + Hk:], dev[:, Hq + Hk:])


@pytest.mark.parametrize("page,order", [(16, "slot"), (48, "head")])
@pytest.mark.parametrize("case", ROTATE, ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}r{c[4]}T{c[7]}")
def test_append_stores_what_rotate_returns(case, page, order):
    dtype, Hq, Hk, D, rotary, inter, norm, T, _ = case
    qkv, pos, w = _rotate_inputs(case, 1)
    _, _, scaling = _rotation(case)
    dev, posd = qkv.cuda(), pos.cuda()
    wd = [None if x is None else x.cuda() for x in w]
    kc, vc = caches(T // page + 3, page, Hk, D, dtype, order, fill=3.0)
    a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, dtype=dtype, rotary_dim=rotary,
                       rope_interleaved=inter, rope_scaling=scaling, q_norm=wd[0], k_norm=wd[1], k_cache=kc, v_cache=vc)
    slots = torch.randperm(kc.shape[0] * page, generator=torch.Generator().manual_seed(2))[:T].to(torch.int32)
    slots[::5] = -1 - slots[::5]  # tokens that go nowhere
    q0, k0 = a.rotate(dev[:, :Hq], dev[:, Hq:Hq + Hk], posd)
    q1 = a.append(dev[:, :Hq], dev[:, Hq:Hq + Hk], dev[:, Hq + Hk:], posd, slots.cuda())
    a.sync()
    assert torch.equal(q0, q1)
    want_k, want_v = torch.full((kc.shape[0] * page, Hk, D), 3.0, dtype=dtype), None
    want_v = want_k.clone()
    keep = slots >= 0
    want_k[slots[keep].long()], want_v[slots[keep].long()] = k0.cpu()[keep], qkv[:, Hq + Hk:][keep]
    assert torch.equal(kc.reshape(-1, Hk, D).cpu(), want_k) and torch.equal(vc.reshape(-1, Hk, D).cpu(), want_v)
    # keys and values without queries
    kc.fill_(3.0), vc.fill_(3.0)
    assert a.append(None, dev[:, Hq:Hq + Hk], dev[:, Hq + Hk:], posd, slots.cuda()) is None
    assert torch.equal(kc.reshape(-1, Hk, D).cpu(), want_k) and torch.equal(vc.reshape(-1, Hk, D).cpu(), want_v)


def test_a_zero_head_and_non_finite_values_stay_in_their_head():
    D = 128
    x = torch.randn(2, 3, D).half()
    x[0, 0] = 0
    x[0, 1, 7] = float("inf")
    x[1, 2, 100] = float("nan")
    a = PagedAttention(num_q_heads=3, num_kv_heads=3, head_dim=D, rotary_dim=64, q_norm=torch.ones(D, device="cuda"))
    q, k = a.rotate(x.cuda(), x.cuda(), torch.tensor([3, 9], dtype=torch.int32, device="cuda"))
    assert (q[0, 0] == 0).all() and torch.isnan(q[0, 1, 7]) and torch.isnan(q[1, 2]).all()
    assert torch.isfinite(q[0, 2]).all() and torch.isfinite(q[1, :2]).all()
    bad = ~torch.isfinite(k[0, 1]).cpu()  # without a norm: the pair of the infinity alone
    assert bad[7] and bad[39] and bad.sum() == 2
    assert (~torch.isfinite(k[1, 2]).cpu()).nonzero().flatten().tolist() == [100]


def test_append_reports_a_slot_beyond_the_cache_and_stores_nothing():
    kc, vc = caches(4, 16, 2, 64, F16, "slot", fill=1.0)
    a = PagedAttention(num_q_heads=2, num_kv_heads=2, head_dim=64, k_cache=kc, v_cache=vc)
    x = torch.randn(3, 2, 64, device="cuda").half()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    a.append(x, x, x, pos, torch.tensor([64, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda"))
    with pytest.raises(capi.MoEError) as e:
        a.sync()
    assert e.value.status == capi.MOE_ERR_INVALID_ARG
    a.sync()  # reported once
    assert (kc.view(64, 2, 64)[:5] == 1).all() and (kc.view(64, 2, 64)[6:] == 1).all()
    assert torch.equal(kc.view(64, 2, 64)[5], x[2])


# --------------------------------------------------------------------- forward

def build(dtype, Hq, Hk, D, page, order, q_lens, own, prefix, seed=0, spare=2, sharp=2.0, keys=None):
    """A filled cache (NaN wherever no token is), its tables and the queries."""
    gen = torch.Generator().manual_seed(seed)
    np_, no = -(-prefix // page), [-(-n // page) for n in own]
    count = np_ + sum(no) + spare
    kc, vc = caches(count, page, Hk, D, dtype, order)
    pages = torch.randperm(count, generator=gen)
    ks, vs, at = [], [], 0
    tables = []
    for n, m in zip([prefix] + list(own), [np_] + no):
        k = (torch.randn(Hk, n, D, generator=gen)).to(dtype) if keys is None else keys(Hk, n, D, gen).to(dtype)
        v = (torch.randn(Hk, n, D, generator=gen) + 0.25).to(dtype)
        mine = pages[at:at + m]
        at += m
        for c, x in ((kc, k), (vc, v)):
            if n:
                full = torch.full((m * page, Hk, D), float("nan"), dtype=dtype)
                full[:n] = x.transpose(0, 1)
                c[mine.cuda()] = full.view(m, page, Hk, D).cuda()
        ks.append(k)
        vs.append(v)
        tables.append(mine.to(torch.int32))
    T = sum(q_lens)
    q = (torch.randn(T, Hq, D, generator=gen) * sharp).to(dtype)
    width = max([len(t) for t in tables[1:]] + [1])
    table = torch.full((len(own), width), -1, dtype=torch.int32)  # what no length reaches is no page
    for b, t in enumerate(tables[1:]):
        table[b, :len(t)] = t
    args = dict(q_offsets=torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda"),
                max_q_len=max(q_lens), seq_lens=torch.tensor(own, dtype=torch.int32, device="cuda"),
                max_seq_len=max(own), block_table=table.cuda(), prefix_len=prefix,
                prefix_pages=tables[0].cuda() if prefix else None)
    a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, dtype=dtype, max_tokens=T, max_seqs=len(own),
                       k_cache=kc, v_cache=vc)
    return a, q, ks, vs, args


FORWARD = {  # dtype, Hq, Hk, D, page, order, query lengths, own keys, prefix, causal
    "one key": (F16, 1, 1, 128, 16, "slot", [1], [1], 0, True),
    "nothing to see": (F16, 4, 2, 64, 16, "slot", [1, 1], [0, 0], 0, True),
    "one row empty": (BF16, 4, 4, 128, 16, "head", [1, 1, 1], [0, 17, 0], 0, True),
    "a prefix of one": (F16, 16, 16, 128, 16, "slot", [1, 1], [0, 3], 1, True),
    "prefix alone": (F16, 16, 2, 128, 32, "head", [1] * 5, [0] * 5, 333, True),
    "page and tile ends": (F16, 8, 8, 128, 64, "slot", [1] * 4, [63, 64, 65, 128], 128, True),
    "sixteen-slot tails": (BF16, 8, 4, 64, 16, "slot", [1] * 6, [15, 16, 17, 127, 129, 1], 47, True),
    "pages of 48": (F16, 12, 4, 96, 48, "head", [1] * 7, [0, 1, 47, 48, 49, 500, 95], 145, True),
    "one page for all": (F16, 4, 4, 128, 1024, "slot", [1] * 3, [700, 1, 1024], 1000, True),
    "heads of 8": (F16, 3, 1, 8, 16, "slot", [1] * 4, [5, 100, 64, 31], 70, True),
    "heads of 40": (BF16, 10, 2, 40, 32, "head", [2, 1, 3], [50, 64, 3], 129, True),
    "heads of 72": (F16, 6, 6, 72, 16, "slot", [1, 4], [130, 9], 64, False),
    "heads of 120": (BF16, 8, 1, 120, 128, "head", [1, 1], [257, 40], 383, True),
    "group of 32": (F16, 32, 1, 128, 64, "slot", [1, 1], [300, 77], 515, True),
    "group of 33": (BF16, 33, 1, 64, 16, "slot", [1, 1], [100, 128], 100, True),
    "drafts": (F16, 32, 8, 128, 16, "slot", [5, 1, 3, 4], [5, 90, 200, 4], 259, True),
    "drafts without a prefix": (BF16, 16, 16, 64, 32, "head", [7, 16, 1], [7, 40, 1], 0, True),
    "more queries than keys": (F16, 8, 8, 128, 16, "slot", [6, 9], [2, 0], 0, True),
    "more queries than keys behind a prefix": (F16, 8, 2, 128, 16, "slot", [6, 40], [2, 0], 20, True),
    "no causality": (BF16, 8, 2, 128, 64, "head", [3, 70], [33, 200], 65, False),
    "a sequence without queries": (F16, 8, 8, 64, 16, "slot", [0, 2, 0, 1], [40, 30, 0, 5], 33, True),
    "a batch of 130": (F16, 4, 4, 64, 16, "slot", [1] * 130, [(37 * i) % 150 for i in range(130)], 200, True),
    "a chunk": (F16, 8, 2, 128, 64, "slot", [130, 1, 64], [130, 300, 100], 300, True),
    "a chunk alone": (BF16, 4, 4, 128, 16, "head", [257], [257], 0, True),
    "a late chunk": (F16, 8, 1, 64, 128, "slot", [100, 33], [1000, 33], 0, True),
    "a long prefix for many": (BF16, 16, 2, 128, 64, "slot", [1] * 40, [i for i in range(40)], 5003, True),
    "a long context for one": (F16, 8, 8, 128, 64, "slot", [1], [9001], 0, True),
    "chunks behind a prefix, blocks of their own": (BF16, 16, 2, 128, 16, "head", [70, 33, 40], [80, 33, 300], 333, True),
    "chunks behind a prefix, no causality": (F16, 8, 1, 96, 32, "slot", [40, 50], [3, 200], 129, False),
    "a chunk that sees the prefix alone": (F16, 4, 1, 64, 16, "slot", [100], [40], 77, True),
    "short chunks behind a prefix": (F16, 8, 2, 64, 64, "slot", [20, 9, 33], [20, 70, 500], 600, True),
    "two thousand tokens": (F16, 2, 1, 64, 16, "slot", [2000], [2100], 130, True),
    "as many groups as there are keys": (BF16, 64, 64, 128, 16, "slot", [1] * 12, [i % 5 for i in range(12)], 0, True),
    "a prefix of many rows beside own keys": (F16, 16, 4, 128, 16, "slot", [1] * 37, [(11 * i) % 90 for i in range(37)], 7301, True),
    "the same in heads of 96": (BF16, 32, 4, 96, 48, "head", [1] * 19, [(7 * i) % 70 for i in range(19)], 7000, False),
    "a prefix of many rows beside drafts": (BF16, 32, 8, 64, 32, "head", [(3 * i) % 6 for i in range(30)], [5 + (13 * i) % 100 for i in range(30)], 2000, True),
    "a prefix of many rows alone": (F16, 16, 2, 128, 128, "slot", [1] * 40, [0] * 40, 700, True),
    "83 tokens after 8940 keys": (F16, 16, 16, 64, 16, "slot", [83], [8940], 0, True),
    "80 tokens of three heads after 9000 keys": (BF16, 48, 16, 64, 64, "head", [80], [9000], 0, True),
    "83 tokens of 128 after 6000 keys": (BF16, 16, 16, 128, 16, "slot", [83], [6000], 0, True),
    "80 tokens of three heads of 128 after 7000 keys": (F16, 48, 16, 128, 32, "slot", [80], [7000], 0, True),
    "a long prefix and 70 tokens each": (F16, 16, 16, 64, 16, "head", [70, 70], [90, 1200], 6000, True),
    "three thousand sequences": (F16, 2, 1, 64, 16, "slot", [1] * 3000, [(7 * i) % 40 for i in range(3000)], 50, True),
    "three thousand behind a long prefix": (BF16, 1, 1, 128, 16, "slot", [1] * 3000, [(5 * i) % 20 for i in range(3000)], 1500, True),
    "the most sequences": (F16, 1, 1, 8, 16, "head", [1] * 4096, [(3 * i) % 35 for i in range(4096)], 0, True),
    "very unequal": (F16, 16, 4, 128, 32, "head", [1] * 9, [1, 4100, 2, 0, 3, 64, 65, 8, 700], 0, True),
}


@pytest.mark.parametrize("name", FORWARD)
def test_forward_matches_the_definition(name):
    dtype, Hq, Hk, D, page, order, q_lens, own, prefix, causal = FORWARD[name]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, page, order, q_lens, own, prefix, seed=len(name))
    out, lse = a.forward(q.cuda(), causal=causal, return_lse=True, **args)
    a.sync()
    want, wlse, tol, ltol = AO.attend(q, ks, vs, q_lens, prefix, own, D ** -0.5, causal)
    within(out, want, tol, "out")
    within(lse, wlse, ltol, "lse")
    # the same bits again, and without the second output
    again = a.forward(q.cuda(), causal=causal, **args)
    assert torch.equal(again, out)


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("slope", [40.0, -40.0, 3.0])
def test_logits_that_grow_or_fall_along_the_keys(rows, slope):
    """The running maximum moves at every tile, or never after the first."""
    q_lens, own = ([1, 1], [700, 300]) if rows == "few" else ([90, 50], [700, 300])
    D = 64

    def keys(Hk, n, D, gen):
        k = torch.randn(Hk, n, D, generator=gen) * 0.3
        k[:, :, 0] += slope * torch.linspace(0, 1, max(n, 1))[None, :n]
        return k

    for dtype in (F16, BF16):
        a, q, ks, vs, args = build(dtype, 4, 2, D, 16, "slot", q_lens, own, 401, seed=5, keys=keys)
        q[..., 0] = 6.0
        out, lse = a.forward(q.cuda(), return_lse=True, **args)
        a.sync()
        want, wlse, tol, ltol = AO.attend(q, ks, vs, q_lens, 401, own, D ** -0.5, True)
        within(out, want, tol, "out")
        within(lse, wlse, ltol, "lse")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,g", [(1, 8), (90, 1), (70, 3)])
def test_logits_that_move_over_many_tiles(D, tokens, g):
    """Each block takes many tiles in a row and moves its reference again and
    again: up, then down, then up by jumps past what FP16 weights can hold."""

    def keys(Hk, n, D, gen):
        k = torch.randn(Hk, n, D, generator=gen) * 0.3
        x = torch.linspace(0, 1, n)
        k[:, :, 0] += 30 * torch.sin(9 * x)[None] + 12 * (torch.arange(n) % 1500 == 700)[None]
        return k

    Hk, n = 16, 7000
    a, q, ks, vs, args = build(F16, Hk * g, Hk, D, 32, "slot", [tokens], [n], 0, seed=7, keys=keys)
    q[..., 0] = 5.0
    out, lse = a.forward(q.cuda(), return_lse=True, **args)
    a.sync()
    want, wlse, tol, ltol = AO.attend(q, ks, vs, [tokens], 0, [n], D ** -0.5, True)
    within(out, want, tol, "out")
    within(lse, wlse, ltol, "lse")


@pytest.mark.parametrize("rows", ["few", "many"])
def test_extreme_logits(rows):
    """Logits of plus and minus tens of thousands: the largest counts almost
    alone, nothing overflows."""
    q_lens, own = ([1, 2], [130, 66]) if rows == "few" else ([80, 60], [130, 66])
    a, q, ks, vs, args = build(F16, 4, 4, 64, 16, "slot", q_lens, own, 70, seed=9, sharp=300.0,
                               keys=lambda Hk, n, D, gen: torch.randn(Hk, n, D, generator=gen) * 100)
    out, lse = a.forward(q.cuda(), return_lse=True, **args)
    a.sync()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # an FP32 logit of this size is off by up to a tenth, and the bounds say so
    want, wlse, tol, ltol = AO.attend(q, ks, vs, q_lens, 70, own, 0.125, True)
    within(lse, wlse, ltol, "lse")
    within(out, want, tol, "out")


@pytest.mark.parametrize("rows", ["few", "many"])
def test_a_query_that_is_not_finite_stays_in_its_row(rows):
    q_lens, own = ([1, 1, 1], [40, 70, 3]) if rows == "few" else ([50, 40, 45], [60, 70, 45])
    a, q, ks, vs, args = build(F16, 8, 4, 128, 16, "slot", q_lens, own, 90, seed=4)
    clean = a.forward(q.cuda(), **args)
    q[1, 3, 5] = float("nan")
    q[2, 0, 0] = float("inf")
    out, lse = a.forward(q.cuda(), return_lse=True, **args)
    a.sync()
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3]) and not torch.isfinite(lse[2, 0])
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[1, 3] = keep[2, 0] = False
    assert torch.equal(out[keep], clean[keep])


def test_strided_queries_and_outputs_and_another_stream():
    dtype, Hq, Hk, D, q_lens, own, prefix = BF16, 8, 2, 64, [1, 3, 1], [20, 33, 129], 75
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, 16, "slot", q_lens, own, prefix, seed=3)
    want = a.forward(q.cuda(), **args)
    wide = torch.randn(5, Hq + 6, D, device="cuda").to(dtype)
    wide[:, 2:2 + Hq] = q.cuda()
    big = torch.full((5, Hq + 3, D), 7.0, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out = a.forward(wide[:, 2:2 + Hq], out=big[:, 1:1 + Hq], **args)
    s.synchronize()
    assert torch.equal(out, want) and (big[:, 0] == 7).all() and (big[:, 1 + Hq:] == 7).all()


def test_lengths_may_change_under_a_captured_graph():
    """One captured append and forward, replayed as the sequences grow."""
    Hq, Hk, D, page = 8, 2, 128, 16
    kc, vc = caches(40, page, Hk, D, F16, "slot")
    table = torch.randperm(36, device="cuda").to(torch.int32).view(3, 12)
    a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, rotary_dim=D, max_tokens=3, max_seqs=3, k_cache=kc,
                       v_cache=vc)
    qkv = torch.zeros(3, Hq + 2 * Hk, D, device="cuda", dtype=F16)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots, lens = torch.zeros_like(pos), torch.zeros_like(pos)
    offs = torch.arange(4, dtype=torch.int32, device="cuda")
    q = torch.empty(3, Hq, D, device="cuda", dtype=F16)
    out, lse = torch.empty_like(q), torch.empty(3, Hq, device="cuda")

    def step():
        a.append(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], pos, slots, q_out=q)
        a.forward(q, q_offsets=offs, max_q_len=1, seq_lens=lens, max_seq_len=12 * page, block_table=table, out=out,
                  lse=lse)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        slots.fill_(-1)
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start = [0, 5, 150]
    ks, vs = [torch.zeros(Hk, 0, D, dtype=F16)], [torch.zeros(Hk, 0, D, dtype=F16)]
    for b, n in enumerate(start):  # what is already there
        k, v = torch.randn(Hk, n, D).half(), torch.randn(Hk, n, D).half()
        at = table[b].long().cpu()[torch.arange(n) // page] * page + torch.arange(n) % page
        kc.view(-1, Hk, D)[at.cuda()], vc.view(-1, Hk, D)[at.cuda()] = k.transpose(0, 1).cuda(), v.transpose(0, 1).cuda()
        ks.append(k)
        vs.append(v)
    inv, m = AO.frequencies(D)
    for n in range(4):
        x = torch.randn(3, Hq + 2 * Hk, D).half()
        p = torch.tensor([b + n for b in start], dtype=torch.int32)
        qkv.copy_(x)
        pos.copy_(p)
        lens.copy_(p + 1)
        slots.copy_(table.cpu()[torch.arange(3), p.long() // page] * page + p % page)
        graph.replay()
        torch.cuda.synchronize()
        qr, kr = AO.norm_rotate(x[:, :Hq], p, D, inv)[0].half(), AO.norm_rotate(x[:, Hq:Hq + Hk], p, D, inv)[0].half()
        for b in range(3):
            # the kernel's own rounded keys are the reference's inputs
            kr_b = kc.view(-1, Hk, D)[slots[b].long()].cpu()
            assert ((kr_b.double() - kr[b].double()).abs() <= 2.0 ** -9 * (1 + kr[b].double().abs())).all()
            ks[1 + b] = torch.cat([ks[1 + b], kr_b[:, None]], 1)
            vs[1 + b] = torch.cat([vs[1 + b], x[b, Hq + Hk:, None]], 1)
        want, wlse, tol, ltol = AO.attend(q.cpu(), ks, vs, [1] * 3, 0, [b + n + 1 for b in start], D ** -0.5, True)
        within(out, want, tol, f"step {n}")
        within(lse, wlse, ltol, f"lse of step {n}")
    a.sync()


def test_a_cache_whose_offsets_pass_32_bits():
    """Pages beyond element 2^32 of a cache of 9 GB a side."""
    Hk, D, page = 8, 128, 64
    count = 72000
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB")
    kc = torch.zeros(count, page, Hk, D, dtype=F16, device="cuda")
    vc = torch.zeros_like(kc)
    a = PagedAttention(num_q_heads=16, num_kv_heads=Hk, head_dim=D, max_tokens=200, max_seqs=2, k_cache=kc, v_cache=vc)
    gen = torch.Generator().manual_seed(1)
    n = 200
    pages = torch.tensor([count - 1, 3, count - 7, 71000], dtype=torch.int32)
    x = torch.randn(n, Hk, D, generator=gen).half()
    v = torch.randn(n, Hk, D, generator=gen).half()
    slots = (pages.long()[torch.arange(n) // page] * page + torch.arange(n) % page).to(torch.int32)
    assert int(slots.max()) * Hk * D > 2 ** 32
    zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
    a.append(None, x.cuda(), v.cuda(), zeros, slots.cuda())
    a.sync()
    assert torch.equal(kc[count - 1].cpu(), x[:64]) and torch.equal(vc[71000][:8].cpu(), v[192:])
    for q_lens, own, prefix in (([1, 1], [n, 40], 0), ([1], [0], n), ([100], [n], 0)):
        q = torch.randn(sum(q_lens), 16, D, generator=gen).half()
        B = len(q_lens)
        out = a.forward(q.cuda(), q_offsets=torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32).cuda(),
                        max_q_len=max(q_lens), seq_lens=torch.tensor(own, dtype=torch.int32).cuda(), max_seq_len=max(own),
                        block_table=pages.repeat(B, 1).cuda(), prefix_len=prefix, prefix_pages=pages.cuda())
        a.sync()
        kt, vt = x.transpose(0, 1), v.transpose(0, 1)
        want, _, tol, _ = AO.attend(q, [kt[:, :prefix]] + [kt[:, :m] for m in own],
                                    [vt[:, :prefix]] + [vt[:, :m] for m in own], q_lens, prefix, own, D ** -0.5, True)
        within(out, want, tol, str((q_lens, own, prefix)))


def test_out_of_range_lengths_offsets_and_pages_are_reported():
    Hq, Hk, D, page = 4, 2, 64, 16
    kc, vc = caches(6, page, Hk, D, F16, "slot", fill=0.5)
    a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, max_tokens=60, max_seqs=2, k_cache=kc, v_cache=vc)

    def run(T=2, offs=(0, 1, 2), lens=(10, 20), table=((0, 1), (2, 3)), prefix=0, pages=(4,), max_q=1):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        q = torch.ones(T, Hq, D, device="cuda").half()
        return a.forward(q, q_offsets=i(offs), max_q_len=max_q, seq_lens=i(lens), max_seq_len=32, block_table=i(table),
                         prefix_len=prefix, prefix_pages=i(pages))

    good = run()
    a.sync()
    assert torch.allclose(good.float(), torch.full_like(good, 0.5).float())
    for bad in (dict(lens=(10, 33)), dict(lens=(-1, 5)), dict(table=((0, 1), (6, 3))), dict(table=((0, 1), (2, -5))),
                dict(prefix=16, pages=(77,)), dict(offs=(0, 2, 2)), dict(offs=(0, 1, 9)), dict(offs=(1, 0, 2)),
                dict(T=60, max_q=40, offs=(0, 20, 60), table=((0, 1), (2, 99))),
                dict(T=60, max_q=40, offs=(0, 50, 60)), dict(T=60, max_q=40, offs=(0, 20, 60), prefix=5, pages=(-1,))):
        run(**bad)
        with pytest.raises(capi.MoEError) as e:
            a.sync()
        assert e.value.status == capi.MOE_ERR_INVALID_ARG, bad
        run()
        a.sync()


def test_no_tokens_is_no_work():
    kc, vc = caches(2, 16, 2, 64, F16, "slot")
    a = PagedAttention(num_q_heads=2, num_kv_heads=2, head_dim=64, k_cache=kc, v_cache=vc)
    e, i = torch.empty(0, 2, 64, device="cuda", dtype=F16), torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = a.rotate(e, e, i)
    assert q.shape == k.shape == (0, 2, 64)
    assert a.append(e, e, e, i, i).shape == (0, 2, 64)
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert a.forward(e, q_offsets=one, max_q_len=1, seq_lens=one[:1], max_seq_len=0).shape == (0, 2, 64)
    a.sync()


def test_refusals():
    lib = capi.lib()
    kc, vc = caches(4, 16, 2, 64, F16, "slot", fill=0.0)
    a = PagedAttention(num_q_heads=4, num_kv_heads=2, head_dim=64, max_tokens=4, max_seqs=2, k_cache=kc, v_cache=vc)
    bare = PagedAttention(num_q_heads=4, num_kv_heads=2, head_dim=64)
    p = torch.zeros(4096, device="cuda").data_ptr()
    INV = capi.MOE_ERR_INVALID_ARG

    def rotate(h=a.handle, q=p, qs=256, k=p, ks=128, pos=p, T=2, qo=p, qos=256, ko=p, kos=128):
        return lib.moe_attn_rotate(h, q, qs, k, ks, pos, T, qo, qos, ko, kos, None)

    for bad in (dict(h=None), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=None, qo=None, k=None, ko=None),
                dict(pos=None), dict(T=-1), dict(T=(1 << 22) + 1), dict(qs=255), dict(qs=248), dict(qos=0), dict(ks=120),
                dict(kos=-128), dict(q=p + 2), dict(ko=p + 8)):
        assert rotate(**bad) == INV, bad
        assert capi.last_error()

    def append(h=a.handle, k=p, v=p, ks=128, vs=128, pos=p, slots=p, q=None, qo=None, T=2):
        return lib.moe_attn_append(h, q, 256, k, ks, v, vs, pos, slots, T, qo, 256, None)

    for bad in (dict(h=bare.handle), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(q=p), dict(vs=64),
                dict(T=-3), dict(v=p + 4)):
        assert append(**bad) == INV, bad

    def forward(h=a.handle, q=p, qs=256, out=p + 8192, os_=256, **kw):
        d = dict(num_tokens=2, num_seqs=2, q_offsets=p, max_q_len=1, seq_lens=p, max_seq_len=16, block_table=p,
                 table_stride=1, prefix_len=0, prefix_pages=None, causal=1)
        d.update(kw)
        return lib.moe_attn_forward(h, q, qs, ctypes.byref(capi.moe_attn_batch_t(**d)), out, os_, None, None)

    for bad in (dict(h=bare.handle), dict(num_tokens=5), dict(num_tokens=-1), dict(num_seqs=3), dict(num_seqs=0),
                dict(q_offsets=None), dict(seq_lens=None), dict(max_q_len=0), dict(max_q_len=3), dict(max_seq_len=17),
                dict(max_seq_len=-1), dict(block_table=None), dict(prefix_len=4), dict(prefix_len=-1), dict(causal=2),
                dict(q=None), dict(out=None), dict(qs=8), dict(os_=257), dict(q=p + 2), dict(table_stride=-1),
                dict(num_seqs=1), dict(prefix_len=(1 << 30), prefix_pages=p)):
        assert forward(**bad) == INV, bad
    assert lib.moe_attn_forward(a.handle, p, 256, None, p, 256, None, None) == INV
    assert lib.moe_attn_sync(None, None) == INV and lib.moe_attn_destroy(None) == capi.MOE_OK
    x = torch.zeros(2, 4, 64, device="cuda")
    with pytest.raises(ValueError):
        a.rotate(x, None, torch.zeros(2, dtype=torch.int32, device="cuda"))  # fp32
    with pytest.raises(ValueError):
        a.rotate(x.half().transpose(0, 1).contiguous().transpose(0, 1), None,
                 torch.zeros(2, dtype=torch.int32, device="cuda"))  # heads not contiguous
    with pytest.raises(ValueError):
        a.rotate(x.half(), None, torch.zeros(2, dtype=torch.int64, device="cuda"))
    a.sync()


# ----------------------------------------------------------- used together

def test_decoder_blocks_behind_a_shared_prompt():
    """Two blocks (append, forward, routed experts) decode behind a prompt that
    all sequences share, and behind copies of it in every sequence's own pages.
    Only the attention is computed another way, so the hidden states agree to
    the rounding of the 16-bit probabilities and outputs, block after block;
    a token whose routing stands on a tie may pick other experts."""
    import importlib.util
    import os

    from w4a16_routed_expert_gb300 import synth

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prefix_decode.py")
    spec = importlib.util.spec_from_file_location("shared_prefix_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    seqs, prompt_len, steps = 9, 301, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    H = synth.TINY.hidden
    prompt = torch.randn(prompt_len, H, generator=gen, device="cuda").half()
    first = torch.randn(seqs, H, generator=gen, device="cuda").half()
    runs = []
    for share in (True, False):
        d = ex.SharedPrefixDecoder(synth.TINY, n_blocks=2, q_heads=8, kv_heads=2, head_dim=64, seqs=seqs,
                                   prompt_len=prompt_len, max_new=steps, share=share)
        out = [d.prefill(prompt)]
        x = first
        for _ in range(steps):
            out.append(d.step(x))
            x = ex.Block.norm(out[-1])
        d.sync()
        runs.append([o.double().cpu() for o in out])
    assert torch.equal(runs[0][0], runs[1][0])  # the prompt's own pass is the same in both
    for a, b in zip(*runs):
        assert torch.isfinite(a).all()
        # each step: probabilities and outputs rounded to 2^-11, then two blocks of
        # products of unit gain; a few times that, relative to the states' size
        rel = (a - b).norm(dim=1) / b.norm(dim=1)
        assert (rel < 0.01).double().mean() >= 0.85 and rel.median() < 0.005, rel
