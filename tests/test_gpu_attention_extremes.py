"""Attention at logits far past what 32 bits hold to a unit: finite, huge, of
both signs, and finite ones behind some that overflowed.

The queries have one component that is not zero (or two whose products add up
to a whole number under 2^24), so every FP32 logit s is exact and the 64-bit
definition says what has to come out. A weight is then off by the rounding of
scale * log2 e and of its exponent, 2^-23 each, times an exponent that is at
most 45 where the weight still counts, and by the exponential's 2^-22: under
2^-16 in all. The rest is the rounding of the weights and of the output to 16
bits (u each) and 2^-32 of the largest value a key where FP16 weights are
subnormal; lse adds the rounding of scale and of scale * s."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attention_oracle as AO  # noqa: E402
from test_gpu_attention import BF16, F16, _cuda, build, within  # noqa: E402,F401
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402

PREFIX, OWN = 401, [700, 300]
Q_LENS = {"few": [1, 2], "many": [90, 50]}


def run(dtype, D, rows, scale, queries, keys, Hq=4, Hk=2):
    """queries(n, gen) and keys(n, gen): the first two components."""
    gen = torch.Generator().manual_seed(1)

    def k_of(heads, n, dim, _):
        k = torch.randn(heads, n, dim, generator=gen)
        if n:
            k[..., 0], k[..., 1] = keys((heads, n), gen)
        return k

    q_lens = Q_LENS[rows]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, 16, "slot", q_lens, OWN, PREFIX, seed=8, keys=k_of)
    q.zero_()
    q[..., 0], q[..., 1] = queries(q.shape[:2], gen)
    if scale is None:
        scale = D ** -0.5
    else:
        a = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, dtype=dtype, max_tokens=q.shape[0],
                           max_seqs=len(OWN), k_cache=a._keep[0], v_cache=a._keep[1], scale=scale)
    out, lse = a.forward(q.cuda(), return_lse=True, **args)
    a.sync()
    want, wlse = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    tol, t0, u = torch.zeros_like(want), 0, AO.UNIT[dtype]
    for b, n in enumerate(q_lens):
        k = torch.cat([ks[0], ks[1 + b]], 1).double().repeat_interleave(Hq // Hk, 0)
        v = torch.cat([vs[0], vs[1 + b]], 1).double().repeat_interleave(Hq // Hk, 0)
        s = torch.einsum("ihd,hjd->hij", q[t0:t0 + n].double(), k) * scale
        hidden = torch.arange(PREFIX + OWN[b]) > (PREFIX + OWN[b] - n + torch.arange(n))[:, None]
        s = s.masked_fill(hidden, -float("inf"))
        z = torch.logsumexp(s, -1)
        p = torch.softmax(s, -1)  # (exp(s - z) would lose ln n beside s in 64 bits)
        o, A = p @ v, p @ v.abs()
        e = (u + 2.0 ** -16) * A + u * o.abs() + k.shape[1] * 2.0 ** -32 * v.abs().max() + 2.0 ** -24
        want[t0:t0 + n], wlse[t0:t0 + n], tol[t0:t0 + n] = o.transpose(0, 1), z.T, e.transpose(0, 1)
        t0 += n
    assert torch.isfinite(wlse).all()
    within(out, want, tol, "out")
    within(lse, wlse, 2.0 ** -21 * (1 + wlse.abs()), "lse")


HUGE = {  # dtype, query component, unit and most units of the key component, scale
    "1e8": (F16, 2.0 ** 15, 16, 2000, None),
    "1e9": (F16, 2.0 ** 15, 16, 2000, 1.0),
    "1e12": (F16, 2.0 ** 15, 16, 2000, 1e3),
    "1e37": (F16, 2.0 ** 15, 16, 2000, 1e28),
    "1e9 of BF16": (BF16, 2.0 ** 15, 2.0 ** 8, 250, None),
    "1e15 of BF16": (BF16, 2.0 ** 25, 2.0 ** 20, 250, None),
    "1e33 of BF16": (BF16, 2.0 ** 52, 2.0 ** 52, 250, None),
}


@pytest.mark.parametrize("rows", Q_LENS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [0, 1, -1])
@pytest.mark.parametrize("name", HUGE)
def test_huge_finite_logits(name, sign, D, rows):
    """The largest keys count alone, and share the weight where several are
    the same: sixteen sizes, so most rows have several. sign: of all logits
    (0: both)."""
    dtype, q0, unit, most, scale = HUGE[name]

    def queries(shape, gen):
        turn = torch.randint(0, 2, shape, generator=gen) * 2 - 1 if sign == 0 else 1
        return q0 * turn / 2.0 ** torch.randint(0, 3, shape, generator=gen), torch.zeros(shape)

    def keys(shape, gen):
        sizes = torch.randint(1, most, (16,), generator=torch.Generator().manual_seed(6)).double()
        if sign == 0:
            sizes[::2] *= -1
        return sizes[torch.randint(0, 16, shape, generator=gen)] * unit * (sign or 1), torch.zeros(shape)

    run(dtype, D, rows, scale, queries, keys)


@pytest.mark.parametrize("rows", Q_LENS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("far", [2.0 ** 20, -2.0 ** 20])
def test_near_logits_far_from_zero(far, dtype, D, rows):
    """Logits a million and a few: what counts is the few."""

    def queries(shape, gen):
        return torch.full(shape, 2.0 ** 10), torch.ones(shape)

    def keys(shape, gen):
        return torch.full(shape, far / 2.0 ** 10), torch.randint(-6, 7, shape, generator=gen).double()

    run(dtype, D, rows, 1.0, queries, keys)


@pytest.mark.parametrize("rows", Q_LENS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("way", ["up", "down", "hill", "valley"])
def test_logits_that_cross_zero_from_afar(way, D, rows):
    """Along the keys of each sequence (and of the prefix) logits run from a
    million below zero to a million above, the other way, up to a few and
    back, or down and back: the reference is far from zero, near it, and far
    again."""

    def queries(shape, gen):
        return 2.0 ** (10 - torch.randint(0, 12, shape, generator=gen)), torch.ones(shape)

    def keys(shape, gen):
        n = shape[1]
        at = torch.arange(n) * 2048 // max(n - 1, 1) - 1024  # -1024 .. 1024
        k = {"up": at, "down": -at, "hill": -at.abs(), "valley": at.abs()}[way]
        return k.expand(shape).double(), torch.randint(-3, 4, shape, generator=gen).double()

    run(F16, D, rows, 1.0, queries, keys)


@pytest.mark.parametrize("rows", Q_LENS)
@pytest.mark.parametrize("D", [64, 128])
def test_finite_logits_behind_an_overflow(D, rows):
    """The prefix's logits are minus infinity in 32 bits (-2^190), those of
    the own keys some -1000: these count alone."""
    first = [True]

    def queries(shape, gen):
        return torch.full(shape, 2.0 ** 100), torch.zeros(shape)

    def keys(shape, gen):
        big, first[0] = first[0], False  # the prefix is asked for first
        return (torch.full(shape, -2.0 ** 90) if big else
                -(1000 + 8 * torch.randint(0, 3, shape, generator=gen).double()) * 2.0 ** -100), torch.zeros(shape)

    run(BF16, D, rows, 1.0, queries, keys)
