"""Plain 64-bit definitions of the attention operators and the error bounds
their tests use (test infrastructure)."""
import numpy as np
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a unit in the last place, relative


def frequencies(rotary, theta=10000.0, kind="none", factor=1.0, original=4096, fast=32.0, slow=1.0):
    """(radians per position of each pair, factor on cosine and sine)."""
    i = np.arange(rotary // 2, dtype=np.float64)
    base = theta * factor ** (rotary / (rotary - 2)) if kind == "ntk" else theta
    inv = base ** (-2 * i / rotary)
    if kind == "linear":
        return inv / factor, 1.0
    if kind != "yarn":
        return inv, 1.0
    pair = {t: rotary * np.log(original / (t * 2 * np.pi)) / (2 * np.log(theta)) for t in (fast, slow)}
    lo, hi = max(np.floor(pair[fast]), 0), min(np.ceil(pair[slow]), rotary - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
    return inv / factor * ramp + inv * (1 - ramp), 0.1 * np.log(factor) + 1


def norm_rotate(x, positions, rotary, inv, m=1.0, interleaved=False, w=None, eps=1e-6):
    """(result, bound): x [T][heads][D] in a 16-bit type, the result in 64
    bits, and how far a kernel that works in FP32 and rounds once may be off:
    the rounding, and 2^-18 of the two products of a pair for the hardware
    sine and cosine (2^-21.4 each), the FP32 norm (eight roundings of 2^-24)
    and the subnormal step."""
    u = UNIT[x.dtype]
    y = x.double()
    if w is not None:
        y = y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    ang = positions.double()[:, None, None] * torch.from_numpy(np.asarray(inv))
    cos, sin = ang.cos() * m, ang.sin() * m
    out, mag = y.clone(), y.abs()
    if rotary:
        ia = torch.arange(0, rotary, 2) if interleaved else torch.arange(rotary // 2)
        ib = ia + 1 if interleaved else ia + rotary // 2
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
        mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * m
    return out, u * out.abs() + 2.0 ** -18 * mag + 2.0 ** -24


def attend(q, keys, values, q_lens, prefix, own, scale, causal):
    """(out, lse, out bound, lse bound) of one batch in 64 bits. keys/values:
    [Hk][n][D] lists, the prefix first and then one per sequence.

    With p_j the weights and A = sum p |v| / sum p: rounding each p to the
    16-bit type costs at most u A (plus 2^-32 max |v| a key where FP16
    probabilities are subnormal: they are kept at 2^7 of the largest),
    rounding the result u |out|; an FP32 logit is off by 2^-21 of
    scale sum |q k|, which moves a weight by as much, relative; sums over n
    keys in FP32, sixteen at a time, by (n / 16 + 8) 2^-23."""
    u = UNIT[q.dtype]
    T, Hq, D = q.shape
    Hk = keys[0].shape[0]
    g = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -np.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for b, n in enumerate(q_lens):
        k = torch.cat([keys[0], keys[1 + b]], 1).double()
        v = torch.cat([values[0], values[1 + b]], 1).double()
        total = prefix + own[b]
        sees = torch.ones(n, total, dtype=torch.bool)
        if causal:
            sees[:, prefix:] = torch.arange(own[b])[None] < (own[b] - n + 1 + torch.arange(n))[:, None]
        some = sees.any(1)
        qb = q[t0:t0 + n].double()
        if total and bool(some.any()):
            kk, vv = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
            qh = qb.transpose(0, 1)  # [Hq][n][D]
            s = (qh @ kk.transpose(1, 2) * scale).masked_fill(~sees, -np.inf)[:, some]
            big = (qh.abs() @ kk.abs().transpose(1, 2) * scale).masked_fill(~sees, 0)[:, some].amax(-1)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            o, A = p @ vv, p @ vv.abs()
            vmax = vv.abs().amax((1, 2))[:, None, None]
            sums = (total / 16 + 8) * 2.0 ** -23
            e = (u + 2 * 2.0 ** -21 * big[..., None] + sums) * A + u * o.abs() + total * 2.0 ** -32 * vmax + 2.0 ** -24
            idx = torch.nonzero(some)[:, 0] + t0
            out[idx], lse[idx], tol[idx] = o.transpose(0, 1), z.T, e.transpose(0, 1)
            ltol[idx] = (2.0 ** -21 * big + sums + 2.0 ** -21 * (1 + z.abs())).T
        t0 += n
    return out, lse, tol, ltol
