"""Plain definitions of the operators around a step over trees of drafted
tokens, and the error bounds their tests use (test infrastructure)."""
import numpy as np
import torch

from attention_oracle import UNIT


def branches(parents):
    """[m][m] truth values: node i's branch holds node j (parents[i] < i)."""
    m = len(parents)
    rows = np.zeros((m, m), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            rows[i] = rows[p]
        rows[i, i] = True
    return rows


def pack(rows, words, junk=None):
    """int32 [m][words] of [m][n] truth values; junk: a generator for the bits
    from n on."""
    m, n = rows.shape
    full = np.zeros((m, words * 32), dtype=np.uint64)
    if junk is not None:
        full[:] = junk.integers(0, 2, full.shape)
    full[:, :n] = rows
    v = (full.reshape(m, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(v.astype(np.uint32).view(np.int32).copy())


def random_tree(rng, m, kind):
    """Parents of m nodes: -1 for the first, then "bushy", "chain" or "line"."""
    p = [-1]
    for i in range(1, m):
        p.append(i - 1 if kind == "line" or (kind == "chain" and rng.random() < 0.75) else int(rng.integers(0, i)))
    return p[:m]


def attend(q, keys, values, q_lens, prefix, own, scale, sees):
    """attention_oracle.attend with sees[b] [n][own[b]]: which own keys each
    query token of sequence b sees. The bounds are derived there."""
    u = UNIT[q.dtype]
    T, Hq, D = q.shape
    g = Hq // keys[0].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -np.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for b, n in enumerate(q_lens):
        k = torch.cat([keys[0], keys[1 + b]], 1).double()
        v = torch.cat([values[0], values[1 + b]], 1).double()
        total = prefix + own[b]
        see = torch.ones(n, total, dtype=torch.bool)
        see[:, prefix:] = torch.from_numpy(np.asarray(sees[b]))
        some = see.any(1)
        if total and bool(some.any()):
            kk, vv = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
            qh = q[t0:t0 + n].double().transpose(0, 1)
            s = (qh @ kk.transpose(1, 2) * scale).masked_fill(~see, -np.inf)[:, some]
            big = (qh.abs() @ kk.abs().transpose(1, 2) * scale).masked_fill(~see, 0)[:, some].amax(-1)
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


def plan(table, ring, state, context, new, page, room, prefix=0, parents=None, words=0):
    """The tables of one step as lists; table and ring are changed in place,
    state is not."""
    F, first, free, held = len(ring), state[0], state[1], list(state[2:])
    off, lens, positions, slots, tree, back, cum, taken = [0], [], [], [], [], [], 0, 0
    for b, m in enumerate(new):
        if m < 0:
            back += table[b][:held[b]]
            held[b] = 0
            off.append(off[-1])
            lens.append(0)
            continue
        need = max(0, -(-(context[b] + m) // page) - held[b])
        cum += need
        ok = need == 0 or cum <= free
        if ok and need:
            taken = cum
            for i in range(need):
                table[b][held[b] + i] = ring[(first + cum - need + i) % F]
            held[b] += need
        lens.append(context[b] + m if ok else 0)
        mine = parents[off[-1]:off[-1] + m] if parents is not None else None
        rows = branches(mine) if mine is not None else None
        for i in range(m):
            key = context[b] + i
            positions.append(prefix + context[b] + (i if rows is None else int(rows[i].sum()) - 1))
            slots.append(table[b][key // page] * page + key % page if ok else -1)
        if rows is not None and m:
            tree += pack(rows, words).tolist()
        off.append(off[-1] + m)
    for k, x in enumerate(back):
        ring[(first + free + k) % F] = x
    pad = room - off[-1]
    return dict(q_offsets=off, seq_lens=lens, positions=positions + [0] * pad, slots=slots + [-1] * pad,
                tree=tree + [[0] * words] * pad, state=[(first + taken) % F, free - taken + len(back)] + held)


def accept(tokens, targets, parents, max_path):
    """The confirmed branch of one tree."""
    path = [0]
    for j in range(1, len(tokens)):
        if len(path) < max_path and parents[j] == path[-1] and tokens[j] == targets[path[-1]]:
            path.append(j)
    return path[:max_path]
