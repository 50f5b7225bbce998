"""Attention over trees on each way that a call can take, and as steps of fixed
room make it: bounds above the lengths, tokens behind the last sequence. Which
way a case takes follows from its sizes (attn_api.cu, attn.h); they stand well
inside what the rules there say."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_oracle as TO  # noqa: E402
from test_gpu_attention import BF16, F16, _cuda, build, within  # noqa: E402,F401
from test_gpu_tree import seen_by  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402

PATHS = {  # dtype, Hq, Hk, D, page, order, nodes, context, prefix, what a token sees, tokens behind, max_q_len, max_seq_len
    # two row groups of the few-row kernel by two key groups, in parts
    "17 to 32 rows of 128": (F16, 2, 2, 128, 16, "slot", [17, 31, 32, 5], [400, 700, 333, 0], 0, "bushy", 0, 32, 732),
    "17 to 32 rows of 96": (BF16, 8, 4, 96, 48, "head", [16, 9, 13, 0], [500, 0, 77, 400], 0, "random", 3, 16, 1000),
    "17 to 32 rows of 128 behind a prefix": (BF16, 12, 6, 128, 32, "slot", [16, 9, 0, 15], [500, 0, 41, 3], 150, "chain", 0, 16, 600),
    "17 to 32 rows of 128 over a long context": (F16, 4, 4, 128, 64, "slot", [31, 20], [4200, 100], 0, "bushy", 0, 32, 5000),
    # in whole groups
    "17 to 32 rows of 128 in whole groups": (F16, 3, 3, 128, 16, "slot", [32, 17, 0, 25], [280, 0, 90, 3], 0, "random", 5, 32, 320),
    "17 to 32 rows of 96 in whole groups": (BF16, 4, 2, 96, 16, "head", [13, 9, 16], [-13, 200, -3], 0, "bushy", 0, 16, 320),
    "17 to 32 rows of 64 in whole groups": (F16, 4, 1, 64, 16, "slot", [8, 5, 7], [150, 0, 303], 0, "chain", 2, 8, 311),
    "few rows of 64 in whole groups": (BF16, 4, 4, 64, 16, "head", [16, 1, 0, 9], [150, 0, 70, 280], 0, "bushy", 7, 16, 320),
    "33 to 64 rows in whole groups, more than there are SMs": (F16, 4, 4, 128, 16, "slot", [(11 * i) % 65 for i in range(42)],
                                                               [(31 * i) % 240 for i in range(42)], 0, "bushy", 4, 64, 320),
    # 33 to 64 rows in parts
    "33 to 64 rows of 128 behind a prefix": (F16, 4, 2, 128, 16, "slot", [32, 20, 5], [300, 900, 0], 77, "bushy", 0, 32, 1000),
    "33 to 64 rows of 64 over a long context": (BF16, 8, 1, 64, 64, "slot", [8, 5], [5000, 60], 0, "bushy", 0, 8, 6000),
    # the prefix on the tcgen05 tiles, the few own rows after it, their join
    "a long prefix, few own rows of 64": (BF16, 32, 8, 64, 32, "head", [(3 * i) % 8 for i in range(40)], [(13 * i) % 100 for i in range(40)],
                                          2500, "bushy", 6, 8, 128),
    "a long prefix, few own rows of 128": (F16, 16, 16, 128, 16, "slot", [(5 * i) % 17 - (i == 10) for i in range(24)], [(31 * i) % 200 for i in range(24)],
                                       4099, "chain", 5, 16, 256),
    "a long prefix, 17 to 32 own rows of 96": (BF16, 16, 8, 96, 48, "head", [(5 * i) % 17 for i in range(20)], [(91 * i) % 500 for i in range(20)],
                                               4000, "bushy", 9, 16, 520),
    "a long prefix and no keys": (F16, 32, 8, 64, 16, "slot", [5] * 30, [-5] * 30, 2000, "bushy", 0, 8, 64),
    # the tcgen05 tiles in whole groups
    "whole groups on the tiles without keys": (F16, 8, 2, 128, 16, "slot", [40, 30], [-40, -30], 0, "random", 3, 40, 100),
    "whole groups on the tiles without keys, of 64": (BF16, 8, 2, 64, 16, "slot", [40, 30], [-40, -30], 0, "random", 3, 40, 100),
    "whole groups of one row tile of 128": (BF16, 32, 4, 128, 16, "slot", [(5 * i) % 17 for i in range(24)], [(87 * i) % 900 for i in range(24)], 0, "bushy",
                                            0, 16, 900),
    "whole groups of one row tile of 64": (F16, 32, 4, 64, 16, "head", [(5 * i) % 17 for i in range(24)], [(37 * i) % 300 for i in range(24)], 0, "bushy",
                                           6, 16, 310),
    # the prefix apart from own keys, both on the tiles
    "a prefix apart from own rows of 128": (F16, 16, 2, 128, 32, "head", [64, 1, 2, 3, 5, 1, 1, 40], [900, 9, 0, 5000, 90, 130, 1, 64], 500, "chain",
                                            3, 64, 6000),
    # fixed room and loose bounds, as a step of up to 32 tokens a sequence has them
    "half full": (F16, 16, 16, 128, 16, "slot", [(7 * i) % 31 for i in range(12)], [(67 * i) % 900 for i in range(12)], 0, "bushy",
                  12 * 32 - sum((7 * i) % 31 for i in range(12)), 32, 4096),
    "half full behind a prefix": (BF16, 16, 4, 64, 16, "head", [(7 * i) % 31 for i in range(12)], [(67 * i) % 900 for i in range(12)], 333, "chain",
                                  12 * 32 - sum((7 * i) % 31 for i in range(12)), 32, 4096),
    "half full of hundreds": (BF16, 8, 2, 128, 16, "slot", [100, 0, 157], [30, 500, 700], 90, "bushy", 3 * 200 - 257, 200, 4096),
}


@pytest.mark.parametrize("name", PATHS)
def test_forward_over_trees_on_every_way(name):
    dtype, Hq, Hk, D, page, order, nodes, context, prefix, kind, pad, most, bound = PATHS[name]
    rng = np.random.default_rng(len(name))
    own, T = [c + m for c, m in zip(context, nodes)], sum(nodes)
    rows = [seen_by(rng, kind, m) for m in nodes]
    sees = [np.concatenate([np.ones((m, max(c, 0)), dtype=bool), r[:, max(-c, 0):]], 1) for m, c, r in zip(nodes, context, rows)]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, page, order, nodes, own, prefix, seed=len(name))
    words = -(-most // 32)
    bits = torch.cat([TO.pack(r, words, rng) for r in rows] + [torch.full((pad, words), -1, dtype=torch.int32)]).cuda()
    room = PagedAttention(num_q_heads=Hq, num_kv_heads=Hk, head_dim=D, dtype=dtype, max_tokens=T + pad, max_seqs=len(nodes),
                          k_cache=a._keep[0], v_cache=a._keep[1])
    table = torch.full((len(nodes), max(-(-bound // page), args["block_table"].shape[1])), -1, dtype=torch.int32, device="cuda")
    table[:, :args["block_table"].shape[1]] = args["block_table"]
    args.update(max_q_len=most, max_seq_len=bound, block_table=table)
    qp = torch.cat([q.cuda(), torch.full((pad, Hq, D), float("nan"), dtype=dtype, device="cuda")])
    out, lse = torch.full_like(qp, 9.0), torch.full((T + pad, Hq), 9.0, device="cuda")
    room.forward(qp, tree=bits, out=out, lse=lse, **args)
    room.sync()
    want, wlse, tol, ltol = TO.attend(q, ks, vs, nodes, prefix, own, D ** -0.5, sees)
    within(out[:T], want, tol, "out")
    within(lse[:T], wlse, ltol, "lse")
    if not prefix:  # (a prefix is everybody's)
        assert (out[T:] == 0).all() and (lse[T:] == -float("inf")).all()
    # the same call again: the same bits, and nothing left of the first in the workspace
    again, alse = torch.full_like(qp, 7.0), torch.full_like(lse, 7.0)
    room.forward(qp, tree=bits, out=again, lse=alse, **args)
    room.sync()
    assert torch.equal(again[:T], out[:T]) and torch.equal(alse[:T], lse[:T])
