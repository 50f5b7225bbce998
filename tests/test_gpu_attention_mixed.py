"""A prompt chunk beside sequences that decode one token each, as a server's
batches are: the same call serves rows by the thousand and rows by the few."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attention_oracle as AO  # noqa: E402
from test_gpu_attention import BF16, F16, _cuda, build, within  # noqa: E402,F401

MIXED = {  # dtype, Hq, Hk, D, page, order, tokens of the chunk, its own keys, other sequences, prefix, causal
    "rows fill a block of each sequence on average": (F16, 8, 1, 64, 64, "slot", 2048, 2048, 63, 700, True),
    "one sequence fewer rows than that": (BF16, 8, 1, 64, 16, "head", 1900, 1900, 63, 700, True),
    "heads of 128": (BF16, 16, 2, 128, 16, "slot", 1100, 1300, 30, 333, True),
    "heads of 96, no causality": (F16, 8, 2, 96, 48, "head", 300, 900, 11, 1000, False),
    "no prefix": (F16, 8, 2, 128, 32, "slot", 700, 700, 40, 0, True),
    "the chunk's keys are the prefix": (BF16, 4, 4, 72, 16, "slot", 500, 0, 20, 900, True),
}


@pytest.mark.parametrize("where", ["first", "last", "between"])
@pytest.mark.parametrize("name", MIXED)
def test_a_chunk_beside_decoding_sequences(name, where):
    dtype, Hq, Hk, D, page, order, tokens, keys, others, prefix, causal = MIXED[name]
    at = {"first": 0, "last": others, "between": others // 3}[where]
    q_lens = [1] * at + [tokens] + [1] * (others - at)
    own = [(37 * i) % 90 for i in range(at)] + [keys] + [(53 * i) % 150 for i in range(others - at)]
    a, q, ks, vs, args = build(dtype, Hq, Hk, D, page, order, q_lens, own, prefix, seed=len(name))
    out, lse = a.forward(q.cuda(), causal=causal, return_lse=True, **args)
    a.sync()
    want, wlse, tol, ltol = AO.attend(q, ks, vs, q_lens, prefix, own, D ** -0.5, causal)
    within(out, want, tol, "out")
    within(lse, wlse, ltol, "lse")
    assert torch.equal(a.forward(q.cuda(), causal=causal, **args), out)
