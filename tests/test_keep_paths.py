"""keep's paths as rows of a wider array, without a GPU: the wrapper hands over
a row's width and its stride apart, so that no word beside the rows is taken
for a node or read behind the array. Tensors and library are stand-ins."""
import pytest

pytest.importorskip("torch")

from test_attention_wrapper import B, ints
from test_tree_wrapper import attn  # noqa: F401


@pytest.fixture
def keep(attn):  # noqa: F811
    attn._lib.moe_attn_keep_strided = lambda *args: attn.calls.append(("moe_attn_keep_strided", args)) or 0

    def call(path, counts):
        attn.keep(path, counts, q_offsets=ints(counts.shape[0] + 1), seq_lens=ints(counts.shape[0]), max_seq_len=32,
                  block_table=ints(counts.shape[0], 2))
        return attn.calls.pop()

    return call


def columns(rows, width, lo, hi):
    t = ints(rows, width)
    t._on_cpu = t._on_cpu[:, lo:hi]
    return t


@pytest.mark.parametrize("width,lo,hi", [(64, 3, 7), (5, 1, 5), (5, 0, 4), (9, 8, 9)])
def test_a_slice_of_columns_hands_over_its_width(keep, width, lo, hi):
    path = columns(B, width, lo, hi)
    name, args = keep(path, ints(B))
    assert name == "moe_attn_keep_strided"
    assert args[8:11] == (path.data_ptr(), width, hi - lo) and args[12] == 7


def test_whole_rows_and_one_row(keep):
    assert keep(ints(B, 4), ints(B))[1][8:10][1] == 4
    name, args = keep(columns(1, 9, 2, 5), ints(1))  # (a single row has no stride)
    assert name == "moe_attn_keep" and args[9] == 3
