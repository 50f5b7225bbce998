"""Named barriers of the few-row attention kernel, read from its source: they
wait without a limit for a fixed number of threads, so no computing warp may
leave between them by itself. (Showing it on a GPU would take a kernel that
hangs.)"""
import os
import re

from w4a16_routed_expert_gb300 import build as B


def part_loop():
    """(depth, inside a for loop, statement) of each barrier, break and return
    in the computing warps' loop over the parts."""
    src = open(os.path.join(B.CSRC, "attn_rows.cu")).read()
    src = re.sub(r"//[^\n]*", "", src[src.index("bool some = next_segment(&s);"):])
    src = src[src.index("while ("):]
    found, loops, statement = [], [], ""
    for token in re.findall(r"[{};]|[^{};]+", src):
        if token == "{":
            loops.append("for (" in statement)
            statement = ""
        elif token == "}":
            loops.pop()
            statement = ""
            if not loops:
                break
        elif token == ";" and statement.count("(") == statement.count(")"):
            if re.search(r"\bbreak\b|\breturn\b|\bbar_\w+\(", statement):
                found.append((len(loops), any(loops), " ".join(statement.split())))
            statement = ""
        else:
            statement += token
    return found


def test_computing_warps_leave_together():
    found = part_loop()
    barriers = [i for i, (_, _, s) in enumerate(found) if "bar_" in s]
    assert len(barriers) >= 4 and all(found[i][0] == 1 for i in barriers)  # none under a condition
    out = [i for i, (_, nested, s) in enumerate(found) if re.search(r"\bbreak\b|\breturn\b", s) and not nested]
    # the one way out of the loop is the first barrier's, where all warps know of each other
    assert out == barriers[:1] and re.search(r"bar_any\(!ok\)", found[out[0]][2]), found
