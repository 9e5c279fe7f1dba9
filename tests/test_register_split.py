"""The kernels' register splits, read from their source.

setmaxnreg is one instruction of a whole warpgroup: all its four warps have to execute the same one. So a call of
warpgroup_regs_inc / warpgroup_regs_dec may stand only behind branches on which no two warps of a warpgroup
differ: comparisons of the warp number by < and >= with multiples of four."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "block_sparse_attention_kunlun_b200", "csrc")
CALL = re.compile(r"warpgroup_regs_(?:inc|dec)<[^>]*>\(\);")
BRANCH = re.compile(r"(\}\s*)?(else\s+)?if (?:constexpr )?\((.*)\) \{$|(\}\s*)?else \{$")


def conditions(text):
    """For each call, the conditions of the branches around it and of the branches tried before those."""
    stack, last, found = [], {}, []  # stack: conditions of each open block; last: of the block closed at a depth
    for line in text.splitlines():
        code = line.split("//")[0].strip()
        if CALL.search(code):
            found.append([c for block in stack for c in block])
            continue
        m = BRANCH.match(code)
        for ch in code[:code.rfind("{")] if m else code:
            if ch == "}":
                closed = stack.pop()
                last[len(stack)] = closed
            elif ch == "{":
                stack.append([])
        if m:
            before = last.get(len(stack), []) if "else" in code.split("(")[0] else []
            stack.append(before + ([m.group(3)] if m.group(3) else []))
    assert not stack
    return found


def splits_a_warpgroup(condition):
    """Whether warps of one warpgroup may differ on a condition."""
    rest = re.sub(r"\bwarp (?:<|>=) (\d+)", lambda m: "" if int(m.group(1)) % 4 == 0 else m.group(0), condition)
    return re.search(r"\b(?:warp|lane|tid|threadIdx)\b", rest) is not None


@pytest.mark.parametrize("name", ["ba_fwd_sm100.cu", "ba_bwd_dq_sm100.cu", "ba_cache_fwd_sm100.cu"])
def test_a_warpgroup_executes_one_register_split(name):
    with open(os.path.join(CSRC, name)) as f:
        calls = conditions(f.read())
    assert len(calls) >= 2
    for c in calls:
        assert not any(splits_a_warpgroup(x) for x in c), c


def test_every_kernel_that_splits_registers_is_read():
    users = {n for n in os.listdir(CSRC) if n.endswith(".cu") and CALL.search(open(os.path.join(CSRC, n)).read())}
    assert users == {"ba_fwd_sm100.cu", "ba_bwd_dq_sm100.cu", "ba_cache_fwd_sm100.cu"}


def test_the_reading_itself():
    good = "void f() {\n if (warp < 4) {\nwarpgroup_regs_inc<A>();\n} else {\nwarpgroup_regs_dec<B>();\n}\n}"
    bad = "void f() {\n if (warp < 12) {\n} else if (warp == kCopy) {\nwarpgroup_regs_dec<B>();\n} else {\n" \
          "warpgroup_regs_dec<B>();\n}\n}"
    assert not any(splits_a_warpgroup(x) for c in conditions(good) for x in c)
    assert [any(splits_a_warpgroup(x) for x in c) for c in conditions(bad)] == [True, True]
