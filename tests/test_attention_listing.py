"""Wait states of attention's direct loads to LDS, read off the compiler's listing of the kernels.

The loads stand in inline assembly, where the compiler places no wait states of its own.  A vector-memory instruction
that reads a scalar register needs five of them behind a vector instruction that wrote it, and a direct load one behind
a write of m0; scalar writes are interlocked otherwise.
"""

import os
import re
import subprocess

import pytest

from weight_only_quantized_wq_amd import build

LOAD = "global_load_lds"


def scalars(text):
    out = set()
    for a, b, c, d in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(m0)\b", text):
        out |= {"m0"} if d else {int(c)} if c else set(range(int(a), int(b) + 1))
    return out


def missing(lines, at):
    """Why the load at lines[at] may come too early, or None.  Looks back through the text, over labels too."""
    need, waits, m0 = scalars(lines[at][len(LOAD):]) | {"m0"}, 0, False
    for text in reversed(lines[max(0, at - 40):at]):
        op = text.split()[0]
        wrote = scalars(text[len(op):].split(",")[0]) & need
        if op.startswith("v_") and wrote and waits < 5:
            return f"{text} with {waits} wait states before {lines[at]}"
        if op.startswith("s_") and "m0" in wrote:
            if waits < 1:
                return f"{text} right before {lines[at]}"
            m0 = True
        if op.startswith(("v_", "s_")):
            need -= wrote
        waits += int(text.split()[1]) + 1 if op == "s_nop" else 1
        if m0 and (waits >= 5 or not need):
            return None
    return None if m0 or waits >= 5 else f"no write of m0 found before {lines[at]}"


def test_the_check_sees_what_it_is_for():
    good = ["s_add_u32 s4, s2, s8", "s_mov_b32 m0, s9", "s_nop 0", f"{LOAD}_dwordx4 v1, s[4:5]"]
    assert missing(good, 3) is None
    assert missing(good[:2] + good[3:], 2)
    assert missing(["s_nop 7", "v_readfirstlane_b32 s5, v2"] + good[1:], 4)
    assert missing(["v_readfirstlane_b32 s5, v2", "s_nop 1"] + good[1:], 4)
    assert missing(["v_readfirstlane_b32 s5, v2", "s_nop 2"] + good[1:], 4) is None
    assert missing(["v_readfirstlane_b32 s4, v2"] + good, 4) is None
    assert missing(["v_readlane_b32 m0, v2, 3", "s_nop 0", f"{LOAD}_dword v[2:3], off"], 2)


def test_direct_loads_have_their_wait_states(tmp_path):
    src = os.path.join(build.HERE, "csrc", "wq_tree_attention.hip")
    out = str(tmp_path / "listing.s")
    try:
        cmd = build.compile_command(src, out)
    except RuntimeError:
        pytest.skip("hipcc is not here")
    cmd[cmd.index("-c")] = "-S"
    subprocess.run(cmd[:1] + ["--cuda-device-only"] + cmd[1:], check=True, capture_output=True, text=True)
    with open(out) as f:
        lines = [t for t in (x.split(";")[0].strip() for x in f) if t and not t.startswith(".") and not t.endswith(":")]
    loads = [i for i, t in enumerate(lines) if t.startswith(LOAD)]
    assert len(loads) >= 200          # 17 kernels, each with the loads of its ring
    assert [w for w in (missing(lines, i) for i in loads) if w] == []
