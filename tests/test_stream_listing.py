"""Wait states of the direct loads to LDS in the MXFP4 and expert-layer kernels, read off the compiler's listing, as for
attention's (test_attention_listing)."""

import os
import subprocess

import pytest

from test_attention_listing import LOAD, missing
from weight_only_quantized_wq_amd import build


@pytest.mark.parametrize("source", ["wq_mx_gemm.hip", "wq_moe_ffn.hip"])
def test_direct_loads_have_their_wait_states(tmp_path, source):
    src = os.path.join(build.HERE, "csrc", source)
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
    assert len(loads) >= 200
    assert [w for w in (missing(lines, i) for i in loads) if w] == []
    # nothing that the kernels keep in registers between their loads is spilled
    assert not [t for t in lines if t.startswith("scratch_")]
