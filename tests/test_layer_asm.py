"""What the layer's hand-written assembly takes for granted about the code around
it, checked on the compiler's listing."""
import os
import re
import shutil
import subprocess

import pytest

from combine_routing_histogram_amd import build as hip_build

# instructions that read or write M0 without naming it
IMPLICIT = re.compile(r"movrel|sendmsg|gws|ttrace|\bs_cmovrel")


def foreign_m0(listing):
    """Lines outside asm blocks that use M0."""
    inside, found = False, []
    for line in listing.splitlines():
        if "ASMSTART" in line:
            inside = True
        elif "ASMEND" in line:
            inside = False
        elif not inside:
            code = line.split(";")[0]
            if re.search(r"\bm0\b", code) or IMPLICIT.search(code):
                found.append(line.strip())
    return found


def test_finder():
    block = ";;#ASMSTART\n\ts_mov_b32 m0, s1\n\t;;#ASMEND\n"
    assert foreign_m0(block + "\tv_mov_b32_e32 v0, v1 ; m0\n") == []
    assert foreign_m0(block + "\ts_mov_b32 m0, s1\n") == ["s_mov_b32 m0, s1"]
    assert foreign_m0("\ts_movrels_b32 s0, s1\n") == ["s_movrels_b32 s0, s1"]


def test_compiler_leaves_m0_alone(tmp_path):
    """load_direct sets M0 in its asm block, which cannot be declared."""
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    out = str(tmp_path / "layer.s")
    cmd = [a for a in hip_build.hipcc_command(out, hip_build.LAYER_SRC)
           if a not in ("-shared", "-fPIC")] + ["--cuda-device-only", "-S"]
    subprocess.run(cmd, check=True, capture_output=True)
    text = open(out).read()
    assert "m0" in text and os.path.getsize(out) > 1 << 20
    assert foreign_m0(text) == []
