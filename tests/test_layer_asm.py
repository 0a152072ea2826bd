"""What the layer's hand-written assembly takes for granted about the code around
it, checked on the compiler's listing."""
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


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "layer.s")
    cmd = [a for a in hip_build.hipcc_command(out, hip_build.LAYER_SRC)
           if a not in ("-shared", "-fPIC")] + ["--cuda-device-only", "-S"]
    subprocess.run(cmd, check=True, capture_output=True)
    text = open(out).read()
    assert len(text) > 1 << 20
    return text


def test_compiler_leaves_m0_alone(listing):
    """load_direct sets M0 in its asm block, which cannot be declared."""
    assert "m0" in listing
    assert foreign_m0(listing) == []


def _sgprs(text):
    found = set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        found |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return found


def short_waits(listing, states=5):
    """Loads in asm blocks that read a scalar register fewer than `states` wait
    states after a vector instruction wrote it.  An instruction is a state, s_nop n
    is n + 1; labels are passed over, so a block reached by falling through counts
    in full."""
    past, inside, found = [], False, []
    for line in listing.splitlines():
        if "ASMSTART" in line:
            inside = True
        elif "ASMEND" in line:
            inside = False
        code = line.split(";")[0].strip()
        if not code or code.startswith(".") or code.endswith(":"):
            continue
        op, _, args = code.partition(" ")
        if inside and op.startswith(("buffer_", "global_")):
            read, waited = _sgprs(args), 0
            for p, pargs in reversed(past):
                if waited >= states:
                    break
                if p.startswith("v_") and _sgprs(pargs.split(",")[0]) & read:
                    found.append(f"{p} {pargs} -> {code}")
                waited += int(pargs) + 1 if p == "s_nop" else 1
        past.append((op, args.strip()))
        del past[:-16]
    return found


def test_wait_finder():
    load = ";;#ASMSTART\n{}\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n;;#ASMEND\n"
    write = "\tv_readfirstlane_b32 s6, v2\n"
    assert short_waits(write + load.format("")) and short_waits(write + load.format("\ts_nop 3\n"))
    assert not short_waits(write + load.format("\ts_nop 4\n"))
    assert short_waits(write + "\ts_mov_b32 s9, s8\n" * 2 + load.format("\ts_nop 1\n"))
    assert not short_waits("\tv_readfirstlane_b32 s8, v2\n" + load.format(""))
    assert not short_waits("\ts_mov_b32 s6, s8\n" + load.format(""))


def test_direct_loads_wait_for_their_descriptor(listing):
    """A memory instruction may read a scalar register five wait states after a
    vector instruction wrote it at the earliest.  Nothing in the hardware sees to
    it, and the compiler does not look into asm blocks."""
    assert short_waits(listing) == []
