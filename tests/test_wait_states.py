"""Memory instructions written in assembly, in the code that the compiler makes of
them: it pads its own instructions, but does not see into assembly (no GPU needed).

gfx9 needs five wait states between a vector instruction that writes a scalar register
and a memory instruction that reads it, and one between a scalar write of m0 and a load
into LDS.  An instruction is one, s_nop N makes N + 1."""
import os
import re
import subprocess

import pytest

from nvfp4_w4a16_mtp_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")

SOURCES = [s for s in build.SOURCES
           if re.search(r'asm\s+volatile\([^;]*(global|buffer|flat)_(load|store)', open(os.path.join(build.CSRC, s)).read())]


def scalars(operand):
    """Scalar registers of an operand."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.fullmatch(r"s\d+|vcc|m0", operand) else set()


def too_early(lines):
    """(line number, text) of memory instructions that come too soon, reading the lines in order."""
    now, valu, m0, bad = 0, {}, -9, []
    for at, line in enumerate(lines, 1):
        text = line.split(";")[0].strip()
        if not text or text.startswith(".") or text.endswith(":"):
            continue
        op, _, rest = text.partition(" ")
        args = [x.strip() for x in rest.split(",")]
        if op == "s_nop":
            now += int(args[0], 0) + 1
            continue
        if op.startswith(("global_", "buffer_", "flat_", "scratch_")):
            read = set().union(*(scalars(y) for x in args for y in x.split()))
            if any(now - valu.get(r, -9) < 6 for r in read) or ("_lds_" in op and now - m0 < 2):
                bad.append((at, text))
        elif op.startswith("v_"):
            wide = "_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64"))
            for x in args[:2 if wide else 1]:
                valu.update({r: now for r in scalars(x)})
        elif op.startswith("s_") and args[0] == "m0":
            m0 = now
        now += 1
    return bad


def test_the_reading_of_listings():
    def run(*lines):
        return [n for n, _ in too_early(lines)]
    base = "\tv_readfirstlane_b32 s5, v1"
    load = "\tglobal_load_lds_dwordx4 v2, s[4:5]"
    m0 = "\ts_mov_b32 m0, s9"
    assert run(base, m0, "\ts_nop 0", load) == [4]
    assert run(base, m0, "\ts_nop 2", load) == [4]
    assert run(base, m0, "\ts_nop 3", load) == []
    assert run("\tv_readlane_b32 s6, v1, 3", m0, "\ts_nop 0", load) == []
    assert run("\tv_cmp_lt_u32_e64 s[4:5], v1, v2", *["\ts_add_i32 s8, s8, 1"] * 4, "\tglobal_load_dword v1, v2, s[4:5] offset:16") == [6]
    assert run("\tv_add_co_u32_e64 v1, s[2:3], v2, v3", "; note", ".LBB0_1:", "\tbuffer_load_dword v1, v2, s[0:3], s3 offen") == [4]
    assert run("\ts_add_u32 s4, s4, s2", m0, load) == [3] and run("\ts_add_u32 s4, s4, s2", m0, "\ts_nop 0", load) == []


def test_a_source_is_found():
    assert "prompt_attn.hip" in SOURCES


@pytest.mark.parametrize("source", SOURCES)
def test_wait_states(source, tmp_path):
    out = str(tmp_path / "out.s")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = open(out).read().splitlines()
    assert sum("_lds_dwordx4" in x for x in lines) > 0
    bad = too_early(lines)
    assert not bad, (len(bad), bad[:5])
