"""Wait states around the direct-to-LDS copies of the built library.

The copies are inline assembly, whose operands the compiler's hazard pass does
not look into, so the instructions around them are read back from the
disassembly. On gfx950 two distances have to be kept:

  a write of m0, then a copy that places its data by m0:  1 wait state
  a VALU write of an SGPR, then a memory operation reading it:  5 wait states"""
import os
import re
import shutil
import subprocess

import pytest

from moe_expert_ffn_persistent_amd import _lib

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")) if p and os.path.exists(p)), None)
MEMORY = ("global_", "buffer_", "flat_", "scratch_")


def sgprs(args):
    out = set()
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", args):
        out |= set(range(int(lo), int(hi) + 1))
    return out | {int(r) for r in re.findall(r"\bs(\d+)\b", args)}


def hazards(lines):
    """(rule, instruction, states between) of every distance that is too short,
    and the number of copies seen. An instruction is a state, s_nop n is n + 1."""
    found, copies = [], 0
    now, m0, written = 0, None, {}   # states so far; when m0 was last written, and each SGPR by a VALU
    for line in lines:
        if line.rstrip().endswith(">:"):   # another function
            m0, written = None, {}
            continue
        m = re.match(r"\s+([a-z]\w+)\s*(.*?)\s*(//.*)?$", line)
        if not m:
            continue
        op, args = m[1], m[2]
        first = args.split(",")[0]
        if op.startswith(MEMORY):
            if "_lds_" in op or re.search(r"\blds\b", args):
                copies += 1
                if m0 is not None and now - m0 < 1:
                    found.append(("m0", line.strip(), now - m0))
            for r in sgprs(args) & set(written):
                if now - written[r] < 5:
                    found.append(("sgpr", line.strip(), now - written[r]))
        now += 1 + (int(args.split()[0], 0) if op == "s_nop" else 0)
        if op.startswith("v_"):
            written.update({r: now for r in sgprs(first)})
        elif op.startswith("s_") and not op.startswith(("s_nop", "s_cmp", "s_bitcmp")):
            for r in sgprs(first):
                written.pop(r, None)
        if first.strip() == "m0" and not op.startswith(MEMORY):
            m0 = now
    return found, copies


def test_the_reader_counts_wait_states():
    near = ["\ts_mov_b32 m0, s35   // 0: BEFC0023", "\tglobal_load_lds_dwordx4 v1, s[60:61]   // 4: DDF48000 003C00AA"]
    assert [f[0] for f in hazards(near)[0]] == ["m0"]
    assert hazards([near[0], "\ts_nop 0", near[1]]) == ([], 1)
    assert hazards([near[0], "\tv_add_u32_e32 v1, v2, v3", near[1]]) == ([], 1)
    lane = "\tv_readfirstlane_b32 s61, v9"
    assert [f[::2] for f in hazards([lane, "\ts_nop 3", near[1]])[0]] == [("sgpr", 4)]
    assert hazards([lane, "\ts_nop 4", near[1]]) == ([], 1)
    assert hazards([lane, "\ts_mov_b32 s61, 0", near[1]]) == ([], 1)
    assert hazards([lane, "\ts_cmp_lt_i32 s61, 4", near[1]])[0]
    assert hazards(["0000 <a>:", *near[:1], "0000 <b>:", near[1]]) == ([], 1)


def test_copies_keep_their_wait_states(tmp_path):
    if not os.path.exists(_lib.LIB_PATH) or OBJDUMP is None:
        pytest.skip("libmoe_ffn.so not built, or no llvm-objdump")
    shutil.copy(_lib.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    total = 0
    for code in sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950")):
        r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", code], cwd=tmp_path, check=True, capture_output=True, text=True)
        found, copies = hazards(r.stdout.splitlines())
        assert not found, f"{code}: {len(found)} of {copies} copies and other memory operations too early, first {found[0]}"
        total += copies
    assert total > 1000
