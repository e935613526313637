"""Wait states in the device code of the built library, without a GPU.

On gfx950 a vector memory instruction may read a scalar register no sooner
than five wait states after a vector instruction wrote it (v_readfirstlane,
v_readlane, a comparison): sooner it may see the register's old value, here
an old offset or half of an old buffer descriptor. The compiler keeps this
distance for the instructions that it knows, but does not look into inline
assembly. Each instruction is one wait state, s_nop N is N + 1.

The gfx950 code objects are taken from the library and disassembled, and
every path through every kernel is followed."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_amd import binding as B
from combine_topk_ids_dest_amd import build as hip_build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
NEED = 5

_LINE = re.compile(r"^\s+(\S+)\s*(.*?)\s*//\s*([0-9A-F]{12,16}):[^<]*(?:<([^+>]+)(?:\+0x([0-9a-f]+))?>)?")
_SYMBOL = re.compile(r"^([0-9a-f]{16}) <(.+)>:$")
_SGPR = re.compile(r"(?<![\w.])(?:s(\d+)|s\[(\d+):(\d+)\]|(vcc_lo|vcc_hi|vcc|m0))(?![\w\[])")
# vector instructions whose second operand is a scalar result (a carry, a flag)
_CARRY = re.compile(r"^v_(add|sub|subrev|addc|subb|subbrev)_co_|^v_div_scale_|^v_mad_(u64_u32|i64_i32)")
_SCALAR_NO_RESULT = re.compile(
    r"^s_(cmp|bitcmp|branch|cbranch|nop|waitcnt|barrier|endpgm|set|sleep|icache|dcache|trap|sendmsg|code_end)")
_MEMORY = re.compile(r"^(buffer|tbuffer|global|flat|scratch|image)_")


def _registers(text):
    found = set()
    for one, lo, hi, name in _SGPR.findall(text):
        if one:
            found.add(int(one))
        elif lo:
            found.update(range(int(lo), int(hi) + 1))
        else:
            found.update({"vcc": ("vcc_lo", "vcc_hi")}.get(name, (name,)))
    return found


def _operands(text):
    return [o.strip() for o in text.split(",")] if text else []


def _parse(listing):
    """[(address, mnemonic, operands as text, branch target or None)]"""
    starts, code = {}, []
    for line in listing.splitlines():
        s = _SYMBOL.match(line)
        if s:
            starts[s.group(2)] = int(s.group(1), 16)
            continue
        m = _LINE.match(line)
        if m:
            target = None
            if m.group(1).startswith(("s_branch", "s_cbranch")):
                target = (m.group(4), int(m.group(5) or "0", 16))
            code.append((int(m.group(3), 16), m.group(1), m.group(2), target))
    return [(a, op, text, None if t is None else starts[t[0]] + t[1]) for a, op, text, t in code]


def _effect(op, text):
    """(registers a scalar instruction writes, a vector instruction writes, a
    memory instruction reads, wait states) of one instruction."""
    ops = _operands(text)
    if op == "s_nop":
        return set(), set(), set(), int(text, 0) + 1
    if op.startswith("v_"):
        writes = _registers(ops[0]) if ops else set()
        if _CARRY.match(op) and len(ops) > 1:
            writes |= _registers(ops[1])
        return set(), writes, set(), 1
    if _MEMORY.match(op):
        return set(), set(), _registers(text), 1
    if op.startswith("s_") and ops and not _SCALAR_NO_RESULT.match(op):
        return _registers(ops[0]), set(), set(), 1
    return set(), set(), set(), 1


def too_early(listing):
    """The memory instructions that, on some path, read a scalar register fewer
    than NEED wait states behind a vector instruction's write of it."""
    code = _parse(listing)
    at = {c[0]: i for i, c in enumerate(code)}
    info = [_effect(op, text) for _, op, text, _ in code]
    ends = {i for i, c in enumerate(code) if c[1] in ("s_endpgm", "s_branch", "s_setpc_b64")}
    first = {0} | {at[c[3]] for c in code if c[3] is not None} | \
            {i + 1 for i, c in enumerate(code) if i in ends or c[3] is not None}
    # by block: wait states since the nearest write of each register, over all ways into it
    entry = {i: {} for i in first if i < len(code)}
    work, bad = list(entry), {}
    while work:
        i = work.pop()
        state = dict(entry[i])
        while True:
            kills, writes, reads, states = info[i]
            early = sorted(str(r) for r in reads if r in state)
            if early:
                bad[i] = f"{code[i][0]:x}: {code[i][1]} {code[i][2]} ({', '.join(early)})"
            state = {r: d + states for r, d in state.items()
                     if r not in kills and d + states < NEED}
            state.update((r, 0) for r in writes)
            target = code[i][3]
            into = [] if target is None else [at[target]]
            if i not in ends and i + 1 < len(code) and (into or i + 1 in first):
                into.append(i + 1)
            for j in into:
                new = dict(entry[j])
                for r, d in state.items():
                    new[r] = min(d, new.get(r, NEED))
                if new != entry[j]:
                    entry[j] = new
                    work.append(j)
            i += 1
            if i - 1 in ends or i in first or i >= len(code):
                break
    return [bad[i] for i in sorted(bad)]


def _snippet(*lines):
    text = "0000000000000000 <k>:\n"
    for n, line in enumerate(lines):
        text += f"\t{line:<58} // {4 * n:012X}: 00000000"
        m = re.match(r"s_c?branch\w* ([0-9]+)$", line)
        text += f" <k+0x{4 * int(m.group(1)):x}>\n" if m else "\n"
    return text


LOAD = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"


@pytest.mark.parametrize("lines,found", [
    (["v_readlane_b32 s9, v0, 3", "s_mov_b32 m0, s2", "s_nop 0", LOAD, "s_endpgm"], 1),
    (["v_readlane_b32 s9, v0, 3", "s_mov_b32 m0, s2", "s_nop 2", LOAD, "s_endpgm"], 1),
    (["v_readlane_b32 s9, v0, 3", "s_mov_b32 m0, s2", "s_nop 3", LOAD, "s_endpgm"], 0),
    (["v_readfirstlane_b32 s6, v0", LOAD, "s_endpgm"], 1),
    (["v_readfirstlane_b32 s8, v0", LOAD, "s_endpgm"], 0),
    (["v_readfirstlane_b32 s6, v0", "s_mov_b32 s6, s2", LOAD, "s_endpgm"], 0),
    (["v_cmp_gt_i32_e64 s[8:9], s4, v7", "s_nop 1", LOAD, "s_endpgm"], 1),
    (["v_add_co_u32_e64 v1, s[8:9], v2, v3", LOAD, "s_endpgm"], 1),
    (["v_add_u32_e32 v1, s9, v2", LOAD, "s_endpgm"], 0),
    # over a branch: one of the two ways is too short
    (["v_readlane_b32 s9, v0, 3", "s_cbranch_scc1 3", "s_nop 4", LOAD, "s_endpgm"], 1),
    (["s_cbranch_scc1 2", "s_endpgm", "s_nop 1", LOAD, "v_readlane_b32 s9, v0, 3", "s_branch 2"], 1),
    (["s_cbranch_scc1 2", "s_endpgm", "s_nop 3", LOAD, "v_readlane_b32 s9, v0, 3", "s_branch 2"], 0),
])
def test_the_check_itself(lines, found):
    assert len(too_early(_snippet(*lines))) == found


def test_no_load_reads_a_scalar_register_too_early(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    if not os.path.exists(B.LIB_PATH):
        hip_build.build()
    lib = str(tmp_path / "lib.so")
    shutil.copy(B.LIB_PATH, lib)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    objects = sorted(glob.glob(lib + ".*gfx950*"))
    assert objects
    loads_to_lds, bad = 0, []
    for path in objects:
        listing = subprocess.run([OBJDUMP, "-d", path], check=True, capture_output=True,
                                 text=True).stdout
        loads_to_lds += listing.count("offen lds")
        bad += too_early(listing)
    assert loads_to_lds > 0                      # the products' loads were seen
    assert not bad, f"{len(bad)} loads, among them {bad[:5]}"
