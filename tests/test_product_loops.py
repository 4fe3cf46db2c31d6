"""The compiled inner loops of the products that stage their operands in shared memory
without registers between (CPU only: hipcc cross-compiles to gfx950 assembly), taken by
their control flow: the natural loop around the matrix instructions, in whatever order
the compiler places its blocks."""
import os
import re

import pytest

from conftest import ROOT
from test_isa_guards import _device_asm, _load

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "zero_sharded_mixed_bucketed_amd", "csrc")

# of a turn of the loop: the wait as written, matrix instructions, loads to shared memory
TURN = {"ring": ("vmcnt(0) lgkmcnt(0)", 64, 16), "slim": ("vmcnt(10) lgkmcnt(0)", 4, 5)}


def _blocks(body):
    """({label: code}, {label: successors}) of a function's assembly; blocks run from label
    to label, and one that does not end in a jump goes on in the next."""
    parts = re.split(r"^(\.LBB\d+_\d+):.*$", body, flags=re.M)
    labels = ["entry"] + parts[1::2]
    code = dict(zip(labels, [parts[0]] + parts[2::2]))
    after = {}
    for label, nxt in zip(labels, labels[1:] + [None]):
        ops = [line.split(";")[0].strip() for line in code[label].splitlines()]
        ops = [op for op in ops if op and not op.startswith(".")]
        to = {op.split()[1] for op in ops if re.match(r"s_c?branch", op)}
        if nxt and not (ops and re.match(r"s_branch|s_endpgm|s_setpc", ops[-1])):
            to.add(nxt)
        after[label] = to & set(labels)
    return code, after


def _loops(after):
    """The natural loops: of each jump back to a block that every way to the jump passes,
    all blocks that reach the jump without passing that block."""
    doms = {b: set(after) for b in after}
    doms["entry"] = {"entry"}
    before = {b: {a for a in after if b in after[a]} for b in after}
    change = True
    while change:
        change = False
        for b in after:
            if b == "entry" or not before[b]:
                continue
            new = {b} | set.intersection(*(doms[a] for a in before[b]))
            if new != doms[b]:
                doms[b], change = new, True
    for a in after:
        for head in after[a] & doms[a]:
            loop, todo = {head}, [a]
            while todo:
                b = todo.pop()
                if b not in loop:
                    loop.add(b)
                    todo += before[b]
            yield head, loop


def _inner_loop(body):
    """The code of the smallest loop that holds all of its matrix instructions' blocks."""
    code, after = _blocks(body)
    mul = {b for b in code if "v_mfma" in code[b]}
    merged = {}
    for head, loop in _loops(after):               # two jumps to one block: one loop
        merged[head] = merged.get(head, set()) | loop
    loops = [loop for loop in merged.values() if mul <= loop]
    assert mul and loops, "no loop around the matrix instructions"
    return "\n".join(code[b] for b in code if b in min(loops, key=len))


def faults(kind, loop):
    """What a turn of the loop holds beside what it should."""
    wait, mfma, loads = TURN[kind]
    found = []
    waits = [w.strip() for w in re.findall(r"s_waitcnt ([^\n;]*vmcnt\(\d+\)[^\n;]*)", loop)]
    if waits != [wait]:
        found.append(f"waits {waits}")
    if loop.count("v_mfma") != mfma:
        found.append(f"{loop.count('v_mfma')} matrix instructions")
    memory = re.findall(r"^\s*((?:buffer|global|flat|scratch)_\w+)[^\n]*?(\blds)?\s*$", loop, re.M)
    if sorted(memory) != [("buffer_load_dwordx4", "lds")] * loads:
        found.append(f"memory {sorted(memory)}")
    if len(re.findall(r"^\s*s_barrier", loop, re.M)) != 1:
        found.append("not one barrier")
    return found


def _compiled(name, out):
    zb = _load("zero_sharded_mixed_bucketed_amd/_build.py")
    asm = _device_asm(os.path.join(CSRC, name), zb.HIP_FLAGS, [os.path.join(ROOT, "include"), CSRC],
                      out)
    for m in re.finditer(r"^(_ZN4zero3act\d+(ring|slim)_kernel\S+):", asm, re.M):
        yield m.group(2), m.group(1), asm[m.end():asm.index(".Lfunc_end", m.end())]


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
@pytest.mark.parametrize("name,kernels", [("gated_ffn.hip", (6, 4)), ("vocab_loss.hip", (6, 4))])
def test_the_loop_holds_its_own_wait_and_loads_and_nothing_else(name, kernels, tmp_path):
    seen = []
    for kind, symbol, body in _compiled(name, str(tmp_path / "k.s")):
        seen.append(kind)
        assert faults(kind, _inner_loop(body)) == [], symbol
    assert (seen.count("ring"), seen.count("slim")) == kernels


LOOP = """
\ts_mov_b32 s0, 0
.LBB0_1:                                ; the loads, placed before the loop's head
\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds
\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds
\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds
\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds
\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds
\ts_cbranch_scc1 .LBB0_4
.LBB0_2:
\ts_waitcnt lgkmcnt(0)
\tv_mfma_f32_32x32x16_f16 a[0:15], v[0:3], v[4:7], a[0:15]
\tv_mfma_f32_32x32x16_f16 a[0:15], v[0:3], v[4:7], a[0:15]
\tv_mfma_f32_32x32x16_f16 a[0:15], v[0:3], v[4:7], a[0:15]
\tv_mfma_f32_32x32x16_f16 a[0:15], v[0:3], v[4:7], a[0:15]
\ts_cbranch_scc0 .LBB0_5
.LBB0_3:                                ; behind the matrix instructions
\ts_waitcnt vmcnt(10) lgkmcnt(0)
\ts_barrier
\ts_branch .LBB0_1
.LBB0_4:
\tv_mov_b32_e32 v1, 0
\ts_branch .LBB0_2
.LBB0_5:
\ts_waitcnt vmcnt(0)
\tglobal_store_dwordx4 v[0:1], v[2:5], off
\ts_endpgm
"""


def test_a_planted_wait_or_load_anywhere_in_the_loop_is_seen():
    assert faults("slim", _inner_loop(LOOP)) == []
    for at, what in (("\ts_cbranch_scc1", "\ts_waitcnt vmcnt(0)\n"),
                     ("\ts_cbranch_scc0", "\tglobal_load_dwordx4 v[2:5], v[0:1], off\n"),
                     ("\ts_barrier", "\ts_waitcnt vmcnt(3)\n"),
                     ("\tv_mov_b32", "\tscratch_load_dword v1, off, off\n"),
                     ("\tv_mov_b32", "\ts_waitcnt vmcnt(0)\n"), ("\tv_mov_b32", "\ts_barrier\n")):
        assert faults("slim", _inner_loop(LOOP.replace(at, what + at, 1))) != [], what
    for gone in ("\ts_waitcnt vmcnt(10) lgkmcnt(0)\n",
                 "\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds\n"):
        assert faults("slim", _inner_loop(LOOP.replace(gone, "", 1))) != [], gone
