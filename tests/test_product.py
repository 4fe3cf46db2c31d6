"""The products' cuts (host arithmetic) and their compiled inner loops (CPU only: hipcc
cross-compiles to gfx950 assembly)."""
import os
import re
import subprocess

import pytest

from conftest import ROOT
from test_isa_guards import _device_asm, _load

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "zero_sharded_mixed_bucketed_amd", "csrc")

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")


def test_cuts_fit_the_grid_and_the_workspace_for_every_count(tmp_path):
    exe = str(tmp_path / "product_plan_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip",
                        os.path.join(ROOT, "tests", "native", "product_plan_check.cpp"),
                        "-Wl,--unresolved-symbols=ignore-all", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "product plan check ok" in r.stdout, r.stdout[-2000:]


WAITS = {"ring": "vmcnt(0) lgkmcnt(0)", "slim": "vmcnt(10) lgkmcnt(0)"}   # as written


def _kernels(asm):
    """(kind, symbol, code from the loop's own wait, or its first matrix instruction, to its
    last) of the products that stage their operands without registers between."""
    for m in re.finditer(r"^(_ZN4zero3act\d+(ring|slim)_kernel\S+):", asm, re.M):
        body = asm[m.end():asm.index(".Lfunc_end", m.end())]
        first = min(body.index("s_waitcnt " + WAITS[m.group(2)]), body.index("v_mfma"))
        yield m.group(2), m.group(1), body[first:body.rindex("v_mfma") + 6]


@pytest.mark.slow
@pytest.mark.parametrize("name", ["gated_ffn.hip", "vocab_loss.hip"])
def test_loads_to_shared_memory_are_waited_for_once_a_stage(name, tmp_path):
    """A wait for memory that the compiler puts into the inner loop (for a load of its own, or
    registers that it keeps in scratch memory) would hold up the stages under way: the loop
    holds the kernel's own wait only, and the kernels use no scratch memory."""
    zb = _load("zero_sharded_mixed_bucketed_amd/_build.py")
    asm = _device_asm(os.path.join(CSRC, name), zb.HIP_FLAGS, [os.path.join(ROOT, "include"), CSRC],
                      str(tmp_path / "k.s"))
    seen = set()
    for kind, symbol, loop in _kernels(asm):
        seen.add(kind)
        waits = [w.strip() for w in re.findall(r"s_waitcnt ([^\n;]*vmcnt\(\d+\)[^\n;]*)", loop)]
        # the block with the own wait may stand behind the matrix instructions
        assert waits in ([WAITS[kind]], []), symbol
        assert len(re.findall("v_mfma", loop)) == (64 if kind == "ring" else 4), symbol
        assert "scratch" not in loop and "global_load" not in loop, symbol
        size = re.search(re.escape(symbol) + r"\.private_seg_size, (\d+)", asm)
        assert size and int(size.group(1)) == 0, symbol
    assert seen == {"ring", "slim"}
