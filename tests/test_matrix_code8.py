"""The machine code of the 8-bit forms of the experts' products, checked as that
of the bf16 ones: waits around assembly statements, and m0 for copies only.
Needs the compiler, no GPU."""
import os
import subprocess

import pytest

from combine_epx_get_amd import build
from tests.test_matrix_code import faults, functions

SOURCES = ["epx_expert_int8.hip", "epx_expert_kept8.hip"]


@pytest.mark.parametrize("source", SOURCES)
def test_waits_around_assembly_statements(source):
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-w", "--cuda-device-only", "-S", os.path.join(build.CSRC, source),
                        "-o", "-"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    kernels = copies = products = 0
    bad = {}
    for name, blocks in functions(r.stdout):
        code = [c for _, block in blocks for c in block]
        kernels += 1
        copies += sum(1 for op, _, inside in code if inside and op.startswith("buffer_"))
        products += sum(1 for op, _, inside in code if inside and op.startswith("v_mfma"))
        assert not [c for c in code if not c[2] and "m0" in c[1]], name
        early = faults(blocks)
        if early:
            bad[name] = sorted(early)[:4]
    print(f"{source}: {kernels} kernels, {copies} copies, {products} matrix instructions in statements")
    assert kernels >= 15 and copies >= 200 and products >= 100
    assert not bad, bad


def test_the_large_weight_gradient_waits_for_its_copies():
    """Its waits allow as many memory operations to be under way as loads of codes and scale bytes follow its last
    copies: at least that many have to stand between the two, or the wait would not reach the copies."""
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-w", "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, "epx_expert_kept8.hip"), "-o", "-"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    memory = ("buffer_", "global_", "flat_", "scratch_")
    checked = 0
    for name, blocks in functions(r.stdout):
        if "wgrad_kept_deep" not in name:
            continue
        for _, code in blocks:
            for at, (op, operands, inside) in enumerate(code):
                if not (inside and op == "s_waitcnt" and "vmcnt(4)" in " ".join(operands)):
                    continue
                loads = 0
                for before in reversed(code[:at]):
                    if before[0].startswith(memory):
                        if before[2]:
                            break
                        loads += 1
                assert loads >= 4, (name, at, loads)
                checked += 1
    assert checked >= 4   # before the loop and in it, for either type of result
