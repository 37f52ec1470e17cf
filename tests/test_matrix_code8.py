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
