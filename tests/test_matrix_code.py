"""The machine code of the experts' products, as built from these sources.

Their copies to LDS and some of their matrix instructions are written as
assembly statements, whose operands the compiler does not time. What it puts
around them is checked here, on the assembly of the two sources, for the waits
of gfx950: 5 between a vector instruction that writes a scalar register and a
memory instruction that reads it, 2 between one that writes a vector register
and a matrix instruction that reads it, and up to 19 between a matrix
instruction and any other use of its result (16 passes; a wait is one
instruction, or n + 1 for "s_nop n"). The copies also set m0, which a statement
cannot name among what it changes: nothing else may use it. Needs the
compiler, no GPU."""
import os
import re
import subprocess

import pytest

from combine_epx_get_amd import build

SOURCES = ["epx_expert_gemm.hip", "epx_expert_mxfp4.hip"]
SCALAR_TO_MEMORY, VECTOR_TO_MATRIX, MATRIX_TO_USE = 5, 2, 19


def registers(operand):
    found = []
    for kind, lo, hi, one in re.findall(r"\b([sva])(?:\[(\d+):(\d+)\]|(\d+)\b)", operand):
        found += [kind + str(n) for n in (range(int(lo), int(hi) + 1) if lo else [int(one)])]
    return found


def operands(text):
    """Operands split at the commas outside brackets."""
    return [o.strip() for o in re.split(r",(?![^\[]*\])", text)] if text else []


def functions(text):
    """(name, blocks): blocks are (label, instructions), an instruction (opcode, operands, its statement's number or 0)."""
    name, blocks, statement, inside = None, [], 0, False
    for line in text.splitlines():
        if "#ASMSTART" in line:
            statement, inside = statement + 1, True
        elif "#ASMEND" in line:
            inside = False
        elif re.match(r"_Z\w+:", line):
            name, blocks = line.split(":")[0], [("entry", [])]
        elif name and re.match(r"(\.LBB\w+|; %bb\.\d+):", line):
            blocks.append((line.split(":")[0], []))
        elif name and line.startswith(".Lfunc_end"):
            yield name, blocks
            name = None
        elif name:
            code = line.split(";")[0].strip()
            if code and not code.startswith("."):
                op, _, rest = code.partition(" ") if " " in code else code.partition("\t")
                blocks[-1][1].append((op.strip(), operands(rest.strip()), statement if inside else 0))


def edges(blocks):
    after = []
    for i, (_, code) in enumerate(blocks):
        to = {o[0] for op, o, inside in code if not inside and (op == "s_branch" or op.startswith("s_cbranch"))}
        if not (code and code[-1][0] in ("s_branch", "s_endpgm")) and i + 1 < len(blocks):
            to.add(blocks[i + 1][0])
        after.append(to)
    index = {label: i for i, (label, _) in enumerate(blocks)}
    return [sorted(index[t] for t in to if t in index) for to in after]


def loops(succ):
    """The number of each block's strongly connected component (blocks reachable from each other)."""
    n = len(succ)
    pred = [[] for _ in range(n)]
    for i, to in enumerate(succ):
        for t in to:
            pred[t].append(i)

    def reach(start, step, within):
        seen, todo = {start}, [start]
        while todo:
            for t in step[todo.pop()]:
                if t not in seen and t in within:
                    seen.add(t)
                    todo.append(t)
        return seen

    component, parts = [0] * n, [set(range(n))]
    number = 0
    while parts:
        part = parts.pop()
        if not part:
            continue
        pivot = min(part)
        down, up = reach(pivot, succ, part), reach(pivot, pred, part)
        both = down & up
        for i in both:
            component[i] = number
        number += 1
        parts += [down - both, up - both, part - down - up]
    return component


def faults(blocks):
    """Uses that come too early, on any path: (instruction, register, waits, kind).

    The state maps (kind, register) to the waits since it was written. A statement that ends in a conditional skip of
    its waits (the last matrix instruction of a step) takes them where the loop ends: on the way out of a loop whose
    latest one was of that form, every result is done."""
    succ = edges(blocks)
    part = loops(succ)
    waiting = {s for _, code in blocks for op, _, s in code if s and op.startswith("s_cbranch")}
    found = set()

    def run(state, code):
        for op, ops, inside in code:
            if inside in waiting and not (op.startswith("v_mfma")):
                continue
            matrix, vector = op.startswith("v_mfma"), op.startswith("v_") and not op.startswith("v_mfma")
            first = [] if not ops or op.startswith(("buffer_", "global_", "scratch_", "ds_")) else registers(ops[0])
            writes = first if matrix or vector or op.startswith("s_") else []
            if vector and ("swap" in op or "_co_" in op) and len(ops) > 1:
                writes = writes + registers(ops[1])
            touched = [r for o in ops for r in registers(o)]
            if inside and op.startswith("buffer_"):
                for r in touched:
                    if r[0] == "s" and state.get(("scalar", r), 99) < SCALAR_TO_MEMORY:
                        found.add((op, r, state[("scalar", r)], "scalar to copy"))
            if inside and matrix:
                for r in touched:
                    if state.get(("vector", r), 99) < VECTOR_TO_MATRIX:
                        found.add((op, r, state[("vector", r)], "vector to matrix"))
            else:
                for r in touched:
                    if state.get(("matrix", r), 99) < MATRIX_TO_USE:
                        found.add((op, r, state[("matrix", r)], "matrix to use"))
            if inside and matrix:
                state[("last", "waits")] = 0 if inside in waiting else 1
            step = int(ops[0], 0) + 1 if op == "s_nop" else 1
            for key in [k for k in state if k[0] != "last"]:
                state[key] += step
                if state[key] >= MATRIX_TO_USE:
                    del state[key]
            for r in writes:
                for kind in ("scalar", "vector", "matrix"):
                    state.pop((kind, r), None)
                if vector:
                    state[("scalar" if r[0] == "s" else "vector", r)] = 0
                elif inside and matrix:
                    state[("matrix", r)] = 0
        return state

    start = [None] * len(blocks)
    start[0] = {}
    todo = [0]
    while todo:
        i = todo.pop()
        end = run(dict(start[i]), blocks[i][1])
        for t in succ[i]:
            state = dict(end)
            if part[t] != part[i] and state.get(("last", "waits")) == 0:
                state = {k: v for k, v in state.items() if k[0] != "matrix"}
            if start[t] is None:
                start[t] = state
                todo.append(t)
                continue
            changed = False
            for k, v in state.items():
                old = start[t].get(k)
                better = old is None or (v > old if k[0] == "last" else v < old)
                if better:
                    start[t][k] = v
                    changed = True
            if changed:
                todo.append(t)
    return found


@pytest.fixture(scope="module", params=SOURCES)
def assembly(request):
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-w", "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, request.param), "-o", "-"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return request.param, r.stdout


def test_waits_around_assembly_statements(assembly):
    source, text = assembly
    kernels = copies = products = 0
    bad = {}
    for name, blocks in functions(text):
        code = [c for _, block in blocks for c in block]
        kernels += 1
        copies += sum(1 for op, _, inside in code if inside and op.startswith("buffer_"))
        products += sum(1 for op, _, inside in code if inside and op.startswith("v_mfma"))
        assert not [c for c in code if not c[2] and "m0" in c[1]], name
        early = faults(blocks)
        if early:
            bad[name] = sorted(early)[:4]
    print(f"{source}: {kernels} kernels, {copies} copies, {products} matrix instructions in statements")
    assert kernels >= 20 and copies >= 300
    assert source != "epx_expert_gemm.hip" or products >= 100
    assert not bad, bad


def test_the_check_sees_what_it_is_for():
    """Early uses of each kind, and the same with the waits."""
    def code(text):
        return faults(next(functions("_Zk:\n" + text + "\ts_endpgm\n.Lfunc_end0:\n"))[1])

    def asm(text):
        return ";#ASMSTART\n" + text + ";#ASMEND\n"

    load = asm("\ts_mov_b32 m0, s9\n\ts_nop 0\n\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds\n")
    assert code("\tv_readfirstlane_b32 s2, v7\n" + load)
    assert not code("\tv_readfirstlane_b32 s2, v7\n\ts_nop 3\n" + load)
    product = "\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n"
    assert code("\tv_mov_b32_e32 v6, v9\n" + asm(product))
    assert not code("\tv_mov_b32_e32 v6, v9\n\ts_nop 1\n" + asm(product))
    assert code(asm(product) + "\tv_accvgpr_read_b32 v9, a2\n")
    assert not code(asm(product) + "\ts_nop 15\n\ts_nop 2\n\tv_accvgpr_read_b32 v9, a2\n")
    loop = ".LBB0_1:\n" + asm(product + "{}") + "\ts_cmp_eq_u32 s1, 0\n\ts_cbranch_scc0 .LBB0_1\n{}\tv_accvgpr_read_b32 v9, a2\n"
    wait = "\ts_nop 15\n\ts_nop 15\n"
    assert code(loop.format("", ""))
    assert not code(loop.format("\ts_cmp_lg_u32 s1, 0\n\ts_cbranch_scc1 2\n" + wait, ".LBB0_2:\n"))
    # a wait behind the loop does not help what comes before it
    assert code(loop.format("", "\tv_accvgpr_read_b32 v8, a3\n" + asm(wait)))
