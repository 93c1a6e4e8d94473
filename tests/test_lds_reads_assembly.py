"""LDS reads that are written as assembly statements: the compiler takes their
registers as written at once, and as free when it sees no later use, while the
read is still under way.  Between a read and the lgkmcnt wait that covers it
nothing may write its registers, nor use them (but for moves, whose copies are
of values that are read again).  Read, over every path, from the assembly that
hipcc writes for the kernels (compiled here for gfx950; no GPU)."""

import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from mxfp4_block_scaled_quant_amd import build as B

SOURCES = ["bmm_a16w4", "gemm_prefill", "gemm_prefill_n128", "gemm_prefill_act", "gemm_prefill_act_n128",
           "gemm_prefill_experts"]
REGISTER = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
NONE = frozenset()
READS = ("ds_read", "ds_bpermute", "ds_permute", "ds_swizzle")
LOADS = ("buffer_load", "global_load", "flat_load", "scratch_load")


def registers(text):
    found = set()
    for kind, first, last, one in REGISTER.findall(text):
        found |= {(kind, i) for i in range(int(first or one), int(last or one) + 1)}
    return frozenset(found)


def kernels(text):
    """(name, [(is_label, text)]) of each kernel of an assembly file."""
    name, code = None, []
    for line in text.split("\n"):
        start = re.match(r"(_Z\w+):", line)
        if start:
            name, code = start.group(1), []
        elif name and line.startswith(".Lfunc_end"):
            yield name, code
            name = None
        elif name:
            line = line.split(";")[0].strip()
            label = re.fullmatch(r"([.\w]+):", line)
            if label:
                code.append((True, label.group(1)))
            elif line and not line.startswith("."):
                code.append((False, line))


def blocks(code):
    """(instructions, following blocks) of each basic block."""
    done, at, current = [], {}, []
    for i, (is_label, line) in enumerate(code):
        if is_label:
            if current:
                done.append(current)
                current = []
            at[line, i] = at[line] = len(done)
        else:
            current.append((i, line))
            if line.startswith(("s_cbranch", "s_branch", "s_endpgm")):
                done.append(current)
                current = []
    if current:
        done.append(current)
    graph = []
    for n, block in enumerate(done):
        i, last = block[-1]
        follows = []
        if last.startswith(("s_cbranch", "s_branch")):
            target = last.split()[-1]
            near = re.fullmatch(r"(\d+)f", target)
            if near:                 # "1f": the next label 1
                place = min(k[1] for k in at if isinstance(k, tuple) and k[0] == near.group(1) and k[1] > i)
                follows.append(at[near.group(1), place])
            else:
                follows.append(at[target])
        if not last.startswith(("s_branch", "s_endpgm")) and n + 1 < len(done):
            follows.append(n + 1)
        graph.append(([line for _, line in block], follows))
    return graph


def step(under_way, lines, faults):
    """The reads under way (oldest first, a set of registers each) after `lines`."""
    under_way = list(under_way)
    for line in lines:
        op, _, operands = line.partition(" ")
        if op == "s_waitcnt":
            count = re.search(r"lgkmcnt\((\d+)\)", line)
            if count:
                under_way = under_way[max(0, len(under_way) - int(count.group(1))):]
            continue
        busy = frozenset().union(*under_way)
        first, _, rest = operands.partition(",")
        if op.startswith(READS):
            if registers(rest) & busy:
                faults.add(line)
            under_way.append(registers(first))
            continue
        writes = registers(first) if op.startswith(("v_",) + LOADS) and not op.startswith("v_cmp") else NONE
        if line.endswith(" lds"):
            writes = NONE
        if writes & busy or (registers(operands) & busy and not op.startswith("v_mov_b")):
            faults.add(line)
        if op.startswith(("ds_", "s_load", "s_buffer_load")):
            under_way.append(NONE)
    return tuple(under_way[-64:])


def faults_of(code):
    """(LDS reads of a kernel, instructions that touch one under way)."""
    graph = blocks(code)
    faults, entry, todo = set(), {0: ()}, [0]
    while todo:
        n = todo.pop()
        out = step(entry[n], graph[n][0], faults)
        for m in graph[n][1]:
            old = entry.get(m)
            new = out
            if old is not None:      # the newest reads side by side
                size = max(len(old), len(out))
                pair = [(NONE,) * (size - len(s)) + s for s in (old, out)]
                new = tuple(a | b for a, b in zip(*pair))
            if new != old:
                entry[m] = new
                todo.append(m)
    return sum(line.startswith("ds_read") for lines, _ in graph for line in lines), faults


def _kernel(*lines):
    return [(line.endswith(":"), line.rstrip(":")) for line in lines + ("s_endpgm",)]


def test_the_reader_finds_what_it_should():
    read, use = "ds_read_b128 v[4:7], v1 offset:16", "v_add_f32_e32 v9, v5, v8"
    assert faults_of(_kernel(read, "s_waitcnt lgkmcnt(0)", use)) == (1, set())
    assert faults_of(_kernel(read, use))[1] == {use}
    assert faults_of(_kernel(read, "v_mov_b32_e32 v6, 0"))[1]
    assert not faults_of(_kernel(read, "v_mov_b32_e32 v10, v6", "s_waitcnt lgkmcnt(0)"))[1]
    assert faults_of(_kernel(read, "ds_read_b32 v9, v4"))[1]
    more = "ds_read_b32 v20, v1"
    assert not faults_of(_kernel(read, more, "s_waitcnt lgkmcnt(1)", use))[1]
    assert faults_of(_kernel(read, more, "s_waitcnt lgkmcnt(2)", use))[1]
    loop = ("s_mov_b32 s0, 0", ".LBB0_1:", "v_mov_b32_e32 v6, 0", read, "s_cbranch_scc0 .LBB0_1")
    assert faults_of(_kernel(*loop))[1]                               # the next turn's write
    near = ("s_cbranch_scc1 1f", read, "1:", use)
    assert faults_of(_kernel(*near))[1] == {use}                       # one of two ways in


@pytest.mark.skipif(not (os.path.exists(B.HIPCC) or shutil.which(B.HIPCC)), reason="needs hipcc")
def test_no_instruction_touches_a_read_under_way(tmp_path):
    def assembly(name):
        out = str(tmp_path / (name + ".s"))
        flags = [*B.FLAGS, *B.FILE_FLAGS.get(name + ".hip", [])]
        r = subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(B.CSRC, name + ".hip"), "-o", out],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return open(out).read()

    with cf.ThreadPoolExecutor(4) as pool:
        texts = list(pool.map(assembly, SOURCES))
    for source, text in zip(SOURCES, texts):
        reads = 0
        for name, code in kernels(text):
            n, faults = faults_of(code)
            reads += n
            assert not faults, (source, name, sorted(faults)[:5])
        assert reads > 0, source
