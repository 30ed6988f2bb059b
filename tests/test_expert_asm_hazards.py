"""The inline MFMAs of the experts' tile kernel and the compiler's schedule around them (CPU only: compiles the kernel file to
gfx950 assembly).  As for the large GEMM: no accumulator write between the zero fill's wait states and the first MFMA, no
accumulator read between the last MFMA and the epilogue's, and a main loop without accumulator copies, spills or a
wait for all vector-memory loads, whose barriers' counts are those of the loads issued since the stage they wait for."""
import os
import re
import subprocess
import tempfile

import pytest

from test_gemm_asm_hazards import ROOT

SRC = os.path.join(ROOT, "dynamic_scaling_scaled_amd", "csrc", "expert_gemm.hip")


@pytest.fixture(scope="module")
def kernels():
    from dynamic_scaling_scaled_amd import _build

    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "expert_gemm.s")
        cmd = [_build.hipcc(), *_build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I", _build.INCLUDE, "-I", _build.CSRC,
               SRC, "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            pytest.fail("hipcc failed:\n" + r.stderr[-2000:])
        s = open(out).read()
    found = {}
    for m in re.finditer(r"^(_ZN\S*k_expert_tile\S*):", s, re.M):
        found[m.group(1)] = s[m.start():s.index(".Lfunc_end", m.start())].split("\n")
    return found


def registers(line):
    """AGPRs that a line names, as bits."""
    found = 0
    for lo, hi, one in re.findall(r"\ba(?:\[(\d+):(\d+)\]|(\d+)\b)", line.split(";")[0]):
        found |= ((1 << int(hi) + 1) - (1 << int(lo))) if lo else 1 << int(one)
    return found


def walk(name, lines):
    """Follows every path: no accumulator is touched by another instruction between the wait states (three s_nop 7)
    and the MFMAs that update it, in either order.  Returns the accumulators of all MFMAs."""
    labels = {m.group(1): k for k, l in enumerate(lines) for m in [re.match(r"^(\.LBB\d+_\d+):", l)] if m}
    starts = sorted({0, *labels.values(), *(k + 1 for k, l in enumerate(lines) if re.search(r"\ts_c?branch", l))})
    state = {s: None for s in starts}  # per block: (registers of MFMAs, of others) since the wait states
    todo, everything = [(0, 0, 0)], 0
    while todo:
        k, mfma, other = todo.pop()
        if state[k] is not None and (mfma | state[k][0], other | state[k][1]) == state[k]:
            continue
        state[k] = (mfma | (state[k] or (0, 0))[0], other | (state[k] or (0, 0))[1])
        mfma, other = state[k]
        while k < len(lines):
            line = lines[k].strip()
            if all(l.strip() == "s_nop 7" for l in lines[k:k + 3]):
                mfma = other = 0
            elif line.startswith("v_mfma"):
                d = registers(line.split(",")[0])
                assert not d & other, (name, k, line)
                mfma |= d
                everything |= d
            else:
                r = registers(line)
                assert not r & mfma, (name, k, line)
                other |= r
            branch = re.match(r"s_(c?)branch\S*\s+(\.LBB\d+_\d+)", line)
            if branch:
                todo.append((labels[branch.group(2)], mfma, other))
                if not branch.group(1):
                    break
            if line.startswith("s_endpgm"):
                break
            k += 1
            if k in state:
                todo.append((k, mfma, other))
                break
    return everything


def loops(lines):
    labels = {m.group(1): k for k, l in enumerate(lines) for m in [re.match(r"^(\.LBB\d+_\d+):", l)] if m}
    for k, l in enumerate(lines):
        m = re.search(r"s_cbranch_\w+\s+(\.LBB\d+_\d+)", l)
        if m and labels.get(m.group(1), len(lines)) < k:
            yield "\n".join(lines[labels[m.group(1)]:k])


def test_every_instantiation_is_there(kernels):
    assert len(kernels) == 8, list(kernels)  # 2 A formats x 2 outputs x tiles of 1 and 4 blocks


def test_accumulator_fences_bracket_the_mfmas(kernels):
    for name, lines in kernels.items():
        acc = walk(name, lines)
        assert bin(acc).count("1") >= 64 * int(re.search(r"Li(\d)EEEv", name).group(1)), name


def test_main_loops_are_clean(kernels):
    for name, lines in kernels.items():
        main = [l for l in loops(lines) if "v_mfma" in l and l.count("\n.LBB") == 0]  # (one block each)
        blocks = int(re.search(r"Li(\d)EEEv", name).group(1))
        counts = []
        for text in main:
            assert "v_accvgpr_mov" not in text and "scratch_" not in text, name
            moved = 0  # (operands may rest in AGPRs; accumulators stay where they are)
            acc = 0
            for line in text.split("\n"):
                if "v_mfma" in line:
                    acc |= registers(line.split(",")[0])
                elif "v_accvgpr" in line:
                    moved |= registers(line)
            assert not moved & acc, name
            assert not re.search(r"vmcnt\(0\)", text), name
            n = text.count("v_mfma")
            assert n % 48 == 0, (name, n)      # three stages of 4 NB x 4 MFMAs
            nb = n // 48
            counts.append(nb)
            assert text.count("s_barrier") == 3, name
            waits = [int(w) for w in re.findall(r"vmcnt\((\d+)\)", text)]
            assert waits.count(16 + 2 * nb) >= 3, (name, nb, waits)
            assert text.count("buffer_load_dwordx4") == 3 * (8 + 2 * nb), (name, nb)
        assert sorted(counts) == list(range(1, blocks + 1)), (name, counts)
