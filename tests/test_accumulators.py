"""The prefill kernels' accumulators in the built library's gfx950 code. Their matrix instructions are inline assembly,
which the compiler knows no hazards of, so every other access to an accumulator register has to lie behind an
accumulator fence (four s_nop 15 in a row): one between it and the matrix instructions before it, and one between it
and those after it."""
import os
import re
import shutil
import subprocess

import pytest

from sparse_rank_linear_prune24_amd import binding

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def registers(text):
    """Accumulator registers that an instruction's text names."""
    found = set()
    for first, last, one in re.findall(r"\ba(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        found |= set(range(int(first), int(last) + 1)) if first else {int(one)}
    return found


def unfenced(instructions):
    """Numbers of the instructions that touch an accumulator with no fence between them and a matrix instruction."""
    matrix = re.compile(r"v_(smfmac|mfma)_")
    accumulators = set()
    for text in instructions:
        if matrix.match(text):
            accumulators |= registers(text.split(",")[0])
    wrong, nops, since = [], 0, []   # since: accesses after the last fence
    after_matrix = False             # a matrix instruction after the last fence
    for i, text in enumerate(instructions):
        nops = nops + 1 if re.match(r"s_nop 15\b", text) else 0
        if nops == 4:
            since, after_matrix = [], False
        elif matrix.match(text):
            wrong += since
            since, after_matrix = [], True
        elif registers(text) & accumulators:
            if after_matrix:
                wrong.append(i)
            since.append(i)
    return accumulators, wrong


def test_the_check_itself():
    mfma, nop, move = "v_smfmac_f32_16x16x64_bf16 a[0:3], v[0:3], v[4:11], v12", "s_nop 15", "v_accvgpr_mov_b32 a1, a7"
    assert unfenced([move] + [nop] * 4 + [mfma, mfma] + [nop] * 4 + ["ds_write_b128 v0, a[0:3]"])[1] == []
    assert unfenced([move] + [nop] * 3 + [mfma])[1] == [0]
    assert unfenced([mfma, move] + [nop] * 4 + [mfma])[1] == [1]
    assert unfenced([mfma] + [nop] * 4 + [move, mfma])[1] == [5]
    assert unfenced([mfma, "v_accvgpr_write_b32 a9, v3", "v_accvgpr_read_b32 v3, a9"])[1] == []   # another register


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no AMD disassembler here")
def test_accumulators_are_touched_behind_fences_only(tmp_path):
    library = shutil.copy(binding.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", library], cwd=tmp_path, check=True, capture_output=True)
    kernels = 0
    for name in sorted(os.listdir(tmp_path)):
        if "gfx950" not in name or os.path.getsize(tmp_path / name) == 0:
            continue
        symbols = subprocess.run([OBJDUMP, "-t", tmp_path / name], check=True, capture_output=True, text=True).stdout
        if "linear_prefill_wide_kernel" not in symbols:
            continue
        code = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", tmp_path / name], check=True,
                              capture_output=True, text=True).stdout
        for part in re.split(r"\n(?=<)", code):
            title, _, body = part.partition("\n")
            if "linear_prefill_wide_kernel" not in title:
                continue
            accumulators, wrong = unfenced([line.split("//")[0].strip() for line in body.split("\n") if line.strip()])
            kernels += 1
            assert len(accumulators) in (64, 128), title
            assert not wrong, f"{title} {len(wrong)} accesses, the first at instruction {wrong[0]}"
    assert kernels >= 12
