"""The forward kernel of the delta rule with one decay per value head moves registers between its warps: by the count that the compiler gave it."""

import os
import re
import subprocess

import pytest

from gated_delta_rule_56_gb300 import build

SOURCE = os.path.join(build.CSRC, "kda_delta_tc.cu")


def _threads_and_registers():
    text = open(SOURCE).read()
    number = lambda name: int(re.search(rf"\b{name} = (\d+)", text).group(1))  # noqa: E731
    warps = dict(chain=number("kChainWarps"), prep=number("kPrepWarps"))
    return text, warps, number("kPrepRegisters"), number("kOtherRegisters")


def test_no_move_of_registers_without_a_check_of_the_compiled_count():
    text, _, _, _ = _threads_and_registers()
    moves = re.findall(r"setmaxnreg\.(inc|dec)[^;]*;\" ::\"n\"\((\w+)\)", text)
    assert sorted(moves) == [("dec", "kOtherRegisters"), ("inc", "kPrepRegisters")] and text.count("setmaxnreg.") == 2
    launch = text[text.index("cudaError_t launch("):]
    assert launch.index("cudaFuncGetAttributes") < launch.index("registers_suffice(registers)") < launch.index("<<<")


@pytest.mark.slow
def test_the_compiled_count_lets_them_move(tmp_path):
    _, warps, prep, other = _threads_and_registers()
    p = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", SOURCE, "-o", str(tmp_path / "x.o")],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    used = [int(n) for n in re.findall(r"delta_tc_kernel.*?Used (\d+) registers", p.stdout + p.stderr, re.S)]
    assert used
    for n in used:
        n = -(-n // 8) * 8
        assert other <= n <= prep
        assert warps["prep"] * (prep - n) <= (28 - warps["prep"] - warps["chain"]) * (n - other)
        assert 28 * 32 * n <= 65536
