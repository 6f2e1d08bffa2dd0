"""The rule of the 4-bit products' kernels (csrc/int4_plan.h, compiled for the host): the
batches of tests/int4_kernels.py run on the kernels they stand for, with reductions of
more blocks a wave than the scales kept at a time."""
import os
import subprocess

from mixture_experts_transformer_moe_amd.build import CSRC
from tests.int4_kernels import E, K, KERNELS, LONG, batch


def test_batches_take_their_kernels(tmp_path):
    exe = tmp_path / "int4_plan"
    src = os.path.join(os.path.dirname(__file__), "int4_plan.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, src, "-o", str(exe)], check=True)
    lines = []
    for mode, group, mean in KERNELS:
        T, rows = batch(mode, mean)[0], mean * E
        assert T * K == rows
        columns = 32 if mode == "gate_up" else 64
        lines.append(f"{mode == 'gate_up':d} {group} {rows} {E} {LONG // 128} 256 {columns} {min(rows, E + rows // 16)}")
    out = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split("\n")
    for (case, kernel), got in zip(KERNELS.items(), out):
        name, ks = got.split()
        assert name == kernel, case
        # the blocks of a wave, in pairs: more than the 8 whose scales are in LDS at a time
        ks, pairs = int(ks), LONG // 256
        assert max(2 * (pairs * (i + 1) // ks) - 2 * (pairs * i // ks) for i in range(ks)) > 8, case
