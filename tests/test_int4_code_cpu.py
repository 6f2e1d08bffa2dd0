"""The assembly of the 4-bit products: where a wave's lanes read what others of it wrote
to LDS, something holds the compiler to that order."""
import os
import re
import subprocess

import pytest

from mixture_experts_transformer_moe_amd import build


def unordered(lines):
    """LDS reads that follow a write, and writes that follow a read, with no barrier (of the
    workgroup, or the compiler's own of the wave) between them."""
    found, last = [], None
    for line in lines:
        if "s_barrier" in line or "wave barrier" in line:
            last = None
        kind = re.match(r"\s*ds_(read|write)", line)
        if kind:
            if last is not None and last != kind[1]:
                found.append(line.strip())
            last = kind[1]
    return found


def test_scan_finds_what_it_looks_for():
    write, read = "\tds_write_b128 v1, v[2:5]", "\tds_read_b32 v1, v2"
    assert unordered([write, read]) and unordered([read, write])
    assert not unordered([write, write, "\t; wave barrier", read, read, "\ts_barrier", write])


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: lines} of int4.hip's kernels, compiled as the library is."""
    out = tmp_path_factory.mktemp("int4") / "int4.s"
    cmd = [build.hipcc(), *build.CFLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, "int4.hip"), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True)
    found, cur = {}, None
    for line in out.read_text().splitlines():
        if label := re.match(r"(_ZN\w+):", line):
            cur = found.setdefault(label[1], [])
        elif line.startswith(".Lfunc_end"):
            cur = None
        elif cur is not None:
            cur.append(line)
    return found


def test_lanes_meet_before_they_read_each_other(kernels):
    rows = {n: k for n, k in kernels.items() if "int4_rows_kernel" in n}
    assert len(rows) == 12                                # gate/up and down, 16 and 32 rows, three groups
    for name, lines in rows.items():
        assert sum("ds_write_b128" in x for x in lines) > 0 and sum("ds_read_b128" in x for x in lines) > 0
        assert not unordered(lines), name
