"""Index arithmetic of the attention kernels, compiled for the host (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "coo_spmm_sparse_gb300", "csrc")


def run(tmp_path, body):
    """Standard output of a program whose main() is `body`."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "index.cu"
    src.write_text(f'#include "{CSRC}/attention.cuh"\n#include <cstdio>\nusing namespace snack;\n'
                   f"int main() {{\n{body}\nreturn 0;\n}}\n")
    exe = tmp_path / "index"
    subprocess.run([nvcc, "-std=c++17", "-o", str(exe), str(src)], check=True, capture_output=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()


def test_query_rows_of_a_tile_of_keys(tmp_path):
    """Rows [first query * group, nq * group): empty for keys in padding, however far behind the
    sequence's end, and never outside 0 .. nq * group."""
    cases = [(1, j0, nq, nk, group) for nq, group in ((32, 32), (1, 1), (2 ** 26 - 200, 31), (0, 8))
             for nk in (0, 1, 40, 2 ** 26, 2 ** 31 - 4097)
             for j0 in (0, 16, 48, 2 ** 26 + 4096, 2 ** 31 - 4112)]
    cases += [(0, j0, nq, nk, group) for _, j0, nq, nk, group in cases]
    body = "".join(f'printf("%d %d\\n", first_query({c}, {j}, {nq}, {nk}) * {g}, {nq} * {g});\n'
                   for c, j, nq, nk, g in cases)
    got = [int(x) for x in run(tmp_path, body)]
    for (causal, j0, nq, nk, group), begin, end in zip(cases, got[::2], got[1::2]):
        first = 0 if not causal else max(0, j0 - nk + nq)
        want = nq if j0 >= nk else first
        assert (begin, end) == (want * group, nq * group) and 0 <= begin <= end
