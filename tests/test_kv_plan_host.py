"""Host checks (no GPU) of what the attention over a shared prefix takes from a plan that does not fit its call."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantised_weight_gb300", "csrc")


@pytest.fixture(scope="module")
def columns(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("plan") / "plan_probe")
    subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "plan_probe.cu"), "-o", exe],
                   check=True, capture_output=True, timeout=300)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout
    return [tuple(int(x) for x in line.split()) for line in out.splitlines()]


def test_tokens_behind_a_prefix_lie_in_the_table(columns):
    """A sequence reads its columns from those it shares on, for the rest of its cut length: none lies behind the row's
    last, whatever length and entry say; a length beyond the table counts as the table."""
    seen = set()
    for log2p, width, held, n, skip, cols in columns:
        page = 1 << log2p
        length = min(max(held, 0), width * page)
        if skip == 0 or n == 0:
            assert cols == 0
        elif skip < 0 or skip % page or skip > length - n + 1:
            assert cols == -1
        else:
            rest = length - cols * page
            assert cols * page == skip and rest >= n - 1 and cols + -(-rest // page) <= width
        seen.add((held > width * page, skip > width * page, cols))
    # an entry of exactly what a length is beyond its table is among them
    assert (True, True, -1) in seen and (True, False, 1) in seen and (False, False, 3) in seen
    assert any(held - skip == width << log2p and skip > 0 and n > 0 for log2p, width, held, n, skip, _ in columns)


def test_the_row_kernel_decides_once():
    """The kernel that adds the prefix asks for the columns in one place, and keeps what it was told."""
    src = open(os.path.join(CSRC, "kv_rows.cuh")).read()
    assert src.count("shared_columns(") == 1 and src.count("a.lens[") == 0
