"""Plans of the row operators' launches, compiled for the CPU (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# co-resident clusters of 1..16 CTAs on a GB300, as the occupancy query reports them
ACTIVE = [304, 152, 97, 74, 58, 46, 38, 36, 30, 28, 23, 23, 19, 14, 14, 14]
FULL, CROSS = 0, 7
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan((batch, H_q, H_kv, d, dtype, pages, page), commands) -> a list of ints a command."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "rows_probe")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "dynamic_sparse_kv_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "rows_probe.cu"), "-o", exe], check=True)

    def run(dims, commands):
        r = subprocess.run([exe, *map(str, [*dims, 152, *ACTIVE])], input="\n".join(commands) + "\n",
                           capture_output=True, text=True, check=True)
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    return run


def test_cross_attention_is_split_by_its_tokens_not_by_the_batch(plan):
    """A query token is a unit: one token on a large handle is split as on a handle of one sequence."""
    for heads in ((28, 4, 128), (10, 10, 128), (8, 2, 64)):
        for n in (300, 2624, 8320):
            for rows in (1, 3, 16, 64, 256):
                own = plan((rows, *heads, BF16, 1024, 16), [f"p {CROSS} {rows} {n}", f"p {FULL} 0 {n}"])
                large = plan((256, *heads, BF16, 1024, 16), [f"p {CROSS} {rows} {n}"])
                assert own[0] == own[1] == large[0], (heads, n, rows, own, large)
    # a handful of tokens spreads its states over the GPU
    assert plan((256, 28, 4, 128, BF16, 1024, 16), [f"p {CROSS} 1 8320"])[0] == [16, 1]


def test_cross_attention_goes_by_token_only_as_far_as_its_worst_case_allows(plan):
    """As many tokens as sequences may be one prompt: its states are then read once a token."""
    def by_token(batch, rows, heads, pages, dtype=BF16):
        return plan((batch, *heads, dtype, pages, 16), [f"c {rows}"])[0][0]
    big = (28, 4, 128)
    assert by_token(16, 16, (10, 10, 128), 164) == 1          # a decode step
    assert by_token(256, 1, big, 520) == 1                    # one token on a large handle
    assert by_token(256, 256, big, 520) == 0                  # 4.4 GB if it is one prompt
    assert by_token(256, 256, (10, 10, 128), 520) == 0
    assert by_token(256, 256, big, 38) == 1                   # short states
    assert by_token(16, 17, big, 10) == 0                     # more tokens than sequences
    assert by_token(256, 256, big, 520, F32) == 1             # the fp32 row kernel takes longer for single tokens
    assert by_token(70000, 70000, (4, 2, 64), 1) == 0         # a grid has 65535 blocks in z
    assert by_token(70000, 70000, (4, 2, 64), 1, F32) == 0
    assert by_token(70000, 65535, (4, 2, 64), 1) == by_token(70000, 65535, (4, 2, 64), 1, F32) == 1
