"""Which split records the merges follow, on the CPU: a record that a call with
a timed-out wait left behind may hold any words, and none of them may lead the
merge past the workspace's slots."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
EDGES = [-2**31, -2**30, -1, 0, 1, 2, 3, 151, 152, 303, 304, 1000, 2**29, 2**30 - 1, 2**30, 2**30 + 1, 2**31 - 2,
         2**31 - 1, 0x3f800000, 0x7f800000]


@pytest.fixture(scope="module")
def follow():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    out_dir = os.path.join(HERE, "native", "_build")  # git-ignored
    os.makedirs(out_dir, exist_ok=True)
    exe = os.path.join(out_dir, "merge_records_dump")
    subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    os.path.join(ROOT, "mla_paged_decode_gb300", "csrc"), "-I", os.path.join(ROOT, "include"),
                    os.path.join(HERE, "native", "merge_records_dump.cu"), "-o", exe], check=True, capture_output=True)

    def run(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_records_are_followed_only_inside_the_slots(follow):
    rng = random.Random(0)
    word = lambda: rng.choice(EDGES) if rng.random() < 0.7 else rng.randint(-2**31, 2**31 - 1)  # noqa: E731
    cases = [(word(), word(), word(), rng.choice([1, 152, 1000, 100_000]), rng.choice([1, 2])) for _ in range(20000)]
    cases += [(x, y, z, 152, s) for x in EDGES for y in EDGES for z in EDGES for s in (1, 2)]
    got = follow(cases)
    assert len(got) == len(cases)
    followed = [0, 0]
    for (x, y, z, bound, stride), (split, pieces) in zip(cases, got):
        # slots of a split: z, and 2 (x + k) for 0 < k < y; there are 2 * bound
        assert split == (y > 1 and x >= 0 and 0 <= z < 2 * bound and 2 * (x + y - 1) < 2 * bound), (x, y, z, bound)
        # slots of pieces: (z + k) * stride + half, k < y, half < stride; there are `bound`
        last = (z + y - 1) * stride + stride - 1
        assert pieces == (y > 0 and z >= 0 and last < bound), (x, y, z, bound, stride)
        followed[0] += split
        followed[1] += pieces
    assert min(followed) > 50
