"""The kernels' own bounds of packed batches (csrc/packed.cuh), compiled for the host: whatever
the offsets hold, no row outside the tensors and no row sums outside their room."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("host") / "packed_places")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run([cc, "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", exe,
                    os.path.join(ROOT, "tests", "host", "packed_places.cpp"),
                    "-I", os.path.join(ROOT, "differentiable_image_quality_gb300", "csrc"),
                    "-I", os.path.join(cuda, "include")], check=True)

    def run(q_rows, k_rows, q, k):
        text = f"{len(q) - 1} {q_rows} {k_rows}\n{' '.join(map(str, q))}\n{' '.join(map(str, k))}\n"
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        room, loose, tight, least, left = map(int, out.split())
        assert 0 <= tight <= room and least == 0 and left == 0
        return room, loose, tight

    return run


def test_sequences_that_share_rows(places):
    """1000 sequences, every other one all 1024 rows again: four times the row sums' room."""
    q = [0, 1024] * 500 + [0]
    k = list(range(1001))
    room, loose, tight = places(1024, 1000, q, k)
    assert loose > 3 * room and tight == room


def test_counts_that_leave_an_int(places):
    rows, n = 2 ** 29, 2000
    room, loose, tight = places(rows, n, [0, rows] * (n // 2) + [0], list(range(n + 1)))
    assert loose > 2 ** 31 and tight == room


@pytest.mark.parametrize("offsets", [[0], [0, 5, 5, 9], [0, 2000], [3, -4, 100, 7], [0, 9, 2, 9],
                                     [-2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 700]])
def test_offsets_out_of_range(places, offsets):
    places(700, 900, offsets, offsets[::-1])


def test_ascending_offsets_keep_their_rows(places):
    rng = random.Random(1)
    for rows in (0, 1, 127, 128, 129, 5000):
        for n in (1, 3, 200):
            q = [0] + sorted(rng.randrange(rows + 1) for _ in range(n))
            room, loose, tight = places(rows, rows, q, q)
            assert loose == tight <= room
