"""Host-only checks of the overlap test of strided arrays (``csrc/overlap.h``),
compiled with the host C++ compiler, against sets of bytes."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "log_domain_sinkhorn_amd", "csrc")


@pytest.fixture(scope="module")
def meets(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("overlap") / "overlap_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "overlap_check.cpp"), "-o", exe], check=True)

    def run(pairs):
        text = "".join(" ".join(map(str, (x[0], *x[1], *x[2], x[3]))) + "\n" for p in pairs for x in p)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split()
        assert len(out) == len(pairs)
        return [x == "1" for x in out]

    return run


def _bytes(x):
    at, step, count, width = x
    return {at + i * step[0] + j * step[1] + k * step[2] + w for i in range(count[0]) for j in range(count[1])
            for k in range(count[2]) for w in range(width)} if at else set()


def test_against_sets_of_bytes(meets):
    rng = random.Random(5)
    pairs = []
    for _ in range(4000):
        p = []
        for _ in range(2):
            count = [rng.randint(0 if rng.random() < 0.02 else 1, 5) for _ in range(3)]
            width = rng.choice([1, 2, 4, 8])
            step = [rng.choice([0, 1, 3, 8, 16, 24, 40, 64, 120, 200, 333]) for _ in range(3)]
            p.append((1000 + rng.randint(0, 300), step, count, width))
        pairs.append(p)
    got = meets(pairs)
    want = [bool(_bytes(a) & _bytes(b)) for a, b in pairs]
    assert got == want and 500 < sum(want) < 3500


def test_layouts_of_one_buffer(meets):
    """[batch][length][heads][width] arrays of 2 bytes an element."""
    B, L, H, d = 4, 1000, 8, 64

    def rows(first, n, total, at=1 << 20):  # of [B][total][H][d]
        return (at + 2 * first * H * d, (2 * total * H * d, 2 * H * d, 2 * d), (B, n, H), 2 * d)

    def heads(first, n, total, at=1 << 20):  # of [B][H][total][d]
        return (at + 2 * first * d, (2 * H * total * d, 2 * d, 2 * total * d), (B, n, H), 2 * d)

    def part(i, of, at=1 << 20):  # of [B][L][of][H][d]
        return (at + 2 * i * H * d, (2 * L * of * H * d, 2 * of * H * d, 2 * d), (B, L, H), 2 * d)

    def column(i, of, at=1 << 20):  # of [B][L][H][of][d]
        return (at + 2 * i * d, (2 * L * H * of * d, 2 * H * of * d, 2 * of * d), (B, L, H), 2 * d)

    cases = [
        (rows(0, L, 2 * L), rows(L, 300, 2 * L), False), (rows(0, L, 2 * L), rows(L - 1, 300, 2 * L), True),
        (heads(0, L, 2 * L), heads(L, 300, 2 * L), False), (heads(0, L, 2 * L), heads(L - 1, 1, 2 * L), True),
        (part(0, 3), part(1, 3), False), (part(1, 3), part(2, 3), False), (part(2, 3), part(2, 3), True),
        (column(0, 2), column(1, 2), False), (column(0, 2), column(0, 2), True),
        # one half of each entry by rows, the other by heads
        (rows(0, L, 2 * L), heads(0, L, L)[:1] + ((4 * L * H * d, 2 * d, 2 * L * d),) + heads(0, L, L)[2:], True),
        (rows(0, L, 2 * L), (heads(0, L, L)[0] + 2 * L * H * d, (4 * L * H * d, 2 * d, 2 * L * d)) + heads(0, L, L)[2:], False),
        # an expanded input, and one far away
        (rows(0, L, L), (1 << 20, (0, 2 * H * d, 2 * d), (B, L, H), 2 * d), True),
        (rows(0, L, L), rows(0, L, L, at=(1 << 20) + 2 * B * L * H * d), False),
        # sizes past 32 bits, and a null array
        ((1 << 40, (1 << 33, 1 << 12, 1 << 8), (1 << 10, 1 << 20, 16), 256), ((1 << 40) + (1 << 32), (1 << 33, 1 << 12, 1 << 8), (1 << 10, 1 << 20, 16), 256), False),
        ((1 << 40, (1 << 33, 1 << 12, 1 << 8), (1 << 10, (1 << 20) + 1, 16), 256), ((1 << 40) + (1 << 32), (1 << 33, 1 << 12, 1 << 8), (1 << 10, 1 << 20, 16), 256), True),
        ((0, (8, 8, 8), (4, 4, 4), 8), (8, (8, 8, 8), (4, 4, 4), 8), False),
    ]
    assert meets([c[:2] for c in cases]) == [c[2] for c in cases]


def test_undecided_within_the_bound_counts_as_overlap(meets):
    # steps without a common one, and no byte in common: even against odd addresses
    a = (1 << 20, (2 * 10007, 2 * 101, 2), (5000, 90, 40), 1)
    b = ((1 << 20) + 1, (2 * 10009, 2 * 103, 2 * 3), (5000, 90, 15), 1)
    assert meets([(a, b)]) == [True]
