"""The cut of trees' keys into shares, on the host (tests/native/tree_cut_check.cpp
runs the arithmetic that a wave of the GPU runs).

A plan launches a workgroup for each share that there can be; a share beyond
them would never be computed.  Whatever the batch, the cut must stay within them.
"""

import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_gemm_decode_amd", "csrc")
ROCM = "/opt/rocm/include"

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM), reason="needs g++ and HIP's headers")


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cut") / "tree_cut_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-Wno-unknown-pragmas", "-isystem", ROCM, "-I", CSRC,
                    os.path.join(HERE, "native", "tree_cut_check.cpp"), "-o", exe], check=True)

    def run(batches):
        """[(kv heads, max_kv, slots, [(blocks, length)])] -> [(shares, longest in tiles, rounds)]"""
        text = "\n".join("%d %d %d %d %s" % (h, m, s, len(b), " ".join("%d %d" % x for x in b)) for h, m, s, b in batches)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(out) == len(batches)
        return out
    return run


def launched(heads, slots, batch):
    """Workgroups that a plan for just these units launches: units / slots + 1/4, rounded up, times the slots."""
    units = heads * sum(blocks for blocks, _ in batch)
    return -(-(4 * units + slots) // (4 * slots)) * slots


def check(cut, batches):
    for (heads, max_kv, slots, batch), (shares, longest, rounds) in zip(batches, cut(batches)):
        most = launched(heads, slots, batch)
        assert shares <= most, (heads, max_kv, slots, batch[:4], len(batch), shares, most)
        assert bool(rounds) == (most // heads * heads > slots)


def test_very_long_contexts(cut):
    """Blocks times keys beyond 2^30: 12 blocks of 134 million keys, 16 of 268 million, 600 of 3.84 million; the largest
    context that a plan takes; many such sequences."""
    check(cut, [(1, 134217728, 768, [(12, 134217728)]), (1, 268435456, 768, [(16, 268435456)]), (1, 3840000, 768, [(600, 3840000)]),
                (1, 2 ** 30, 768, [(1, 2 ** 30)]), (1, 2 ** 30, 512, [(16, 2 ** 30)] * 30), (2, 2 ** 30, 512, [(3, 2 ** 29 + i) for i in range(64)]),
                (8, 2 ** 30, 512, [(1, 2 ** 30 - i * 2 ** 20) for i in range(512)]), (1, 2 ** 30, 768, [(8388608, 2 ** 30)]),
                (128, 50000000, 512, [(40, 50000000), (1, 128)])])


def test_random_batches(cut):
    r = random.Random(5)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** r.random()))
    batches = []
    for _ in range(4000):
        n, top = spread(1, 512), spread(129, 2 ** 30)
        lens = [r.randint(0, top) if r.random() < 0.5 else min(top, spread(1, top)) for _ in range(n)]
        most = spread(1, 5000)
        batches.append((r.choice([1, 2, 4, 5, 8, 16, 64, 200]), top, r.choice([512, 768]),
                        [(0 if r.random() < 0.1 else r.randint(1, most), x) for x in lens]))
        # (the plan refuses what needs 2^24 workgroups)
        if launched(batches[-1][0], batches[-1][2], batches[-1][3]) >= 2 ** 24:
            batches.pop()
    check(cut, batches)


def test_ordinary_batches_fill_the_card(cut):
    """A batch that can be cut takes most of the workgroups launched, and no share is more than a tile above twice the even one."""
    r = random.Random(6)
    batches = []
    for _ in range(500):
        top = r.randint(2000, 60000)
        batches.append((r.choice([1, 2, 8]), top, 512, [(r.randint(1, 3), r.randint(1000, top)) for _ in range(r.randint(1, 64))]))
    for (heads, top, slots, batch), (shares, longest, _) in zip(batches, cut(batches)):
        most = launched(heads, slots, batch) // heads
        tiles = sum(b * -(-x // 64) for b, x in batch)
        units = sum(b for b, _ in batch)
        assert longest <= max(2, tiles // max(1, most - units) + 2), (heads, top, batch[:4], shares, longest, most)
