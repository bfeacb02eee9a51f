"""Which partial results the join of a tree's shares reads, on the host.

Whatever cu_q holds, they lie among those of the workgroups launched: sequences
that overlap can count more shares than 32 bits hold, so that a count before a
sequence comes out negative or small.
"""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_gemm_decode_amd", "csrc")
ROCM = "/opt/rocm/include"

CASES = [  # shares before the sequence, block, shares of a unit, KV heads, launched; first share
    ((0, 0, 4, 1, 512), 0), ((100, 3, 4, 8, 1024), 112), ((127, 0, 1, 4, 512), -1), ((124, 0, 4, 4, 512), 124), ((125, 0, 4, 4, 512), -1),
    ((0, 0, 1, 1, 512), -1),                            # a unit that was not cut
    ((-5, 0, 4, 1, 512), -1), ((-5, 2, 4, 1, 512), 3), ((-2147483648, 0, 2, 1, 512), -1),
    ((2147483647, 0, 2, 1, 512), -1), ((2147483600, 20, 100, 65536, 512), -1),
    ((0, 8388607, 8388608, 1, 16777215), -1), ((0, 8388607, 512, 1, 16777215), -1),
    ((500, 8388607, 257, 1, 512), -1), ((0, 0, 2147483647, 64, 512), -1), ((100, 0, -7, 1, 512), -1),
]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM), reason="needs g++ and HIP's headers")
def test_shares_are_among_those_launched(tmp_path):
    exe = str(tmp_path / "tree_share_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-Wno-unknown-pragmas", "-isystem", ROCM, "-I", CSRC,
                    os.path.join(HERE, "native", "tree_share_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c, _ in CASES), capture_output=True, text=True, check=True)
    assert len(r.stdout.split()) == len(CASES) and [int(x) for x in r.stdout.split()] == [want for _, want in CASES]
