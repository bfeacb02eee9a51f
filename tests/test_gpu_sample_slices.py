"""Sampling of rows that several workgroups share: special values that fill whole
slices, maxima far apart, borders among equal entries of several slices; and
vocabularies of more than 512 slices.  Tolerances as in test_gpu_sample.py: a
mass is a sum of steps of 2^-34, half a step and 3 10^-12 off an entry, which is
within 2^-34 of itself.
"""

import pytest
import torch

from tests.gpu_util import requires_gpu
from tests.test_gpu_sample import INF, NAN, RULES, check, run, special_rows

pytestmark = [pytest.mark.gpu, requires_gpu]
SLICE = 4096            # the shortest; others are twice and four times as long
N = 5 * SLICE - 469


def slice_rows(n):
    """special_rows, and rows that differ by slice."""
    g = torch.Generator().manual_seed(10)
    x = torch.randn(18, n, generator=g)
    part = torch.arange(n) // SLICE
    x[0, part == 0] = -INF
    x[1, part == 4] = NAN
    x[2, 2 * SLICE + 77] = INF                              # one value, in the middle
    x[3, SLICE - 1:SLICE + 1] = INF                         # on both sides of a border
    x[4] = -INF
    x[4, 3 * SLICE:3 * SLICE + 9] = INF                     # nothing else in the row
    x[5, part == 3] += 1e6
    x[6, part != 1] += 1e6
    x[7] -= 100.0 * part                                    # 800 buckets apart at T = 1
    x[8] = x[8].clamp(-0.05, 0.05) - 63.9 * (part % 2)      # 511 or 512 buckets apart
    x[9] = torch.where(part % 2 == 0, NAN, -INF)
    x[9, n - 1] = -3.0                                      # the last entry alone
    x[10] = 1.0 - (part >= 3).float()                       # equal ones over three slices, then over two
    x[11] = torch.where(torch.arange(n) % SLICE == SLICE - 1, 2.0, -2.0)
    x[12, part < 4] = NAN
    x[13] = 20.0 * x[13] - 1e4 * (4 - part)                 # the last slice alone weighs
    x[14] = (x[14] * 4).round() / 4                         # few values, in all slices
    x[15, part > 0] = torch.finfo(torch.float32).min
    x[16] = 1e-3 * x[16] + 300.0
    x[17] = torch.where(part % 2 == 0, 0.0, -0.0)
    return torch.cat([special_rows(n)[:20], x])


def problem(bf16, repeat=1):
    x = slice_rows(N).repeat(repeat, 1)
    noise = torch.empty(x.shape).exponential_(generator=torch.Generator().manual_seed(4)).clamp_min(1e-20)
    return (x.to(torch.bfloat16) if bf16 else x).cuda(), noise.cuda()


def columns(rules, each):
    return {k: [r[i] for r in rules for _ in range(each)] for i, k in enumerate(("temperature", "top_k", "top_p", "min_p"))}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rule", range(len(RULES)))
def test_slices_of_special_values(rule, bf16):
    """Five slices a row."""
    x, noise = problem(bf16)
    rules = columns([RULES[rule]], len(x))
    check(x, noise, *run(x, noise, **rules), **rules)


MORE = [(0.5, 9000, 0.6, 0.0), (1.0, 4097, 1.0, 0.0), (1.0, 8193, 0.7, 1e-3), (2.0, 0, 0.45, 0.0), (1.0, 12289, 1.0, 0.0),
        (0.01, 5000, 0.999, 0.0), (30.0, 0, 0.97, 0.2)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kinds", [5, 7])
def test_slices_of_other_lengths(kinds, bf16):
    """190 rows have three slices of twice the shortest length, 266 two of four times that."""
    x, noise = problem(bf16, kinds)
    rules = columns(MORE[:kinds], len(x) // kinds)
    check(x, noise, *run(x, noise, **rules), **rules)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("spread", [3.0, 0.05])
@pytest.mark.parametrize("rule", [(0.8, 0, 0.9, 0.0), (1.0, 70000, 0.8, 0.0), (1.2, 0, 1.0, 0.05), (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0)])
def test_more_than_512_slices(rule, spread, bf16):
    n = 2200003
    g = torch.Generator().manual_seed(6)
    x = spread * torch.randn(1, n, generator=g)
    x[0, 700 * 3000:] += spread             # what lies in the last slices weighs too
    noise = torch.empty(1, n).exponential_(generator=g).clamp_min(1e-20).cuda()
    x = (x.to(torch.bfloat16) if bf16 else x).cuda()
    rules = columns([rule], 1)
    check(x, noise, *run(x, noise, **rules), **rules)


def test_the_longest_vocabulary():
    n = 1 << 24
    g = torch.Generator().manual_seed(7)
    x = (2.0 * torch.randn(1, n, generator=g)).to(torch.bfloat16).cuda()
    x[0, n - 3] = 9.0
    noise = torch.empty(1, n).exponential_(generator=g).clamp_min(1e-20).cuda()
    rules = columns([(0.9, 10 ** 7, 0.7, 0.0)], 1)
    check(x, noise, *run(x, noise, **rules), **rules)
