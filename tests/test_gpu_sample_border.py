"""Top-p limits that fall between the sums of two buckets.

The kernels find the border of what top-p keeps by the masses of buckets of an
eighth of T.  These rows have a first entry of weight 1, two in the next bucket,
and a tail that brings p times the whole mass, less the 10^-10 that the search
allows, to the number right above the first bucket's.  By the definition
(p * sum = 1 + 10^-10) the first two entries are kept.
"""

import numpy as np
import pytest
import torch

from tests.gpu_util import requires_gpu
from tests.test_gpu_sample import check, run

pytestmark = [pytest.mark.gpu, requires_gpu]
P = 0.25


def weight(l):
    """exp(l) as the kernels sum it: in its bucket a multiple of 2^-34 from a polynomial, times the bucket's factor."""
    x = l.astype(np.float64) * 8.0
    f, p = x - np.floor(x), 2.54348632162432e-07
    for c in (9.53864143867337e-06, 0.0003058076755491678, 0.007339162402444752, 0.11742663303627268, 0.9394130628109114):
        p = p * f + c
    y = (0.5 + np.floor(x)) * (0.125 * 1.44269504088896340736)
    n, e = np.rint(y), 1.0 / 39916800.0
    g = (y - n) * 0.69314718055994530942
    for d in (3628800.0, 362880.0, 40320.0, 5040.0, 720.0, 120.0, 24.0, 6.0, 2.0, 1.0, 1.0):
        e = e * g + 1.0 / d
    return np.rint(p * 2.0 ** 34) / 2.0 ** 34 * np.ldexp(e, n.astype(int))


def rows(n, seed, width=16):
    r = np.random.default_rng(seed)
    x = np.full((n, width), -np.inf, np.float32)
    x[:, 0] = 0
    x[:, 1:3] = -r.uniform(0.01, 0.12, (n, 2))
    x[:, 3] = -r.uniform(1.0, 2.0, n)
    have = weight(x[:, 0]) + (weight(x[:, 1]) + weight(x[:, 2])) + weight(x[:, 3])
    target = (weight(x[:, 0]) + 2.0 ** -52) / (P * (1 - 1e-10))
    for i in range(4, width):       # entries that are not above what is left
        left = target - have
        some = left > 2.0 ** -53
        l = np.minimum(np.log(np.where(some, left, 1.0)), -0.3).astype(np.float32)
        for _ in range(3):
            l = np.where(weight(l) > left, np.nextafter(l, np.float32(-np.inf)), l)
        x[:, i] = np.where(some, l, -np.inf)
        have = have + np.where(some, weight(l), 0.0)
    return x


def test_a_limit_between_two_buckets():
    x = rows(1500, 1)
    want = np.zeros(x.shape, bool)
    want[:, 0] = True
    want[np.arange(len(x)), 1 + (x[:, 2] > x[:, 1])] = True
    # (masses are off by half a step of 2^-34 an entry: within half of what separates the limit from the first entry)
    assert (np.abs(P * np.exp(x.astype(np.float64)).sum(1) - 1 - 1e-10) < 5e-11).all()
    logits = torch.from_numpy(x).cuda()
    noise = torch.empty(x.shape).exponential_(generator=torch.Generator().manual_seed(2)).clamp_min(1e-20).cuda()
    rules = dict(top_p=[P] * len(x))
    got = run(logits, noise, **rules)
    assert np.array_equal(got[2] > 0, want), int(((got[2] > 0).sum(1) > 2).sum())
    check(logits, noise, *got, **rules)
