"""Workspaces of a server's largest batch serve its smaller ones: the sizes asked
for never fall as a batch grows (CPU: queries alone)."""

import pytest

import quantized_gemm_decode_amd as ql


def rises(size, values):
    """size(v) for rising v does not fall; the first pair where it does, or None."""
    last = None
    for v in values:
        n = size(v)
        if last is not None and n < last[1]:
            return last, (v, n)
        last = v, n
    return None


SAMPLE_VOCABS = (1, 100, 4096, 4097, 8193, 16385, 32001, 50257, 128256, 151936, 1 << 20, (1 << 22) + 1, 1 << 24)


@pytest.mark.parametrize("vocab", SAMPLE_VOCABS)
def test_sampling_rows(vocab):
    size = lambda r: ql.qlinear_sample_workspace_bytes(r, vocab)    # noqa: E731
    assert rises(size, range(1, 1200)) is None
    assert rises(size, [1200 + 97 * i for i in range(600)] + [65535]) is None


@pytest.mark.parametrize("rows", (1, 2, 5, 8, 26, 27, 31, 64, 127, 128, 256, 511, 512, 513, 4000, 65535))
def test_sampling_vocabularies(rows):
    steps = sorted({1, 7} | {k * 4096 + d for k in range(1, 4097) for d in (-1, 0, 1) if k * 4096 + d <= 1 << 24})
    assert rises(lambda v: ql.qlinear_sample_workspace_bytes(rows, v), steps) is None
