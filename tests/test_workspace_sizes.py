"""Workspaces of a server's largest batch serve its smaller ones: the sizes asked
for never fall as a batch grows (CPU: queries alone)."""

import ctypes

import pytest

import quantized_gemm_decode_amd as ql
from quantized_gemm_decode_amd._lib import QLLora


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


def lora(adapters, rank, k, slices):
    return QLLora(None, None, None, slices * rank * k, slices * 64 * rank, k, (ctypes.c_int64 * 4)(*([64] * slices)), adapters, rank,
                  slices)


@pytest.mark.parametrize("adapters,rank,k,slices", [(8, 16, 4096, 3), (32, 16, 4096, 3), (1, 8, 512, 1), (4, 32, 5120, 2), (0, 16, 4096, 1),
                                                    (500, 128, 17408, 4), (65536, 64, 28672, 1), (3, 8, 8, 1), (2, 16, 1 << 20, 1),
                                                    (16, 64, 2048, 4)])
def test_adapter_tokens(adapters, rank, k, slices):
    s = lora(adapters, rank, k, slices)
    size = lambda t: ql.lib().qlinear_lora_workspace_bytes(ctypes.byref(s), t)      # noqa: E731
    assert rises(size, range(1, 40000)) is None
    assert rises(size, [40000 + 9973 * i for i in range(1600)] + [1 << 24]) is None


def test_adapter_sizes_hold_what_a_call_needs():
    """The chunks of K that a call makes (see lora_shape), for every token, slice and rank in binary32."""
    for adapters, rank, k, slices in ((8, 16, 4096, 3), (40, 64, 17408, 2), (2, 128, 100000, 4)):
        for tokens in list(range(1, 300)) + [1000, 4096, 4097, 16384, 16385, 100000]:
            blocks, wide = -(-tokens // 64), tokens > 64
            slots = 2 if wide else max(1, min(tokens, adapters + 1 + tokens // 16))
            chunks = max(1, min(-(-k // 512), 1024 // (blocks * slots * -(-slices * rank // 64))))
            chunk = (-(-k // chunks) + 255) // 256 * 256
            s = lora(adapters, rank, k, slices)
            need = -(-k // chunk) * tokens * slices * rank * 4
            assert ql.lib().qlinear_lora_workspace_bytes(ctypes.byref(s), tokens) >= need, (adapters, rank, k, slices, tokens)


@pytest.mark.parametrize("vocab", (1, 1023, 2048, 4096, 32001, 151936, 1 << 20, 1 << 30))
def test_verification_sequences(vocab):
    size = lambda b: ql.qlinear_verify_workspace_bytes(b, vocab)    # noqa: E731
    assert rises(size, range(1, 3000)) is None
    assert rises(size, [3000 + 97 * i for i in range(600)] + [65535]) is None


@pytest.mark.parametrize("batch", (1, 2, 3, 7, 64, 100, 511, 512, 513, 1024, 65535))
def test_verification_vocabularies(batch):
    steps = sorted({1, 7} | {k * m + d for k in range(1, 3000) for m in (1024, 4092) for d in (-1, 0, 1, 4, 5)})
    assert rises(lambda v: ql.qlinear_verify_workspace_bytes(batch, v), steps) is None
