"""Adapters whose inner sums reach the end of binary32's range."""

import pytest
import torch

import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]
BF16 = torch.bfloat16


@pytest.mark.parametrize("rank", [8, 24, 64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sums_above_the_largest_bf16_number(rank, sign):
    """1.998 2^127 rounds to infinity as bf16, not as binary32: out = 2^-100 of it, to 2^-16 and a rounding (2^-8)."""
    K, N = 64, 72
    x = torch.zeros(2, K)
    x[:, 0], x[:, 1] = 2.0 ** 63, sign * 2.0 ** 63
    x[:, 0] *= sign
    x[1] = 0.0
    a = torch.zeros(1, rank, K)
    a[0, 3, 0], a[0, 3, 1] = 1.9921875 * 2.0 ** 64, 0.005859375 * 2.0 ** 64
    b = torch.zeros(1, N, rank)
    b[0, :, 3] = 2.0 ** -100 * (1 + torch.arange(N) % 3)
    x, a, b = (t.to(BF16).cuda() for t in (x, a, b))
    y = torch.ones(2, N, dtype=BF16, device="cuda")
    stack = ql.LoraStack(a, b)
    out = torch.zeros_like(y)
    ql.qlinear_lora(stack, x, y, torch.zeros(2, dtype=torch.int32, device="cuda"), ql.lora_workspace(stack, 2), out=out)
    inner = (x[0].double().cpu() * a[0, 3].double().cpu()).sum()
    assert abs(inner) > torch.finfo(BF16).max and abs(inner) < torch.finfo(torch.float32).max
    want = 1.0 + inner * b[0, :, 3].double().cpu()
    assert ((out[0].double().cpu() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20)).all(), out[0, :4].tolist()
    assert torch.equal(out[1], y[1])


@pytest.mark.parametrize("rank", [8, 24, 64])
def test_infinite_and_nan_sums(rank):
    """As 32 bits have them: infinity, its negative, NaN; a zero of B beside an infinity is NaN."""
    K, N = 64, 64
    x = torch.zeros(4, K)
    x[0, 5], x[1, 5], x[2, 5], x[3, 5] = float("inf"), -float("inf"), float("nan"), 1.0
    a, b = torch.ones(1, rank, K), torch.ones(1, N, rank)
    b[0, 7] = 0.0
    b[0, 9] = -1.0
    x, a, b = (t.to(BF16).cuda() for t in (x, a, b))
    y = torch.ones(4, N, dtype=BF16, device="cuda")
    stack = ql.LoraStack(a, b)
    ql.qlinear_lora(stack, x, y, torch.zeros(4, dtype=torch.int32, device="cuda"), ql.lora_workspace(stack, 4))
    inf = float("inf")
    rest = [n for n in range(N) if n not in (7, 9)]
    assert (y[0, rest] == inf).all() and y[0, 9] == -inf and torch.isnan(y[0, 7])
    assert (y[1, rest] == -inf).all() and y[1, 9] == inf and torch.isnan(y[1, 7])
    assert torch.isnan(y[2]).all()
    assert (y[3, rest] == 1 + rank).all() and y[3, 7] == 1 and y[3, 9] == 1 - rank
