"""Low-rank adapters beside a projection on the GPU against the oracle in 64 bits.

Tolerance, from the operator's arithmetic (u = 2^-24): the first sum loses at
most (K + 64) u of |A| |x|, twice that counting the matrix core's truncated
alignment; it enters the second product as two bf16 numbers, off by 2^-16 of it
and the scale's u; the second sum loses (2 R + 4) u, twice that, of |B| |h|; y's
addition u; then one rounding to bf16 (2^-8).
"""

import numpy as np
import pytest
import torch

import oracle.requests as ref
import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]
U = 2.0 ** -24
BF16 = torch.bfloat16


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


class Problem:
    def __init__(self, seed, adapters, n_adapters, rank, k, widths, x_pad=0, y_pad=0, scales=True, pool=1):
        g = torch.Generator().manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g)

        T, wide = len(adapters), sum(widths)
        x = randn(T, k)
        x[:, :2] *= 10
        self.x = torch.zeros(T, k + x_pad, dtype=BF16)
        self.x[:, :k] = x.to(BF16)
        self.x = self.x.cuda()[:, :k]
        self.y_all = (randn(T, wide + y_pad)).to(BF16).cuda()
        self.y = self.y_all[:, :wide]
        self.a = (randn(n_adapters, pool, len(widths) * rank, k) * k ** -0.5).to(BF16).cuda()[:, pool - 1]
        self.b = (randn(n_adapters, pool, wide, rank)).to(BF16).cuda()[:, pool - 1]
        self.scales = (0.5 + torch.rand(n_adapters, generator=g)).cuda() if scales else None
        self.widths, self.rank, self.k = widths, rank, k
        self.adapters = torch.tensor(adapters, dtype=torch.int32)
        self.stack = ql.LoraStack(self.a, self.b, self.scales, widths)

    def run(self, inplace=False, stream=None):
        y = self.y_all.clone()[:, :self.y.shape[1]]
        out = y if inplace else torch.full((y.shape[0], y.shape[1] + 8), 7.0, dtype=BF16, device="cuda")[:, :y.shape[1]]
        ws = ql.lora_workspace(self.stack, len(self.adapters))
        ws.fill_(255)
        ql.qlinear_lora(self.stack, self.x, y, self.adapters.cuda(), ws, out=None if inplace else out, stream=stream)
        torch.cuda.synchronize()
        return out

    def check(self, out):
        want, first, second = ref.lora(f64(self.x), f64(self.y), self.adapters.tolist(), f64(self.a), f64(self.b),
                                       f64(self.scales), self.widths)
        d = 2 * (self.k + 64) * U * first + second * (2.0 ** -16 + U + 2 * (2 * self.rank + 4) * U)
        tol = d + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + 2 * U * np.abs(f64(self.y)) + 1e-38
        err = np.abs(f64(out) - want)
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(err / tol)))
        none = (self.adapters < 0) | (self.adapters >= self.a.shape[0])
        assert torch.equal(out[none.cuda()], self.y[none.cuda()])


CASES = [  # adapters of the tokens, adapters, rank, K, widths, x_pad, y_pad, pool
    ([0], 1, 8, 64, [64], 0, 0, 1),
    ([0], 3, 16, 4096, [4096, 1024, 1024], 0, 0, 1),
    ([2], 3, 16, 8, [8], 8, 8, 2),                                            # the smallest sizes
    ([-1], 3, 16, 128, [128], 0, 0, 1),
    ([1, 1, 0, 5, 2, 1, -1, 7], 6, 16, 520, [136, 72], 0, 0, 1),              # 5, 7: no such adapter
    (list(range(64)), 64, 32, 256, [200], 0, 64, 1),                          # a full block of distinct adapters
    ([i % 3 for i in range(33)], 3, 64, 1000, [72, 64, 8], 24, 0, 3),         # more tokens of one adapter than a tile
    ([3] * 64, 4, 128, 512, [128], 0, 0, 1),
    ([0, 1] * 20, 2, 24, 384, [64, 56, 64, 40], 0, 0, 1),                     # a rank between; four slices
    ([i // 30 for i in range(65)], 3, 16, 256, [264], 0, 0, 1),               # one token beyond a block
    ([i // 90 - 1 for i in range(450)], 5, 16, 640, [128, 64], 8, 8, 2),      # prompts; the first without an adapter
    ([(i * 7) % 11 for i in range(200)], 11, 40, 192, [72], 0, 0, 1),         # mixed up
    ([1] * 130, 2, 128, 128, [64], 0, 0, 1),
    ([i // 50 for i in range(150)], 3, 8, 72, [16], 0, 0, 1),
    ([0] * 100 + [1] * 29, 2, 64, 2048, [320], 0, 0, 1),
    ([0, 1, -1], 2, 88, 328, [88, 24], 0, 0, 1),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("inplace", [False, True])
def test_lora(i, inplace):
    adapters, n, rank, k, widths, x_pad, y_pad, pool = CASES[i]
    p = Problem(i, adapters, n, rank, k, widths, x_pad, y_pad, scales=i % 4 != 3, pool=pool)
    p.check(p.run(inplace))


def test_neighbouring_columns_stay():
    """What lies beside out's columns is not written."""
    p = Problem(77, [0, 1, 0], 2, 16, 128, [72], y_pad=8)
    out = torch.full((3, 80), 7.0, dtype=BF16, device="cuda")
    ql.qlinear_lora(p.stack, p.x, p.y, p.adapters.cuda(), ql.lora_workspace(p.stack, 3), out=out[:, :72])
    assert (out[:, 72:] == 7).all()
    p.check(out[:, :72])


@pytest.mark.parametrize("tokens", [12, 140])
def test_nonfinite_weights_reach_their_own_tokens_only(tokens):
    p = Problem(5, [i % 3 for i in range(tokens)], 3, 16, 256, [64])
    want = p.run()
    p.a[1, 3, 5] = float("inf")
    p.b[1, 7, 2] = float("nan")
    p.x[2, 9] = float("nan")
    got = p.run()
    ok = torch.ones(tokens, dtype=torch.bool)
    ok[1::3] = False
    ok[2] = False
    assert torch.equal(got[ok.cuda()], want[ok.cuda()])
    assert not torch.isfinite(got[1]).all() and torch.isnan(got[2]).all()


def test_no_tokens_and_no_adapters():
    p = Problem(6, [0], 1, 16, 64, [64])
    none = torch.zeros(0, 64, dtype=BF16, device="cuda")
    ql.qlinear_lora(p.stack, none, none, torch.zeros(0, dtype=torch.int32, device="cuda"), ql.lora_workspace(p.stack, 0))
    empty = ql.LoraStack(p.a[:0], p.b[:0])
    out = torch.zeros_like(p.y)
    ql.qlinear_lora(empty, p.x, p.y, torch.tensor([0], dtype=torch.int32).cuda(), ql.lora_workspace(empty, 1), out=out)
    assert torch.equal(out, p.y)


def test_results_repeat_and_replay():
    """The same bits in every run, on another stream, and in every replay of a captured call with new inputs between."""
    p = Problem(8, [i % 5 - 1 for i in range(48)], 4, 16, 1024, [256, 64])
    first = p.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(first, p.run(stream=side))
    ws, out, ad = ql.lora_workspace(p.stack, 48), torch.zeros_like(p.y), p.adapters.cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ql.qlinear_lora(p.stack, p.x, p.y, ad, ws, out=out)
    for i in range(4):
        p.x.mul_(-1.0 if i else 1.0)
        ad.copy_(torch.roll(ad, i))
        p.adapters = ad.cpu()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        p.check(out)
        assert torch.equal(out, p.run())
