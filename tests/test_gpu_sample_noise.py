"""Sampling with noise far from one: scores of weights that binary32 holds as
subnormal numbers.  Tolerance as in test_gpu_sample.py (a score is rounded twice)
and a step of 2^-149 of the weight."""

import numpy as np
import pytest
import torch

import oracle.requests as ref
from tests.gpu_util import requires_gpu
from tests.test_gpu_sample import U, run

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("rules", [{}, dict(top_k=3000), dict(top_p=0.999999)])
@pytest.mark.parametrize("bf16", [False, True])
def test_small_weights_over_small_noise(rules, bf16):
    """Weights of 2^-126 and less beside small and large noise, from the kernels' first entries to their last."""
    n, rows = 9001, 64
    g = torch.Generator().manual_seed(3)
    x = -50.0 * torch.rand(rows, n, generator=g)
    noise = 2.0 ** (20 + 20 * torch.rand(rows, n, generator=g))
    x[:, 7] = 0.0
    for i in range(rows):           # one entry of 2^-126 .. 2^-140 of the largest, whose score is the best
        x[i, 130 * i + 300] = -87.5 - 0.15 * i
        noise[i, 130 * i + 300] = 2.0 ** -124
    x = (x.to(torch.bfloat16) if bf16 else x).cuda()
    all_rows = {k: [v] * rows for k, v in rules.items()}
    tokens, _, _ = run(x, noise.cuda(), probs=False, **all_rows)
    for i in range(rows):
        score, want = ref.sample(x[i].float().cpu().numpy(), noise[i].numpy(), **{k: np.float32(v) for k, v in rules.items()})
        step = 2.0 ** -149 / noise[i, int(score.argmax())].item()
        assert want[tokens[i]] > 0 and score[tokens[i]] >= score.max() * (1 - 4 * U) - step, (i, int(tokens[i]), int(score.argmax()))
