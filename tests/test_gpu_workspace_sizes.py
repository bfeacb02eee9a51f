"""Smaller calls in the workspace of a larger one: the same results, and nothing
behind it is written."""

import pytest
import torch

import quantized_gemm_decode_amd as ql
from tests import test_gpu_lora as lora, test_gpu_sample as sample
from tests.gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]
GUARD = 1 << 20


def guarded(size):
    """A workspace of just that size, and the memory behind it."""
    buf = torch.full((size + GUARD,), 255, dtype=torch.uint8, device="cuda")
    return buf[:size], buf[size:]


@pytest.mark.parametrize("rows,vocab,most_rows,most_vocab", [(127, 32001, 128, 32001), (26, 151936, 27, 151936), (63, 128256, 64, 128256),
                                                           (64, 114688, 64, 114689), (1, 20000, 30, 40000)])
def test_sampling(rows, vocab, most_rows, most_vocab):
    logits, noise = sample.problem(rows, rows, vocab, True)
    want = sample.run(logits, noise, probs=False, **sample.columns(rows))
    ws, behind = guarded(ql.qlinear_sample_workspace_bytes(most_rows, most_vocab))
    tokens, logs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in sample.columns(rows).items()}
    ql.qlinear_sample(logits, noise, tokens, ws, logprobs=logs, **dev)
    assert (tokens.cpu().numpy() == want[0]).all() and (logs.double().cpu().numpy() == want[1]).all()
    assert (behind == 255).all()


@pytest.mark.parametrize("tokens,most,k", [(4096, 4097, 4096), (1, 2000, 4096), (64, 65, 8192), (300, 5000, 2048)])
def test_adapters(tokens, most, k):
    p = lora.Problem(tokens, [i // 40 % 5 - 1 for i in range(tokens)], 4, 16, k, [64, 64, 64])
    want = p.run()
    ws, behind = guarded(ql.qlinear_lora_workspace_bytes(p.stack, most))
    out = torch.zeros_like(p.y)
    ql.qlinear_lora(p.stack, p.x, p.y, p.adapters.cuda(), ws, out=out)
    assert torch.equal(out, want) and (behind == 255).all()


@pytest.mark.parametrize("batch,vocab,most", [(512, 3000, 513), (8, 32001, 9), (6, 151936, 7)])
def test_verification(batch, vocab, most):
    """Without drafts the next token is argmax p / noise."""
    g = torch.Generator().manual_seed(vocab)
    probs = torch.rand(batch, vocab, generator=g).cuda()
    noise = torch.ones(batch, vocab, device="cuda")
    ws, behind = guarded(ql.qlinear_verify_workspace_bytes(most, vocab))
    out, accepted = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((batch, 2), (batch,)))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    ql.qlinear_verify_draft(probs, None, none, torch.zeros(batch + 1, dtype=torch.int32, device="cuda"),
                            torch.zeros(0, device="cuda"), noise, out, accepted, ws)
    assert torch.equal(out[:, 0].long(), probs.argmax(-1)) and not accepted.any() and (out[:, 1] == -1).all()
    assert (behind == 255).all()
