"""The serving example: a prompt's chunk and speculative steps (captured and
not) of a one-layer model, against the model in 64 bits on its final texts."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("speculative_serving", os.path.join(ROOT, "examples", "speculative_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(model, text):
    """Logits after every token of `text`, from the unquantized weights, float64 on the CPU."""
    H, Hk, D = model.q_heads, model.kv_heads, model.head_dim
    w = {n: t.double().cpu() for n, t in model.weights.items()}
    x = model.embedding.cpu()[torch.tensor(text)].double()
    heads = (x @ w["qkv"].T).view(len(text), H + 2 * Hk, D)
    table = model.cos_sin.cpu()[:len(text)].double()
    cos, sin = table[:, None, :D // 2], table[:, None, D // 2:]

    def rotate(t, weight):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double().cpu()
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    q, k, v = rotate(heads[:, :H], model.q_norm), rotate(heads[:, H:H + Hk], model.k_norm), heads[:, H + Hk:]
    hidden = torch.ones(len(text), len(text), dtype=torch.bool).triu(1)
    a = torch.empty(len(text), H, D, dtype=torch.float64)
    for h in range(H):
        kh, vh = k[:, h * Hk // H], v[:, h * Hk // H]
        a[:, h] = (q[:, h] @ kh.T * D ** -0.5).masked_fill(hidden, float("-inf")).softmax(-1) @ vh
    return (x + a.reshape(len(text), H * D) @ w["o"].T) @ w["head"].T


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("capture", [False, True])
def test_speculative_serving_follows_the_model(capture, e4m3):
    """Every logits row of an accepted token stays within the noise of the
    8-bit formats: an E4M3 rounding has a relative error of 2^-4 at most and
    0.037 root mean square if it is spread evenly over a binade's widest step
    (2^-3 / sqrt(12)).  A linear's output has two of them (0.051).  Along the
    path: V (with its cache rounding 0.063), O's input 0.051 and the head's
    0.051, and the scores, whose q and k errors of up to 0.063 each move
    logits of size ~1 by 0.09 and with it the weights; in quadrature 0.14.  A
    wrong position, page or length gives an error of the size of 1: the bound
    is 0.25 of the root mean square."""
    ex = load_example()
    model = ex.Model(q_heads=8, kv_heads=2, head_dim=64, vocab=1024, max_pos=512)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(1024, (n,), generator=g).tolist() for n in (130, 17, 64)]
    for p in prompts:
        p += p[:8]                                     # something for the drafts to find
    server = ex.Server(model, prompts, 3, 24, page_size=16, e4m3=e4m3, temperature=0.7)
    rows = []                                          # (sequence, position, logits)
    for c, part in enumerate(server.prefill(150, logits=True)):      # chunks of 50 tokens a sequence
        part = list(part.float().cpu())
        for b, p in enumerate(prompts):
            for i in range(50 * c, min(50 * (c + 1), len(p) - 1)):
                rows.append((b, i, part.pop(0)))
        assert not part
    accepted = []
    for _ in range(8):
        before = [len(t) for t in server.text]
        accepted += server.step(capture)
        logits = server.logits.float().cpu().view(len(prompts), 4, -1)
        for b, n in enumerate(before):
            rows += [(b, n - 1 + i, logits[b, i]) for i in range(len(server.text[b]) - n)]
        assert all(0 <= m <= 3 for m in accepted[-3:])
        assert [len(t) - n - 1 for t, n in zip(server.text, before)] == accepted[-3:]
    refs = [reference(model, t) for t in server.text]
    for b, i, got in rows:
        want = refs[b][i]
        err = (got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert err < 0.25, (b, i, float(err))
