"""The example of a server with adapters and trees of drafts: the four operators of
a step one after the other (captured and not), against the model in 64 bits."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("tree_serving", os.path.join(ROOT, "examples", "tree_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rms(x):
    return float(x.square().mean().sqrt())


def reference(model, text, adapter):
    """(logits, keys, values) of every token of `text`, float64 on the CPU."""
    H, Hk, D = model.q_heads, model.kv_heads, model.head_dim
    w = {n: t.double().cpu() for n, t in model.weights.items()}
    x = model.embedding.cpu()[torch.tensor(text)].double()
    y = x @ w["qkv"].T
    if adapter >= 0:
        s = model.adapters
        a, b, rank = s.a[adapter].double().cpu(), s.b[adapter].double().cpu(), s.b.shape[2]
        down = x @ a.T
        n = 0
        for j, width in enumerate(s.widths):
            y[:, n:n + width] += float(s.scales[adapter]) * (down[:, j * rank:(j + 1) * rank] @ b[n:n + width].T)
            n += width
    heads = y.view(len(text), H + 2 * Hk, D)
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
    return (x + a.reshape(len(text), H * D) @ w["o"].T) @ w["head"].T, k, v


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("capture", [False, True])
def test_trees_follow_the_model(capture, e4m3):
    """Logits at the nodes of each accepted branch, and the keys and values that
    the cache holds at last, stay within the noise of the 8-bit formats: 0.037 of
    the root mean square for one E4M3 rounding (2^-3 / sqrt(12)), two of them in a
    linear's output and one in the cache, 0.14 along the whole path.  A wrong
    adapter, position, page or place gives an error of the size of 1: the
    bound is 0.25.  An adapter's own part is bf16's (0.4 % of a term).  Greedy rows
    draw the first largest logit, and a row of top_k 2 one of its two largest,
    exactly.  A greedy row's log-probability is that of its one entry's weight, 1,
    over the same weight's mass in the sums: a number of steps of 2^-34, at
    least exp(-1/16) of them, so rounded by 2^-35 / 0.939 = 3.1e-11 at most, and of
    a series off by 3e-12: below 4e-11."""
    ex = load_example()
    model = ex.Model(adapters=3, rank=8, q_heads=8, kv_heads=2, head_dim=64, vocab=1024, max_pos=512)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(1024, (n,), generator=g).tolist() for n in (130, 17, 64, 70)]
    for p in prompts:
        p += p[:8]                                     # something for the drafts to find
    adapter = [1, -1, 2, 1]
    rules = [dict(temperature=0.0), dict(temperature=0.8, top_p=0.9), dict(top_k=2), dict(temperature=0.0)]
    server = ex.Server(model, prompts, adapter, rules, 3, 4, 60, page_size=16, e4m3=e4m3)
    server.prefill(200)                                # chunks of 50 tokens a sequence
    n = server.nodes
    assert n == 13
    rows = []                                          # (sequence, position, logits)
    for _ in range(10):
        before = [len(t) for t in server.text]
        accepted = server.step(capture)
        logits = server.logits.float().cpu().view(4, n, -1)
        drawn, logprobs = server.sampled.cpu().view(4, n), server.logprobs.cpu().view(4, n)
        for b in (0, 3):
            assert drawn[b].tolist() == logits[b].numpy().argmax(-1).tolist()
            assert float(logprobs[b].abs().max()) < 4e-11
        two = logits[2].topk(2).values[:, 1]
        assert (logits[2].gather(1, drawn[2].long()[:, None])[:, 0] >= two).all()
        tokens, parents = server.trees.tokens.cpu().view(4, n), server.trees.parents.cpu().view(4, n)
        for b in range(4):
            assert 0 <= accepted[b] <= 4 and len(server.text[b]) == before[b] + accepted[b] + 1
            assert int(server.new_lens[b]) == len(server.text[b]) - 1
            node = 0                                   # down the branch again, by the text
            for i in range(accepted[b] + 1):
                rows.append((b, before[b] - 1 + i, logits[b, node]))
                draw = server.text[b][before[b] + i]
                assert draw == int(drawn[b, node])
                below = [c for c in range(n) if int(parents[b, c]) == node and int(tokens[b, c]) == draw]
                assert (i < accepted[b]) <= bool(below)
                node = below[0] if below else -1
    for b, text in enumerate(server.text):
        want, k, v = reference(model, text, adapter[b])
        for c, i, got in rows:
            if c == b:
                assert rms(got.double() - want[i]) < 0.25 * rms(want[i]), (b, i)
        held = len(text) - 1                           # the newest token is not in the cache yet
        at = torch.arange(held)
        slots = server.page_table.cpu()[b, at // 16].long() * 16 + at % 16
        for cache, exact in ((server.cache.k, k), (server.cache.v, v)):
            got = cache.float().cpu().view(-1, 2, 64)[slots].double()
            err = (got - exact[:held]).square().mean((1, 2)).sqrt() / exact[:held].square().mean((1, 2)).sqrt()
            assert float(err.max()) < 0.25, (b, int(err.argmax()), float(err.max()))
