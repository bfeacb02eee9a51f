"""Sampling on the GPU against the oracle in 64 bits.

What is kept has to be the same set; tolerances (u = 2^-24): a score w / noise
is rounded twice, so the token's score is within 4 u of the best one; a
probability is rounded once, from a mass that is a sum of steps of 2^-36 (half
a step each, and 10^-11 of a weight): u of it + 2^-33; its logarithm u of
itself + 2^-33 relative in its argument.
"""

import numpy as np
import pytest
import torch

import oracle.requests as ref
import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


def run(logits, noise, probs=True, stream=None, **rules):
    rows, vocab = logits.shape
    tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    logs = torch.full((rows,), 7.0, device="cuda")
    p = torch.full((rows, vocab), 7.0, device="cuda") if probs else None
    ws = ql.sample_workspace(rows, vocab)
    ws.fill_(255)
    dev = {k: None if v is None else torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda()
           for k, v in rules.items()}
    ql.qlinear_sample(logits, noise, tokens, ws, logprobs=logs, probs=p, stream=stream, **dev)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), logs.double().cpu().numpy(), None if p is None else p.double().cpu().numpy()


def check(logits, noise, tokens, logs, probs, **rules):
    x, e = logits.float().cpu().numpy(), noise.cpu().numpy()
    for i in range(len(x)):
        mine = {k: None if v is None else np.float32(v[i]) if k != "top_k" else v[i] for k, v in rules.items()}
        score, want = ref.sample(x[i], e[i], **mine)
        if not want.any():
            assert tokens[i] == -1 and np.isneginf(logs[i]) and (probs is None or not probs[i].any()), i
            continue
        t = int(tokens[i])
        assert 0 <= t < len(want) and want[t] > 0, (i, t, mine)
        assert score[t] >= score.max() * (1 - 4 * U), (i, t, int(score.argmax()))
        if (score >= score.max() * (1 - 4 * U)).sum() == 1:
            assert t == int(score.argmax())
        assert abs(logs[i] - np.log(want[t])) <= U * abs(np.log(want[t])) + 2.0 ** -33, (i, logs[i], np.log(want[t]))
        if probs is not None:
            # a weight below the range of binary32 may be 0
            assert np.array_equal(probs[i] > 0, want.astype(np.float32) > 0) or (
                np.abs(probs[i] - want)[(probs[i] > 0) != (want.astype(np.float32) > 0)] < 1e-44).all(), i
            assert (np.abs(probs[i] - want) <= U * want + 2.0 ** -33 * want + 1e-45).all(), i


RULES = [  # temperature, top_k, top_p, min_p
    (1.0, 0, 1.0, 0.0), (0.0, 50, 0.9, 0.1), (0.7, 1, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0),
    (0.6, 40, 0.8, 0.0), (1.0, 0, 1.0, 0.05), (0.9, 30, 1.0, 0.02), (0.8, 0, 0.95, 0.01), (1.0, 100, 0.5, 0.3),
    (NAN, 3, 0.5, 0.1), (-1.0, 0, 1.0, 0.0), (1e4, 0, 0.3, 0.0), (INF, 7, 1.0, 0.0), (1e-3, 0, 0.9, 0.0),
    (1e-20, 5, 0.9, 0.5), (1.0, 0, 0.0, 0.0), (1.0, 0, -1.0, 0.0), (1.0, 0, NAN, NAN), (1.0, -5, 2.0, -1.0),
    (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, 3.0), (2.0, 10 ** 9, 0.99, 0.0), (5.0, 5000, 0.999, 1e-6), (1.0, 0, 1e-30, 0.0),
    (INF, 0, 0.5, 0.0), (1.0, 0, 0.999999, 0.0), (1e30, 2500, 0.7, 0.9),
]


def columns(rows):
    r = [RULES[i % len(RULES)] for i in range(rows)]
    return dict(temperature=[x[0] for x in r], top_k=[x[1] for x in r], top_p=[x[2] for x in r], min_p=[x[3] for x in r])


def problem(seed, rows, vocab, bf16, spread=2.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(rows, vocab + pad, generator=g)
    noise = torch.empty(rows, vocab).exponential_(generator=g).clamp_min(1e-20)
    return (x.to(torch.bfloat16) if bf16 else x).cuda()[:, :vocab], noise.cuda()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 255, 2047, 2048, 2049, 4001, 32001])
def test_rules(vocab, bf16):
    logits, noise = problem(vocab, len(RULES), vocab, bf16, pad=vocab % 2)
    rules = columns(len(RULES))
    check(logits, noise, *run(logits, noise, **rules), **rules)


@pytest.mark.parametrize("rows,vocab,bf16,spread", [(84, 50257, True, 3.0), (80, 50257, False, 0.05), (3, 151936, True, 2.0),
                                                    (56, 70001, False, 20.0)])
def test_many_entries(rows, vocab, bf16, spread):
    """Both lengths of a slice; flat rows, whose border has more candidates than a workgroup holds."""
    logits, noise = problem(vocab, rows, vocab, bf16, spread)
    rules = columns(rows)
    check(logits, noise, *run(logits, noise, **rules), **rules)


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", None])
def test_single_rules(name):
    """Rules that no row has are NULL."""
    logits, noise = problem(3, len(RULES), 5003, False)
    rules = {k: v for k, v in columns(len(RULES)).items() if k == name}
    check(logits, noise, *run(logits, noise, **rules), **rules)
    tokens, logs, _ = run(logits, noise, probs=False, **rules)
    check(logits, noise, tokens, logs, None, **rules)


def special_rows(n):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(24, n, generator=g)
    x[0] = 0.25                                     # all alike
    x[1] = -INF                                     # nothing
    x[2] = NAN
    x[3, :] = -INF
    x[3, n // 2] = -40.0                            # one entry
    x[4, ::2] = -INF                                # a mask
    x[5, 1::3] = NAN
    x[6, 5] = x[6, n - 2] = INF
    x[7] = torch.where(torch.arange(n) % 2 == 0, 0.0, -0.0)
    x[8] = x[8].round()                             # a few values, many entries each
    x[9] = torch.finfo(torch.float32).min           # masks of the type's lowest value
    x[9, 3] = 1.0
    x[10] = x[10] * 1e5
    x[11] = x[11] * 1e30
    x[12] = torch.finfo(torch.float32).max
    x[13] = 1e-40 * x[13]                           # subnormal
    x[14] = torch.linspace(-60, 0, n)
    x[15] = torch.linspace(50000, 50001, n)
    x[16, :7] = 30.0                                # equal ones at the top
    x[17] = -1e7
    x[17, ::5] = -1e7 + 1
    x[18] = 3e38
    x[18, :9] = -3e38
    x[19] = torch.arange(n).flip(0) * 1e-7
    return x


@pytest.mark.parametrize("rule", range(len(RULES)))
def test_special_rows(rule):
    n = 3001
    x = special_rows(n)
    noise = torch.empty(24, n).exponential_(generator=torch.Generator().manual_seed(4)).clamp_min(1e-20).cuda()
    t, k, p, m = RULES[rule]
    rules = dict(temperature=[t] * 24, top_k=[k] * 24, top_p=[p] * 24, min_p=[m] * 24)
    check(x.cuda(), noise, *run(x.cuda(), noise, **rules), **rules)


def test_ties_go_to_the_lowest_index():
    """Equal logits are kept from the lowest index on; equal scores give the lowest."""
    x = torch.zeros(4, 9001, device="cuda")
    noise = torch.ones(4, 9001, device="cuda")
    rules = dict(top_k=[1, 4000, 0, 0], top_p=[1.0, 1.0, 0.5, 1.0])
    tokens, logs, probs = run(x, noise, **rules)
    assert tokens.tolist() == [0] * 4
    kept = [1, 4000, 4501, 9001]            # 4500 entries before it weigh 4500 < 4500.5
    for i, n in enumerate(kept):
        assert (probs[i, :n] > 0).all() and not probs[i, n:].any(), i
    # exactly on the border: the second of two equal entries has half before it
    two, e = torch.zeros(1, 2, device="cuda"), torch.tensor([[5.0, 1e-3]], device="cuda")
    assert run(two, e, top_p=[0.5])[2].tolist() == [[1.0, 0.0]]


@pytest.mark.parametrize("bf16", [False, True])
def test_strided_rows_at_any_alignment(bf16):
    base, noise = problem(12, 6, 2501, bf16, pad=40)
    rules = columns(6)
    for off in range(1, 9):
        wide = torch.zeros(6, 2560, dtype=base.dtype, device="cuda")
        wide[:, off:off + 2501] = base
        wide[:, :off] = wide[:, off + 2501:] = INF      # beside the row: not looked at
        x = wide[:, off:off + 2501]
        check(x, noise, *run(x, noise, **rules), **rules)


def test_draws_follow_the_probabilities():
    """40,000 draws among 5 kept entries: each count within 5 standard deviations."""
    rows = 40000
    row = torch.tensor([1.0, 0.5, 0.0, -0.5, -1.0] + [-3.0] * 12)
    g = torch.Generator().manual_seed(0)
    noise = torch.empty(rows, 17).exponential_(generator=g).clamp_min(1e-20).cuda()
    x = row.cuda().expand(rows, 17).contiguous()
    tokens, _, _ = run(x, noise, probs=False, top_k=[5] * rows)
    p = torch.softmax(row[:5].double(), 0).numpy()
    n = np.bincount(tokens, minlength=17)
    assert not n[5:].any() and (np.abs(n[:5] - rows * p) <= 5 * np.sqrt(rows * p * (1 - p))).all()


def test_repeat_streams_and_replays():
    logits, noise = problem(31, 28, 9001, True)
    rules = columns(28)
    first = run(logits, noise, **rules)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(logits, noise, stream=side, **rules)
    assert all(np.array_equal(x, y) for x, y in zip(first, again))
    tokens, logs = torch.zeros(28, dtype=torch.int32, device="cuda"), torch.zeros(28, device="cuda")
    probs, ws = torch.zeros(28, 9001, device="cuda"), ql.sample_workspace(28, 9001)
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda() for k, v in rules.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ql.qlinear_sample(logits, noise, tokens, ws, logprobs=logs, probs=probs, **dev)
    for i in range(4):
        logits.copy_(torch.roll(logits, i, 1))
        ws.fill_(255 - i)
        graph.replay()
        torch.cuda.synchronize()
        want = run(logits, noise, **rules)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(probs.double().cpu().numpy(), want[2])
        assert np.array_equal(logs.double().cpu().numpy(), want[1])


def test_probabilities_serve_the_verification():
    """The target's and the draft's filtered distributions into the verification: a draft that the target keeps
    with certainty is accepted, one that it does not keep is not."""
    vocab = 1000
    logits, _ = problem(8, 4, vocab, True)
    noise = torch.ones(4, vocab, device="cuda")
    probs = torch.zeros(4, vocab, device="cuda")
    tokens, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), ql.sample_workspace(4, vocab)
    k = torch.tensor([1, 5, 1, 5], dtype=torch.int32, device="cuda")
    ql.qlinear_sample(logits, noise, tokens, ws, top_k=k, probs=probs)
    drafts = torch.stack([logits[0].argmax(), logits[2].argmin()]).int()
    out, accepted = (torch.empty(2, 2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"))
    ql.qlinear_verify_draft(probs, None, drafts, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"),
                            torch.tensor([0.5, 0.0], device="cuda"), noise[:2].contiguous(), out, accepted,
                            ql.verify_workspace(2, vocab))
    assert accepted.tolist() == [1, 0] and out[0].tolist() == [int(drafts[0]), int(tokens[1])]
    assert out[1].tolist() == [int(tokens[2]), -1]
