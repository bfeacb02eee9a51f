"""Adapters, sampling, trees and their commit: infinities, offsets beyond 32 bits,
two streams at once, two graphs over one workspace."""

import pytest
import torch

import quantized_gemm_decode_amd as ql
from tests import test_gpu_lora as lora, test_gpu_sample as sample
from tests.gpu_util import requires_gpu
from tests.test_gpu_tree import Tree

pytestmark = [pytest.mark.gpu, requires_gpu]
BF16 = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rank", [8, 24, 64])
def test_an_infinite_activation_is_an_infinite_sum(rank):
    """Positive weights: every column of an infinite token is +inf, of a negative one -inf."""
    p = lora.Problem(9, [0, 1, 0, 1, -1], 2, rank, 128, [64, 72])
    p.a.copy_(p.a.abs() + 0.01)
    p.b.copy_(p.b.abs() + 0.01)
    p.x[1, 9], p.x[2, 70], p.x[4, 3] = float("inf"), -float("inf"), float("inf")
    out = p.run()
    assert (out[1] == float("inf")).all() and (out[2] == -float("inf")).all()
    assert torch.isfinite(out[[0, 3]]).all() and torch.equal(out[4], p.y[4])


@pytest.mark.parametrize("tokens", [10, 70])
def test_adapters_far_apart(tokens):
    """Rows and adapters more than 2^32 bytes apart: the same bits as close together."""
    p = lora.Problem(21, [i % 3 - 1 for i in range(tokens)], 2, 16, 256, [64, 72])
    step, wide = 2 ** 32 // (tokens - 2) // 8 * 8, 136

    def far(t, step):
        big = torch.empty((t.shape[0] - 1) * step + t[0].numel(), dtype=BF16, device="cuda")
        view = big.as_strided(t.shape, (step, *t.stride()[1:]))
        view.copy_(t)
        return view
    a, b = far(p.a.contiguous(), 2 ** 32), far(p.b.contiguous(), 2 ** 32)
    out = far(torch.zeros_like(p.y), step)
    stack = ql.LoraStack(a, b, p.scales, p.widths)
    ql.qlinear_lora(stack, far(p.x, step), far(p.y, step), p.adapters.cuda(), ql.lora_workspace(stack, tokens), out=out)
    assert out.stride(0) * (tokens - 1) * 2 > 2 ** 32 and out.shape[1] == wide
    assert torch.equal(out.contiguous(), p.run())


def test_logits_far_apart():
    logits, noise = sample.problem(31, 4, 5003, True)
    big = torch.empty(3 * 2 ** 30 + 5003, dtype=BF16, device="cuda").as_strided((4, 5003), (2 ** 30, 1))
    big.copy_(logits)
    rules = dict(temperature=[0.8, 1.0, 0.0, 1.3], top_k=[0, 50, 0, 900], top_p=[0.9, 1.0, 1.0, 0.95], min_p=[0.0, 0.0, 0.0, 0.001])
    got, want = sample.run(big, noise, **rules), sample.run(logits, noise, **rules)
    assert all((x == y).all() for x, y in zip(got, want))


@pytest.mark.parametrize("new", [[5, 4], [60, 33]])
def test_trees_and_their_commit_on_far_pages(new):
    """Pages behind 2^32 bytes of a cache: the same bits as in a small one."""
    p = Tree(41, new, [700, 333], 8, 2, 128, 16, False)
    pages, first = p.cache.k.shape[0], 2 ** 32 // (16 * 2 * 128 * 2) + 5
    big = [torch.empty(first + pages, 16, 2, 128, dtype=BF16, device="cuda") for _ in range(2)]
    near = [t.contiguous().clone() for t in (p.cache.k, p.cache.v)]
    for b, t in zip(big, near):
        b[first:].copy_(t)
    want, want_ls = p.run(p.plan())
    old = p.cache.k, p.cache.v
    small, far = ql.PagedCache(*near), ql.PagedCache(*big)
    p.cache, table = far, p.table
    p.table = table + first
    out, ls = p.run(p.plan())
    assert torch.equal(out, want) and torch.equal(ls, want_ls)
    T, cu = sum(new), [0, new[0], sum(new)]
    parents = i32([-1, 0, 1, 1, 3] + [-1] * (new[0] - 5) + [-1, 0, 0, 2] + [-1] * (new[1] - 4))
    names, drawn = torch.arange(T, dtype=torch.int32, device="cuda"), torch.full((T,), -9, dtype=torch.int32, device="cuda")
    drawn[0], drawn[1], drawn[3], drawn[cu[1]], drawn[cu[1] + 2] = 1, 3, 4, cu[1] + 2, cu[1] + 3
    for cache, tab in ((small, table), (far, p.table)):
        outs, accepted, lens = torch.zeros(2, 5, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([0, 0])
        ql.qlinear_tree_commit([cache], tab.cuda(), p.lens.cuda(), i32(cu), names, parents, drawn, outs, accepted, lens)
        assert accepted.tolist() == [3, 2] and lens.tolist() == [700 - new[0] + 4, 333 - new[1] + 3]
    for b, t, before in zip(big, near, old):
        # (bits: what lies beyond the sequences is NaN)
        assert torch.equal(b[first:].view(torch.int16), t.view(torch.int16))
        assert not torch.equal(t.view(torch.int16), before.contiguous().view(torch.int16))


def test_two_streams_at_once():
    """Calls of both streams with workspaces of their own, one behind the other without waits between the streams."""
    p = [lora.Problem(51 + i, [(j + i) % 4 - 1 for j in range(64)], 3, 16, 2048, [512, 256]) for i in range(2)]
    s = [sample.problem(61 + i, 24, 40000, True) for i in range(2)]
    trees = [Tree(71 + i, [33, 20], [900, 1400], 8, 2, 128, 16, False) for i in range(2)]
    want = [(p[i].run(), sample.run(*s[i])[0], trees[i].run(trees[i].plan())[0]) for i in range(2)]
    ad = [x.adapters.cuda() for x in p]
    outs = [(torch.zeros_like(p[i].y), torch.zeros(24, dtype=torch.int32, device="cuda"), torch.zeros_like(want[i][2])) for i in range(2)]
    ws = [(ql.lora_workspace(p[i].stack, 64), ql.sample_workspace(24, 40000)) for i in range(2)]
    plans = [t.plan() for t in trees]
    spaces = [x.new_workspace() for x in plans]
    dev = [(t.table.cuda(), t.lens.cuda(), t.cu.cuda()) for t in trees]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            ql.qlinear_lora(p[i].stack, p[i].x, p[i].y, ad[i], ws[i][0], out=outs[i][0], stream=streams[i])
            ql.qlinear_sample(s[i][0], s[i][1], outs[i][1], ws[i][1], stream=streams[i])
            ql.qlinear_tree_attention(plans[i], trees[i].q, trees[i].cache, *dev[i], trees[i].dev_sees, outs[i][2],
                                      workspace=spaces[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and (outs[i][1].cpu().numpy() == want[i][1]).all()
        assert torch.equal(outs[i][2], want[i][2])


def test_graphs_share_a_workspace():
    """Two captured runs of other sizes over one workspace, replayed in turn on one stream."""
    p = [lora.Problem(81, [j % 4 - 1 for j in range(50)], 3, 16, 1024, [256]), lora.Problem(82, [j % 2 for j in range(200)], 2, 32, 512, [128])]
    s = [sample.problem(83, 3, 30011, False), sample.problem(84, 40, 9000, True)]
    trees = [Tree(85, [40, 20], [900, 1400], 8, 2, 128, 16, False), Tree(86, [3, 64, 9], [2000, 70, 500], 8, 2, 128, 16, False)]
    plans = [t.plan() for t in trees]
    ad = [x.adapters.cuda() for x in p]
    size = max([max(ql.qlinear_lora_workspace_bytes(x.stack, len(x.adapters)) for x in p)] +
               [max(ql.qlinear_sample_workspace_bytes(*x[0].shape) for x in s)] + [x.workspace_bytes for x in plans])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(p[i].y), torch.zeros(len(s[i][0]), dtype=torch.int32, device="cuda"),
             torch.zeros(trees[i].T, 8, 128, dtype=BF16, device="cuda")) for i in range(2)]
    dev = [(t.table.cuda(), t.lens.cuda(), t.cu.cuda()) for t in trees]
    graphs = []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ql.qlinear_lora(p[i].stack, p[i].x, p[i].y, ad[i], ws, out=outs[i][0])
            ql.qlinear_sample(s[i][0], s[i][1], outs[i][1], ws)
            ql.qlinear_tree_attention(plans[i], trees[i].q, trees[i].cache, *dev[i], trees[i].dev_sees, outs[i][2], workspace=ws)
        graphs.append(g)
    want = [(p[i].run(), sample.run(*s[i])[0], trees[i].run(plans[i])[0]) for i in range(2)]
    for turn in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for i in (0, 1, 1, 0)[turn:turn + 2]:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set((0, 1, 1, 0)[turn:turn + 2]):
            assert torch.equal(outs[i][0], want[i][0]) and (outs[i][1].cpu().numpy() == want[i][1]).all()
            assert torch.equal(outs[i][2], want[i][2])
