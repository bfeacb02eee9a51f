"""Attention for trees of drafted tokens and the commit of a branch, on the GPU
against the oracle in 64 bits.

Attention's tolerance is that of test_gpu_serving.py's chunks (weights rounded
to bf16).  A commit moves bytes: exact.
"""

import numpy as np
import pytest
import torch

import oracle.requests as ref
import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu
from tests.test_gpu_serving import Problem, f64

pytestmark = [pytest.mark.gpu, requires_gpu]
U = 2.0 ** -24
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def random_parents(n, rng, wide=4):
    return [-1] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, n)]


def ancestors(parents, words):
    m = np.zeros((len(parents), words), np.uint64)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i // 64] |= np.uint64(1 << (i % 64))
    return m


class Tree(Problem):
    def __init__(self, seed, new, *args, words=None, kind="tree", **kw):
        super().__init__(seed, new, *args, **kw)
        rng = np.random.default_rng(seed)
        words = words or max(1, -(-max(new) // 64))
        rows = []
        for n in new:
            if kind == "tree":
                rows.append(ancestors(random_parents(n, rng), words) if n else np.zeros((0, words), np.uint64))
            elif kind == "any":         # any set of nodes, bits beyond them too
                rows.append(rng.integers(0, 2 ** 64, (n, words), dtype=np.uint64))
            else:                       # the context alone
                rows.append(np.zeros((n, words), np.uint64))
        self.sees = np.concatenate(rows)
        self.dev_sees = torch.from_numpy(self.sees.view(np.int64)).cuda()

    def plan(self, max_q=None, max_kv=None, tokens=None, scale=None):
        return ql.qlinear_tree_attention_plan(self.cache, self.hq, len(self.kv), tokens or self.T,
                                              max_q or max(self.new), max_kv or max(self.kv), scale)

    def run(self, plan, lse=True, stream=None):
        out = torch.full((self.T, self.hq, self.D), 9.0, dtype=BF16, device="cuda")
        ls = torch.full((self.T, self.hq), 9.0, device="cuda") if lse else None
        ql.qlinear_tree_attention(plan, self.q, self.cache, self.table.cuda(), self.lens.cuda(), self.cu.cuda(),
                                  self.dev_sees, out, ls, plan.new_workspace(), stream)
        torch.cuda.synchronize()
        return out, ls

    def check(self, out, ls, scale=None):
        r = ref.tree_attention(f64(self.q), self.k_host, self.v_host, self.table.numpy(), self.kv, self.cu.numpy(),
                               self.sees, self.page, scale or self.D ** -0.5, None if self.ks is None else f64(self.ks),
                               None if self.vs is None else f64(self.vs))
        n = max(max(self.kv), 1)
        d = 2 * self.D * U * r["reach"] + 8 * U * (r["reach"] + 1)
        tol = r["weight"] * (2.0 ** -8 + 2 * d + n * U)[..., None] + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(r["out"]) + 1e-38
        err = np.abs(f64(out) - r["out"])
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(err / tol)))
        if ls is not None:
            e = f64(ls)
            empty = np.isneginf(r["lse"])
            assert np.array_equal(np.isneginf(e), empty)
            lt = d + n * U + 4 * U * np.abs(np.where(empty, 0, r["lse"])) + 4 * U
            with np.errstate(invalid="ignore"):
                assert (empty | (np.abs(e - r["lse"]) <= lt)).all()


CASES = [  # new, kv, hq, hk, D, page, e4m3, order, kind
    ([1], [1], 4, 1, 128, 16, False, "token", "tree"),                       # a root alone, no context
    ([5], [5], 4, 2, 64, 16, False, "token", "tree"),                        # a tree without context
    ([7, 3], [300, 77], 8, 2, 128, 16, False, "token", "tree"),              # few rows: the decode kernel
    ([4, 8, 1], [41, 1030, 9], 8, 2, 64, 32, True, "head", "tree"),
    ([8], [95], 16, 4, 128, 16, True, "token", "any"),
    ([26], [1031], 32, 8, 128, 16, False, "token", "tree"),
    ([64, 1, 33], [64, 700, 150], 8, 2, 128, 16, False, "token", "tree"),
    ([63, 20], [1000, 97], 10, 2, 128, 48, True, "token", "tree"),           # group 5
    ([64, 64], [500, 66], 8, 2, 64, 64, True, "head", "any"),
    ([40, 2], [90, 2100], 12, 4, 64, 16, False, "token", "any"),
    ([100, 65], [800, 65], 4, 1, 128, 16, False, "token", "tree"),           # more nodes than a word's bits
    ([150], [421], 4, 2, 64, 16, True, "token", "any"),
    ([12, 0, 40], [12, 9, 0], 4, 2, 128, 16, False, "token", "tree"),        # no nodes; nothing cached
    ([9, 30], [4, 20], 4, 2, 64, 16, False, "token", "any"),                 # more nodes than cached tokens
    ([3, 50], [3, 50], 4, 2, 128, 16, False, "token", "none"),               # rows that see nothing
    ([2], [2], 4, 2, 64, 16, False, "token", "none"),
    ([30], [3000], 24, 1, 128, 32, True, "token", "tree"),                   # one KV head, many rows
    ([20, 31, 5], [60, 64, 33], 4, 2, 128, 16, False, "token", "any"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_tree_attention(i):
    new, kv, hq, hk, D, page, e4m3, order, kind = CASES[i]
    p = Tree(700 + i, new, kv, hq, hk, D, page, e4m3, order, q_pad=64 if i % 2 else 0, kind=kind)
    out, ls = p.run(p.plan())
    p.check(out, ls)


@pytest.mark.parametrize("max_q,max_kv,words", [(None, 40000, 1), (300, None, 5), (None, None, 3)])
def test_bounds_may_be_loose(max_q, max_kv, words):
    p = Tree(3, [40, 6, 23], [700, 90, 1500], 8, 2, 128, 16, False, words=words)
    cols = -(-max(max_kv or 0, 1500) // 16)
    p.table = torch.nn.functional.pad(p.table, (0, max(0, cols - p.table.shape[1])), value=-7)
    out, ls = p.run(p.plan(max_q=max_q, max_kv=max_kv))
    p.check(out, ls)


@pytest.mark.parametrize("new", [[8, 3], [40, 33]])
def test_a_chain_is_causal_attention(new):
    """Nodes in a row, each seeing those before it: the same bits as qlinear_attention's."""
    p = Tree(11, new, [120, 90], 8, 2, 128, 16, False)      # (short enough that both are cut alike)
    p.dev_sees = torch.cat([torch.tensor([(1 << (i + 1)) - 1 for i in range(n)]) for n in new])[:, None].cuda()
    out, ls = p.run(p.plan())
    want, want_ls = Problem.run(p, Problem.plan(p))
    assert torch.equal(out, want) and torch.equal(ls, want_ls)


@pytest.mark.parametrize("new,kv", [(6, 40), (40, 70), (70, 200)])
@pytest.mark.parametrize("D,e4m3", [(128, False), (64, True)])
def test_nonfinite_keys_and_values_stay_with_the_rows_that_see_them(new, kv, D, e4m3):
    p = Tree(5, [new], [kv], 8, 2, D, 16, e4m3)
    want, _ = p.run(p.plan())
    node = new // 2
    at = kv - new + node
    page, place = int(p.table[0, at // 16]), at % 16
    nan = torch.tensor(float("nan")).to(p.v.dtype).view(torch.uint8 if e4m3 else torch.int16).cuda()
    p.v.view(nan.dtype)[page, place, :, 3] = nan
    got, _ = p.run(p.plan())
    sees = torch.from_numpy((p.sees[:, node // 64] >> np.uint64(node % 64)) & np.uint64(1)).bool().cuda()
    assert sees.any() and not sees.all()
    assert torch.equal(got[~sees], want[~sees]) and torch.isnan(got[sees][:, :, 3]).all()
    rest = [d for d in range(D) if d != 3]
    assert torch.equal(got[sees][:, :, rest], want[sees][:, :, rest])
    p.k.view(nan.dtype)[page, place, :, 5] = nan
    got, _ = p.run(p.plan())
    assert torch.equal(got[~sees], want[~sees]) and torch.isnan(got[sees]).all()


@pytest.mark.parametrize("batch,nodes,kv,D,hq,hk", [(70, 34, 260, 64, 4, 1), (9, 40, 3000, 128, 8, 2), (3, 200, 900, 64, 4, 4),
                                                    (40, 36, 700, 128, 16, 4), (520, 33, 140, 64, 2, 2)])
def test_many_trees(batch, nodes, kv, D, hq, hk):
    """More sequences than lanes, keys cut into many shares, more units than the card holds, batches that are not cut."""
    new = [(nodes, 1, nodes // 2, 0, nodes - 1)[i % 5] for i in range(batch)]
    p = Tree(60 + batch, new, [nodes + (i * 7919) % kv for i in range(batch)], hq, hk, D, 16, False)
    out, ls = p.run(p.plan())
    p.check(out, ls)


def test_cu_q_that_is_none_stays_inside():
    """Sequences that overlap or run backwards: some rows are computed, nothing outside out is written."""
    p = Tree(4, [40] * 8, [900] * 8, 8, 2, 128, 16, False)
    want, _ = p.run(p.plan())
    plan = p.plan()
    wide = torch.full((p.T + 2, 8, 128), 9.0, dtype=BF16, device="cuda")
    cu = torch.tensor([0, 320, 0, 320, -5, 10 ** 6, 7, 320, 320], dtype=torch.int32, device="cuda")
    ws = plan.new_workspace()
    ql.qlinear_tree_attention(plan, p.q, p.cache, p.table.cuda(), p.lens.cuda(), cu, p.dev_sees, wide[1:-1], workspace=ws)
    torch.cuda.synchronize()
    assert (wide[0] == 9).all() and (wide[-1] == 9).all()
    assert torch.equal(p.run(plan)[0], want)


def test_tree_attention_replays():
    p = Tree(14, [20, 33, 1], [260, 500, 31], 8, 2, 128, 16, True)
    plan = p.plan(max_kv=600)
    p.table = torch.nn.functional.pad(p.table, (0, 8))
    table, lens, cu, ws = p.table.cuda(), p.lens.cuda(), p.cu.cuda(), plan.new_workspace()
    out = torch.zeros(p.T, 8, 128, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ql.qlinear_tree_attention(plan, p.q, p.cache, table, lens, cu, p.dev_sees, out, workspace=ws)
    for i in range(4):
        p.q.mul_(-1.0)
        if i == 2:      # other trees and lengths
            p.kv = [230, 490, 20]
            p.lens = torch.tensor(p.kv, dtype=torch.int32)
            lens.copy_(p.lens)
            p.dev_sees.copy_(p.dev_sees.flip(0))
            p.sees = p.dev_sees.cpu().numpy().view(np.uint64)
        if ws is not None:
            ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        p.check(out, None)


# ------------------------------------------------------------------ commit

class Commit:
    def __init__(self, seed, nodes, kv, layers, hk, D, page, e4m3, order="token", accept=0.8):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        need = [-(-x // page) for x in kv]
        pages = sum(need) + 3
        perm = torch.randperm(pages, generator=g)
        self.table = torch.full((len(kv), max(max(need), 1) + 2), -(2 ** 31), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        self.page, self.kv, self.e4m3 = page, kv, e4m3
        kind = torch.uint8 if e4m3 else torch.int16
        self.raw = []
        for _ in range(2 * layers):
            x = torch.randint(-100, 100, (pages, page, hk, D), generator=g).to(kind).cuda()
            self.raw.append(x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if order == "head" else x)
        dt = E4M3 if e4m3 else BF16
        self.caches = [ql.PagedCache(self.raw[2 * i].view(dt), self.raw[2 * i + 1].view(dt)) for i in range(layers)]
        self.parents, self.tokens, self.sampled = [], [], []
        for n in nodes:
            parents = random_parents(n, rng, 6) if n else []
            tokens = rng.integers(0, 50, n)
            draws = rng.integers(0, 50, n)
            for i in range(n):          # most nodes draw one of their children's tokens
                below = [j for j in range(n) if parents[j] == i]
                if below and rng.random() < accept:
                    draws[i] = tokens[below[int(rng.integers(len(below)))]]
            self.parents += parents
            self.tokens += tokens.tolist()
            self.sampled += draws.tolist()
        self.cu = torch.tensor([0] + list(nodes)).cumsum(0).to(torch.int32)

    def run(self, depth, new_lens=True, stream=None, **kw):
        batch = len(self.kv)
        dev = [torch.tensor(x, dtype=torch.int32).cuda() for x in (self.tokens, self.parents, self.sampled)]
        out = torch.full((batch, depth + 1), 77, dtype=torch.int32, device="cuda")
        accepted = torch.full((batch,), 77, dtype=torch.int32, device="cuda")
        lens = torch.full((batch,), 77, dtype=torch.int32, device="cuda") if new_lens else None
        before = [x.clone() for x in self.raw]
        ql.qlinear_tree_commit(self.caches, self.table.cuda(), torch.tensor(self.kv, dtype=torch.int32).cuda(),
                               self.cu.cuda(), *dev, out, accepted, lens, stream=stream, **kw)
        torch.cuda.synchronize()
        t, n, l, moves = ref.tree_commit(self.tokens, self.parents, self.sampled, self.cu.tolist(), self.kv, depth)
        assert np.array_equal(out.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
        assert lens is None or np.array_equal(lens.cpu().numpy(), l)
        for got, old in zip(self.raw, before):
            want = old.clone()
            for b, pairs in enumerate(moves):
                for src, dst in pairs:
                    if dst >= 0:
                        s, d = ((int(self.table[b, x // self.page]), x % self.page) for x in (src, dst))
                        want[d] = old[s]
            assert torch.equal(got, want)
        return n


COMMITS = [  # nodes, kv, layers, hk, D, page, e4m3, order, depth
    ([1], [1], 1, 1, 64, 16, False, "token", 0),
    ([1, 5], [30, 5], 1, 2, 128, 16, False, "token", 4),
    ([13, 2, 7, 0, 30], [300, 17, 16, 40, 31], 2, 8, 128, 16, False, "head", 8),
    ([64, 64, 64], [64, 200, 100], 3, 4, 64, 48, True, "token", 20),
    ([64, 3], [80, 3], 2, 1, 64, 16, True, "head", 1),                        # stopped by max_depth
    ([100, 200, 65], [150, 200, 90], 1, 2, 128, 32, False, "token", 30),      # more nodes than lanes
    ([40] * 70, list(range(40, 110)), 5, 2, 64, 16, False, "token", 10),
    ([20], [60], 40, 1, 64, 16, True, "token", 9),                            # more layers than a launch takes
    ([12, 9], [70, 50], 0, 1, 64, 16, False, "token", 5),                     # no cache: the walk alone
    ([8, 40], [60, 200], 1, 3, 256, 16, False, "token", 12),
]


@pytest.mark.parametrize("i", range(len(COMMITS)))
def test_tree_commit(i):
    nodes, kv, layers, hk, D, page, e4m3, order, depth = COMMITS[i]
    c = Commit(40 + i, nodes, kv, layers, hk, D, page, e4m3, order)
    n = c.run(depth, new_lens=i % 3 != 1)
    if max(nodes) > 5 and depth > 1:
        assert n.max() > 1


def test_long_chains_move_in_order():
    """Every node's only child draws on: rows move onto places that later rows leave."""
    c = Commit(2, [60], [100], 1, 2, 128, 16, False)
    c.parents = [-1] + [max(0, i - 2) for i in range(1, 60)]      # two interleaved chains
    c.tokens = list(range(60))
    c.sampled = [min(i + 2, 59) if i else 1 for i in range(60)]   # 0 -> 1 -> 3 -> 5 ...
    assert c.run(64)[0] == 30


def test_broken_trees_and_tables_stay_inside():
    """Parents that point to themselves or ahead, pages outside the cache, more nodes than cached tokens."""
    c = Commit(3, [6, 6], [40, 4], 1, 2, 64, 16, False)
    c.parents = [0, 1, 5, 5, 0, 4] * 2
    c.tokens = [7] * 12
    c.sampled = [7] * 12
    c.table[0] = torch.where(torch.arange(c.table.shape[1]) == 2, 10 ** 6, -3).int()
    before = [x.clone() for x in c.raw]
    dev = [torch.tensor(x, dtype=torch.int32).cuda() for x in (c.tokens, c.parents, c.sampled)]
    out, acc = torch.zeros(2, 5, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ql.qlinear_tree_commit(c.caches, c.table.cuda(), torch.tensor(c.kv, dtype=torch.int32).cuda(), c.cu.cuda(), *dev, out, acc)
    torch.cuda.synchronize()
    assert acc.tolist() == [2, 2] and out.tolist() == [[7, 7, 7, -1, -1]] * 2      # 0 -> 4 -> 5
    # sequence 1: node 4 stands at 4 - 6 + 4 = 2 and would move to -1; node 5 moves from 3 to 0
    p = int(c.table[1, 0])
    for got, old in zip(c.raw, before):
        old[p, 0] = old[p, 3]
        assert torch.equal(got, old)


def test_commit_on_a_stream_and_replayed():
    c = Commit(9, [20, 31], [100, 64], 2, 2, 64, 16, False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(8, stream=side)
    dev = [torch.tensor(x, dtype=torch.int32).cuda() for x in (c.tokens, c.parents, c.sampled)]
    out, acc = torch.zeros(2, 9, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    table, kv, cu = c.table.cuda(), torch.tensor(c.kv, dtype=torch.int32).cuda(), c.cu.cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ql.qlinear_tree_commit(c.caches, table, kv, cu, *dev, out, acc)
    rng = np.random.default_rng(1)
    for _ in range(3):
        draws = rng.permutation(np.array(c.sampled))
        dev[2].copy_(torch.from_numpy(draws.astype(np.int32)))
        before = [x.clone() for x in c.raw]
        graph.replay()
        torch.cuda.synchronize()
        after = [x.clone() for x in c.raw]
        for x, y in zip(c.raw, before):
            x.copy_(y)
        c.sampled = draws.tolist()
        c.run(8)
        assert all(torch.equal(x, y) for x, y in zip(after, c.raw))
