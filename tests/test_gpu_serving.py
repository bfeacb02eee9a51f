"""The serving operators on the GPU against the oracle in 64 bits.

Tolerances, derived from the operators' arithmetic (u = 2^-24 is binary32's
unit roundoff; bf16, of 8 significant bits, rounds by at most 2^-8 of a value,
E4M3, of 4, by 2^-4 of it or half its smallest step 2^-9):

* norm and rotation: the sum of squares, its root and the products lose at
  most (dim + 16) u of |n_a| + |n_b|; then one rounding to the output's type.
* attention: a score's products and sums lose at most dim u of reach = max_j
  scale sum_d |q_d k_jd|, twice that counting the matrix core's truncated
  alignment; the exponent's argument is rounded, 4 u of it.  A weight is off by
  the exponential of that and by P's rounding to bf16 (2^-8); sums over n keys
  lose at most n u.  All of it scales with weight = sum_j p_j |v_j|; then one
  rounding to bf16.
"""

import numpy as np
import pytest
import torch

import oracle.serving as ref
import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]
U = 2.0 ** -24
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


# ------------------------------------------------------------------ norm and rotation, append

def head_inputs(seed, T, hq, hk, D, norm, pad=0):
    """q, k, v as columns of one QKV output, `pad` unused columns after them."""
    g = torch.Generator().manual_seed(seed)
    x = randn(g, T, hq + 2 * hk, D)
    x[:, :, :2] *= 10.0
    wide = torch.zeros(T, (hq + 2 * hk) * D + pad, dtype=BF16)
    wide[:, :(hq + 2 * hk) * D] = x.reshape(T, -1).to(BF16)
    wide = wide.cuda()
    heads = wide[:, :(hq + 2 * hk) * D].unflatten(1, (hq + 2 * hk, D))
    w = [(1 + 0.3 * randn(g, D)).to(BF16).cuda() if norm else None for _ in range(2)]
    return heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:], w[0], w[1]


def check_rounded(got, y, size, D, what):
    tol = 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -8) + (D + 16) * U * size + 1e-38
    bad = ~(np.abs(got - y) <= tol) & ~(np.isnan(got) & np.isnan(y))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist())


def check_codes(codes, scale, y, size, D, what):
    """codes [tokens, heads, dim] of y / scale[head]."""
    s = np.ones(y.shape[1]) if scale is None else f64(scale)
    t = np.clip(y / s[None, :, None], -448, 448)
    got = f64(codes)
    tol = np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10) * (1 + 2.0 ** -10) + (D + 16) * U * size / s[None, :, None]
    bad = ~(np.abs(got - t) <= tol) & ~(np.isnan(got) & np.isnan(t))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist())


NORM_CASES = [  # T, hq, hk, D, rot, norm, interleaved, pad, in place
    (1, 32, 8, 128, 128, True, False, 0, False),
    (5, 40, 8, 128, 128, True, False, 64, True),
    (3, 7, 1, 64, 64, True, True, 8, False),
    (4, 28, 4, 128, 64, False, False, 0, True),
    (2, 3, 3, 256, 128, True, True, 0, False),
    (33, 4, 2, 256, 256, True, False, 16, True),
    (7, 5, 1, 64, 16, False, True, 0, False),
    (2, 16, 16, 128, 0, True, False, 0, False),
    (1030, 3, 1, 64, 32, True, False, 0, False),
    (2, 4, 0, 128, 128, True, False, 0, False),
]


@pytest.mark.parametrize("T,hq,hk,D,rot,norm,inter,pad,inplace", NORM_CASES)
def test_qk_norm_rope(T, hq, hk, D, rot, norm, inter, pad, inplace):
    q, k, _, qw, kw = head_inputs(T * 31 + D, T, hq, hk, D, norm, pad)
    table = ql.rope_table(97, rot) if rot else None
    pos = torch.randint(0, 97, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    eps = 1e-5
    want = [ref.norm_rope(f64(x), f64(w), pos.cpu().numpy(), None if table is None else f64(table), rot, inter, eps)
            for x, w in ((q, qw), (k, kw))]
    qo, ko = (q, k) if inplace else (torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous())
    ql.qlinear_qk_norm_rope(q, k, pos, table, qo, ko, qw, kw, eps=eps, interleaved=inter)
    torch.cuda.synchronize()
    check_rounded(f64(qo), *want[0], D, "q")
    check_rounded(f64(ko), *want[1], D, "k")


def test_positions_outside_the_table_give_nan_rows():
    q, k, _, qw, kw = head_inputs(1, 4, 2, 1, 64, True)
    table = ql.rope_table(10, 64)
    pos = torch.tensor([9, 10, -1, 1 << 40]).cuda()
    qo, ko = torch.zeros_like(q).contiguous(), torch.zeros_like(k).contiguous()
    ql.qlinear_qk_norm_rope(q, k, pos, table, qo, ko, qw, kw)
    assert torch.isfinite(qo[0]).all() and torch.isfinite(ko[0]).all()
    assert torch.isnan(qo[1:]).all() and torch.isnan(ko[1:]).all()


def new_cache(pages, page, hk, D, e4m3, order="token", fill=3.0):
    """A cache tensor whose pages hold tokens of all heads ("token") or heads of all tokens ("head")."""
    dt = E4M3 if e4m3 else BF16
    if order == "head":
        return torch.full((pages, hk, page, D), fill).to(dt).cuda().permute(0, 2, 1, 3)
    return torch.full((pages, page, hk, D), fill).to(dt).cuda()


APPEND_CASES = [  # T, hq, hk, D, rot, norm, page, e4m3, order, with q
    (1, 32, 8, 128, 128, True, 16, False, "token", True),
    (9, 64, 8, 128, 128, True, 16, True, "token", True),
    (17, 6, 2, 64, 32, False, 48, True, "head", True),
    (40, 4, 4, 64, 64, True, 32, False, "head", False),
    (3, 2, 1, 256, 256, True, 64, True, "token", True),
    (300, 3, 1, 128, 64, True, 16, False, "token", False),
]


@pytest.mark.parametrize("T,hq,hk,D,rot,norm,page,e4m3,order,with_q", APPEND_CASES)
def test_qkv_append(T, hq, hk, D, rot, norm, page, e4m3, order, with_q):
    q, k, v, qw, kw = head_inputs(T + page, T, hq, hk, D, norm)
    table = ql.rope_table(512, rot)
    g = torch.Generator().manual_seed(9)
    pos = torch.randint(0, 512, (T,), generator=g).cuda()
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    skip = torch.rand(T, generator=g) < 0.2 if T > 1 else torch.zeros(T, dtype=torch.bool)
    given = torch.where(skip, torch.tensor(-1), slots)
    if T > 4:
        given[int(skip.int().argmin())] = pages * page      # beyond the cache: writes nothing either
    kc, vc = (new_cache(pages, page, hk, D, e4m3, order) for _ in range(2))
    ks = (0.05 + 0.02 * torch.rand(hk, generator=g)).cuda() if e4m3 else None
    vs = (0.05 + 0.02 * torch.rand(hk, generator=g)).cuda() if e4m3 else None
    before = [x.clone() for x in (kc, vc)]
    cache = ql.PagedCache(kc, vc, ks, vs)
    qo = torch.zeros(T, hq, D, dtype=BF16, device="cuda") if with_q else None
    ql.qlinear_qkv_append(q if with_q else None, k, v, pos, given.cuda(), table, qo, cache, qw, kw)
    torch.cuda.synchronize()
    p = pos.cpu().numpy()
    if with_q:
        check_rounded(f64(qo), *ref.norm_rope(f64(q), f64(qw), p, f64(table), rot, False, 1e-6), D, "q")
    ok = (given >= 0) & (given < pages * page)
    at, rows = given[ok].cuda(), ok.nonzero()[:, 0].numpy()
    y, size = ref.norm_rope(f64(k), f64(kw), p, f64(table), rot, False, 1e-6)
    for got, old, y, size, s, what in ((kc, before[0], y, size, ks, "k"),
                                       (vc, before[1], f64(v), np.abs(f64(v)), vs, "v")):
        got, old = got.view(torch.uint8 if e4m3 else torch.int16), old.view(torch.uint8 if e4m3 else torch.int16)
        got, old = (x.contiguous().flatten(0, 1) for x in (got, old))
        rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert torch.equal(got[rest], old[rest]), "slots that were not given changed"
        new = got[at].view(E4M3 if e4m3 else BF16)
        if e4m3:
            check_codes(new, s, y[rows], size[rows], D, what)
        else:
            check_rounded(f64(new), y[rows], size[rows], D, what)


def test_append_saturates_and_keeps_nan():
    """E4M3 codes beyond 448 saturate; a NaN value stays one and no neighbour changes."""
    T, D = 1, 64
    k = torch.zeros(T, 1, D, dtype=BF16)
    k[0, 0, :6] = torch.tensor([1e6, -1e6, float("nan"), 448.0, float("inf"), 1.0])
    k = k.cuda()
    kc, vc = new_cache(2, 16, 1, D, True), new_cache(2, 16, 1, D, True)
    ql.qlinear_qkv_append(None, k, k, torch.zeros(T, dtype=torch.int64).cuda(), torch.tensor([17]).cuda(), None, None,
                          ql.PagedCache(kc, vc))
    row = kc.float()[1, 1, 0].cpu()
    assert row[:6].nan_to_num(nan=-1.0).tolist() == [448.0, -448.0, -1.0, 448.0, 448.0, 1.0]
    assert (row[6:] == 0).all()


# ------------------------------------------------------------------ attention

class Problem:
    def __init__(self, seed, new, kv, hq, hk, D, page, e4m3, order="token", spare=3, q_pad=0, table_pad=2):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hk, self.D, self.page, self.e4m3 = hq, hk, D, page, e4m3
        self.new, self.kv = new, kv
        need = [-(-x // page) for x in kv]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g)
        cols = max(max(need), 1) + table_pad
        self.table = torch.full((len(kv), cols), -(2 ** 31), dtype=torch.int32)   # beyond a sequence: never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        dt = E4M3 if e4m3 else BF16
        k, v = ((randn(g, pages, page, hk, D) * (16 if e4m3 else 1)).to(dt) for _ in range(2))
        # what no sequence owns is NaN
        own = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(kv):
            for i in range(need[b]):
                own[self.table[b, i], :min(page, n - i * page)] = True
        nan = torch.tensor(float("nan")).to(dt).view(torch.uint8 if e4m3 else torch.int16)
        for x in (k, v):
            x.view(nan.dtype)[~own] = nan
        self.k_host, self.v_host = f64(k), f64(v)
        if order == "head":
            k, v = (x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v))
        self.k, self.v = k.cuda(), v.cuda()
        self.ks = (0.05 + 0.02 * torch.rand(hk, generator=g)).cuda() if e4m3 else None
        self.vs = (0.05 + 0.02 * torch.rand(hk, generator=g)).cuda() if e4m3 else None
        self.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        T = int(self.cu[-1])
        self.T = T
        wide = torch.zeros(T, hq * D + q_pad, dtype=BF16)
        wide[:, :hq * D] = (1.5 * randn(g, T, hq * D)).to(BF16)
        self.q = wide.cuda()[:, :hq * D].unflatten(1, (hq, D))
        self.cache = ql.PagedCache(self.k, self.v, self.ks, self.vs)
        self.lens = torch.tensor(kv, dtype=torch.int32)

    def plan(self, causal=True, window=0, scale=None, max_q=None, max_kv=None, tokens=None):
        return ql.qlinear_attention_plan(self.cache, self.hq, len(self.kv), tokens or self.T,
                                         max_q or max(self.new), max_kv or max(self.kv), causal, window, scale)

    def run(self, plan, lse=True, stream=None):
        out = torch.full((self.T, self.hq, self.D), 9.0, dtype=BF16, device="cuda")
        ls = torch.full((self.T, self.hq), 9.0, device="cuda") if lse else None
        ql.qlinear_attention(plan, self.q, self.cache, self.table.cuda(), self.lens.cuda(), self.cu.cuda(), out, ls,
                             plan.new_workspace(), stream)
        torch.cuda.synchronize()
        return out, ls

    def check(self, out, ls, causal=True, window=0, scale=None):
        scale = scale or self.D ** -0.5
        r = ref.attention(f64(self.q), self.k_host, self.v_host, self.table.numpy(), self.kv, self.cu.numpy(),
                          self.page, scale, causal, window, None if self.ks is None else f64(self.ks),
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


ATTEND_CASES = [  # new, kv, hq, hk, D, page, e4m3, order, causal, window
    ([1], [1], 4, 1, 128, 16, False, "token", True, 0),                       # the first token
    ([1], [1031], 32, 8, 128, 16, False, "token", True, 0),                   # odd length, chunks
    ([1, 1, 1, 1], [17, 4096, 2, 300], 8, 2, 128, 32, False, "head", True, 0),
    ([1, 1, 1], [65, 777, 31], 10, 2, 128, 48, True, "token", True, 0),       # group 5, pages of 48
    ([1, 1], [2049, 130], 14, 2, 64, 64, True, "head", True, 0),              # group 7
    ([5, 5, 5], [517, 5, 64], 32, 8, 128, 16, False, "token", True, 0),       # drafted tokens
    ([8, 3], [300, 3], 16, 16, 64, 16, False, "token", True, 0),              # one query head a KV head
    ([2, 7], [900, 40], 24, 1, 128, 32, True, "token", True, 0),              # one KV head
    ([1, 0, 3], [40, 9, 0], 4, 2, 128, 16, False, "token", True, 0),          # no new tokens; an empty context
    ([6, 4], [3, 4], 4, 2, 64, 16, False, "token", True, 0),                  # more new tokens than cached ones
    ([4, 4], [200, 33], 4, 2, 128, 16, True, "token", False, 0),              # not causal
    ([1, 1], [1500, 70], 8, 2, 128, 16, False, "token", True, 100),           # a window
    ([9, 2], [600, 90], 8, 2, 64, 16, True, "token", True, 1),                # a window of the token itself
    ([40], [40], 8, 2, 128, 16, False, "token", True, 0),                     # a whole prompt
    ([129, 1, 70], [300, 513, 70], 8, 2, 128, 16, False, "token", True, 0),   # chunks and a single token
    ([100, 257], [1000, 260], 12, 4, 128, 16, True, "head", True, 0),
    ([260], [777], 6, 2, 64, 32, True, "token", True, 200),
    ([131], [400], 5, 1, 64, 16, False, "token", False, 0),
    ([300], [2000], 4, 1, 128, 48, False, "token", True, 333),
    ([40, 1], [9000, 8500], 4, 1, 128, 16, False, "token", True, 0),          # many pages a wave
    ([33], [4500], 4, 1, 64, 32, True, "head", True, 4200),
]


@pytest.mark.parametrize("i", range(len(ATTEND_CASES)))
def test_attention(i):
    new, kv, hq, hk, D, page, e4m3, order, causal, window = ATTEND_CASES[i]
    p = Problem(100 + i, new, kv, hq, hk, D, page, e4m3, order, q_pad=64 if i % 2 else 0)
    out, ls = p.run(p.plan(causal, window))
    p.check(out, ls, causal, window)


@pytest.mark.parametrize("max_q,max_kv", [(None, 40000), (64, None), (500, 5000), (2000, 2000)])
def test_attention_plan_bounds_may_be_loose(max_q, max_kv):
    """A plan made for longer sequences than the call's gives the same rows."""
    p = Problem(5, [1, 6, 3], [700, 90, 1500], 8, 2, 128, 16, False)
    cols = -(-max(max_kv or 0, 1500) // 16)
    p.table = torch.nn.functional.pad(p.table, (0, max(0, cols - p.table.shape[1])), value=-7)
    out, ls = p.run(p.plan(max_q=max_q, max_kv=max_kv))
    p.check(out, ls)


@pytest.mark.parametrize("new", [[1, 2], [40, 1]])
def test_attention_without_any_context(new):
    """max_kv = 0: a page table without columns; every row is zero, its lse -inf."""
    p = Problem(9, new, [0, 0], 4, 2, 64, 16, False)
    p.table = torch.zeros(2, 0, dtype=torch.int32)
    out, ls = p.run(p.plan(max_kv=0))
    assert not out.any() and torch.isneginf(ls).all()


@pytest.mark.parametrize("D,e4m3,batch,kv", [(64, False, 130, 90), (128, True, 200, 40), (64, False, 40, 420), (64, True, 64, 33),
                                             (128, False, 64, 66), (128, False, 65, 66)])
def test_attention_many_sequences(D, e4m3, batch, kv):
    """More sequences than a wave holds, more tiles than there are slots, and
    slots that lie in one sequence each; some sequences have no new token."""
    new = [(0, 1, 1, 2, 3)[i % 5] for i in range(batch)]
    p = Problem(50 + batch, new, [3 + (i * 7919) % kv for i in range(batch)], 16, 8, D, 16, e4m3)
    out, ls = p.run(p.plan())
    p.check(out, ls)


def test_attention_batch_of_chunks_and_many_short_sequences():
    """Sequences of few rows beside chunks, with contexts (by the plan's bound)
    long enough that they get a launch of their own."""
    new, kv = [40, 1, 9, 1, 3, 0, 1], [300, 1500, 700, 40, 65, 20, 1]
    p = Problem(21, new, kv, 8, 2, 128, 16, True)
    p.table = torch.nn.functional.pad(p.table, (0, 3750 - p.table.shape[1]), value=-7)
    plan = p.plan(max_kv=60000)
    assert plan.facts["stream_rows"] == 16 and plan.facts["tile_rows"] == 128
    out, ls = p.run(plan)
    p.check(out, ls)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv,window", [(5, 70, 0), (40, 130, 0), (150, 200, 33), (7, 150, 40)])
def test_non_finite_values_reach_only_rows_that_see_them(new, kv, window, D, e4m3):
    """One infinite and some NaN entries of K and V at tokens that some new
    tokens see: every other row stays as without them, to the bit."""
    p = Problem(31, [new], [kv], 4, 2, D, 16, e4m3)
    plan = p.plan(window=window)
    clean, _ = p.run(plan)
    bad_k, bad_v = kv - 2, kv - new // 2                    # K of the last token but one, V of one in the middle
    nan = torch.tensor(float("nan")).to(p.k.dtype).cuda()
    for x, at, head, dims in ((p.k, bad_k, 0, (5,)), (p.v, bad_v, 1, (3, D - 1))):
        page = int(p.table[0, at // 16])
        for d in dims:
            x[page, at % 16, head, d] = nan if e4m3 or d != 3 else float("inf")
    got, _ = p.run(plan)
    pos = torch.arange(kv - new, kv)

    def sees(at):
        return (pos >= at) & ((pos - at < window) if window else True)
    for t in range(new):
        k_seen, v_seen = bool(sees(bad_k)[t]), bool(sees(bad_v)[t])
        for h in range(4):
            if h // 2 == 0:
                assert torch.isnan(got[t, h]).all() if k_seen else torch.equal(got[t, h], clean[t, h]), (t, h)
            else:
                hit = torch.zeros(D, dtype=torch.bool, device="cuda")
                hit[[3, D - 1]] = v_seen
                assert not torch.isfinite(got[t, h][hit]).any(), (t, h)
                assert torch.equal(got[t, h][~hit], clean[t, h][~hit]), (t, h)


def test_attention_scale_and_rows_outside():
    """A given scale; rows of q that no sequence owns stay as they were."""
    p = Problem(6, [3, 2], [100, 50], 4, 2, 128, 16, False)
    p.q = torch.cat([p.q, p.q[:2]])
    p.T += 2
    out, ls = p.run(p.plan(scale=0.02))
    assert (out[-2:] == 9.0).all() and (ls[-2:] == 9.0).all()
    p.T -= 2
    p.q, out, ls = p.q[:-2], out[:-2], ls[:-2]
    p.check(out, ls, scale=0.02)


@pytest.mark.parametrize("new,kv", [([1, 1], [3000, 500]), ([200, 1], [700, 900])])
def test_attention_repeats_to_the_bit_on_a_stream_and_in_a_graph(new, kv):
    p = Problem(7, new, kv, 8, 2, 128, 16, False)
    plan = p.plan()
    out, ls = p.run(plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again, ls2 = p.run(plan, stream=s)
    assert torch.equal(out, again) and torch.equal(ls, ls2)
    ws, got = plan.new_workspace(), torch.zeros_like(out)
    table, lens, cu = p.table.cuda(), p.lens.cuda(), p.cu.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ql.qlinear_graph_begin(s)
        ql.qlinear_attention(plan, p.q, p.cache, table, lens, cu, got, workspace=ws, stream=s)
        graph = ql.qlinear_graph_end(s)
    for i in range(3):
        with torch.cuda.stream(s):
            got.fill_(5.0)
            graph.launch(s)
        s.synchronize()
        assert torch.equal(got, out), i
        p.run(plan)     # eager work between the replays
    # the lengths are read on the device: the same graph serves the next step
    p.lens[0] = p.kv[0] = kv[0] - 30
    lens.copy_(p.lens)
    with torch.cuda.stream(s):
        graph.launch(s)
    s.synchronize()
    p.check(got, None)


def test_attention_beyond_32_bit_offsets():
    """A cache of more than 4 GiB a tensor, its used pages at the far end."""
    page, hk, D, pages = 64, 8, 128, (1 << 32) // (64 * 8 * 128 * 2) + 40
    k = torch.empty(pages, page, hk, D, dtype=BF16, device="cuda")
    v = torch.empty(pages, page, hk, D, dtype=BF16, device="cuda")
    p = Problem(8, [1, 20], [500, 70], 16, hk, D, page, False)
    first = pages - p.k.shape[0]
    k[first:], v[first:] = p.k, p.v
    p.table[p.table >= 0] += first
    p.k_host = np.lib.stride_tricks.as_strided(p.k_host, p.k_host.shape, p.k_host.strides)
    p.cache = ql.PagedCache(k, v)
    out, ls = p.run(p.plan())
    p.table[p.table >= 0] -= first
    p.check(out, ls)


def test_attention_over_an_appended_cache():
    """Append, then attend, on one stream with no synchronisation between: each
    token sees itself and its past as if the whole sequence had been given at once."""
    hq, hk, D, page, n = 8, 2, 128, 16, 50
    q, k, v, qw, kw = head_inputs(11, n, hq, hk, D, True)
    table = ql.rope_table(64, D)
    kc, vc = (new_cache(5, page, hk, D, False, fill=float("nan")) for _ in range(2))
    cache = ql.PagedCache(kc, vc)
    pages = torch.tensor([[3, 0, 4, 1]], dtype=torch.int32)
    pos = torch.arange(n)
    slots = pages[0, pos // page].long() * page + pos % page
    out = torch.zeros(n, hq, D, dtype=BF16, device="cuda")
    qr = torch.zeros(n, hq, D, dtype=BF16, device="cuda")
    tab = pages.cuda()
    for a, b in ((0, 33), (33, 34), (34, 50)):
        ql.qlinear_qkv_append(q[a:b], k[a:b], v[a:b], pos[a:b].cuda(), slots[a:b].cuda(), table, qr[a:b], cache, qw, kw)
        plan = ql.qlinear_attention_plan(cache, hq, 1, b - a, b - a, b)
        ql.qlinear_attention(plan, qr[a:b], cache, tab, torch.tensor([b], dtype=torch.int32).cuda(),
                             torch.tensor([0, b - a], dtype=torch.int32).cuda(), out[a:b], None, plan.new_workspace())
    torch.cuda.synchronize()
    r = ref.attention(f64(qr), f64(kc), f64(vc), pages.numpy(), [n], np.array([0, n]), page, D ** -0.5)
    tol = r["weight"] * (2.0 ** -8 + 2.0 ** -12) + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(r["out"]) + 1e-30
    assert (np.abs(f64(out) - r["out"]) <= tol).all()


def test_binding_refusals():
    """Tensors that do not fit are refused by name before anything is launched;
    the library's own refusals come as QLinearError."""
    q, k, v, qw, kw = head_inputs(1, 4, 4, 2, 64, True)
    pos, table = torch.zeros(4, dtype=torch.int64).cuda(), ql.rope_table(8, 64)
    qo, ko = torch.zeros_like(q).contiguous(), torch.zeros_like(k).contiguous()

    def norm(**kw_):
        d = dict(q=q, k=k, positions=pos, cos_sin=table, q_out=qo, k_out=ko, q_weight=qw, k_weight=kw)
        d.update(kw_)
        return ql.qlinear_qk_norm_rope(*d.values())
    for name, bad in (("q", q.float()), ("q", q.cpu()), ("k", k[:3]), ("q_out", qo[:, :3]), ("k_out", ko.transpose(0, 2)),
                      ("positions", pos.int()), ("positions", pos[:3]), ("q_weight", qw[:60]), ("k_weight", kw.float()),
                      ("cos_sin", table.double()), ("cos_sin", ql.rope_table(8, 128)), ("q", 3), ("q", q[0])):
        with pytest.raises(ValueError, match=name):
            norm(**{name: bad})
    with pytest.raises(ql.QLinearError) as e:
        norm(q=torch.zeros(4, 4, 72, dtype=BF16, device="cuda")[:, :, 4:68])    # 8 bytes off
    assert e.value.status == 5
    p = Problem(1, [1, 1], [900, 40], 4, 2, 64, 16, False)
    plan = p.plan()
    args = dict(plan=plan, q=p.q, cache=p.cache, page_table=p.table.cuda(), seq_lens=p.lens.cuda(), cu_q=p.cu.cuda(),
                out=torch.zeros(2, 4, 64, dtype=BF16, device="cuda"), lse=None, workspace=plan.new_workspace())
    for name, bad in (("q", p.q[:1]), ("page_table", p.table.cuda()[:, :50]), ("page_table", p.table.cuda().long()),
                      ("seq_lens", p.lens.cuda()[:1]), ("cu_q", p.cu.cuda()[:2]), ("workspace", None),
                      ("workspace", plan.new_workspace()[:-1]), ("out", args["out"].float()),
                      ("lse", torch.zeros(7, device="cuda"))):
        with pytest.raises(ValueError, match=name):
            ql.qlinear_attention(*dict(args, **{name: bad}).values())
    x = verify_inputs(1, [2, 1], 50)
    dev = [None if t is None else (torch.from_numpy(t) if isinstance(t, np.ndarray) else t).cuda() for t in x]
    out, acc = torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    ws = ql.verify_workspace(2, 50)
    for i, name, bad in ((0, "target_probs", dev[0][:-1]), (1, "draft_probs", dev[1].half()), (3, "cu_drafts", dev[3][:2]),
                         (4, "uniforms", dev[4][:2]), (5, "noise", dev[5][0])):
        with pytest.raises(ValueError, match=name):
            ql.qlinear_verify_draft(*dev[:i], bad, *dev[i + 1:], out, acc, ws)
    with pytest.raises(ValueError, match="out_tokens"):
        ql.qlinear_verify_draft(*dev, out[:1], acc, ws)


# ------------------------------------------------------------------ draft verification

def verify_inputs(seed, counts, vocab, spread=0.6, certain=False):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(counts), len(counts)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    target = torch.softmax(2.5 * randn(g, n + b, vocab), -1)
    rows = torch.tensor([i + s for s in range(b) for i in range(int(cu[s]), int(cu[s + 1]))], dtype=torch.int64)
    draft = torch.softmax(torch.log(target[rows]) + spread * randn(g, n, vocab), -1) if n else torch.zeros(0, vocab)
    tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32) if n else torch.zeros(0, dtype=torch.int32)
    u = torch.rand(n, generator=g)
    noise = -torch.log(torch.rand(b, vocab, generator=g).clamp_min(1e-20)) + 1e-10
    return target, None if certain else draft, tokens, cu, u, noise


def run_verify(target, draft, tokens, cu, u, noise, max_drafts):
    b, vocab = noise.shape
    out = torch.full((b, max_drafts + 1), 99, dtype=torch.int32, device="cuda")
    acc = torch.full((b,), 99, dtype=torch.int32, device="cuda")
    ql.qlinear_verify_draft(target.cuda(), None if draft is None else draft.cuda(), tokens.cuda(),
                            torch.from_numpy(cu).cuda(), u.cuda(), noise.cuda(), out, acc, ql.verify_workspace(b, vocab))
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy()


@pytest.mark.parametrize("counts,vocab,certain", [([3], 5, False), ([1], 1, False), ([4, 0, 5, 2], 1000, False),
                                                  ([3, 3, 3], 32001, False), ([5, 1], 4099, True), ([0, 0], 77, False),
                                                  ([70, 2], 129, False), ([2] * 40, 2053, False)])
def test_verify_draft(counts, vocab, certain):
    for seed in range(4):
        x = verify_inputs(seed + vocab, counts, vocab, certain=certain, spread=0.2 if seed % 2 else 0.8)
        most = max(counts) + seed % 2
        want = ref.verify(*(None if t is None else np.asarray(t) for t in x), most)
        got = run_verify(*x, most)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), (seed, got, want)


def test_verify_draft_edges():
    """Equal distributions accept everything; zero target probability never
    accepts; ties take the lowest index; NaN and a token outside the vocabulary
    count as nothing; p - q nowhere positive falls back to p."""
    V = 300
    flat = torch.full((2, V), 1.0 / V)
    ones = torch.ones(1, V)
    zero = np.array([0, 1], np.int32)
    x = (flat, flat[:1].clone(), torch.tensor([7], dtype=torch.int32), zero, torch.tensor([0.999]), ones)
    assert run_verify(*x, 1)[0].tolist() == [[7, 0]]
    t = flat.clone()
    t[0, 7] = 0.0
    out, acc = run_verify(t, flat[:1], torch.tensor([7], dtype=torch.int32), zero, torch.tensor([0.0]), ones, 1)
    assert acc.tolist() == [0] and out.tolist() == [[0, -1]]        # p <= q everywhere: p itself, lowest index
    t = flat.clone()
    t[0, :5] = float("nan")
    t[0, 200] = 0.5
    out, acc = run_verify(t, flat[:1], torch.tensor([3], dtype=torch.int32), zero, torch.tensor([0.0]), ones, 1)
    assert acc.tolist() == [0] and out.tolist() == [[200, -1]]
    for bad in (-1, V, 2 ** 31 - 1):
        out, acc = run_verify(flat, flat[:1], torch.tensor([bad], dtype=torch.int32), zero, torch.tensor([0.0]), ones, 1)
        assert acc.tolist() == [0] and out.tolist() == [[0, -1]]


def test_verify_draft_follows_the_target():
    """Over many draws the first token's frequencies are the target's, whatever the draft's."""
    V, B = 5, 40000
    g = torch.Generator().manual_seed(1)
    p, q = torch.tensor([0.1, 0.35, 0.05, 0.3, 0.2]), torch.tensor([0.3, 0.1, 0.4, 0.15, 0.05])
    tokens = torch.multinomial(q, B, replacement=True, generator=g).to(torch.int32)
    noise = torch.empty(B, V).exponential_(generator=g).clamp_min(1e-20)
    out, _ = run_verify(p.expand(2 * B, V).contiguous(), q.expand(B, V).contiguous(), tokens,
                        np.arange(B + 1, dtype=np.int32), torch.rand(B, generator=g), noise, 1)
    freq = np.bincount(out[:, 0], minlength=V) / B
    # five standard deviations of a frequency near 0.35 over 40,000 draws
    assert np.abs(freq - p.numpy()).max() < 5 * np.sqrt(0.35 * 0.65 / B), freq


# ------------------------------------------------------------------ edges of the arguments and of the values

def test_an_empty_table_gives_nan_rows():
    """No position is known where the table has no row: every rotated row is NaN, and nothing is read."""
    q, k, _, qw, kw = head_inputs(2, 3, 2, 1, 64, True)
    pos = torch.tensor([0, 5, -1]).cuda()
    qo, ko = torch.zeros_like(q).contiguous(), torch.zeros_like(k).contiguous()
    ql.qlinear_qk_norm_rope(q, k, pos, ql.rope_table(0, 64), qo, ko, qw, kw)
    assert torch.isnan(qo).all() and torch.isnan(ko).all()


def test_a_cache_on_another_device_is_refused():
    q, k, v, qw, kw = head_inputs(1, 2, 4, 2, 64, True)
    p = Problem(1, [1, 1], [90, 40], 4, 2, 64, 16, False)
    plan = p.plan()
    out = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    pos, slots, table = torch.zeros(2, dtype=torch.int64).cuda(), torch.tensor([0, 1]).cuda(), ql.rope_table(8, 64)
    p.cache.device_index = torch.cuda.current_device() + 1
    with pytest.raises(ValueError, match="cache"):
        ql.qlinear_qkv_append(q, k, v, pos, slots, table, torch.zeros_like(q), p.cache, qw, kw)
    with pytest.raises(ValueError, match="cache"):
        ql.qlinear_qkv_append(None, k, v, pos, slots, table, None, p.cache, qw, kw)
    with pytest.raises(ValueError, match="cache"):
        ql.qlinear_attention(plan, p.q, p.cache, p.table.cuda(), p.lens.cuda(), p.cu.cuda(), out,
                             workspace=plan.new_workspace())


@pytest.mark.parametrize("batch,D,e4m3,max_q,max_kv", [(130, 64, False, None, None), (70, 128, True, 500, 3000),
                                                       (5, 64, False, 2000, 9000), (200, 64, True, 41, 4000)])
def test_attention_of_chunks_in_ragged_batches(batch, D, e4m3, max_q, max_kv):
    """Many sequences of none, few and many new tokens, bounds far above them,
    with keys in one chunk and in several."""
    new = [(0, 40, 1, 9, 0, 33, 130 if max_q != 41 else 41)[i % 7] for i in range(batch)]
    p = Problem(90 + batch, new, [max(3, n) + (i * 7919) % 200 for i, n in enumerate(new)], 4, 2, D, 16, e4m3)
    cols = -(-(max_kv or 0) // 16)
    p.table = torch.nn.functional.pad(p.table, (0, max(0, cols - p.table.shape[1])), value=-7)
    plan = p.plan(max_q=max_q, max_kv=max_kv)
    assert plan.facts["tile_rows"] == 128
    out, ls = p.run(plan)
    p.check(out, ls)


NAN_SCORE_CASES = [(2, 40, 40, 0), (3, 3000, 3000, 0), (40, 200, 200, 0), (40, 9000, 9000, 0), (6, 300, 300, 20)]


@pytest.mark.parametrize("new,kv,max_kv,window", NAN_SCORE_CASES)
def test_lse_of_rows_whose_scores_are_nan(new, kv, max_kv, window):
    """A row of NaN scores has a NaN output and a NaN lse (-inf says that a row
    sees nothing); the other rows keep theirs."""
    p = Problem(61, [new], [kv], 4, 2, 64, 16, False)
    plan = p.plan(window=window, max_kv=max_kv)
    clean, clean_lse = p.run(plan)
    q = p.q
    p.q = q.clone()
    p.q[new - 1, 1, 7] = float("nan")
    out, lse = p.run(plan)
    p.q = q
    hit = torch.zeros(new, 4, dtype=torch.bool, device="cuda")
    hit[new - 1, 1] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    out[hit], lse[hit] = clean[hit], clean_lse[hit]
    p.check(out, lse, window=window)


@pytest.mark.parametrize("new,kv", [(5, 70), (6, 3000), (40, 130), (40, 9000)])
def test_lse_of_rows_that_see_a_nan_key(new, kv):
    p = Problem(62, [new], [kv], 4, 2, 128, 16, True)
    plan = p.plan()
    out, clean = p.run(plan)
    at = kv - 2
    p.k[int(p.table[0, at // 16]), at % 16, 1, 9] = torch.tensor(float("nan")).to(E4M3).cuda()
    _, lse = p.run(plan)
    hit = torch.zeros(new, 4, dtype=torch.bool, device="cuda")
    hit[new - 2:, 2:] = True
    assert torch.isnan(lse[hit]).all()
    lse[hit] = clean[hit]
    p.check(out, lse)


def test_verify_draft_counts_nan_draft_probabilities_as_zero():
    """At the drafted token (accepted where the target's is positive), elsewhere
    in a rejected row (the whole of p is left there), and with certain drafts after it."""
    V = 300
    nan, zero = float("nan"), np.array([0, 1], np.int32)
    flat, ones = torch.full((2, V), 1.0 / V), torch.ones(1, V)
    q = flat[:1].clone()
    q[0, 7] = nan
    x = (flat, q, torch.tensor([7], dtype=torch.int32), zero, torch.tensor([0.999]), ones)
    out, acc = run_verify(*x, 1)
    assert acc.tolist() == [1] and out.tolist() == [[7, 0]]
    t = flat.clone()
    t[0, 7] = 0.0                                            # 0 < 0 is false: rejected
    assert run_verify(t, *x[1:], 1)[1].tolist() == [0]
    t, q = flat.clone(), flat[:1].clone()
    t[0, 3], t[0, 250], q[0, 250] = 0.0, 1.5 / V, nan        # left: 1.5 / V at 250, nothing elsewhere
    out, acc = run_verify(t, q, torch.tensor([3], dtype=torch.int32), zero, torch.tensor([0.5]), ones, 1)
    assert acc.tolist() == [0] and out.tolist() == [[250, -1]]
    for seed in range(3):
        target, draft, tokens, cu, u, noise = verify_inputs(seed, [3, 2, 4], 801, spread=0.8)
        draft[torch.rand(draft.shape, generator=torch.Generator().manual_seed(seed)) < 0.2] = nan
        want = ref.verify(*(np.asarray(y) for y in (target, draft, tokens, cu, u, noise)), 4)
        got = run_verify(target, draft, tokens, cu, u, noise, 4)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), (seed, got, want)


@pytest.mark.parametrize("new,kv", [([8], [5]), ([6, 1], [3, 900]), ([200, 4], [100, 700])])
def test_a_window_as_long_as_can_be_is_no_window(new, kv):
    """More new tokens than cached ones beside it: positions below zero minus the window do not wrap."""
    p = Problem(71, new, kv, 4, 2, 64, 16, False)
    for window in (2 ** 31 - 1, 2 ** 31 - 6, 2 ** 40 + 5):
        out, ls = p.run(p.plan(window=window))
        p.check(out, ls)


def test_verify_many_sequences_of_a_tiny_vocabulary():
    counts, V = [i % 3 for i in range(1500)], 3
    x = verify_inputs(5, counts, V, spread=0.8)
    want = ref.verify(*(np.asarray(t) for t in x), 2)
    got = run_verify(*x, 2)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_rows_of_another_length_are_refused():
    """Probabilities of a padded vocabulary, and an lse of other heads, hold
    enough elements but not where the call would read or write them."""
    target, draft, tokens, cu, u, noise = verify_inputs(3, [2, 1], 50)
    dev = [torch.nn.functional.pad(target, (0, 14)).cuda(), torch.nn.functional.pad(draft, (0, 14)).cuda(), tokens.cuda(),
           torch.from_numpy(cu).cuda(), u.cuda(), noise.cuda()]
    out, acc = torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    ws = ql.verify_workspace(2, 50)
    for i, name in ((0, "target_probs"), (1, "draft_probs")):
        x = list(dev)
        x[1 - i] = (target, draft)[1 - i].cuda()
        with pytest.raises(ValueError, match=name):
            ql.qlinear_verify_draft(*x, out, acc, ws)
    p = Problem(1, [3, 2], [90, 40], 4, 2, 64, 16, False)
    plan = p.plan()
    with pytest.raises(ValueError, match="lse"):
        ql.qlinear_attention(plan, p.q, p.cache, p.table.cuda(), p.lens.cuda(), p.cu.cuda(),
                             torch.zeros(5, 4, 64, dtype=BF16, device="cuda"), torch.zeros(4, 5, device="cuda"),
                             plan.new_workspace())


def test_page_table_as_columns_of_a_wider_one():
    p = Problem(12, [1, 2, 40], [500, 33, 90], 8, 2, 128, 16, False)
    want, lse = p.run(p.plan())
    wide = torch.full((3, p.table.shape[1] + 5), -9, dtype=torch.int32)
    wide[:, 2:-3] = p.table
    out, got = torch.zeros_like(want), torch.zeros_like(lse)
    plan = p.plan()
    args = (p.lens.cuda(), p.cu.cuda(), out, got, plan.new_workspace())
    ql.qlinear_attention(plan, p.q, p.cache, wide.cuda()[:, 2:-3], *args)
    assert torch.equal(out, want) and torch.equal(got, lse)
    with pytest.raises(ValueError, match="page_table"):
        ql.qlinear_attention(plan, p.q, p.cache, p.table.cuda().T.contiguous().T, *args)


def test_attention_mixed_batch_of_wide_groups():
    """More query heads a KV head than the decode share of a mixed batch takes rows."""
    p = Problem(23, [50, 1, 1, 2, 0, 1], [300, 1500, 40, 65, 20, 1], 24, 1, 64, 16, False)
    p.table = torch.nn.functional.pad(p.table, (0, 3750 - p.table.shape[1]), value=-7)
    out, ls = p.run(p.plan(max_kv=60000))
    p.check(out, ls)


@pytest.mark.parametrize("D,e4m3", [(64, False), (128, False), (64, True), (128, True)])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [17, 60, 2000]), ([5, 2, 4], [40, 300, 25]), ([1], [4001])])
def test_decode_weights_are_not_held_in_bf16(new, kv, D, e4m3):
    """The decode kernel's weights enter the product with V to 2^-16 of a
    weight: only the output's own rounding is bf16's."""
    p = Problem(81 + D, new, kv, 8, 2, D, 16, e4m3)
    out, _ = p.run(p.plan())
    assert p.plan().facts["tile_rows"] == 0
    r = ref.attention(f64(p.q), p.k_host, p.v_host, p.table.numpy(), p.kv, p.cu.numpy(), 16, D ** -0.5, True, 0,
                      None if p.ks is None else f64(p.ks), None if p.vs is None else f64(p.vs))
    d = 2 * D * U * r["reach"] + 8 * U * (r["reach"] + 1)
    tol = r["weight"] * (2.0 ** -16 + 2 * d + 2 * max(kv) * U)[..., None] + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(r["out"]) + 1e-38
    err = np.abs(f64(out) - r["out"])
    assert (err <= tol).all(), (int((err > tol).sum()), err.size, float((err / tol).max()))


def test_decode_and_append_beyond_32_bit_offsets():
    """The decode kernel, and rows appended to the last pages, in a cache of more than 4 GiB a tensor."""
    page, hk, D, pages = 64, 8, 128, (1 << 32) // (64 * 8 * 128 * 2) + 40
    k = torch.empty(pages, page, hk, D, dtype=BF16, device="cuda")
    v = torch.empty(pages, page, hk, D, dtype=BF16, device="cuda")
    p = Problem(8, [1, 4], [500, 70], 16, hk, D, page, False)
    first = pages - p.k.shape[0]
    k[first:], v[first:] = p.k, p.v
    p.table[p.table >= 0] += first
    p.cache = ql.PagedCache(k, v)
    plan = p.plan()
    assert plan.facts["tile_rows"] == 0 and k.element_size() * k.stride(0) * first > 1 << 32
    out, ls = p.run(plan)
    p.table[p.table >= 0] -= first
    p.check(out, ls)
    q, nk, nv, qw, kw = head_inputs(4, 3, 2, hk, D, True)
    slots = torch.tensor([pages * page - 1, (pages - 1) * page, first * page + 5])
    table, pos = ql.rope_table(16, D), torch.tensor([3, 15, 0])
    before = [x[first:].clone() for x in (k, v)]
    ql.qlinear_qkv_append(None, nk, nv, pos.cuda(), slots.cuda(), table, None, p.cache, qw, kw)
    torch.cuda.synchronize()
    y, size = ref.norm_rope(f64(nk), f64(kw), pos.numpy(), f64(table), D, False, 1e-6)
    at = (slots - first * page).cuda()
    check_rounded(f64(k[first:].flatten(0, 1)[at]), y, size, D, "k")
    assert torch.equal(v[first:].flatten(0, 1)[at], nv)
    rest = torch.ones((pages - first) * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    for x, old in zip((k, v), before):
        got, old = (t.flatten(0, 1).view(torch.int16)[rest] for t in (x[first:], old))
        assert torch.equal(got, old), "slots that were not given changed"
