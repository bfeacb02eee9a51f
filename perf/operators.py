"""Operators around the quantized linears of a serving step: what is measured of them.

Between the QKV and the O projection of a layer, a serving step normalises and
rotates the heads of the queries and keys, appends keys and values to a paged
cache and attends over it; after the last layer it checks drafted tokens
against the target's probabilities.  Head layouts are those of the workloads
of this repository: QKV widths 6144 = (32 + 2*8)*128 (8B class), 7168 =
(40 + 2*8)*128 (14B class) and 10240 = (64 + 2*8)*128 (32B class), with
64-wide heads as the second head size.
"""

import torch

own = False     # False: the plain form; True: the framework's operators

PAGE_TABLE_SLACK = 3        # page-table columns beyond the longest sequence, as a server over-allocates
ACCEPT = 0.75               # about this share of drafted tokens is accepted (what prepare's draft model gives)


def listed():
    return [
        # a decode step of the 8B class: eight running sequences, one new token each; launch latency counts
        dict(name="norm_rope_8", op="norm_rope", tokens=8, q_heads=32, kv_heads=8, dim=128, rot=128, norm=True,
             interleaved=False, max_pos=8192),
        # a long prefill chunk of the 14B class: streaming, bandwidth counts
        dict(name="norm_rope_8191", op="norm_rope", tokens=8191, q_heads=40, kv_heads=8, dim=128, rot=128, norm=True,
             interleaved=False, max_pos=16384),
        # a decode step of the 32B class appending one token to each of 32 sequences
        dict(name="append_32", op="append", tokens=32, q_heads=64, kv_heads=8, dim=128, rot=128, norm=True,
             interleaved=False, max_pos=8192, cache="bf16", page=16, pages=2048),
        # a prefill chunk of the 8B class written as E4M3
        dict(name="append_4096_e4m3", op="append", tokens=4096, q_heads=32, kv_heads=8, dim=128, rot=128, norm=True,
             interleaved=False, max_pos=16384, cache="e4m3", page=16, pages=1024),
        # one interactive user of the 8B class: one token over a short context; latency counts
        dict(name="attend_1x1031", op="attend", batch=1, new=1, even=True, kv=1031, kv_min=1031, q_heads=32, kv_heads=8,
             dim=128, cache="bf16", page=16, window=0),
        # a full decode batch of the 32B class over contexts of different lengths
        dict(name="attend_32x8190", op="attend", batch=32, new=1, even=True, kv=8190, kv_min=1021, q_heads=64,
             kv_heads=8, dim=128, cache="bf16", page=16, window=0),
        # a large decode batch of the 14B class over an E4M3 cache
        dict(name="attend_64x16001_e4m3", op="attend", batch=64, new=1, even=True, kv=16001, kv_min=4003, q_heads=40,
             kv_heads=8, dim=128, cache="e4m3", page=32, window=0),
        # the forward that checks four drafted tokens a sequence (five new rows each), 8B class
        dict(name="attend_draft_16x5", op="attend", batch=16, new=5, even=True, kv=4099, kv_min=515, q_heads=32,
             kv_heads=8, dim=128, cache="bf16", page=16, window=0),
        # a prefill chunk of 2048 tokens at the end of a 10,240-token context, 8B class; matrix products count
        dict(name="attend_chunk_2048", op="attend", batch=1, new=2048, even=True, kv=10240, kv_min=10240, q_heads=32,
             kv_heads=8, dim=128, cache="bf16", page=16, window=0),
        # chunks and single tokens mixed in one batch, 64-wide heads over an E4M3 cache, a sliding window
        dict(name="attend_mixed_e4m3", op="attend", batch=12, new=701, even=False, kv=4097, kv_min=701, q_heads=32,
             kv_heads=8, dim=64, cache="e4m3", page=64, window=2048),
        # two interactive users, three drafted tokens each, a small vocabulary
        dict(name="verify_2x3", op="verify", batch=2, drafts=3, vocab=32001),
        # a full batch of drafted tokens against a large vocabulary
        dict(name="verify_64x5", op="verify", batch=64, drafts=5, vocab=151936),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    heads = rng.choice([(32, 8, 128), (40, 8, 128), (64, 8, 128), (32, 8, 64), (16, 16, 128), (28, 4, 128), (24, 1, 64)])
    op = rng.choice(["norm_rope", "append", "attend", "attend", "attend", "verify"])
    base = dict(op=op, q_heads=heads[0], kv_heads=heads[1], dim=heads[2])
    if op in ("norm_rope", "append"):
        d = dict(base, tokens=log_int(1, 8000), rot=rng.choice([heads[2], heads[2], heads[2] // 2]),
                 norm=rng.random() < 0.75, interleaved=rng.random() < 0.25, max_pos=16384)
        if op == "append":
            page = rng.choice([16, 32, 64, 48])
            d.update(cache=rng.choice(["bf16", "e4m3"]), page=page, pages=-(-d["tokens"] // page) + log_int(8, 500))
        return d
    if op == "verify":
        return dict(op=op, batch=log_int(1, 64), drafts=rng.randint(1, 5), vocab=log_int(4001, 151936))
    cache, page = rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 48])
    kv = log_int(17, 16000)
    if rng.random() < 0.6:       # decode, drafted tokens included
        most = 64 * 16001 * 8 * 128 // (kv * heads[1] * heads[2] * (1 if cache == "e4m3" else 2))
        new, batch, even = min(kv, rng.choice([1, 1, 2, 3, 4, 5, 7, 8])), max(1, min(most, log_int(1, 64))), True
    else:                        # chunks, alone or mixed with single tokens
        kv = min(kv, 10240)
        new = min(kv, log_int(9, 2048))
        new = max(1, min(new, 2048 * 10240 * 32 // (kv * heads[0])))
        batch = max(1, min(12, 2048 * 10240 * 32 // (new * kv * heads[0]), log_int(1, 12)))
        even = rng.random() < 0.5
    return dict(base, batch=batch, new=new, even=even, kv=kv, kv_min=max(new, log_int(max(1, kv // 8), kv)), cache=cache,
                page=page, window=rng.choice([0, 0, 0, log_int(64, 4096)]))


def _lengths(c):
    """(new tokens, context length with them) of every sequence: spread evenly over the case's ranges."""
    b = c["batch"]
    kv = [c["kv"] - (c["kv"] - c["kv_min"]) * i // max(1, b - 1) for i in range(b)]
    new = [c["new"] if c["even"] or i % 3 == 0 else 1 if i % 3 == 1 else 1 + c["new"] * i // b for i in range(b)]
    return [min(n, k) for n, k in zip(new, kv)], kv


def _visible(c, n, kv):
    """Number of (new token, key) pairs that causality and the window leave of one sequence."""
    w = c["window"] or kv
    return sum(min(w, kv - n + i + 1) for i in range(n))


def work(c):
    d = c.get("dim", 0)
    if c["op"] == "norm_rope":
        rows = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return dict(bytes=rows * d * 4 + c["tokens"] * (c["rot"] * 4 + 8), flops=rows * d * 8)
    if c["op"] == "append":
        rows, kv = c["tokens"] * (c["q_heads"] + c["kv_heads"]), c["tokens"] * c["kv_heads"] * d
        size = 1 if c["cache"] == "e4m3" else 2
        return dict(bytes=c["tokens"] * c["q_heads"] * d * 4 + 2 * kv * (2 + size) + c["tokens"] * (c["rot"] * 4 + 16),
                    flops=rows * d * 8)
    if c["op"] == "attend":
        size = 1 if c["cache"] == "e4m3" else 2
        new, kv = _lengths(c)
        seen = [k if not c["window"] else min(k, n - 1 + c["window"]) for n, k in zip(new, kv)]
        return dict(bytes=2 * sum(seen) * c["kv_heads"] * d * size + 4 * sum(new) * c["q_heads"] * d
                    + sum(-(-k // c["page"]) for k in seen) * 4,
                    flops=4 * d * c["q_heads"] * sum(_visible(c, n, k) for n, k in zip(new, kv)))
    rejected = 1 - ACCEPT ** c["drafts"]    # only a rejected sequence needs a row of the draft's probabilities
    return dict(bytes=c["batch"] * c["vocab"] * 4 * (2 + rejected) + c["batch"] * (c["drafts"] * 16 + 8),
                flops=c["batch"] * c["vocab"] * 4)


def _rope_table(c):
    half = c["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    s = dict(case=c)
    if c["op"] in ("norm_rope", "append"):
        t, hq, hk, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
        # the QKV projection's output rows: queries, keys and values side by side, a few large channels
        x = randn(t, hq + 2 * hk, d)
        x[:, :, torch.randperm(d, generator=g, device="cuda")[:max(1, d // 50)]] *= 8.0
        qkv = x.to(torch.bfloat16)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                 positions=torch.randint(0, c["max_pos"], (t,), generator=g, device="cuda", dtype=torch.int64),
                 table=_rope_table(c),
                 q_weight=(1 + 0.2 * randn(d)).to(torch.bfloat16) if c["norm"] else None,
                 k_weight=(1 + 0.2 * randn(d)).to(torch.bfloat16) if c["norm"] else None,
                 q_out=torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda"))
        if c["op"] == "norm_rope":
            s["k_out"] = torch.zeros(t, hk, d, dtype=torch.bfloat16, device="cuda")
            return s
        shape = (c["pages"], c["page"], hk, d)
        # a cache in use: every slot of it holds some token already
        k, v = (randn(*shape).to(torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16) for _ in range(2))
        scales = c["cache"] == "e4m3"
        s.update(slots=torch.randperm(c["pages"] * c["page"], generator=g, device="cuda")[:t].to(torch.int64), k_cache=k,
                 v_cache=v, k_scale=0.05 + 0.01 * randn(hk).abs() if scales else None,
                 v_scale=0.05 + 0.01 * randn(hk).abs() if scales else None)
    elif c["op"] == "attend":
        new, kv = _lengths(c)
        hq, hk, d, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        need = [-(-k // page) for k in kv]
        pages = sum(need) + 5
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(c["batch"], max(need) + PAGE_TABLE_SLACK, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        scales = c["cache"] == "e4m3"
        shape = (pages, page, hk, d)
        k, v = (torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        if scales:
            k, v = ((x * 16).to(torch.float8_e4m3fn) for x in (k, v))
        cu = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        s.update(q=(1.5 * randn(sum(new), hq, d)).to(torch.bfloat16), k_cache=k, v_cache=v,
                 k_scale=0.06 + 0.01 * randn(hk).abs() if scales else None,
                 v_scale=0.06 + 0.01 * randn(hk).abs() if scales else None, page_table=table,
                 seq_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"), cu_q=cu, max_q=max(new), max_kv=max(kv),
                 out=torch.zeros(sum(new), hq, d, dtype=torch.bfloat16, device="cuda"))
    else:
        b, n, vocab = c["batch"], c["drafts"], c["vocab"]
        # a target model's distributions, and a draft model's that are near to them
        logits = 2.5 * randn(b, n + 1, vocab)
        target = torch.softmax(logits, -1)
        draft = torch.softmax(logits[:, :n] + 0.6 * randn(b, n, vocab), -1).reshape(b * n, vocab)
        s.update(target=target.reshape(b * (n + 1), vocab), draft=draft,
                 tokens=torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32),
                 cu_drafts=torch.arange(0, b * n + 1, n, dtype=torch.int32, device="cuda"),
                 uniforms=torch.rand(b * n, generator=g, device="cuda"),
                 noise=torch.empty(b, vocab, device="cuda").exponential_(generator=g).clamp_min(1e-20),
                 out_tokens=torch.zeros(b, n + 1, dtype=torch.int32, device="cuda"),
                 accepted=torch.zeros(b, dtype=torch.int32, device="cuda"))
    if own:
        import quantized_gemm_decode_amd as ql
        if c["op"] in ("append", "attend"):
            s["cache"] = ql.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "attend":
            s["plan"] = ql.qlinear_attention_plan(s["cache"], c["q_heads"], c["batch"], s["q"].shape[0], s["max_q"],
                                                  s["max_kv"], window=c["window"])
            s["workspace"] = s["plan"].new_workspace()
        if c["op"] == "verify":
            s["workspace"] = ql.verify_workspace(c["batch"], c["vocab"])
    return s


EPS = 1e-6


def _norm_rope(x, weight, s):
    """Root-mean-square norm of each head, then the rotation of its first `rot` channels, in 32 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot, half = c["rot"], c["rot"] // 2
    cs = s["table"][s["positions"]][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_norm_rope(s):
    s["q_out"].copy_(_norm_rope(s["q"], s["q_weight"], s))
    s["k_out"].copy_(_norm_rope(s["k"], s["k_weight"], s))
    return s["q_out"], s["k_out"]


def _store(cache, slots, x, scale):
    """Rows of 32-bit values into a cache's slots, rounded to its type."""
    if scale is None:
        cache.view(-1, *cache.shape[2:])[slots] = x.to(cache.dtype)
    else:
        codes = (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        cache.view(torch.uint8).view(-1, *cache.shape[2:])[slots] = codes.view(torch.uint8)


def _plain_append(s):
    s["q_out"].copy_(_norm_rope(s["q"], s["q_weight"], s))
    _store(s["k_cache"], s["slots"], _norm_rope(s["k"], s["k_weight"], s), s["k_scale"])
    _store(s["v_cache"], s["slots"], s["v"].float(), s["v_scale"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gather(cache, table, scale, length):
    """The cached rows of every sequence as [batch, kv heads, length, dim] in 32 bits."""
    e4m3 = cache.dtype == torch.float8_e4m3fn
    x = (cache.view(torch.uint8) if e4m3 else cache)[table.long()]
    x = (x.view(torch.float8_e4m3fn) if e4m3 else x).flatten(1, 2)[:, :length].float()
    return (x if scale is None else x * scale[:, None]).transpose(1, 2)


def _plain_attend(s):
    c = s["case"]
    b, hq, hk, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    n, length, dev = s["max_q"], s["max_kv"], s["q"].device
    width = -(-length // c["page"])
    k = _gather(s["k_cache"], s["page_table"][:, :width], s["k_scale"], length)
    v = _gather(s["v_cache"], s["page_table"][:, :width], s["v_scale"], length)
    cu, kv = s["cu_q"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, hq // hk * n, d)
    scores = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    at = kv[:, None] - new[:, None] + i                                     # position of each new token
    j = torch.arange(length, device=dev)
    sees = (j <= at[:, :, None]) & (i < new[:, None])[:, :, None]
    if c["window"]:
        sees &= j > at[:, :, None] - c["window"]
    scores = scores.view(b, hk, hq // hk, n, length).masked_fill(~sees[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(p.view(b, hk, hq // hk * n, length), v)
    o = o.view(b, hk, hq // hk, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, hq, d)
    keep = (i < new[:, None]).reshape(-1).nonzero()[:, 0]                   # the new tokens in their order
    s["out"].copy_(o[keep])
    return s["out"]


def _plain_verify(s):
    c = s["case"]
    b, n, vocab = c["batch"], c["drafts"], c["vocab"]
    seq = torch.arange(b, device="cuda")
    target, draft = s["target"].view(b, n + 1, vocab), s["draft"].view(b, n, vocab)
    tokens = s["tokens"].view(b, n).long()
    p = target[:, :n].gather(2, tokens[..., None])[..., 0]
    q = draft.gather(2, tokens[..., None])[..., 0]
    ok = s["uniforms"].view(b, n) * q < p
    accepted = ok.int().cumprod(1).sum(1)
    row = target[seq, accepted]
    other = draft[seq, accepted.clamp(max=n - 1)]
    left = torch.where((accepted < n)[:, None], (row - other).clamp_min(0), row)
    weight = torch.where((left > 0).any(1)[:, None], left, row)     # nothing left of the difference: the target itself
    chosen = (weight / s["noise"]).argmax(1)
    i = torch.arange(n + 1, device="cuda")
    padded = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(i < accepted[:, None], padded, torch.where(i == accepted[:, None], chosen[:, None], -1))
    s["out_tokens"].copy_(out)
    s["accepted"].copy_(accepted)
    return s["out_tokens"], s["accepted"]


def _own(s):
    import quantized_gemm_decode_amd as ql
    c = s["case"]
    if c["op"] == "norm_rope":
        ql.qlinear_qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["q_out"], s["k_out"], s["q_weight"],
                                s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return s["q_out"], s["k_out"]
    if c["op"] == "append":
        ql.qlinear_qkv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["table"], s["q_out"], s["cache"],
                              s["q_weight"], s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "attend":
        ql.qlinear_attention(s["plan"], s["q"], s["cache"], s["page_table"], s["seq_lens"], s["cu_q"], s["out"],
                             workspace=s["workspace"])
        return s["out"]
    ql.qlinear_verify_draft(s["target"], s["draft"], s["tokens"], s["cu_drafts"], s["uniforms"], s["noise"],
                            s["out_tokens"], s["accepted"], s["workspace"])
    return s["out_tokens"], s["accepted"]


PLAIN = dict(norm_rope=_plain_norm_rope, append=_plain_append, attend=_plain_attend, verify=_plain_verify)


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_heads(x, weight, s):
    """Norm and rotation as multiplications of complex numbers."""
    c = s["case"]
    x = x.double()
    if weight is not None:
        x = weight.double() * x / (x.square().sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
    half = c["rot"] // 2
    t = s["table"].double().index_select(0, s["positions"])
    turn = torch.complex(t[:, :half], t[:, half:]).unsqueeze(1)
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (
        slice(0, half), slice(half, c["rot"]))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_cache(cache, scale, slots, x):
    y = cache.double().flatten(0, 1)
    y[slots] = x if scale is None else (x / scale.double().view(1, -1, 1)).clamp(-448, 448)
    return y.view(cache.shape)


def _exact_attend(s):
    c = s["case"]
    g, hk, d = c["q_heads"] // c["kv_heads"], c["kv_heads"], c["dim"]
    new, kv = _lengths(c)
    out, first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, length) in enumerate(zip(new, kv)):
        at = torch.arange(length, device="cuda")
        page, slot = s["page_table"][b].long()[at // c["page"]], at % c["page"]
        pos = torch.arange(length - n, length, device="cuda")
        hidden = at[None, :] > pos[:, None]
        if c["window"]:
            hidden |= at[None, :] <= pos[:, None] - c["window"]
        for h in range(hk):
            ks, vs = ((x.view(torch.uint8)[page, slot, h].view(x.dtype) if x.dtype == torch.float8_e4m3fn
                       else x[page, slot, h]).double() for x in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                ks, vs = ks * s["k_scale"][h].double(), vs * s["v_scale"][h].double()
            q = s["q"][first:first + n, h * g:(h + 1) * g].double().transpose(0, 1)
            a = (q @ ks.T / d ** 0.5).masked_fill(hidden, float("-inf")).softmax(-1)
            out[first:first + n, h * g:(h + 1) * g] = (a @ vs).transpose(0, 1)
        first += n
    return out


def _exact_verify(s):
    c = s["case"]
    n = c["drafts"]
    tokens, counts = torch.full((c["batch"], n + 1), -1, dtype=torch.int32), []
    for b in range(c["batch"]):
        i = 0
        while i < n:
            x, row = int(s["tokens"][b * n + i]), b * n + i
            if float(s["uniforms"][row]) * float(s["draft"][row, x]) >= float(s["target"][b * (n + 1) + i, x]):
                break
            tokens[b, i] = x
            i += 1
        p = s["target"][b * (n + 1) + i].double()
        if i < n:
            left = (p - s["draft"][b * n + i].double()).clamp_min(0)
            p = left if bool((left > 0).any()) else p
        tokens[b, i] = int((p / s["noise"][b].double()).argmax())
        counts.append(i)
    return tokens, torch.tensor(counts, dtype=torch.int32)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        return _exact_heads(s["q"], s["q_weight"], s), _exact_heads(s["k"], s["k_weight"], s)
    if c["op"] == "append":
        return (_exact_heads(s["q"], s["q_weight"], s),
                _exact_cache(s["k_cache"], s["k_scale"], s["slots"], _exact_heads(s["k"], s["k_weight"], s)),
                _exact_cache(s["v_cache"], s["v_scale"], s["slots"], s["v"].double()))
    return _exact_attend(s) if c["op"] == "attend" else _exact_verify(s)
