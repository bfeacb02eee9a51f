"""Operators of a server of many requests with tree-shaped drafts: what is measured of them.

A step of such a server runs the shared projections with each request's
low-rank adapter beside them, attends from a tree of drafted tokens over the
cache, draws a token at every node of the tree from the head's logits, and
commits the branch that the draws agree with: its tokens are given out and
its keys and values move to the places behind the context.  Widths are those
of the workloads of this repository: hidden 4096 with QKV 6144 = 4096 + 2*1024
(8B class), hidden 5120 with QKV 7168 and gate_up 34816 = 2*17408 (14B class),
QKV 10240 (32B class).
"""

import torch

own = False     # False: the plain form; True: the framework's operators

PAGE_TABLE_SLACK = 3        # page-table columns beyond the longest sequence, as a server over-allocates


def listed():
    return [
        # a decode step of the 8B class, eight requests with an adapter each, merged QKV; launch latency counts
        dict(name="lora_8", op="lora", tokens=8, runs=1, adapters=16, rank=16, k=4096, widths="4096,1024,1024", pad=0),
        # a full decode batch of the 14B class, merged gate and up, few adapters shared by many requests
        dict(name="lora_64", op="lora", tokens=64, runs=1, adapters=24, rank=32, k=5120, widths="17408,17408", pad=0),
        # prompt chunks of some requests, 8B class, merged QKV; streaming, bandwidth counts
        dict(name="lora_4093", op="lora", tokens=4093, runs=700, adapters=8, rank=16, k=4096, widths="4096,1024,1024",
             pad=0),
        # one interactive user, a small vocabulary; latency counts
        dict(name="sample_1", op="sample", rows=1, vocab=32001, type="f32", rules="all", probs=False),
        # a full batch with a large vocabulary, every request with rules of its own
        dict(name="sample_64_bf16", op="sample", rows=64, vocab=151936, type="bf16", rules="mixed", probs=False),
        # the target's and the draft's distributions for the verification of drafted tokens
        dict(name="sample_probs_40", op="sample", rows=40, vocab=128256, type="f32", rules="top_p", probs=True),
        # one interactive user of the 8B class with a tree of 25 drafted tokens; latency counts
        dict(name="tree_1x26", op="tree", batch=1, nodes=26, even=True, kv=1031, kv_min=1031, q_heads=32, kv_heads=8,
             dim=128, cache="bf16", page=16),
        # a batch of the 8B class over contexts of different lengths
        dict(name="tree_16x32", op="tree", batch=16, nodes=32, even=True, kv=4099, kv_min=515, q_heads=32, kv_heads=8,
             dim=128, cache="bf16", page=16),
        # a large batch of the 14B class, trees of up to 63 drafts, an E4M3 cache; matrix products count
        dict(name="tree_32x64_e4m3", op="tree", batch=32, nodes=64, even=False, kv=8190, kv_min=1021, q_heads=40,
             kv_heads=8, dim=128, cache="e4m3", page=32),
        # the commit of a few interactive users in one layer's cache; latency counts
        dict(name="commit_4x13", op="commit", batch=4, nodes=13, layers=1, kv=1031, kv_min=300, kv_heads=8, dim=128,
             cache="bf16", page=16),
        # a full batch's commit in the caches of eight layers
        dict(name="commit_64x64", op="commit", batch=64, nodes=64, layers=8, kv=1023, kv_min=300, kv_heads=8, dim=128,
             cache="bf16", page=16),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["lora", "lora", "sample", "sample", "tree", "tree", "commit"])
    if op == "lora":
        k = rng.choice([2048, 4096, 5120, 12288])
        widths = rng.choice(["4096,1024,1024", "5120,1024,1024", "8192,1024,1024", "4096", "5120", "1000",
                             "12288,12288", "17408,17408"])
        wide = sum(map(int, widths.split(",")))
        tokens = min(log_int(1, 4093), 4093 * (4096 + 2 * 6144) // (k + 2 * wide))
        adapters, rank = log_int(1, 32), rng.choice([8, 16, 16, 32, 64])
        return dict(op=op, tokens=tokens, runs=1 if tokens <= 128 else log_int(64, 2000), adapters=adapters, rank=rank,
                    k=k, widths=widths, pad=rng.choice([0, 0, 64]))
    if op == "sample":
        rows = log_int(1, 64)
        probs = rng.random() < 0.4
        return dict(op=op, rows=rows, vocab=min(log_int(4001, 151936), 151936 * 32 // rows if probs else 151936),
                    type=rng.choice(["f32", "bf16"]), rules=rng.choice(["all", "mixed", "mixed", "top_k", "top_p", "none"]),
                    probs=probs)
    page = rng.choice([16, 32, 64, 48])
    cache = rng.choice(["bf16", "e4m3"])
    nodes = rng.randint(3, 64)
    if op == "commit":
        return dict(op=op, batch=log_int(1, 64), nodes=nodes, layers=rng.randint(1, 8), kv=log_int(200, 1023),
                    kv_min=100, kv_heads=rng.choice([8, 4, 1]), dim=rng.choice([128, 64]), cache=cache, page=page)
    heads = rng.choice([(32, 8, 128), (40, 8, 128), (64, 8, 128), (32, 8, 64), (16, 16, 128), (28, 4, 128), (24, 1, 64)])
    kv = log_int(80, 8190)
    most = 32 * 64 * 8190 * 40 * 128 // (2 * kv * nodes * heads[0] * heads[2])
    return dict(op=op, batch=max(1, min(most, log_int(1, 32))), nodes=nodes, even=rng.random() < 0.5, kv=kv,
                kv_min=max(nodes, log_int(max(1, kv // 8), kv)), q_heads=heads[0], kv_heads=heads[1], dim=heads[2],
                cache=cache, page=page)


def _widths(c):
    return [int(w) for w in c["widths"].split(",")]


def _lengths(c):
    """(nodes, context length with them) of every sequence: spread evenly over the case's ranges."""
    b = c["batch"]
    kv = [c["kv"] - (c["kv"] - c["kv_min"]) * i // max(1, b - 1) for i in range(b)]
    new = [c["nodes"] if c.get("even", False) or i % 3 == 0 else 1 + c["nodes"] * i // b for i in range(b)]
    return [min(n, k) for n, k in zip(new, kv)], kv


def _tree(n):
    """Parents of a drafted tree of n nodes, node 0 the newest token: the likeliest chain first, then branches of
    two nodes, each hanging off the chain, one place later than the last."""
    chain = min(n, 7)
    parents = list(range(-1, chain - 1))
    while len(parents) < n:
        i = len(parents) - chain
        parents.append((i // 2) % chain if i % 2 == 0 else len(parents) - 1)
    return parents


def _ancestors(parents):
    """Bit masks of the nodes that each node sees: itself and those above it."""
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    return [m - (1 << 64) if m >> 63 else m for m in masks]


def _accepted_path(n, seq):
    """The nodes that sequence `seq` of a batch accepts: some of the chain, in two of three also a branch off it."""
    parents = _tree(n)
    chain = min(n, 7)
    path = list(range(1, min(chain, 1 + seq % 5)))
    if seq % 3:
        off = [i for i in range(chain, n) if parents[i] == (path[-1] if path else 0)]
        if off:
            path.append(off[-1])
            path += [i for i in range(off[-1] + 1, n) if parents[i] == off[-1]][:1]
    return path


def work(c):
    if c["op"] == "lora":
        t, k, w, s = c["tokens"], c["k"], sum(_widths(c)), len(_widths(c))
        used = min(c["adapters"], -(-t // c["runs"]))
        return dict(bytes=2 * t * (k + 2 * w) + 4 * t + used * c["rank"] * 2 * (s * k + w),
                    flops=2 * t * c["rank"] * (s * k + w))
    if c["op"] == "sample":
        size = 4 if c["type"] == "f32" else 2
        return dict(bytes=c["rows"] * c["vocab"] * (size + (4 if c["rules"] == "none" else 0) + (4 if c["probs"] else 0)),
                    flops=c["rows"] * c["vocab"] * 8)
    size = 1 if c["cache"] == "e4m3" else 2
    new, kv = _lengths(c)
    if c["op"] == "commit":
        moved = sum(sum(i != d for d, i in enumerate(_accepted_path(n, b), 1)) for b, n in enumerate(new))
        return dict(bytes=4 * moved * c["layers"] * c["kv_heads"] * c["dim"] * size + 12 * sum(new) + 64 * c["batch"],
                    flops=0)
    pairs = sum(n * (k - n) + sum(bin(m & (2 ** 64 - 1)).count("1") for m in _ancestors(_tree(n))) for n, k in zip(new, kv))
    return dict(bytes=2 * sum(kv) * c["kv_heads"] * c["dim"] * size + 4 * sum(new) * c["q_heads"] * c["dim"]
                + sum(-(-k // c["page"]) for k in kv) * 4 + 8 * sum(new), flops=4 * c["dim"] * c["q_heads"] * pairs)


def _rules(c, rand):
    """Sampling rules of every row, as requests bring them: [rows] tensors, or None where no row has one."""
    r = c["rows"]
    ones = torch.ones(r, device="cuda")
    t = 0.5 + 0.7 * rand(r)
    k = (5 + 60 * rand(r)).int()
    p = 0.8 + 0.18 * rand(r)
    m = 0.02 + 0.06 * rand(r)
    if c["rules"] == "none":
        return dict(temperature=t, top_k=None, top_p=None, min_p=None)
    if c["rules"] == "top_k":
        return dict(temperature=t, top_k=k, top_p=None, min_p=None)
    if c["rules"] == "top_p":
        return dict(temperature=t, top_k=None, top_p=p, min_p=None)
    if c["rules"] == "all":
        return dict(temperature=t, top_k=k, top_p=p, min_p=m)
    kind = torch.arange(r, device="cuda") % 6       # greedy; no rule; top-k; top-p; top-k and top-p; min-p
    return dict(temperature=torch.where(kind == 0, 0 * ones, t), top_k=torch.where((kind == 2) | (kind == 4), k, 0 * k),
                top_p=torch.where((kind == 3) | (kind == 4), p, ones), min_p=torch.where(kind == 5, m, 0 * ones))


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)

    s = dict(case=c)
    if c["op"] == "lora":
        t, k, widths, a, r = c["tokens"], c["k"], _widths(c), c["adapters"], c["rank"]
        wide = sum(widths)
        # the projection's input with a few large channels, and its output, as columns of a wider buffer
        x = randn(t, k)
        x[:, torch.randperm(k, generator=g, device="cuda")[:k // 100]] *= 8.0
        rows = randn(t, wide + c["pad"]).to(torch.bfloat16)
        runs = -(-t // c["runs"])
        which = torch.randint(0, a, (runs,), generator=g, device="cuda", dtype=torch.int32)
        which = torch.where(rand(runs) < 0.1, -1, which)                    # some requests have no adapter
        s.update(x=x.to(torch.bfloat16), y=rows[:, :wide], adapters=which.repeat_interleave(c["runs"])[:t].contiguous(),
                 a=(randn(a, len(widths) * r, k) * k ** -0.5).to(torch.bfloat16),
                 b=(0.3 * randn(a, wide, r)).to(torch.bfloat16), scales=0.5 + rand(a),
                 out=torch.zeros(t, wide + c["pad"], dtype=torch.bfloat16, device="cuda")[:, :wide])
    elif c["op"] == "sample":
        r, v = c["rows"], c["vocab"]
        # rows of flat and of confident distributions
        logits = (1.0 + 2.0 * rand(r, 1)) * randn(r, v)
        logits[:, :8] += 6.0 * rand(r, 1)
        logits = logits.gather(1, torch.randperm(v, generator=g, device="cuda").expand(r, v))
        s.update(logits=logits.to(torch.bfloat16) if c["type"] == "bf16" else logits,
                 noise=torch.empty(r, v, device="cuda").exponential_(generator=g).clamp_min(1e-20),
                 tokens=torch.zeros(r, dtype=torch.int32, device="cuda"), logprobs=torch.zeros(r, device="cuda"),
                 probs=torch.zeros(r, v, device="cuda") if c["probs"] else None, **_rules(c, rand))
    else:
        new, kv = _lengths(c)
        hk, d, page = c["kv_heads"], c["dim"], c["page"]
        need = [-(-k // page) for k in kv]
        pages = sum(need) + 5
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        host = torch.zeros(c["batch"], max(need) + PAGE_TABLE_SLACK, dtype=torch.int64)
        at = 0
        for b, n in enumerate(need):
            host[b, :n] = torch.arange(at, at + n)
            at += n
        inside = torch.arange(host.shape[1], device="cuda") < torch.tensor(need, device="cuda")[:, None]
        table = torch.where(inside, order[host.cuda()], torch.zeros_like(order[:1]))
        scales = c["cache"] == "e4m3"
        shape = (c.get("layers", 1), pages, page, hk, d)
        k, v = (torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        if scales:
            k, v = ((x * 16).to(torch.float8_e4m3fn) for x in (k, v))
        s.update(k_cache=k, v_cache=v, k_scale=0.06 + 0.01 * randn(hk).abs() if scales else None,
                 v_scale=0.06 + 0.01 * randn(hk).abs() if scales else None, page_table=table,
                 seq_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                 cu=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(), max_q=max(new), max_kv=max(kv))
        if c["op"] == "tree":
            sees = [m for n in new for m in _ancestors(_tree(n))]
            s.update(q=(1.5 * randn(sum(new), c["q_heads"], d)).to(torch.bfloat16),
                     sees=torch.tensor(sees, dtype=torch.int64)[:, None].cuda(),
                     out=torch.zeros(sum(new), c["q_heads"], d, dtype=torch.bfloat16, device="cuda"))
        else:
            parents, wanted = [], []
            for b, n in enumerate(new):
                path = [0] + _accepted_path(n, b)
                want = [-1] * n                              # the node that each node's draw names
                for x, y in zip(path, path[1:]):
                    want[x] = y
                parents += _tree(n)
                wanted += want
            t = sum(new)
            tokens = torch.randperm(151936, generator=g, device="cuda")[:2 * t].int()   # no token twice
            first = s["cu"][:-1].long().repeat_interleave(torch.tensor(new, device="cuda"))
            want = torch.tensor(wanted, device="cuda")
            s.update(parents=torch.tensor(parents, dtype=torch.int32).cuda(), node_tokens=tokens[:t].contiguous(),
                     sampled=torch.where(want >= 0, tokens[(first + want).clamp_min(0)], tokens[t:]).contiguous(),
                     out_tokens=torch.zeros(c["batch"], DEPTH + 1, dtype=torch.int32, device="cuda"),
                     accepted=torch.zeros(c["batch"], dtype=torch.int32, device="cuda"),
                     new_lens=torch.zeros(c["batch"], dtype=torch.int32, device="cuda"))
    if own:
        import quantized_gemm_decode_amd as ql
        if c["op"] == "lora":
            s["stack"] = ql.LoraStack(s["a"], s["b"], s["scales"], _widths(c))
            s["workspace"] = ql.lora_workspace(s["stack"], c["tokens"])
        elif c["op"] == "sample":
            s["workspace"] = ql.sample_workspace(c["rows"], c["vocab"])
        else:
            s["caches"] = [ql.PagedCache(k, v, s["k_scale"], s["v_scale"]) for k, v in zip(s["k_cache"], s["v_cache"])]
        if c["op"] == "tree":
            s["plan"] = ql.qlinear_tree_attention_plan(s["caches"][0], c["q_heads"], c["batch"], s["q"].shape[0],
                                                       s["max_q"], s["max_kv"])
            s["workspace"] = s["plan"].new_workspace()
    return s


DEPTH = 8       # most tokens that a commit accepts


def _plain_lora(s):
    c = s["case"]
    a, r, widths = c["adapters"], c["rank"], _widths(c)
    h = torch.matmul(s["x"].float(), s["a"].float().view(-1, c["k"]).T).view(-1, a, len(widths), r)
    mine = s["adapters"][:, None] == torch.arange(a, device="cuda")
    h = h * (mine * s["scales"])[:, :, None, None]                          # adapters other than a token's own: 0
    parts, n = [], 0
    for j, w in enumerate(widths):
        b = s["b"][:, n:n + w].float().transpose(1, 2).reshape(a * r, w)
        parts.append(torch.matmul(h[:, :, j].reshape(-1, a * r), b))
        n += w
    s["out"].copy_(s["y"].float() + torch.cat(parts, 1))
    return s["out"]


def _plain_sample(s):
    c = s["case"]
    rows, v = c["rows"], c["vocab"]
    value, index = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    rank = torch.arange(v, device="cuda")
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    # 64 bits: whether an entry is kept depends on sums over the whole row
    w = torch.exp((value - value[:, :1]).double() / torch.where(greedy, torch.ones_like(t), t))
    keep = torch.ones(rows, v, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        mass = torch.where(keep, w, torch.zeros_like(w)).cumsum(1)
        keep &= (mass - w < p * mass[:, -1:]) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep = torch.where(greedy, rank == 0, keep | (rank == 0))
    w = torch.where(keep, w, torch.zeros_like(w))
    at = (w.float() / s["noise"].gather(1, index)).argmax(1, keepdim=True)
    w = w / w.sum(1, keepdim=True)
    s["tokens"].copy_(index.gather(1, at)[:, 0])
    s["logprobs"].copy_(w.gather(1, at)[:, 0].log())
    if s["probs"] is None:
        return s["tokens"], s["logprobs"]
    s["probs"].scatter_(1, index, w.float())
    return s["tokens"], s["logprobs"], s["probs"]


def _gather(cache, table, scale, length):
    """The cached rows of every sequence as [batch, kv heads, length, dim] in 32 bits."""
    e4m3 = cache.dtype == torch.float8_e4m3fn
    x = (cache.view(torch.uint8) if e4m3 else cache)[table.long()]
    x = (x.view(torch.float8_e4m3fn) if e4m3 else x).flatten(1, 2)[:, :length].float()
    return (x if scale is None else x * scale[:, None]).transpose(1, 2)


def _plain_tree(s):
    c = s["case"]
    b, hq, hk, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    n, length, dev = s["max_q"], s["max_kv"], s["q"].device
    width = -(-length // c["page"])
    k = _gather(s["k_cache"][0], s["page_table"][:, :width], s["k_scale"], length)
    v = _gather(s["v_cache"][0], s["page_table"][:, :width], s["v_scale"], length)
    cu, kv = s["cu"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, hq // hk * n, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    node = torch.arange(length, device=dev) - (kv - new)[:, None]           # of each key: its node, < 0 in the context
    bits = s["sees"][:, 0][rows][:, :, None] >> node.clamp(0, 63)[:, None] & 1
    sees = (node < 0)[:, None] | (bits == 1) & (node < new[:, None])[:, None]
    scores = scores.view(b, hk, hq // hk, n, length).masked_fill(~sees[:, None, None], float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, hq // hk * n, length), v)
    o = o.view(b, hk, hq // hk, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, hq, d)
    keep = (i < new[:, None]).reshape(-1).nonzero()[:, 0]                   # the nodes in their order
    s["out"].copy_(o[keep])
    return s["out"]


def _plain_commit(s):
    c = s["case"]
    cu, kv = s["cu"].long(), s["seq_lens"].long()
    new, n = cu[1:] - cu[:-1], s["max_q"]
    i = torch.arange(n, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=s["parents"].shape[0] - 1)
    parents, tokens, sampled = s["parents"].long()[at], s["node_tokens"][at], s["sampled"][at]
    there = i < new[:, None]
    node, alive = torch.zeros_like(new), torch.ones_like(new, dtype=torch.bool)
    path, out = [], []
    for _ in range(DEPTH):      # one node further down the tree
        draw = sampled.gather(1, node[:, None])
        hit = (parents == node[:, None]) & (tokens == draw) & there & alive[:, None]
        out.append(torch.where(alive, draw[:, 0], -1))
        alive = hit.any(1)
        node = torch.where(alive, hit.int().argmax(1), node)
        path.append(torch.where(alive, node, -1))
    out.append(torch.where(alive, sampled.gather(1, node[:, None])[:, 0], -1))
    path = torch.stack(path, 1)
    accepted = (path >= 0).sum(1)
    s["out_tokens"].copy_(torch.stack(out, 1))
    s["accepted"].copy_(accepted)
    s["new_lens"].copy_(kv - new + 1 + accepted)
    first = (kv - new)[:, None]
    depth = torch.arange(1, DEPTH + 1, device="cuda").expand_as(path)
    src, dst = first + path.clamp_min(0), first + torch.where(path >= 0, depth, 0)     # what is not accepted: 0 to 0
    src, dst = (s["page_table"].long().gather(1, x // c["page"]) * c["page"] + x % c["page"] for x in (src, dst))
    for cache in (s["k_cache"], s["v_cache"]):
        x = cache.view(torch.uint8) if c["cache"] == "e4m3" else cache
        x = x.view(c["layers"], -1, c["kv_heads"], c["dim"])
        x[:, dst.flatten()] = x[:, src.flatten()]
    return s["out_tokens"], s["accepted"], s["new_lens"], s["k_cache"], s["v_cache"]


def _own(s):
    import quantized_gemm_decode_amd as ql
    c = s["case"]
    if c["op"] == "lora":
        ql.qlinear_lora(s["stack"], s["x"], s["y"], s["adapters"], s["workspace"], out=s["out"])
        return s["out"]
    if c["op"] == "sample":
        ql.qlinear_sample(s["logits"], s["noise"], s["tokens"], s["workspace"], temperature=s["temperature"],
                          top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], logprobs=s["logprobs"],
                          probs=s["probs"])
        return (s["tokens"], s["logprobs"]) if s["probs"] is None else (s["tokens"], s["logprobs"], s["probs"])
    if c["op"] == "tree":
        ql.qlinear_tree_attention(s["plan"], s["q"], s["caches"][0], s["page_table"], s["seq_lens"], s["cu"], s["sees"],
                                  s["out"], workspace=s["workspace"])
        return s["out"]
    ql.qlinear_tree_commit(s["caches"], s["page_table"], s["seq_lens"], s["cu"], s["node_tokens"], s["parents"],
                           s["sampled"], s["out_tokens"], s["accepted"], s["new_lens"])
    return s["out_tokens"], s["accepted"], s["new_lens"], s["k_cache"], s["v_cache"]


PLAIN = dict(lora=_plain_lora, sample=_plain_sample, tree=_plain_tree, commit=_plain_commit)


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_lora(s):
    c = s["case"]
    r, y = c["rank"], s["y"].double()
    for i in range(c["adapters"]):
        mine = (s["adapters"] == i).nonzero()[:, 0]
        if mine.numel() == 0:
            continue
        x, n = s["x"][mine].double(), 0
        for j, w in enumerate(_widths(c)):
            down = s["a"][i, j * r:(j + 1) * r].double()
            up = s["b"][i, n:n + w].double()
            y[mine, n:n + w] += s["scales"][i].double() * ((x @ down.T.contiguous()) @ up.T.contiguous())
            n += w
    return y


def _exact_sample(s):
    c = s["case"]
    tokens, logs, probs = [], [], torch.zeros(c["rows"], c["vocab"], dtype=torch.float64)
    for i in range(c["rows"]):
        row = s["logits"][i].double().cpu()
        t = float(s["temperature"][i])
        order = torch.argsort(row, descending=True, stable=True)
        if t <= 0:
            order = order[:1]
            t = 1.0
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            order = order[:int(s["top_k"][i])]
        p = torch.softmax(row[order] / t, 0)
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            before = p.cumsum(0) - p
            n = max(1, int((before < float(s["top_p"][i])).sum()))
            order, p = order[:n], p[:n]
        if s["min_p"] is not None:
            n = max(1, int((p >= float(s["min_p"][i]) * p[0]).sum()))
            order, p = order[:n], p[:n]
        p = p / p.sum()
        probs[i, order] = p
        score = p / s["noise"][i].cpu().double()[order]
        tokens.append(int(order[score == score.max()].min()))
        logs.append(float(probs[i, tokens[-1]].log()))
    tokens, logs = torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)
    return (tokens, logs, probs) if c["probs"] else (tokens, logs)


def _exact_tree(s):
    c = s["case"]
    g, hk, d = c["q_heads"] // c["kv_heads"], c["kv_heads"], c["dim"]
    new, kv = _lengths(c)
    out, first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, length) in enumerate(zip(new, kv)):
        at = torch.arange(length, device="cuda")
        page, slot = s["page_table"][b].long()[at // c["page"]], at % c["page"]
        hidden = torch.zeros(n, length, dtype=torch.bool)
        parents = _tree(n)
        for i in range(n):
            above, j = set(), i
            while j >= 0:
                above.add(j)
                j = parents[j]
            hidden[i, length - n:] = torch.tensor([j not in above for j in range(n)])
        hidden = hidden.cuda()
        for h in range(hk):
            ks, vs = ((x[0].view(torch.uint8)[page, slot, h].view(x.dtype) if x.dtype == torch.float8_e4m3fn
                       else x[0][page, slot, h]).double() for x in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                ks, vs = ks * s["k_scale"][h].double(), vs * s["v_scale"][h].double()
            q = s["q"][first:first + n, h * g:(h + 1) * g].double().transpose(0, 1)
            a = (q @ ks.T.contiguous() / d ** 0.5).masked_fill(hidden, float("-inf")).softmax(-1)
            out[first:first + n, h * g:(h + 1) * g] = (a @ vs).transpose(0, 1)
        first += n
    return out


def _exact_commit(s):
    c = s["case"]
    new, kv = _lengths(c)
    tokens, counts, lens = torch.full((c["batch"], DEPTH + 1), -1, dtype=torch.int32), [], []
    names, parents, draws, table = (s[x].tolist() for x in ("node_tokens", "parents", "sampled", "page_table"))
    src, dst, first = [], [], 0
    for b, (n, length) in enumerate(zip(new, kv)):
        node, base, depth = 0, length - n, 0
        while True:
            tokens[b, depth] = draws[first + node]
            below = [i for i in range(n) if parents[first + i] == node and names[first + i] == draws[first + node]]
            if not below or depth == DEPTH:
                break
            node, depth = below[0], depth + 1
            src.append(table[b][(base + node) // c["page"]] * c["page"] + (base + node) % c["page"])
            dst.append(table[b][(base + depth) // c["page"]] * c["page"] + (base + depth) % c["page"])
        counts.append(depth)
        lens.append(base + 1 + depth)
        first += n
    caches = []
    for cache in (s["k_cache"], s["v_cache"]):
        x = cache.clone()
        flat = x.view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16).view(c["layers"], -1, c["kv_heads"], c["dim"])
        old = flat.clone()
        for i, j in zip(src, dst):
            flat[:, j] = old[:, i]
        caches.append(x)
    return (tokens, torch.tensor(counts, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32), *caches)


def exact(c, seed):
    s = prepare(c, seed)
    return dict(lora=_exact_lora, sample=_exact_sample, tree=_exact_tree, commit=_exact_commit)[c["op"]](s)
