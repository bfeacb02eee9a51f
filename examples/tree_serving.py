"""Serving many requests, each with its own adapter and sampling rules, from trees
of drafted tokens.

    python examples/tree_serving.py [--batch 8] [--prompt 600] [--tokens 64] [--branches 3] [--depth 4]

The model is that of speculative_serving.py, with low-rank adapters beside its
query, key and value projection:

    x   = embedding[token]
    qkv = QKV(x) + adapter of the request (x)               quantized linear, qlinear_lora
    q, cache = norm + rotation of q and k; k, v -> cache    qlinear_qkv_append
    a   = attention(q, cache), each node its own branch     qlinear_tree_attention
    y   = x + O(a);  logits = head(y)                       quantized linears
    token at every node, by the request's rules             qlinear_sample
    the branch that the drawn tokens follow stays           qlinear_tree_commit

Each step feeds a sequence's newest token and branches of drafts below it (what
followed the newest token's last occurrences).  The tokens drawn down the tree are
given out as far as drafts follow them; the accepted drafts' keys and values move
together behind the context, where the next step goes on.  Steps have one shape,
so they are captured once and replayed.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import quantized_gemm_decode_amd as ql  # noqa: E402
import speculative_serving as base  # noqa: E402

BF16 = torch.bfloat16


class Model(base.Model):
    def __init__(self, adapters=16, rank=16, seed=0, device="cuda", **sizes):
        super().__init__(seed=seed, device=device, **sizes)
        g = torch.Generator(device=device).manual_seed(seed + 1)
        D, hidden = self.head_dim, self.q_heads * self.head_dim
        widths = [hidden, self.kv_heads * D, self.kv_heads * D]
        a = torch.randn(adapters, 3 * rank, hidden, generator=g, device=device) * hidden ** -0.5
        b = torch.randn(adapters, sum(widths), rank, generator=g, device=device) * rank ** -0.5
        scales = 0.5 + 0.5 * torch.rand(adapters, generator=g, device=device)
        self.adapters = ql.LoraStack(a.to(BF16), b.to(BF16), scales, widths)

    def forward(self, batch, logits=True):
        """As the base's, with each token's adapter (batch.adapters)."""
        H, Hk, D = self.q_heads, self.kv_heads, self.head_dim
        x = self.embedding[batch.tokens]
        y = self.qkv(x)
        ql.qlinear_lora(self.adapters, x, y, batch.adapters, batch.lora)
        heads = y.view(-1, H + 2 * Hk, D)
        q, k, v = heads[:, :H], heads[:, H:H + Hk], heads[:, H + Hk:]
        ql.qlinear_qkv_append(q, k, v, batch.positions, batch.slots, self.cos_sin, q, batch.cache, self.q_norm, self.k_norm)
        a = torch.empty(len(x), H, D, dtype=BF16, device=x.device)
        batch.attend(q, a)
        y = x + self.o(a.view(len(x), H * D))
        return self.head(y) if logits else None


class Chunk(base.Batch):
    """Chunks of prompts: new[b] tokens of sequence b, whose adapter is adapter[b]."""

    def __init__(self, model, cache, page_table, new, max_kv, adapter):
        super().__init__(model, cache, page_table, new, max_kv)
        self.adapters = torch.tensor(adapter, dtype=torch.int32)[self.row_seq].to(page_table.device)
        self.lora = ql.lora_workspace(model.adapters, sum(new), page_table.device)

    def attend(self, q, out):
        ql.qlinear_attention(self.plan, q, self.cache, self.page_table, self.seq_lens, self.cu_q, out, workspace=self.workspace)


class Trees(Chunk):
    """One step: a tree of the same shape for every sequence (parents, -1 the root's)."""

    def __init__(self, model, cache, page_table, parents, max_kv, adapter):
        n, batch, dev = len(parents), len(adapter), page_table.device
        super().__init__(model, cache, page_table, [n] * batch, max_kv, adapter)
        depth, sees = [0] * n, [1] * n
        for i, p in enumerate(parents[1:], 1):
            depth[i], sees[i] = depth[p] + 1, sees[p] | 1 << i
        words = -(-n // 64)
        bits = [[(m >> 64 * w & (1 << 64) - 1) - (m >> 64 * w + 63 & 1) * (1 << 64) for w in range(words)] for m in sees]
        self.sees = torch.tensor(bits * batch, dtype=torch.int64, device=dev)
        self.parents = torch.tensor(parents * batch, dtype=torch.int32, device=dev)
        self.depth = torch.tensor(depth * batch)
        self.node_tokens = torch.zeros(n * batch, dtype=torch.int32, device=dev)
        self.plan = ql.qlinear_tree_attention_plan(cache, model.q_heads, batch, n * batch, n, max_kv)
        self.workspace = self.plan.new_workspace(dev)

    def attend(self, q, out):
        ql.qlinear_tree_attention(self.plan, q, self.cache, self.page_table, self.seq_lens, self.cu_q, self.sees, out,
                                  workspace=self.workspace)

    def set(self, tokens, lengths):
        """Nodes lie one after the other behind the context and are rotated at their depths."""
        super().set(tokens, lengths)
        self.positions.copy_(torch.tensor(lengths)[self.row_seq] + self.depth)
        self.node_tokens.copy_(self.tokens)


class Server:
    """Fixed sequences with an adapter and rules each; trees of `branches` chains of `depth` drafts."""

    def __init__(self, model, prompts, adapter, rules, branches, depth, new_tokens, page_size=64, e4m3=True, seed=0):
        B, dev = len(prompts), model.embedding.device
        self.model, self.adapter, self.branches, self.depth = model, list(adapter), branches, depth
        self.text = [list(p) for p in prompts]
        parents = [-1] + [0 if d == 0 else b * depth + d for b in range(branches) for d in range(depth)]
        self.nodes = n = len(parents)
        self.max_kv = max_kv = max(len(p) for p in prompts) + new_tokens + n + depth
        columns = -(-max_kv // page_size)
        dtype = torch.float8_e4m3fn if e4m3 else BF16
        shape = (B * columns + 1, page_size, model.kv_heads, model.head_dim)
        self.cache = ql.PagedCache(torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev))
        order = torch.randperm(B * columns, generator=torch.Generator().manual_seed(seed))
        self.page_table = order.view(B, columns).int().to(dev)
        self.trees = Trees(model, self.cache, self.page_table, parents, max_kv, self.adapter)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.noise = torch.ones(B * n, model.vocab, device=dev)
        kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
        off = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
        self.rules = {k: torch.tensor([r.get(k, off[k]) for r in rules for _ in range(n)], dtype=t, device=dev)
                      for k, t in kinds.items()}
        self.sampled = torch.zeros(B * n, dtype=torch.int32, device=dev)
        self.logprobs = torch.zeros(B * n, device=dev)
        self.scratch = ql.sample_workspace(B * n, model.vocab, dev)
        self.out_tokens = torch.zeros(B, depth + 1, dtype=torch.int32, device=dev)
        self.accepted, self.new_lens = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2))
        self.graph = None

    def prefill(self, tokens=8192):
        """The prompts' tokens but the last, which the first step feeds."""
        todo = [len(t) - 1 for t in self.text]
        share = max(1, tokens // len(todo))
        for at in range(0, max(todo), share):
            new = [min(max(n - at, 0), share) for n in todo]
            done = [min(at, n) for n in todo]
            chunk = Chunk(self.model, self.cache, self.page_table, new, min(at + share, max(todo)), self.adapter)
            chunk.set([t for text, d, n in zip(self.text, done, new) for t in text[d:d + n]], done)
            self.model.forward(chunk, logits=False)

    def _draft(self, text):
        """What followed the newest token's last occurrences, one branch each."""
        found = [i for i in range(len(text) - 1) if text[i] == text[-1]][-self.branches:][::-1]
        out = []
        for b in range(self.branches):
            after = text[(found[b] if b < len(found) else len(text) - 2 - b) + 1:]
            out += [after[i % len(after)] for i in range(self.depth)]
        return out

    def _run(self):
        self.logits = self.model.forward(self.trees)
        ql.qlinear_sample(self.logits, self.noise, self.sampled, self.scratch, logprobs=self.logprobs, **self.rules)
        ql.qlinear_tree_commit([self.cache], self.page_table, self.trees.seq_lens, self.trees.cu_q, self.trees.node_tokens,
                               self.trees.parents, self.sampled, self.out_tokens, self.accepted, self.new_lens, self.max_kv)

    def step(self, capture=True):
        """One step of every sequence; returns the accepted drafts of each."""
        if max(map(len, self.text)) - 1 + self.nodes > self.max_kv:
            raise ValueError("a sequence has no room for another step")
        nodes = [t for text in self.text for t in text[-1:] + self._draft(text)]
        self.trees.set(nodes, [len(t) - 1 for t in self.text])
        self.noise.exponential_(generator=self.gen)
        if capture and self.graph is None:
            side = torch.cuda.Stream()                  # plans, buffers and workspaces exist before the capture
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._run()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._run()
        if capture:
            self.graph.replay()
        else:
            self._run()
        accepted = self.accepted.tolist()
        for text, n, out in zip(self.text, accepted, self.out_tokens.tolist()):
            text += out[:n + 1]
        return accepted


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--branches", type=int, default=3)
    ap.add_argument("--depth", type=int, default=4)
    args = ap.parse_args()
    ql.load_default_table()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(model.vocab, (max(2, args.prompt - 7 * b),), generator=g).tolist() for b in range(args.batch)]
    rules = [(dict(temperature=0.0), dict(temperature=0.7, top_p=0.9), dict(top_k=40), dict(temperature=1.2, min_p=0.05))[b % 4]
             for b in range(args.batch)]
    server = Server(model, prompts, [b % 17 - 1 for b in range(args.batch)], rules, args.branches, args.depth, args.tokens)
    server.prefill()
    steps = kept = 0
    while max(len(t) - len(p) for t, p in zip(server.text, prompts)) < args.tokens:
        kept += sum(server.step())
        steps += 1
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        server.graph.replay()
    end.record()
    end.synchronize()
    print("%d steps of %d sequences: %d tokens, %.2f accepted drafts a step and sequence; %.0f us a step on the device"
          % (steps, args.batch, sum(map(len, server.text)) - sum(map(len, prompts)), kept / steps / args.batch,
             begin.elapsed_time(end) * 1e3 / 20))


if __name__ == "__main__":
    main()
