"""Serving a small model with speculative decoding: the quantized linears and
the operators between them, as a server would call them.

    python examples/speculative_serving.py [--batch 8] [--prompt 600] [--tokens 64] [--drafts 4]

The model is one attention layer between an embedding and a head, with random
weights (and likely successors) in FP8_Dynamic:

    x   = embedding[token]
    qkv = QKV(x)                                            quantized linear
    q, cache = norm + rotation of q and k; k, v -> cache    qlinear_qkv_append
    a   = attention(q, cache)                               qlinear_attention
    y   = x + O(a);  logits = head(y)                       quantized linears
    tokens = drafts accepted against softmax(logits)        qlinear_verify_draft

The prompts of all sequences go in as batches of chunks.  Each later step feeds a
sequence's newest token and its drafts (a draft is what followed the newest
token's last occurrence), appends all of them, and keeps as many as the target
accepts; what the cache holds of rejected ones lies beyond the sequence's
length and is written over by the next step.  Steps have one shape, so they are
captured once and replayed.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_decode_amd as ql  # noqa: E402

BF16 = torch.bfloat16


class Linear:
    """A quantized weight with a plan and buffers per token count."""

    def __init__(self, w):
        self.N, self.K = w.shape
        codes, self.scale = ql.quantize_weight(ql.FP8_DYNAMIC, w)
        self.packed = ql.pack_weight(codes)
        self.calls = {}

    def __call__(self, x):
        M = x.shape[0]
        if M not in self.calls:
            plan = ql.qlinear_plan_layouts(ql.FP8_DYNAMIC, M, self.N, self.K, 1, 2)
            self.calls[M] = (plan, ql.act_buffer(plan), ql.act_scale_buffer(plan), plan.new_workspace())
        plan, codes, scales, workspace = self.calls[M]
        y = torch.empty(M, self.N, dtype=BF16, device=x.device)
        ql.qlinear_forward(plan, x, codes, scales, self.packed, self.scale, y, workspace)
        return y


class Model:
    def __init__(self, q_heads=32, kv_heads=8, head_dim=128, vocab=32000, max_pos=16384, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(BF16)
        self.q_heads, self.kv_heads, self.head_dim, self.vocab = q_heads, kv_heads, head_dim, vocab
        hidden = q_heads * head_dim
        self.embedding = randn(vocab, hidden, scale=1.0)
        self.weights = dict(qkv=randn((q_heads + 2 * kv_heads) * head_dim, hidden, scale=hidden ** -0.5),
                            o=randn(hidden, hidden, scale=2 * hidden ** -0.5),
                            head=randn(vocab, hidden, scale=hidden ** -0.5))
        # likely successors, in cycles of 16 tokens: a text that drafts can foresee
        token = torch.arange(vocab, device=device)
        before = torch.where(token % 16 == 0, (token + 15).clamp(max=vocab - 1), token - 1)
        self.weights["head"] += 12 / hidden * self.embedding[before]
        self.qkv, self.o, self.head = (Linear(self.weights[n]) for n in ("qkv", "o", "head"))
        self.q_norm, self.k_norm = randn(head_dim, scale=0.1) + 1, randn(head_dim, scale=0.1) + 1
        self.cos_sin = ql.rope_table(max_pos, head_dim, device=device)

    def forward(self, batch, logits=True):
        """Logits of the batch's tokens (None if not asked for); their keys and
        values go into the cache."""
        H, Hk, D = self.q_heads, self.kv_heads, self.head_dim
        x = self.embedding[batch.tokens]
        heads = self.qkv(x).view(-1, H + 2 * Hk, D)
        q, k, v = heads[:, :H], heads[:, H:H + Hk], heads[:, H + Hk:]
        ql.qlinear_qkv_append(q, k, v, batch.positions, batch.slots, self.cos_sin, q, batch.cache, self.q_norm, self.k_norm)
        a = torch.empty(len(x), H, D, dtype=BF16, device=x.device)
        ql.qlinear_attention(batch.plan, q, batch.cache, batch.page_table, batch.seq_lens, batch.cu_q, a,
                             workspace=batch.workspace)
        y = x + self.o(a.view(len(x), H * D))
        return self.head(y) if logits else None


class Batch:
    """One step's device arrays: new[b] new tokens of sequence b."""

    def __init__(self, model, cache, page_table, new, max_kv):
        self.cache, self.page_table, self.new = cache, page_table, new
        n, dev = sum(new), page_table.device
        self.tokens, self.positions, self.slots = (torch.zeros(n, dtype=torch.int64, device=dev) for _ in range(3))
        self.seq_lens = torch.zeros(len(new), dtype=torch.int32, device=dev)
        self.cu_q = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
        self.plan = ql.qlinear_attention_plan(cache, model.q_heads, len(new), n, max(new), max_kv)
        self.workspace = self.plan.new_workspace(dev)
        self.row_seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
        self.row_at = torch.cat([torch.arange(m) for m in new])

    def set(self, tokens, lengths):
        """`tokens` (all sequences', in order) follow `lengths` tokens of each sequence."""
        lengths = torch.tensor(lengths)
        pos = lengths[self.row_seq] + self.row_at
        size = self.cache.page_size
        self.tokens.copy_(torch.as_tensor(tokens))
        self.positions.copy_(pos)
        self.slots.copy_(self.page_table.cpu()[self.row_seq, pos // size].long() * size + pos % size)
        self.seq_lens.copy_(lengths + torch.tensor(self.new))


class Server:
    """Fixed sequences, `drafts` drafted tokens a step, room for new_tokens each."""

    def __init__(self, model, prompts, drafts, new_tokens, page_size=64, e4m3=True, temperature=1.0, seed=0):
        B, dev = len(prompts), model.embedding.device
        self.model, self.drafts, self.temperature = model, drafts, temperature
        self.text = [list(p) for p in prompts]
        self.max_kv = max_kv = max(len(p) for p in prompts) + new_tokens + 2 * drafts + 2
        columns = -(-max_kv // page_size)
        dtype = torch.float8_e4m3fn if e4m3 else BF16
        shape = (B * columns + 1, page_size, model.kv_heads, model.head_dim)
        self.cache = ql.PagedCache(torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev))
        order = torch.randperm(B * columns, generator=torch.Generator().manual_seed(seed))
        self.page_table = order.view(B, columns).int().to(dev)
        self.batch = Batch(model, self.cache, self.page_table, [drafts + 1] * B, max_kv)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.draft_tokens = torch.zeros(B * drafts, dtype=torch.int32, device=dev)
        self.cu_drafts = torch.arange(B + 1, dtype=torch.int32, device=dev) * drafts
        self.uniforms = torch.zeros(B * drafts, device=dev)
        self.noise = torch.ones(B, model.vocab, device=dev)
        self.out_tokens = torch.zeros(B, drafts + 1, dtype=torch.int32, device=dev)
        self.accepted = torch.zeros(B, dtype=torch.int32, device=dev)
        self.scratch = ql.verify_workspace(B, model.vocab, dev)
        self.graph = None

    def _probs(self, logits):
        return torch.softmax(logits.float() / self.temperature, dim=-1)

    def prefill(self, tokens=8192, logits=False):
        """The prompts' tokens but the last, which the first step feeds, in
        chunks of at most about `tokens`; returns their logits if asked for."""
        B, todo, out = len(self.text), [len(t) - 1 for t in self.text], []
        share = max(1, tokens // B)
        for at in range(0, max(todo), share):
            new = [min(max(n - at, 0), share) for n in todo]
            done = [min(at, n) for n in todo]
            batch = Batch(self.model, self.cache, self.page_table, new, min(at + share, max(todo)))
            batch.set([t for text, d, n in zip(self.text, done, new) for t in text[d:d + n]], done)
            out.append(self.model.forward(batch, logits))
        return out

    def _draft(self, text):
        """What followed the newest token's last occurrence, as often as needed."""
        last = max((i for i in range(len(text) - 1) if text[i] == text[-1]), default=-1)
        after = text[last + 1:]
        return [after[i % len(after)] for i in range(self.drafts)]

    def _run(self):
        self.logits = self.model.forward(self.batch)
        ql.qlinear_verify_draft(self._probs(self.logits), None, self.draft_tokens, self.cu_drafts, self.uniforms,
                                self.noise, self.out_tokens, self.accepted, self.scratch)

    def step(self, capture=True):
        """One step of every sequence; returns the accepted drafts of each."""
        if max(map(len, self.text)) + self.drafts > self.max_kv:
            raise ValueError("a sequence has no room for another step")
        drafts = [self._draft(t) for t in self.text]
        self.batch.set([t for text, d in zip(self.text, drafts) for t in text[-1:] + d], [len(t) - 1 for t in self.text])
        self.draft_tokens.copy_(torch.tensor(drafts, dtype=torch.int32).view(-1))
        self.uniforms.uniform_(generator=self.gen)
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
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.7)
    args = ap.parse_args()
    ql.load_default_table()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(model.vocab, (max(2, args.prompt - 7 * b),), generator=g).tolist() for b in range(args.batch)]
    server = Server(model, prompts, args.drafts, args.tokens, temperature=args.temperature)
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
