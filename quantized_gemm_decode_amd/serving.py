"""The serving operators around the linears (C ABI section "Serving operators"
of ``include/qlinear.h``): norm and rotation of the query and key heads, append
to a paged cache, attention over it (for trees of drafted tokens too),
verification of drafted tokens and commit of a tree's branch, low-rank adapters
beside a projection, sampling.

Tensors keep torch's shapes and strides: heads are ``[tokens, heads,
head_dim]`` views (the query columns of a QKV projection's output as they
stand), caches ``[pages, page_size, kv_heads, head_dim]`` in any order of the
first three.  Only the last dimension has to be contiguous.
"""

import ctypes
import importlib.util
import os

import torch

from . import _lib
from ._lib import QLAttentionFacts, QLAttentionShape, QLKvCache, QLLora

KV_BF16, KV_E4M3 = 0, 1
KV_DTYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3}


def _lib_check(status, where):
    if status != 0:
        from . import QLinearError
        raise QLinearError(status, where)


_module = None


def _binding():
    """The compiled binding (built with the library; there is no other path)."""
    global _module
    if _module is None:
        path = os.path.join(_lib.PKG, "_binding.so")
        if not os.path.exists(path):
            raise OSError("_binding.so is not built (%s); run python -m quantized_gemm_decode_amd.build" % path)
        _lib.load()
        spec = importlib.util.spec_from_file_location("quantized_gemm_decode_amd._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _module = module
    return _module


def _stream(stream):
    """None stays None: the current stream of the call's device."""
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


class PagedCache:
    """Keys and values of many sequences in pages of page_size tokens.

    k, v: [pages, page_size, kv_heads, head_dim], bf16 or float8_e4m3fn, any
    strides with a contiguous last dimension; k_scale, v_scale: binary32
    [kv_heads] for E4M3 (value = code * scale), None = 1.  The tensors stay the
    caller's; the object keeps them alive.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise ValueError("cache %s must be a [pages, page_size, kv_heads, head_dim] tensor" % name)
            if t.dtype not in KV_DTYPES:
                raise ValueError("cache %s has dtype %s, expected bfloat16 or float8_e4m3fn" % (name, t.dtype))
            if t.stride(3) != 1:
                raise ValueError("cache %s must have contiguous heads" % name)
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("cache k and v differ in shape, dtype or device")
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if s is not None and (s.dtype != torch.float32 or not s.is_contiguous() or s.numel() != k.shape[2]
                                  or s.device != k.device):
                raise ValueError("%s must be a contiguous float32 [kv_heads] tensor on the cache's device" % name)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_type = KV_DTYPES[k.dtype]
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        ptr = [None if t is None else t.data_ptr() for t in (k, v, k_scale, v_scale)]
        self.struct = QLKvCache(*ptr, *k.stride()[:3], *v.stride()[:3], self.num_pages, self.kv_type, self.page_size,
                                self.kv_heads, self.head_dim)
        self.address = ctypes.addressof(self.struct)
        self.on_gpu, self.device_index = k.is_cuda, k.get_device()


def rope_table(max_pos, rot_dim, base=1e4, device="cuda"):
    """cos_sin [max_pos, rot_dim] (binary32): cosines, then sines, of pos * base^(-2i / rot_dim)."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * i / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def qlinear_qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, stream=None):
    """q_out, k_out = per-head norm (weights given) and rotation (cos_sin
    given) of q and k; outputs may be the inputs."""
    st = (_module or _binding()).qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight, eps, interleaved,
                                              _stream(stream))
    if st:
        _lib_check(st, "qlinear_qk_norm_rope")


def qlinear_qkv_append(q, k, v, positions, slots, cos_sin, q_out, cache, q_weight=None, k_weight=None, eps=1e-6,
                       interleaved=False, stream=None):
    """Norm and rotation of q into q_out (both may be None) and of k into the
    cache, v into the cache as it is, at slots (page * page_size + place)."""
    if not cache.on_gpu:
        raise ValueError("the cache must be on the GPU")
    st = (_module or _binding()).qkv_append(q, k, v, positions, slots, cos_sin, q_out, cache.address, cache.device_index,
                                            q_weight, k_weight, eps, interleaved, _stream(stream))
    if st:
        _lib_check(st, "qlinear_qkv_append")


class AttentionPlan:
    """Owner of a ql_attention_plan handle (host object)."""

    _make = "qlinear_attention_plan"

    def __init__(self, shape):
        self.shape = shape
        h = ctypes.c_void_p()
        _lib_check(getattr(_lib.load(), self._make)(ctypes.byref(shape), ctypes.byref(h)), self._make)
        self.handle = h
        self.workspace_bytes = int(_lib.load().qlinear_attention_workspace_bytes(h))
        # what a call is checked against, in the binding's order
        self._args = (h.value, shape.batch, shape.tokens, shape.q_heads, shape.head_dim,
                      -(-shape.max_kv // shape.page_size), self.workspace_bytes)

    def __del__(self):
        h = getattr(self, "handle", None)
        try:
            if h is not None and h.value and _lib._lib is not None:
                _lib._lib.qlinear_attention_plan_destroy(h)
        except Exception:       # interpreter shutdown: module globals may be gone
            pass
        self.handle = None

    @property
    def facts(self):
        f = QLAttentionFacts()
        _lib_check(_lib.load().qlinear_attention_plan_info(self.handle, ctypes.byref(f)), "qlinear_attention_plan_info")
        return {n: getattr(f, n) for n, _ in QLAttentionFacts._fields_}

    def new_workspace(self, device="cuda"):
        """Device memory for the partial results (any contents), None if none is needed."""
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device) if self.workspace_bytes else None


def qlinear_attention_plan(cache, q_heads, batch, tokens, max_q, max_kv, causal=True, window=0, scale=None):
    """Plan for `tokens` new tokens of `batch` sequences, at most max_q of one
    sequence, over contexts of at most max_kv tokens (the new ones included)."""
    return AttentionPlan(QLAttentionShape(batch, tokens, max_q, max_kv, q_heads, cache.kv_heads, cache.head_dim,
                                          cache.page_size, cache.kv_type, bool(causal),
                                          max(-1, min(window, 2 ** 31 - 1)), scale or 0.0))


def qlinear_attention(plan, q, cache, page_table, seq_lens, cu_q, out, lse=None, workspace=None, stream=None):
    """out = attention of the new tokens q over the cache (see qlinear.h);
    page_table int32 [batch, columns], seq_lens int32 [batch], cu_q int32 [batch + 1]."""
    if not cache.on_gpu:
        raise ValueError("the cache must be on the GPU")
    st = (_module or _binding()).attention(*plan._args, q, cache.address, cache.device_index, page_table, seq_lens, cu_q, out,
                                           lse, workspace, _stream(stream))
    if st:
        _lib_check(st, "qlinear_attention")


class TreeAttentionPlan(AttentionPlan):
    """The same for trees of drafted tokens."""

    _make = "qlinear_tree_attention_plan"

    def __init__(self, shape):
        super().__init__(shape)
        self._words = -(-min(shape.max_q, shape.tokens) // 64)


def qlinear_tree_attention_plan(cache, q_heads, batch, tokens, max_q, max_kv, scale=None):
    """Plan for trees of drafted tokens: `tokens` nodes of `batch` sequences, at
    most max_q of one, over contexts of at most max_kv tokens (the nodes included)."""
    return TreeAttentionPlan(QLAttentionShape(batch, tokens, max_q, max_kv, q_heads, cache.kv_heads, cache.head_dim,
                                              cache.page_size, cache.kv_type, True, 0, scale or 0.0))


def qlinear_tree_attention(plan, q, cache, page_table, seq_lens, cu_q, sees, out, lse=None, workspace=None, stream=None):
    """qlinear_attention for the nodes of trees: sees int64 [tokens, words], the
    new tokens of its sequence that each node sees, one a bit (see qlinear.h)."""
    if not isinstance(plan, TreeAttentionPlan):
        raise ValueError("the plan is not for trees")
    if not cache.on_gpu:
        raise ValueError("the cache must be on the GPU")
    st = (_module or _binding()).tree_attention(*plan._args, q, cache.address, cache.device_index, page_table, seq_lens, cu_q,
                                                out, lse, workspace, _stream(stream), sees, plan._words)
    if st:
        _lib_check(st, "qlinear_tree_attention")


def qlinear_tree_commit(caches, page_table, seq_lens, cu_q, node_tokens, parents, sampled, out_tokens, accepted,
                        new_lens=None, max_kv=None, stream=None):
    """Follow the drawn tokens down each sequence's tree, give them out and move
    the accepted nodes' keys and values behind the context in every cache of the
    list (see qlinear.h); out_tokens int32 [batch, max_depth + 1].  max_kv: bound
    of the cached lengths, None: what the page table's columns hold."""
    st = (_module or _binding()).tree_commit(caches, page_table, max_kv, seq_lens, cu_q, node_tokens, parents, sampled,
                                             out_tokens, accepted, new_lens, _stream(stream))
    if st:
        _lib_check(st, "qlinear_tree_commit")


def qlinear_verify_workspace_bytes(batch, vocab):
    return int(_lib.load().qlinear_verify_workspace_bytes(batch, vocab))


def verify_workspace(batch, vocab, device="cuda"):
    """Device memory for qlinear_verify_draft (any contents), with up to that many sequences and entries."""
    return torch.empty(max(16, qlinear_verify_workspace_bytes(batch, vocab)), dtype=torch.uint8, device=device)


def qlinear_verify_draft(target_probs, draft_probs, draft_tokens, cu_drafts, uniforms, noise, out_tokens, accepted,
                         workspace, stream=None):
    """Accept drafted tokens against the target's probabilities and draw the
    next token (see qlinear.h); out_tokens int32 [batch, max_drafts + 1]."""
    st = (_module or _binding()).verify_draft(target_probs, draft_probs, draft_tokens, cu_drafts, uniforms, noise,
                                              out_tokens, accepted, workspace, _stream(stream))
    if st:
        _lib_check(st, "qlinear_verify_draft")


class LoraStack:
    """Low-rank adapters of one projection.

    a: [adapters, slices * rank, in_features], b: [adapters, out_features,
    rank], bf16 with contiguous adapters (views of a pool of all layers may
    have any stride between adapters); scales: binary32 [adapters] or None = 1;
    widths: the columns of each slice of a merged projection (query, key and
    value; gate and up), None: one slice.  The tensors stay the owner's.
    """

    def __init__(self, a, b, scales=None, widths=None):
        for t, name in ((a, "a"), (b, "b")):
            if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype != torch.bfloat16:
                raise ValueError("%s must be a bfloat16 tensor of three dimensions" % name)
            if t.numel() and not t[0].is_contiguous():
                raise ValueError("%s must have contiguous adapters" % name)
        widths = [b.shape[1]] if widths is None else [int(w) for w in widths]
        if not 1 <= len(widths) <= 4 or sum(widths) != b.shape[1]:
            raise ValueError("widths must be 1 to 4 numbers that add up to b's %d rows" % b.shape[1])
        if a.shape[0] != b.shape[0] or a.shape[1] != len(widths) * b.shape[2] or a.device != b.device:
            raise ValueError("a and b differ in adapters, rank or device")
        if scales is not None and (scales.dtype != torch.float32 or not scales.is_contiguous()
                                   or scales.numel() != a.shape[0] or scales.device != a.device):
            raise ValueError("scales must be a contiguous float32 [adapters] tensor on a's device")
        self.a, self.b, self.scales, self.widths = a, b, scales, widths
        self.struct = QLLora(a.data_ptr(), b.data_ptr(), None if scales is None else scales.data_ptr(), a.stride(0),
                             b.stride(0), a.shape[2], (ctypes.c_int64 * 4)(*widths), a.shape[0], b.shape[2], len(widths))
        self.address = ctypes.addressof(self.struct)
        self.on_gpu, self.device_index, self.out_features = a.is_cuda, a.get_device(), b.shape[1]


def qlinear_lora_workspace_bytes(stack, tokens):
    return int(_lib.load().qlinear_lora_workspace_bytes(ctypes.byref(stack.struct), tokens))


def lora_workspace(stack, tokens, device="cuda"):
    """Device memory for qlinear_lora with up to `tokens` tokens (any contents)."""
    return torch.empty(max(16, qlinear_lora_workspace_bytes(stack, tokens)), dtype=torch.uint8, device=device)


def qlinear_lora(stack, x, y, adapters, workspace, out=None, stream=None):
    """out (None: y itself) = y + scale B A x of each token's adapter (int32
    [tokens]; outside the stack, as -1: y as it is)."""
    if not stack.on_gpu:
        raise ValueError("the stack must be on the GPU")
    st = (_module or _binding()).lora(stack.address, stack.device_index, stack.out_features, x, y, adapters, out, workspace,
                                      _stream(stream))
    if st:
        _lib_check(st, "qlinear_lora")


def qlinear_sample_workspace_bytes(rows, vocab):
    return int(_lib.load().qlinear_sample_workspace_bytes(rows, vocab))


def sample_workspace(rows, vocab, device="cuda"):
    """Device memory for qlinear_sample (any contents), with up to that many rows and entries."""
    return torch.empty(max(16, qlinear_sample_workspace_bytes(rows, vocab)), dtype=torch.uint8, device=device)


def qlinear_sample(logits, noise, tokens, workspace, temperature=None, top_k=None, top_p=None, min_p=None, logprobs=None,
                   probs=None, stream=None):
    """tokens (int32 [rows]) drawn from logits (float32 or bfloat16 [rows,
    vocab]) with exponential noise under each row's rules (see qlinear.h);
    logprobs and probs of the kept entries where given."""
    st = (_module or _binding()).sample(logits, noise, tokens, workspace, temperature, top_k, top_p, min_p, logprobs, probs,
                                        _stream(stream))
    if st:
        _lib_check(st, "qlinear_sample")
