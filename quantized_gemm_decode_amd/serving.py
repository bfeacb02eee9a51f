"""The serving operators around the linears (C ABI section "Serving operators"
of ``include/qlinear.h``): norm and rotation of the query and key heads, append
to a paged cache, attention over it, verification of drafted tokens.

Tensors keep torch's shapes and strides: heads are ``[tokens, heads,
head_dim]`` views (the query columns of a QKV projection's output as they
stand), caches ``[pages, page_size, kv_heads, head_dim]`` in any order of the
first three.  Only the last dimension has to be contiguous.
"""

import ctypes

import torch

from . import _lib
from ._lib import QLAttentionFacts, QLAttentionShape, QLKvCache, QLNormRope, QLRows

KV_BF16, KV_E4M3 = 0, 1
KV_DTYPES = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3}


def _lib_check(status, where):
    if status != 0:
        from . import QLinearError
        raise QLinearError(status, where)


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _flat(t, name, dtype, numel):
    """Address of a contiguous tensor of at least numel elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.numel() < numel:
        raise ValueError("%s holds %d elements; this call needs at least %d" % (name, t.numel(), numel))
    return t.data_ptr()


def _rows(t, name, heads_dim=None):
    """ql_rows of a bf16 [tokens, heads, head_dim] tensor with contiguous heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise ValueError("%s has dtype %s, expected torch.bfloat16" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 3 or (heads_dim is not None and tuple(shape) != heads_dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(shape), heads_dim or "[tokens, heads, head_dim]"))
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise ValueError("%s must have contiguous heads" % name)
    return QLRows(t.data_ptr(), st[0], st[1])


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
        self.ref = ctypes.byref(self.struct)

    def _check_device(self):
        if not self.k.is_cuda:
            raise ValueError("the cache must be on the GPU")


def _rule(table, q_weight, k_weight, head_dim, eps, interleaved):
    rot, max_pos, at = 0, 0, None
    if table is not None:
        if table.dim() != 2:
            raise ValueError("cos_sin must be a [max_pos, rot_dim] tensor")
        max_pos, rot = table.shape
        at = _flat(table, "cos_sin", torch.float32, 0)
    return QLNormRope(None if q_weight is None else _flat(q_weight, "q_weight", torch.bfloat16, head_dim),
                      None if k_weight is None else _flat(k_weight, "k_weight", torch.bfloat16, head_dim),
                      at, max_pos, rot, bool(interleaved), eps)


def rope_table(max_pos, rot_dim, base=1e4, device="cuda"):
    """cos_sin [max_pos, rot_dim] (binary32): cosines, then sines, of pos * base^(-2i / rot_dim)."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * i / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def qlinear_qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6,
                         interleaved=False, stream=None):
    """q_out, k_out = per-head norm (weights given) and rotation (cos_sin
    given) of q and k; outputs may be the inputs."""
    tokens, q_heads, dim = q.shape
    kv_heads = k.shape[1]
    rq, ro = _rows(q, "q"), _rows(q_out, "q_out", (tokens, q_heads, dim))
    rk, rp = _rows(k, "k", (tokens, kv_heads, dim)), _rows(k_out, "k_out", (tokens, kv_heads, dim))
    rule = _rule(cos_sin, q_weight, k_weight, dim, eps, interleaved)
    byref = ctypes.byref
    _lib_check(_lib.load().qlinear_qk_norm_rope(
        byref(rule), tokens, q_heads, kv_heads, dim, byref(rq), byref(rk),
        _flat(positions, "positions", torch.int64, tokens), byref(ro), byref(rp), _stream(stream, q.device)),
        "qlinear_qk_norm_rope")


def qlinear_qkv_append(q, k, v, positions, slots, cos_sin, q_out, cache, q_weight=None, k_weight=None, eps=1e-6,
                       interleaved=False, stream=None):
    """Norm and rotation of q into q_out (both may be None) and of k into the
    cache, v into the cache as it is, at slots (page * page_size + place)."""
    tokens, dim = k.shape[0], cache.head_dim
    cache._check_device()
    rk = _rows(k, "k", (tokens, cache.kv_heads, dim))
    rv = _rows(v, "v", (tokens, cache.kv_heads, dim))
    q_heads, rq, ro = 0, None, None
    byref = ctypes.byref
    if q is not None:
        q_heads = q.shape[1]
        rq = byref(_rows(q, "q", (tokens, q_heads, dim)))
        ro = byref(_rows(q_out, "q_out", (tokens, q_heads, dim)))
    rule = _rule(cos_sin, q_weight, k_weight, dim, eps, interleaved)
    _lib_check(_lib.load().qlinear_qkv_append(
        byref(rule), tokens, q_heads, rq, byref(rk), byref(rv), _flat(positions, "positions", torch.int64, tokens),
        _flat(slots, "slots", torch.int64, tokens), ro, cache.ref, _stream(stream, k.device)), "qlinear_qkv_append")


class AttentionPlan:
    """Owner of a ql_attention_plan handle (host object)."""

    def __init__(self, shape):
        self.shape = shape
        h = ctypes.c_void_p()
        _lib_check(_lib.load().qlinear_attention_plan(ctypes.byref(shape), ctypes.byref(h)), "qlinear_attention_plan")
        self.handle = h
        self.workspace_bytes = int(_lib.load().qlinear_attention_workspace_bytes(h))
        self._q = (shape.tokens, shape.q_heads, shape.head_dim)
        self._columns = -(-shape.max_kv // shape.page_size)

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
                                          cache.page_size, cache.kv_type, bool(causal), window, scale or 0.0))


def qlinear_attention(plan, q, cache, page_table, seq_lens, cu_q, out, lse=None, workspace=None, stream=None):
    """out = attention of the new tokens q over the cache (see qlinear.h);
    page_table int32 [batch, columns], seq_lens int32 [batch], cu_q int32 [batch + 1]."""
    s = plan.shape
    cache._check_device()
    rq, ro = _rows(q, "q", plan._q), _rows(out, "out", plan._q)
    if page_table.dim() != 2 or page_table.shape[0] < s.batch or page_table.shape[1] < plan._columns:
        raise ValueError("page_table has shape %s; this plan needs at least (%d, %d)"
                         % (tuple(page_table.shape), s.batch, plan._columns))
    if workspace is None:
        if plan.workspace_bytes:
            raise ValueError("this plan needs a workspace")
        at = None
    else:
        at = _flat(workspace, "workspace", torch.uint8, plan.workspace_bytes)
    _lib_check(_lib.load().qlinear_attention(
        plan.handle, ctypes.byref(rq), cache.ref, _flat(page_table, "page_table", torch.int32, 0), page_table.shape[1],
        _flat(seq_lens, "seq_lens", torch.int32, s.batch), _flat(cu_q, "cu_q", torch.int32, s.batch + 1),
        ctypes.byref(ro), None if lse is None else _flat(lse, "lse", torch.float32, s.tokens * s.q_heads), at,
        _stream(stream, q.device)), "qlinear_attention")


def qlinear_verify_workspace_bytes(batch, vocab):
    return int(_lib.load().qlinear_verify_workspace_bytes(batch, vocab))


def verify_workspace(batch, vocab, device="cuda"):
    """Device memory for qlinear_verify_draft (any contents)."""
    return torch.empty(max(16, qlinear_verify_workspace_bytes(batch, vocab)), dtype=torch.uint8, device=device)


def qlinear_verify_draft(target_probs, draft_probs, draft_tokens, cu_drafts, uniforms, noise, out_tokens, accepted,
                         workspace, stream=None):
    """Accept drafted tokens against the target's probabilities and draw the
    next token (see qlinear.h); out_tokens int32 [batch, max_drafts + 1]."""
    n_drafts = draft_tokens.shape[0]
    batch, vocab = noise.shape
    columns = out_tokens.shape[1]
    f32, i32 = torch.float32, torch.int32
    _lib_check(_lib.load().qlinear_verify_draft(
        batch, n_drafts, columns - 1, vocab, _flat(target_probs, "target_probs", f32, (n_drafts + batch) * vocab),
        None if draft_probs is None else _flat(draft_probs, "draft_probs", f32, n_drafts * vocab),
        _flat(draft_tokens, "draft_tokens", i32, n_drafts), _flat(cu_drafts, "cu_drafts", i32, batch + 1),
        _flat(uniforms, "uniforms", f32, n_drafts), _flat(noise, "noise", f32, batch * vocab),
        _flat(out_tokens, "out_tokens", i32, batch * columns), _flat(accepted, "accepted", i32, batch),
        _flat(workspace, "workspace", torch.uint8, qlinear_verify_workspace_bytes(batch, vocab)),
        _stream(stream, noise.device)), "qlinear_verify_draft")
