"""Host checks of the serving operators (CPU: no kernel is launched): refused
arguments and their status codes, plans and workspaces, the binding's checks."""

import ctypes

import pytest
import torch

import quantized_gemm_decode_amd as ql
from quantized_gemm_decode_amd import _lib
from quantized_gemm_decode_amd._lib import QLAttentionShape, QLKvCache, QLNormRope, QLRows

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 5
A = 1 << 20     # an address that no call of these tests reads
ref = ctypes.byref


def rows(data=A, token=1024, head=128):
    return ref(QLRows(data, token, head))


def cache(**kw):
    d = dict(k=A, v=A, k_scale=None, v_scale=None, k_page_stride=16384, k_token_stride=1024, k_head_stride=128,
             v_page_stride=16384, v_token_stride=1024, v_head_stride=128, num_pages=4, type=0, page_size=16, kv_heads=8,
             head_dim=128)
    d.update(kw)
    return QLKvCache(*[d[f] for f, _ in QLKvCache._fields_])


def rule(**kw):
    d = dict(q_weight=None, k_weight=None, cos_sin=A, max_pos=100, rot_dim=128, interleaved=0, eps=1e-6)
    d.update(kw)
    return QLNormRope(*[d[f] for f, _ in QLNormRope._fields_])


def norm(tokens=4, q_heads=8, kv_heads=2, dim=128, r=None, q=None, k=None, pos=A, qo=None, ko=None):
    return ql.lib().qlinear_qk_norm_rope(ref(r or rule()), tokens, q_heads, kv_heads, dim, q or rows(), k or rows(), pos,
                                         qo or rows(), ko or rows(), None)


def append(c=None, tokens=4, q_heads=8, r=None, q=None, k=None, v=None, pos=A, slots=A, qo=None):
    return ql.lib().qlinear_qkv_append(ref(r or rule()), tokens, q_heads, q or rows(), k or rows(), v or rows(), pos,
                                       slots, qo or rows(), ref(c or cache()), None)


def test_norm_rope_refusals():
    assert norm(tokens=0) == OK and norm(q_heads=0, kv_heads=0) == OK
    assert norm(tokens=-1) == INVALID and norm(q_heads=-1) == INVALID
    assert norm(tokens=(1 << 24) + 1) == UNSUPPORTED
    assert norm(dim=96) == UNSUPPORTED
    for bad in (dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=-16), dict(interleaved=2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(max_pos=-1), dict(cos_sin=None)):
        assert norm(r=rule(**bad)) == INVALID, bad
    assert norm(r=rule(q_weight=A + 8)) == ALIGN and norm(r=rule(cos_sin=A + 2)) == ALIGN
    assert norm(pos=None) == INVALID and norm(pos=A + 4) == ALIGN
    assert norm(q=rows(data=None)) == INVALID and norm(ko=rows(data=A + 8)) == ALIGN
    assert norm(q=rows(token=1028)) == ALIGN and norm(k=rows(head=-128)) == INVALID
    assert "head" in ql.lib().qlinear_last_error().decode() or "strides" in ql.lib().qlinear_last_error().decode()


def test_append_refusals():
    assert append(tokens=0) == OK
    for bad, st in ((dict(type=2), INVALID), (dict(page_size=8), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
                    (dict(page_size=16384), UNSUPPORTED), (dict(kv_heads=0), INVALID), (dict(num_pages=0), INVALID),
                    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=A + 8), ALIGN),
                    (dict(k_token_stride=1028), ALIGN), (dict(v_head_stride=-128), INVALID), (dict(k_scale=A), INVALID),
                    (dict(type=1, k_token_stride=1032), ALIGN), (dict(type=1, v_scale=A + 2), ALIGN),
                    (dict(v_token_stride=1 << 27), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED)):
        assert append(cache(**bad)) == st, bad
    assert append(slots=None) == INVALID and append(slots=A + 4) == ALIGN
    assert append(k=rows(data=None)) == INVALID and append(v=rows(token=3)) == ALIGN
    assert append(r=rule(rot_dim=24)) == INVALID


def shape(**kw):
    d = dict(batch=4, tokens=4, max_q=1, max_kv=1000, q_heads=32, kv_heads=8, head_dim=128, page_size=16, kv_type=0,
             causal=1, window=0, scale=0.0)
    d.update(kw)
    return QLAttentionShape(*[d[f] for f, _ in QLAttentionShape._fields_])


def plan_status(**kw):
    h = ctypes.c_void_p()
    st = ql.lib().qlinear_attention_plan(ref(shape(**kw)), ref(h))
    assert bool(h.value) == (st == OK)
    ql.lib().qlinear_attention_plan_destroy(h)
    return st


def test_attention_plan_refusals():
    assert plan_status() == OK and plan_status(batch=0) == OK and plan_status(max_kv=0) == OK
    for bad in (dict(batch=-1), dict(max_q=-1), dict(q_heads=30), dict(q_heads=0), dict(kv_heads=0), dict(kv_type=2),
                dict(causal=2), dict(window=-1), dict(causal=0, window=5), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(scale=-0.1)):
        assert plan_status(**bad) == INVALID, bad
    for bad in (dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=40), dict(max_kv=(1 << 30) + 1),
                dict(tokens=(1 << 24) + 1), dict(batch=65537)):
        assert plan_status(**bad) == UNSUPPORTED, bad
    assert ql.lib().qlinear_attention_plan(None, ref(ctypes.c_void_p())) == INVALID
    assert ql.lib().qlinear_attention_plan(ref(shape()), None) == INVALID


def test_attention_plan_facts():
    def facts(**kw):
        p = ql.AttentionPlan(shape(**kw))
        f = p.facts
        assert f["workspace_bytes"] == p.workspace_bytes
        return f
    one = facts(batch=1, tokens=1, max_kv=32)
    assert one["stream_rows"] == 16 and one["tile_rows"] == 0 and one["workspace_bytes"] == 0
    # up to 64 sequences of at most two tiles of 32 keys are not cut either
    assert facts(batch=64, tokens=64, max_kv=64)["workspace_bytes"] == 0
    assert facts(batch=64, tokens=64, max_kv=65)["workspace_bytes"] > 0 < facts(batch=65, tokens=65, max_kv=64)["workspace_bytes"]
    long = facts(batch=1, tokens=1, max_kv=100000)
    # two partial results a slot: outputs, maxima and sums of every row of every KV head
    assert long["workspace_bytes"] == 2 * 8 * long["slots"] * 16 * (128 + 2) * 4
    assert long == facts(batch=300, tokens=300, max_kv=5000)      # neither lengths nor batch enter
    assert facts(batch=2, tokens=10, max_q=5)["stream_rows"] == 32 and facts(batch=1, tokens=8, max_q=8)["stream_rows"] == 32
    chunk = facts(batch=1, tokens=9, max_q=9)
    assert chunk["stream_rows"] == 0 and chunk["tile_rows"] == 128 and chunk["row_blocks"] == 1
    both = facts(batch=3, tokens=200, max_q=190, max_kv=100000)    # single tokens with long contexts beside a chunk
    assert both["stream_rows"] == 16 and both["tile_rows"] == 128 and both["row_blocks"] == 6
    assert facts(batch=3, tokens=200, max_q=190)["stream_rows"] == 0           # with short ones: one launch
    cut = facts(batch=1, tokens=64, max_q=64, max_kv=100000)
    assert cut["splits"] * cut["chunk"] >= 100000 and cut["splits"] > 4
    near = facts(batch=1, tokens=64, max_q=64, max_kv=100000, window=500)      # a window bounds a unit's keys
    assert near["splits"] * near["chunk"] < 1000
    assert facts(batch=0)["row_blocks"] == 0


def run(plan, c=None, q=None, table=A, stride=1000, lens=A, cu=A, out=None, lse=None, ws=A):
    return ql.lib().qlinear_attention(plan, q or rows(), ref(c or cache()), table, stride, lens, cu, out or rows(), lse, ws,
                                      None)


def test_attention_refusals():
    p = ql.AttentionPlan(shape(max_kv=8000, batch=2))
    h = p.handle
    assert run(None) == INVALID
    assert run(h, cache(kv_heads=4)) == INVALID and run(h, cache(page_size=32)) == INVALID
    assert run(h, cache(type=1)) == INVALID and run(h, cache(head_dim=64)) == INVALID
    assert run(h, q=rows(data=None)) == INVALID and run(h, out=rows(data=A + 4)) == ALIGN
    assert run(h, table=None) == INVALID and run(h, lens=None) == INVALID and run(h, cu=A + 2) == ALIGN
    assert run(h, stride=499) == INVALID
    assert p.workspace_bytes > 0 and run(h, ws=None) == INVALID and run(h, ws=A + 8) == ALIGN
    empty = ql.AttentionPlan(shape(batch=0))
    assert run(empty.handle, q=rows(data=None), table=None, ws=None) == OK


def verify(batch=2, n=6, most=3, vocab=100, **kw):
    d = dict(target=A, draft=A, tokens=A, cu=A, u=A, noise=A, out=A, acc=A, ws=A)
    d.update(kw)
    return ql.lib().qlinear_verify_draft(batch, n, most, vocab, *[d[k] for k in d], None)


def test_verify_refusals():
    assert verify(batch=0) == OK
    assert verify(batch=-1) == INVALID and verify(vocab=0) == INVALID and verify(vocab=-1) == INVALID
    assert verify(batch=65536) == UNSUPPORTED and verify(vocab=(1 << 30) + 1) == UNSUPPORTED
    for k in ("target", "tokens", "cu", "u", "noise", "out", "acc", "ws"):
        assert verify(**{k: None}) == INVALID, k
        assert verify(**{k: A + 2}) == ALIGN, k
    assert ql.qlinear_verify_workspace_bytes(2, 0) == 0
    assert ql.qlinear_verify_workspace_bytes(1, 150000) % 16 == 0


def test_binding_refuses_what_it_can_see():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for bad in (lambda: ql.PagedCache(k, k.half()), lambda: ql.PagedCache(k[0], k[0]),
                lambda: ql.PagedCache(k, k[:2]), lambda: ql.PagedCache(k.transpose(2, 3), k.transpose(2, 3)),
                lambda: ql.PagedCache(k, k, torch.zeros(3)), lambda: ql.PagedCache(k.float(), k.float())):
        with pytest.raises(ValueError):
            bad()
    c = ql.PagedCache(k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), k)
    assert (c.struct.k_head_stride, c.struct.k_token_stride) == (16 * 64, 64)
    with pytest.raises(ValueError, match="GPU"):
        ql.qlinear_qkv_append(None, k[0], k[0], None, None, None, None, c)
    with pytest.raises(ValueError, match="q must be"):
        ql.qlinear_qk_norm_rope(k[0], k[0], None, None, k[0], k[0])
    assert set(f for f, _ in QLRows._fields_) == {"data", "token_stride", "head_stride"}


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structures against the C compiler's."""
    import shutil
    import subprocess
    import os
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not available")
    names = dict(ql_rows=QLRows, ql_kv_cache=QLKvCache, ql_norm_rope=QLNormRope, ql_attention_shape=QLAttentionShape,
                 ql_attention_facts=_lib.QLAttentionFacts)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "qlinear.h"\nint main(void) {\n' + "".join(
        'printf("%%d\\n", (int)sizeof(%s));\n' % n for n in names) + "return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(s) for s in names.values()]


def test_attention_workspace_follows_the_rows_there_are():
    """Partial results are kept for rows that exist: a binary32 output, maximum
    and sum for each chunk, whatever the longest sequence's bound is."""
    def facts(**kw):
        return ql.AttentionPlan(shape(**kw)).facts
    for kw in (dict(batch=32, tokens=2079, max_q=2048, max_kv=32768), dict(batch=16, tokens=2367, max_q=2048, max_kv=32768),
               dict(batch=256, tokens=8447, max_q=8192, max_kv=65536), dict(batch=1, tokens=64, max_q=64, max_kv=32768)):
        f = facts(**kw)
        decode = 2 * 8 * f["slots"] * 16 * (128 + 2) * 4 if f["stream_rows"] else 0
        tile = kw["tokens"] * 32 * f["splits"] * (128 + 2) * 4 if f["splits"] > 1 else 0
        assert f["workspace_bytes"] == decode + tile, kw
    # a bound of more new tokens than the call has tokens is that many
    assert facts(batch=1, tokens=64, max_q=8192, max_kv=32768) == facts(batch=1, tokens=64, max_q=64, max_kv=32768)
    assert facts(batch=1, tokens=5, max_q=100)["tile_rows"] == 0


def test_attention_plans_that_no_grid_holds_are_refused():
    """2^24 workgroups of 256 threads are 2^32 threads, one more than a launch takes."""
    most = dict(tokens=1 << 18, max_q=128, max_kv=64, q_heads=4096, kv_heads=4096)
    assert plan_status(batch=4095, **most) == OK
    assert plan_status(batch=4096, **most) == UNSUPPORTED
    assert "workgroups" in ql.lib().qlinear_last_error().decode()


def test_verify_workspace_of_tiny_vocabularies():
    """Every row has a slice, however many sequences there are and short the row is."""
    for batch in (1, 1024, 1025, 65535):
        for vocab in (1, 3, 4, 1023):
            assert ql.qlinear_verify_workspace_bytes(batch, vocab) >= 8 * batch, (batch, vocab)


def test_attention_plan_of_wide_groups_in_mixed_batches():
    """A token of more query heads a KV head than the decode share takes rows has
    nothing to do there: no launch and no workspace for it."""
    mixed = dict(batch=32, tokens=231, max_q=200, max_kv=80000)
    wide = ql.AttentionPlan(shape(q_heads=32, kv_heads=1, **mixed)).facts
    assert wide["stream_rows"] == 0 and wide["slots"] == 0 and wide["tile_rows"] == 128
    assert ql.AttentionPlan(shape(q_heads=16, kv_heads=1, **mixed)).facts["stream_rows"] == 16
