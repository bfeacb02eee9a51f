"""Host checks of the operators of a server of many requests (CPU: no kernel is
launched): refused arguments and their status codes, sizes, the binding's
checks."""

import ctypes

import pytest
import torch

import quantized_gemm_decode_amd as ql
from quantized_gemm_decode_amd._lib import QLLora, QLSampling
from tests.test_serving_host import A, ALIGN, INVALID, OK, UNSUPPORTED, cache, ref, rows, shape

NAN = float("nan")


def stack(**kw):
    d = dict(a=A, b=A, scales=None, a_adapter_stride=3 * 16 * 256, b_adapter_stride=200 * 16, in_features=256,
             widths=(ctypes.c_int64 * 4)(136, 64), adapters=4, rank=16, slices=2)
    if "widths" in kw:
        kw["widths"] = (ctypes.c_int64 * 4)(*kw["widths"])
    d.update(kw)
    return QLLora(*[d[f] for f, _ in QLLora._fields_])


def lora(s=None, tokens=5, x=A, xs=256, y=A, ys=200, ad=A, out=A + 4096, os=200, ws=A):
    return ql.lib().qlinear_lora(ref(s or stack()), tokens, x, xs, y, ys, ad, out, os, ws, None)


def test_lora_refusals():
    assert lora(tokens=0, x=None, ws=None) == OK
    assert lora(tokens=-1) == INVALID and lora(tokens=(1 << 24) + 1) == UNSUPPORTED
    assert ql.lib().qlinear_lora(None, 1, A, 256, A, 200, A, A, 200, A, None) == INVALID
    for bad, st in ((dict(adapters=-1), INVALID), (dict(adapters=65537), UNSUPPORTED), (dict(slices=0), UNSUPPORTED),
                    (dict(slices=5), UNSUPPORTED), (dict(rank=0), UNSUPPORTED), (dict(rank=12), UNSUPPORTED),
                    (dict(rank=136), UNSUPPORTED), (dict(in_features=0), UNSUPPORTED), (dict(in_features=252), UNSUPPORTED),
                    (dict(in_features=(1 << 20) + 8), UNSUPPORTED), (dict(widths=(136, 60)), UNSUPPORTED),
                    (dict(widths=(136, 0)), UNSUPPORTED), (dict(widths=(-8, 200)), UNSUPPORTED),
                    (dict(a_adapter_stride=-8), INVALID), (dict(a_adapter_stride=2 * 16 * 256 - 8), INVALID),
                    (dict(b_adapter_stride=200 * 16 - 8), INVALID), (dict(b_adapter_stride=200 * 16 + 4), ALIGN),
                    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(a=A + 8), ALIGN), (dict(b=A + 2), ALIGN),
                    (dict(scales=A + 2), ALIGN)):
        assert lora(stack(**bad)) == st, bad
        if st == UNSUPPORTED:
            assert ql.lib().qlinear_lora_workspace_bytes(ref(stack(**bad)), 5) == 0
    for k in ("x", "y", "ad", "out", "ws"):
        assert lora(**{k: None}) == INVALID, k
        assert lora(**{k: A + 2}) == ALIGN, k
    assert lora(xs=248) == INVALID and lora(ys=192) == INVALID and lora(os=-8) == INVALID and lora(xs=260) == ALIGN
    assert lora(out=A, os=208) == INVALID           # y with another stride
    assert ql.lib().qlinear_lora_workspace_bytes(None, 5) == 0
    assert ql.lib().qlinear_lora_workspace_bytes(ref(stack()), 0) == 0


def test_lora_workspace():
    """A binary32 sum of every token, rank and slice for each part of K."""
    for tokens in (1, 5, 64, 65, 4000):
        n = ql.lib().qlinear_lora_workspace_bytes(ref(stack(in_features=4096, a_adapter_stride=32 * 4096)), tokens)
        assert n > 0 and n % (tokens * 2 * 16 * 4) == 0 and n // (tokens * 2 * 16 * 4) <= 16
    # what no grid holds
    assert lora(stack(widths=(1 << 20, 1 << 20), b_adapter_stride=(1 << 21) * 16), tokens=1 << 24, ys=1 << 21,
                os=1 << 21) == UNSUPPORTED


def test_lora_binding():
    bf = torch.bfloat16
    a, b = torch.zeros(3, 32, 64, dtype=bf), torch.zeros(3, 72, 16, dtype=bf)
    s = ql.LoraStack(a, b, widths=(64, 8))
    assert (s.struct.rank, s.struct.slices, s.struct.in_features, list(s.struct.widths)[:2]) == (16, 2, 64, [64, 8])
    pool = torch.zeros(3, 5, 32, 64, dtype=bf)
    assert ql.LoraStack(pool[:, 2], b, widths=(64, 8)).struct.a_adapter_stride == 5 * 32 * 64
    for bad in (lambda: ql.LoraStack(a, b), lambda: ql.LoraStack(a, b, widths=(64, 16)), lambda: ql.LoraStack(a.float(), b),
                lambda: ql.LoraStack(a[:2], b, widths=(64, 8)), lambda: ql.LoraStack(a.transpose(1, 2), b, widths=(64, 8)),
                lambda: ql.LoraStack(a, b, torch.zeros(2), (64, 8)), lambda: ql.LoraStack(a, b, torch.zeros(3).double(), (64, 8)),
                lambda: ql.LoraStack(a, b, widths=(8,) * 9), lambda: ql.LoraStack(a[0], b[0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="GPU"):
        ql.qlinear_lora(s, a[0], a[0], None, None)


def sample(rows_=2, vocab=100, rules=None, stride=None, kind=0, logits=A, noise=A, tokens=A, logs=A, probs=A, ws=A):
    return ql.lib().qlinear_sample(rules, rows_, vocab, logits, vocab if stride is None else stride, kind, noise, tokens,
                                   logs, probs, ws, None)


def test_sample_refusals():
    assert sample(rows_=0, logits=None) == OK
    assert sample(rows_=-1) == INVALID and sample(vocab=0) == INVALID and sample(vocab=-1, stride=5) == INVALID
    assert sample(rows_=65536) == UNSUPPORTED and sample(vocab=(1 << 24) + 1) == UNSUPPORTED
    assert sample(kind=2) == INVALID and sample(stride=99) == INVALID and sample(stride=-1) == INVALID
    for k in ("logits", "noise", "tokens", "ws"):
        assert sample(**{k: None}) == INVALID, k
    for k in ("logits", "noise", "tokens", "logs", "probs", "ws"):
        assert sample(**{k: A + 2}) == ALIGN, k
    assert sample(kind=1, logits=A + 1) == ALIGN
    for i in range(4):
        assert sample(rules=ref(QLSampling(*[A + 2 if j == i else None for j in range(4)]))) == ALIGN
    assert ql.qlinear_sample_workspace_bytes(0, 100) == 0 and ql.qlinear_sample_workspace_bytes(1, 0) == 0
    for r, v in ((1, 1), (3, 2049), (64, 151936)):
        n = ql.qlinear_sample_workspace_bytes(r, v)
        assert n % 16 == 0 and n >= 8 * r * v


def test_sample_binding():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="logits must be"):
        ql.qlinear_sample(x, x, x, x)
    with pytest.raises(ValueError, match="logits must be"):
        ql.qlinear_sample(None, x, x, x)


def tree_plan(**kw):
    h = ctypes.c_void_p()
    st = ql.lib().qlinear_tree_attention_plan(ref(shape(**kw)), ref(h))
    assert bool(h.value) == (st == OK)
    return st, h


def test_tree_attention_refusals():
    assert tree_plan(causal=0)[0] == INVALID and tree_plan(window=5)[0] == INVALID
    assert tree_plan(head_dim=96)[0] == UNSUPPORTED and tree_plan(q_heads=30)[0] == INVALID
    lib = ql.lib()
    st, h = tree_plan(batch=2, tokens=200, max_q=100, max_kv=8000)

    def run(p, sees=A, words=2, table=A, ws=A, stride=1000):
        return lib.qlinear_tree_attention(p, rows(), ref(cache()), table, stride, A, A, sees, words, rows(), None, ws, None)

    assert run(None) == INVALID
    assert run(h, sees=None) == INVALID and run(h, sees=A + 4) == ALIGN and run(h, words=1) == INVALID
    assert run(h, words=-1) == INVALID and run(h, stride=499) == INVALID and run(h, ws=None) == INVALID
    # a plan of one kind serves only its own call
    other = ql.AttentionPlan(shape(batch=2, tokens=200, max_q=100, max_kv=8000))
    assert run(other.handle) == INVALID and "trees" in lib.qlinear_last_error().decode()
    assert lib.qlinear_attention(h, rows(), ref(cache()), A, 1000, A, A, rows(), None, A, None) == INVALID
    lib.qlinear_attention_plan_destroy(h)
    k = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    c = ql.PagedCache(k, k)
    with pytest.raises(ValueError, match="trees"):
        ql.qlinear_tree_attention(other, k, c, k, k, k, k, k)
    plan = ql.qlinear_tree_attention_plan(c, 32, 2, 200, 100, 8000)
    f = plan.facts
    assert f["tile_rows"] == 128 and f["stream_rows"] == 0 and plan._words == 2
    # two workgroups a compute unit, each with the binary32 outputs of 128 rows in 256 lanes, a maximum and sum for each
    # lane; where the keys were cut
    assert f["workspace_bytes"] == 512 * (128 * 128 + 2 * 256) * 4 + 16
    few = ql.qlinear_tree_attention_plan(c, 32, 2, 16, 8, 8000)
    assert few.facts["stream_rows"] == 32 and few.facts["tile_rows"] == 0
    # contexts of two tiles, or more sequences than are cut: no join
    assert ql.qlinear_tree_attention_plan(c, 32, 2, 200, 100, 128).workspace_bytes == 0
    assert ql.qlinear_tree_attention_plan(c, 32, 513, 51300, 100, 8000).workspace_bytes == 0
    wide = ql.qlinear_tree_attention_plan(c, 32, 64, 64 * 33, 33, 8000).facts       # 130 * 8 units: three times 512
    assert wide["workspace_bytes"] == 3 * 512 * (128 * 128 + 2 * 256) * 4 + 64 * 8
    with pytest.raises(ValueError, match="GPU"):
        ql.qlinear_tree_attention(plan, k, c, k, k, k, k, k)


def commit(batch=2, tokens=9, depth=4, max_kv=100, caches=None, n=1, table=A, stride=7, lens=A, cu=A, names=A, parents=A,
           sampled=A, out=A, acc=A, new=A + 64):
    return ql.lib().qlinear_tree_commit(batch, tokens, depth, max_kv, ref(caches or cache()) if n else None, n, table, stride,
                                        lens, cu, names, parents, sampled, out, acc, new, None)


def test_tree_commit_refusals():
    assert commit(batch=0) == OK
    for k in ("batch", "tokens", "depth", "max_kv", "n"):
        assert commit(**{k: -1}) == INVALID, k
    assert commit(batch=65537) == UNSUPPORTED and commit(depth=1025) == UNSUPPORTED and commit(n=4097) == UNSUPPORTED
    assert commit(tokens=(1 << 24) + 1) == UNSUPPORTED and commit(max_kv=(1 << 30) + 1) == UNSUPPORTED
    for k in ("table", "lens", "cu", "names", "parents", "sampled", "out", "acc"):
        assert commit(**{k: None}) == INVALID, k
        assert commit(**{k: A + 2}) == ALIGN, k
    assert commit(new=A + 2) == ALIGN and commit(new=A) == INVALID and commit(stride=6) == INVALID
    assert commit(caches=cache(head_dim=80)) == UNSUPPORTED and commit(caches=cache(page_size=24)) == UNSUPPORTED
    assert commit(caches=cache(k=None)) == INVALID and commit(caches=cache(v=A + 8)) == ALIGN
    two = (type(cache()) * 2)(cache(), cache(page_size=32))
    assert ql.lib().qlinear_tree_commit(2, 9, 4, 100, two, 2, A, 7, A, A, A, A, A, A, A, None, None) == INVALID
    assert "pages" in ql.lib().qlinear_last_error().decode()


def test_tree_commit_binding():
    x = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="node_tokens"):
        ql.qlinear_tree_commit([], x, x, x, x, x, x, x, x)


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structures against the C compiler's."""
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not available")
    names = dict(ql_lora=QLLora, ql_sampling=QLSampling)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "qlinear.h"\nint main(void) {\n' + "".join(
        'printf("%%d\\n", (int)sizeof(%s));\n' % n for n in names) + "return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(s) for s in names.values()]
