"""Trees of drafts over contexts of more than 2^27 keys: every row is written.

All pages of the context are one page of the cache, so a row that sees the
context alone has the softmax over that page's keys.  Tolerance (u = 2^-24): of
the sum of weights times |v|, 2^-8 for the weights and as much of the result for
its rounding, as for other chunks; a sum's parts are added one after the other, 8
keys each at least, in shares of the keys that the cut makes: u twice for each; scores' errors as there.
"""

import numpy as np
import pytest
import torch

import quantized_gemm_decode_amd as ql
from tests.gpu_util import requires_gpu
from tests.test_gpu_serving import f64

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("nodes,hq,pages,shares", [(64, 24, 16384, 32), (70, 8, 128, 32)])
def test_every_row_of_a_long_context(nodes, hq, pages, shares):
    """64 nodes of 24 heads over 134 million keys need fewer than 768 workgroups; a shorter context beside it."""
    page, D = 8192, 64
    g = torch.Generator().manual_seed(nodes)
    k, v = ((4 * torch.randn(2, page, 1, D, generator=g)).to(torch.float8_e4m3fn).cuda() for _ in range(2))
    cache = ql.PagedCache(k, v)
    q = (0.1 * torch.randn(nodes, hq, D, generator=g)).to(torch.bfloat16).cuda()
    length = pages * page + nodes
    table = torch.zeros(1, pages + 1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([length], [0, nodes]))
    sees = torch.zeros(nodes, -(-nodes // 64), dtype=torch.int64, device="cuda")
    out = torch.full((nodes, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nodes, hq), 9.0, device="cuda")
    plan = ql.qlinear_tree_attention_plan(cache, hq, 1, nodes, nodes, length)
    ql.qlinear_tree_attention(plan, q, cache, table, lens, cu, sees, out, lse, plan.new_workspace())
    torch.cuda.synchronize()
    kk, vv, s = f64(k)[0, :, 0], f64(v)[0, :, 0], D ** -0.5
    x = s * np.einsum("thd,kd->thk", f64(q), kk)
    top = x.max(-1, keepdims=True)
    e = np.exp(x - top)
    total = e.sum(-1, keepdims=True)
    want, weight = (e / total) @ vv, (e / total) @ np.abs(vv)
    u, adds = 2.0 ** -24, length / shares / 8
    reach = (np.einsum("thd,kd->thk", np.abs(f64(q)), np.abs(kk)) * s).max(-1)
    d = 2 * D * u * reach + 8 * u * (reach + 1)         # of a score
    tol = weight * (2.0 ** -8 + 2 * d[..., None] + 2 * adds * u) + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(want)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (int((err > tol).sum()), np.argwhere(err > tol)[:4].tolist())
    want_lse = (top + np.log(total * pages))[..., 0]
    assert (np.abs(f64(lse) - want_lse) <= d + 2 * adds * u + 4 * u * np.abs(want_lse) + 4 * u).all()
