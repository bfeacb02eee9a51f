"""Pins of the serving oracle: closed forms and independent restatements on
small inputs (CPU)."""

import numpy as np
import pytest
import torch

from oracle import serving as ref


def test_rotation_is_a_rotation_and_norm_gives_unit_mean_square():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    ang = rng.uniform(0, 6, (10, 32))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([0, 9, 4])
    for inter in (False, True):
        y, size = ref.norm_rope(x, None, pos, table, 64, inter, 0.0)
        a = np.arange(32) * 2 if inter else np.arange(32)
        b = a + 1 if inter else a + 32
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang[pos])[:, None]
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
        assert np.allclose(size[..., a], np.abs(x[..., a]) + np.abs(x[..., b]))
    y, _ = ref.norm_rope(x, np.ones(64), pos, table, 64, False, 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    y, _ = ref.norm_rope(x, None, np.array([0, 10, -1]), table, 64, False, 0.0)
    assert np.isfinite(y[0]).all() and np.isnan(y[1:]).all()
    y, _ = ref.norm_rope(x, None, pos, table[:, :16], 16, False, 0.0)
    assert np.array_equal(y[..., 16:], x[..., 16:])


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_attention_against_torch_softmax(causal, window):
    """The paged loops against one dense softmax over the gathered sequence."""
    rng = np.random.default_rng(1)
    H, hk, D, page, L, n = 4, 2, 8, 16, 21, 6
    k, v = rng.standard_normal((2, 4, page, hk, D))
    table, q = np.array([[2, 0, 9]]), rng.standard_normal((n, H, D))
    r = ref.attention(q, k, v, table, [L], np.array([0, n]), page, 0.3, causal, window)
    kk, vv = (torch.from_numpy(np.concatenate([x[2], x[0]])[:L]) for x in (k, v))
    i, j = torch.arange(L - n, L)[:, None], torch.arange(L)
    hide = torch.zeros(n, L, dtype=torch.bool)
    if causal:
        hide |= j > i
    if window:
        hide |= j <= i - window
    for h in range(H):
        s = (torch.from_numpy(q[:, h]) @ kk[:, h // 2].T * 0.3).masked_fill(hide, float("-inf"))
        assert np.allclose(r["out"][:, h], (s.softmax(-1) @ vv[:, h // 2]).numpy())
        assert np.allclose(r["lse"][:, h], torch.logsumexp(s, -1).numpy())


def test_attention_rows_that_see_nothing():
    k = np.zeros((1, 16, 1, 4))
    r = ref.attention(np.ones((3, 1, 4)), k, k, np.array([[0]]), [1], np.array([0, 3]), 16, 1.0)
    assert (r["out"][:2] == 0).all() and np.isneginf(r["lse"][:2, 0]).all() and np.isfinite(r["lse"][2, 0])


def test_verify_accepts_and_draws_by_hand():
    f = np.float32
    target = np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7], [0.3, 0.3, 0.4]], f)
    draft = np.array([[0.5, 0.5, 0.0], [0.6, 0.4, 0.0]], f)
    one = np.ones((1, 3), f)
    args = (np.array([0, 2], np.int32),)
    # both accepted: the last row decides
    out, acc = ref.verify(target, draft, np.array([0, 1]), *args, np.array([0.9, 0.4], f), one, 2)
    assert acc.tolist() == [2] and out.tolist() == [[0, 1, 2]]
    # the second rejected (0.6 * 0.4 >= 0.2): p - q = (-, -, 0.7)
    out, acc = ref.verify(target, draft, np.array([0, 1]), *args, np.array([0.9, 0.6], f), one, 2)
    assert acc.tolist() == [1] and out.tolist() == [[0, 2, -1]]
    # the first rejected, certain drafts: p without the drafted token, ties to the lowest index
    out, acc = ref.verify(target, None, np.array([0, 1]), *args, np.array([0.9, 0.6], f), one, 2)
    assert acc.tolist() == [0] and out.tolist() == [[1, -1, -1]]
    # noise reorders the draw
    out, _ = ref.verify(target, None, np.array([0, 1]), *args, np.array([0.9, 0.6], f), np.array([[1, 1, 0.5]], f), 2)
    assert out.tolist() == [[2, -1, -1]]
