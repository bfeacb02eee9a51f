"""The oracle of the request operators against definitions written another way."""

import numpy as np

import oracle.requests as ref
from oracle import serving


def test_lora_is_a_merged_weight():
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(4, 12)), rng.normal(size=(4, 10))
    a, b = rng.normal(size=(3, 4, 12)), rng.normal(size=(3, 10, 2))
    out, _, _ = ref.lora(x, y, [2, -1, 0, 3], a, b, np.array([1.0, 2.0, 3.0]), [6, 4])
    for t, i in ((0, 2), (2, 0)):
        w = np.concatenate([b[i, :6] @ a[i, :2], b[i, 6:] @ a[i, 2:]]) * (1, 2, 3)[i]
        assert np.allclose(out[t], y[t] + w @ x[t], rtol=1e-12, atol=1e-12)
    assert (out[[1, 3]] == y[[1, 3]]).all()


def test_sampling_rules():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    e = np.ones(5)

    def kept(**kw):
        return np.flatnonzero(ref.sample(l, e, **kw)[1]).tolist()

    assert kept() == [0, 1, 2, 3, 4] and kept(top_k=2) == [1, 2] and kept(top_k=4) == [0, 1, 2, 3]
    assert kept(top_p=0.39) == [1] and kept(top_p=0.5) == [1, 2] and kept(top_p=0.7) == [1, 2, 3]
    assert kept(top_k=2, top_p=0.67) == [1, 2] and kept(top_k=2, top_p=0.66) == [1]     # of the first two's mass
    assert kept(min_p=0.45) == [1, 2, 3] and kept(min_p=0.55) == [1] and kept(min_p=7.0) == [1]
    assert kept(temperature=0.0) == [1] and kept(temperature=0.5, min_p=0.45) == [1]
    s, p = ref.sample(l, np.array([1.0, 9.0, 1.0, 1.0, 1.0]), top_k=3)
    assert int(s.argmax()) == 2 and np.allclose(p, [0, 0.5, 0.25, 0.25, 0])
    assert not ref.sample([-np.inf, np.nan], e[:2])[1].any()
    assert ref.sample([np.inf, 1.0, np.inf], e[:3])[1].tolist() == [0.5, 0.0, 0.5]


def test_tree_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(3, 4, 2, 8)), rng.normal(size=(3, 4, 2, 8))
    table, lens, cu = np.array([[2, 0], [1, 0]]), [7, 4], [0, 3, 5]
    sees = np.array([[1], [3], [7], [1], [3]], np.uint64)
    got = ref.tree_attention(q, k, v, table, lens, cu, sees, 4, 0.3)
    want = serving.attention(q, k, v, table, lens, cu, 4, 0.3)
    for x in ("out", "lse", "weight"):
        assert np.allclose(got[x], want[x])


def test_commit_walk():
    #        0 -> 1 -> 3, 0 -> 2 -> 4 -> 5
    parents, tokens = [-1, 0, 0, 1, 2, 4], [9, 5, 6, 7, 8, 3]
    out, n, lens, moves = ref.tree_commit(tokens, parents, [6, 0, 8, 0, 1, 2], [0, 6], [20], 4)
    assert out.tolist() == [[6, 8, 1, -1, -1]] and n.tolist() == [2] and lens.tolist() == [17]
    assert moves == [[(16, 15), (18, 16)]]
    out, n, _, _ = ref.tree_commit(tokens, parents, [6, 0, 8, 0, 3, 2], [0, 6], [20], 1)
    assert out.tolist() == [[6, 8]] and n.tolist() == [1]
