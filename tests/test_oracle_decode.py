"""Pins of the decode-step oracle: hand-worked values, closed forms and invariants (CPU only)."""

import numpy as np
import pytest
import torch

import oracle
from tests import decode_cases as dc


def test_w4_weight_by_hand():
    # k: 0..3 in bytes 0x91 (k0 = 1, k1 = 9) and 0xf0 (k2 = 0, k3 = 15); one group of 4
    codes = np.array([[0x91, 0xf0]], dtype=np.uint8)
    w = oracle.w4_weight(codes, np.array([[2.0]]))
    assert np.array_equal(w, [[2 * (1 - 8), 2 * (9 - 8), 2 * (0 - 8), 2 * (15 - 8)]])
    w = oracle.w4_weight(codes, np.array([[2.0]]), np.array([[9]], dtype=np.uint8))
    assert np.array_equal(w, [[-16, 0, -18, 12]])
    # two groups of 2, each its own scale and zero point
    w = oracle.w4_weight(codes, np.array([[1.0, 10.0]]), np.array([[0, 15]], dtype=np.uint8))
    assert np.array_equal(w, [[1, 9, -150, 0]])


def test_linear_w4_by_hand():
    codes = np.array([[0x91, 0xf0], [0x88, 0x88]], dtype=np.uint8)
    y = oracle.linear_w4(np.array([[1.0, 2.0, 3.0, 4.0]]), codes, np.array([[1.0], [5.0]]))
    assert np.array_equal(y, [[-7 + 2 - 24 + 28, 0]])


def test_rope_by_hand():
    # a quarter turn of pair 0, a half turn of pair 1; the fifth element passes
    x, cos, sin = np.array([1.0, 2, 3, 4, 5]), [0.0, -1.0], [1.0, 0.0]
    assert np.array_equal(oracle.rope_head(x, cos, sin), [-3, -2, 1, -4, 5])
    assert np.array_equal(oracle.rope_head(x, cos, sin, interleaved=True), [-2, 1, -3, -4, 5])
    # the norm: mean square 4, weights 1, 2
    u = oracle.rope_head(np.array([2.0, -2.0]), [1.0], [0.0], w=np.array([1.0, 2.0]), eps=0.0)
    assert np.allclose(u, [1, -2], rtol=0, atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_scores_depend_on_the_distance_alone(inter):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 16))
    tab = dc.table(50, 16, 100.0).double().numpy()
    turn = lambda x, p: oracle.rope_head(x, tab[p, :8], tab[p, 8:], interleaved=inter)
    assert np.isclose(turn(q, 30) @ turn(k, 12), turn(q, 45) @ turn(k, 27), rtol=0, atol=1e-5)
    assert np.isclose(np.linalg.norm(turn(q, 7)), np.linalg.norm(q), atol=1e-6)


def test_append_places_by_hand():
    T, D = 4, 2
    q = np.arange(8.0).reshape(T, D)
    kc = np.zeros((2, 2, 1, D))
    qo, k, v = oracle.rope_append(q, q, q + 100, np.array([[1.0, 0.0]]), [0, 0, 1, 0], [3, -1, 0, 1], kc, kc)
    assert np.isnan(qo[2]).all() and np.array_equal(qo[[0, 1, 3]], q[[0, 1, 3]])
    assert np.array_equal(k[:, :, 0], [[[0, 0], [6, 7]], [[0, 0], [0, 1]]])
    assert np.array_equal(v[:, :, 0], [[[0, 0], [106, 107]], [[0, 0], [100, 101]]])


def test_attention_by_hand():
    # two places, scores 0 and log 3: weights 1/4 and 3/4; a prefix of one place, one of its own
    kc = np.zeros((2, 2, 1, 2))
    vc = np.zeros((2, 2, 1, 2))
    kc[1, 0, 0], kc[0, 1, 0] = [0, 1], [np.log(3.0), 0]
    vc[1, 0, 0], vc[0, 1, 0] = [4, 8], [0, -8]
    own = np.array([[7, 0]])  # page 7 lies outside the cache: its two places are masked
    o, lse, spread = oracle.prefix_attention(np.array([[1.0, 0.0]]), kc, vc, [0, 1], None, np.array([[1]]), [1],
                                             own, [4], 1.0)
    # own list: places (0, 0) and (0, 1): scores 0 and log 3, so weights 1, 1, 3 of 5
    assert np.allclose(o, [[4 / 5, 8 / 5 - 24 / 5]]) and np.allclose(lse, np.log(5.0))
    assert np.allclose(spread, [[4 / 5, 32 / 5]])


def test_attention_equals_one_list():
    """A prefix and own keys give what one list of all keys gives, and a library softmax agrees."""
    c = dc.Attn(4, "bf16", 3, [3], 4, 2, 16, 4, [11], [5, 0, 9])
    o, lse, _ = oracle.prefix_attention(*c.args())
    for t in range(3):
        n, m = int(c.prefix_lens[0]), int(c.own_lens[t])
        at = [(int(c.prefix_pages[0, j // 4]), j % 4) for j in range(n)]
        at += [(int(c.own_pages[t, j // 4]), j % 4) for j in range(m)]
        pg, pl = map(torch.tensor, zip(*at))
        for h in range(4):
            s = c.scale * c.k[pg, pl, h // 2].double() @ c.q[t, h * 16:h * 16 + 16].double()
            assert np.isclose(lse[t, h], torch.logsumexp(s, 0).item())
            assert np.allclose(o[t, h * 16:h * 16 + 16], (torch.softmax(s, 0) @ c.v[pg, pl, h // 2].double()).numpy())


def test_attention_empty_rows():
    c = dc.Attn(4, "bf16", 4, [2, 1], 2, 1, 8, 4, [0, 3], [0, 5, 0, 0], perm=False, indptr0=0)
    o, lse, _ = oracle.prefix_attention(*c.args())
    assert np.array_equal(o[0], np.zeros(16)) and np.all(lse[0] == -np.inf)
    assert np.all(np.isfinite(lse[1:3])) and np.isnan(o[3]).all()  # row 3 has no segment
