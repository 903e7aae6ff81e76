"""Pins of the oracle of the calls on several sequences (no GPU)."""
import numpy as np
import pytest

from oracle import paged


def test_tables_worked_example():
    # pages of 4 rows; sequence 0 has 6 rows in pages 3, 1; sequence 1 has 4 rows in page 0
    table = [[3, 1, -1, -1], [0, -1, -1, -1]]
    r = paged.page_tables(table, [6, 4], None, [3, 1], 6, 4)
    assert r["table"][0] == [3, 1, 2, None] and r["table"][1] == [0, 4, None, None]
    assert r["slots"] == [1 * 4 + 2, 1 * 4 + 3, 2 * 4, 4 * 4] and r["position"] == [6, 7, 8, 4]
    assert r["sequence"] == [0, 0, 0, 1] and r["first"] == [0, 3, 4] and r["last"] == [8, 4] and r["length"] == [9, 5]
    assert r["result"] == [0, 4, 0, 2, 1, 0, 0, 0]  # only page 5 is left


def test_beams_that_go_on_from_one_share_its_full_pages():
    table = [[3, 1, -1], [0, 2, -1]]
    r = paged.page_tables(table, [6, 6], [0, 0], None, 6, 4)
    assert r["table"] == [[3, 1, None], [3, 0, None]]  # the dropped beam's pages 0 and 2 are free
    assert r["copies"] == [(1, 0, 2)] and r["result"][:5] == [0, 2, 1, 1, 3]


def test_a_row_that_stands_still_keeps_its_page_from_those_that_grow():
    table = [[3, 1], [0, 2]]
    r = paged.page_tables(table, [6, 6], [0, 0], [0, 1], 6, 4)
    assert r["copies"] == [(1, 0, 2)] and r["length"] == [6, 7] and r["last"] == [-1, 6]


@pytest.mark.parametrize("kw,status", [(dict(add=[20, 0]), 2), (dict(add=[5, 5], max_new=9), 3), (dict(add=[9, 9]), 1),
                                       (dict(parent=[0, 0], add=[1, 1], copies_given=False), 4)])
def test_tables_failures_grow_nothing(kw, status):
    kw = dict(dict(parent=None), **kw)
    r = paged.page_tables([[3, 1, -1, -1], [0, -1, -1, -1]], [6, 4], pages=5, page_rows=4, **kw)
    assert r["result"][0] == status and r["slots"] == [] and r["copies"] == []
    assert r["length"][0] == 6


def test_window_gives_pages_up():
    table = [[4, 3, 2, 1]]
    r = paged.page_tables(table, [13], None, None, 8, 4, window=5, n_sink=2)
    # the token at 13 sees 9..13 and 0, 1: page 1 (rows 4..7) is dead, page 2 (rows 8..11) is not
    assert r["table"][0] == [4, -1, 2, 1]


def test_attention_is_a_dense_masked_softmax():
    rng = np.random.default_rng(3)
    pages, R, G, D, H, n = 9, 4, 2, 8, 6, 3
    key, value = (rng.standard_normal(pages * R * G * D).astype(np.float16) for _ in range(2))
    table = np.array([[5, 2, 7], [1, -1, 8], [0, 3, 4]])
    position = [9, 11, 2]
    q = rng.standard_normal((n, H * D)).astype(np.float32)
    k, v = (rng.standard_normal((n, G * D)).astype(np.float32) for _ in range(2))
    out, stored = paged.paged_attention(key, value, pages, R, G, D, False, table, position, q, H, 0.3, k, v, window=6, n_sink=1)
    assert stored == [(7, 1), (8, 3), (0, 2)]
    flat = key.reshape(-1, G, D).astype(np.float64), value.reshape(-1, G, D).astype(np.float64)
    for i in range(n):
        seen = [p for p in range(position[i]) if (position[i] - p < 6 or p < 1) and table[i, p // R] >= 0]
        slots = [table[i, p // R] * R + p % R for p in seen]
        for h in range(H):
            K = np.vstack([flat[0][slots, h // 3], k[i].reshape(G, D)[h // 3].astype(np.float16)])
            V = np.vstack([flat[1][slots, h // 3], v[i].reshape(G, D)[h // 3].astype(np.float16)])
            a = np.exp(0.3 * K @ q[i].reshape(H, D)[h].astype(np.float64))
            assert np.allclose(out[i].reshape(H, D)[h], (a / a.sum()) @ V, atol=1e-12)


def test_beam_selection_by_brute_force():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 11)).astype(np.float32)
    score = np.array([-1.0, -2.0, -0.5, -np.inf], np.float32)
    p, t, s, e = paged.beam_select(x, score, 2, 2, 5, np.array([0, 1, 0, 0]), 3)
    lp = x - np.log(np.exp(x.astype(np.float64)).sum(1, keepdims=True))
    first = sorted([(-1.0 + lp[0, v], 0, v) for v in range(11)] + [(-2.0, 1, 3)], key=lambda b: -b[0])[:5]
    assert [b[1] for b in first] == list(p[:5]) and [b[2] for b in first] == list(t[:5])
    assert np.allclose([b[0] for b in first], s[:5])
    assert set(p[5:]) == {2} and np.array_equal(t[5:], np.argsort(-x[2], kind="stable")[:5])
    assert all(e[i] == (t[i] == 3 or p[i] == 1) for i in range(10))


def test_beam_selection_without_enough_ways_on():
    p, t, s, e = paged.beam_select(np.zeros((2, 2), np.float32), np.array([0.0, -np.inf]), 1, 2, 4)
    assert list(p) == [0, 0, -1, -1] and list(t) == [0, 1, -1, -1] and list(e) == [0, 0, 1, 1]
    assert np.allclose(s[:2], -np.log(2)) and np.isneginf(s[2:]).all()
