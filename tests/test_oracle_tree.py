"""Pins of the oracle's speculative step: tree attention, draft verification,
and the append of accepted rows (CPU)."""
import numpy as np
import pytest

import oracle
from tests.tree_util import BINARY, CHAIN, STAR, TWO, depths, drafted, logits, parents, plane


def brute_attention(ring, key, value, kvh, D, hm, q, k, v, H, scale, parent, window, n_sink, sink, gate):
    """Dense masked softmax in numpy over every slot row gathered in logical order."""
    M, cap = q.shape[0], ring.capacity

    def rows(buf, cap, hm, slots):
        f = buf.view(np.float16).astype(np.float64)
        return f.reshape(kvh, cap, D)[:, slots] if hm else f.reshape(cap, kvh, D)[slots].transpose(1, 0, 2)

    d = np.array(depths(parent))
    end = ring.origin_logical + ring.len
    slots = (ring.origin_physical + np.arange(ring.len)) % cap
    pos = [ring.origin_logical + np.arange(ring.len), end + d]
    r16 = lambda t: t.astype(np.float16).astype(np.float64).reshape(M, kvh, D).transpose(1, 0, 2)  # noqa: E731
    K, V = [rows(key, cap, hm, slots), r16(k)], [rows(value, cap, hm, slots), r16(v)]
    anc = np.eye(M, dtype=bool)
    for i in range(1, M):
        anc[i] |= anc[parent[i]]
    allowed = [np.ones((M, ring.len), bool), anc]
    if sink is not None:
        sr, sk, sv, shm = sink
        sp = sr.origin_logical + np.arange(sr.len)
        keep = (sp < n_sink) & (sp < ring.origin_logical)
        ss = ((sr.origin_physical + np.arange(sr.len)) % sr.capacity)[keep]
        K.append(rows(sk, sr.capacity, shm, ss))
        V.append(rows(sv, sr.capacity, shm, ss))
        pos.append(sp[keep])
        allowed.append(np.ones((M, keep.sum()), bool))
    K, V, pos, allowed = np.concatenate(K, 1), np.concatenate(V, 1), np.concatenate(pos), np.concatenate(allowed, 1)
    if window:
        allowed &= ((end + d)[:, None] - pos[None] < window) | (pos[None] < n_sink)
    out = np.empty((M, H, D))
    for i in range(M):
        see = allowed[i]
        for h in range(H):
            g = h // (H // kvh)
            s = scale * (K[g][see] @ q[i].reshape(H, D)[h].astype(np.float64))
            e = np.exp(s - s.max())
            out[i, h] = (e / e.sum()) @ V[g][see]
    if gate is not None:
        out /= 1 + np.exp(-gate.reshape(M, H, D).astype(np.float64))
    return out.reshape(M, H * D)


@pytest.mark.parametrize("M,H,kvh,D,n,cap,origin,hm,window,n_sink,kind", [
    (1, 2, 1, 3, 0, 4, 0, False, 0, 0, CHAIN), (1, 4, 2, 8, 9, 9, 5, False, 4, 0, CHAIN),
    (5, 4, 2, 8, 20, 32, 0, True, 7, 3, BINARY), (16, 6, 3, 5, 40, 40, 25, False, 12, 6, TWO),
    (16, 2, 2, 4, 3, 8, 0, False, 2, 0, CHAIN), (7, 2, 1, 6, 11, 16, 0, True, 1, 2, STAR),
    (6, 2, 1, 6, 11, 16, 0, False, 3, 14, CHAIN)])
@pytest.mark.parametrize("with_sink", [False, True])
def test_tree_attention_brute_force(M, H, kvh, D, n, cap, origin, hm, window, n_sink, kind, with_sink):
    rng = np.random.default_rng(M * 100 + n)
    ring, key, value = plane(rng, cap, kvh, D, n, origin, hm)
    sink = None
    if with_sink:
        sr, sk, sv = plane(rng, 9, kvh, D, 8, 0, not hm, physical=4)
        sink = (sr, sk, sv, not hm)
    p = parents(kind, M)
    q, gate = rng.standard_normal((M, H * D)).astype(np.float32), rng.standard_normal((M, H * D)).astype(np.float32)
    k, v = (rng.standard_normal((M, kvh * D)).astype(np.float32) for _ in range(2))
    got = oracle.tree_attention(ring, key, value, kvh * D, D, hm, q, k, v, H, 0.3, p, window, n_sink, sink, gate)
    want = brute_attention(ring, key, value, kvh, D, hm, q, k, v, H, 0.3, p, window, n_sink, sink, gate)
    # the oracle rounds once to binary32
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-12)


def test_tree_attention_of_a_chain_is_token_by_token_attention():
    """Row i of a chain gives what a single token gives after rows 0..i-1 were appended to the ring."""
    rng = np.random.default_rng(3)
    M, H, kvh, D, n, cap = 6, 4, 2, 8, 30, 64
    ring, key, value = plane(rng, cap, kvh, D, n, 0, False, fill=0)
    q = rng.standard_normal((M, H * D)).astype(np.float32)
    k, v = (rng.standard_normal((M, kvh * D)).astype(np.float32) for _ in range(2))
    tree = oracle.tree_attention(ring, key, value, kvh * D, D, False, q, k, v, H, 0.25, window=17)
    for i in range(M):
        one = oracle.tree_attention(ring, key, value, kvh * D, D, False, q[i:i + 1], k[i:i + 1], v[i:i + 1], H, 0.25,
                                    window=17)
        assert np.allclose(one[0], tree[i], rtol=2e-7, atol=1e-9)
        assert oracle.kv_write(ring, key, value, kvh * D, D, False, k[i:i + 1], v[i:i + 1], n + i)[0] == 0


def test_tree_attention_one_row_returns_its_value():
    rng = np.random.default_rng(4)
    ring, key, value = plane(rng, 4, 1, 6, 0, 0, False)
    v = rng.standard_normal((1, 6)).astype(np.float32)
    out = oracle.tree_attention(ring, key, value, 6, 6, False, np.ones((1, 12)), np.ones((1, 6)), v, 2, 1.0)
    assert np.array_equal(out.reshape(2, 6), np.tile(v.astype(np.float16).astype(np.float32), (2, 1)))


# ----------------------------------------------------------------- verification
def test_verify_hand_worked():
    """p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4) at the root, one child of token 1: it is accepted below p/q = 1/2;
    after a rejection only token 0 is left."""
    target = np.log(np.array([[2, 1, 1], [1, 1, 2]], np.float64)).astype(np.float32)
    draft = np.log(np.array([[1, 2, 1], [1, 1, 1]], np.float64)).astype(np.float32)
    v = lambda u0, u1, **kw: oracle.tree_verify(target, [0, 1], 1.0, [u0, u1], **kw).tolist()  # noqa: E731
    assert v(0.3, 0.49, draft=draft) == [2, 1, 0, 1]     # accepted; row 1's p = (1/4, 1/4, 1/2)
    assert v(0.2, 0.49, draft=draft) == [2, 0, 0, 1]
    assert v(0.6, 0.49, draft=draft) == [2, 2, 0, 1]
    assert v(0.99, 0.51, draft=draft) == [1, 0, 0, -1]   # max(p - q, 0) = (1/4, 0, 0)
    # drafts taken as certain: accepted below p(1) = 1/4; then (2/3, 0, 1/3)
    assert v(0.3, 0.24) == [2, 1, 0, 1]
    assert v(0.66, 0.26) == [1, 0, 0, -1]
    assert v(0.67, 0.26) == [1, 2, 0, -1]
    assert oracle.tree_verify(target, [0, 0], 0.0).tolist() == [2, 2, 0, 1]
    assert oracle.tree_verify(target, [0, 1], 0.0).tolist() == [1, 0, 0, -1]


@pytest.mark.parametrize("kind,M,with_draft", [(STAR, 5, True), (BINARY, 4, True), (CHAIN, 3, True), (STAR, 5, False)])
def test_verify_keeps_the_target_distribution(kind, M, with_draft):
    """Whatever the drafter, the first new token is distributed as the target's row: the frequencies of 40,000 draws
    stay within 5 standard deviations for each of 6 tokens."""
    rng = np.random.default_rng(11)
    V, N, parent = 6, 40000, parents(kind, M)
    target, draft = (rng.standard_normal((M, V)).astype(np.float32) for _ in range(2))
    count = np.zeros(V)
    for _ in range(N):
        tokens = drafted(rng, draft, parent, 1.0) if with_draft else np.array([0, 3, 1, 3, 5][:M], np.int32)
        u = rng.random(M).astype(np.float32)
        r = oracle.tree_verify(target, tokens, 1.0, u, draft if with_draft else None, parent)
        count[tokens[r[3]] if r[0] > 1 else r[1]] += 1
    p = np.exp(target[0].astype(np.float64))
    p /= p.sum()
    assert np.all(np.abs(count / N - p) <= 5 * np.sqrt(p * (1 - p) / N))


def test_verify_tokens_outside_the_vocabulary_are_rejected():
    rng = np.random.default_rng(5)
    t, d = logits(rng, 3, 50), logits(rng, 3, 50)
    for draft in (None, d):
        r = oracle.tree_verify(t, [0, 50, -1], 1.0, [0.5, 0.0, 0.0], draft, parents(STAR, 3))
        assert r[0] == 1 and 0 <= r[1] < 50


def test_commit_is_ring_writes_of_the_accepted_rows():
    """The append of rows path of a tree is one ring write per row (what the GPU call is held to)."""
    rng = np.random.default_rng(6)
    ring, key, value = plane(rng, 8, 1, 4, 8, 3, False, fill=0)
    k, v = (rng.standard_normal((5, 4)).astype(np.float32) for _ in range(2))
    before = key.copy()
    for j, i in enumerate([0, 2, 4]):
        assert oracle.kv_write(ring, key, value, 4, 4, False, k[i:i + 1], v[i:i + 1], 11 + j)[0] == 0
    assert (ring.len, ring.origin_logical, ring.origin_physical) == (8, 6, 6)
    slots = [3, 4, 5]
    assert np.array_equal(key.reshape(8, 4)[slots], k[[0, 2, 4]].astype(np.float16).view(np.uint16))
    rest = [s for s in range(8) if s not in slots]
    assert np.array_equal(key.reshape(8, 4)[rest], before.reshape(8, 4)[rest])
