"""The speculative step on the GPU against the fp64 oracle: attention of tree rows over a plane, draft verification,
the append of accepted rows, and the three together."""
import ctypes

import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import check_canary, dev, host, nan_like
from tests.tree_util import BINARY, CHAIN, STAR, TWO, drafted, logits, parents, plane

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import quantized_weight_streaming_q4_gb300 as mu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mu.build()
    mu.lib()
    torch.cuda.init()


def to_dev16(a):
    return dev(a.view(np.int16))


def kv_plane(ring, key, value, kvh, D, hm):
    return mu.KvPlane(key.data_ptr(), value.data_ptr(), ring.capacity, ring.len, ring.origin_logical,
                      ring.origin_physical, kvh * D, D, int(hm), 0)


# ------------------------------------------------------------------ attention
def attention_bound(q, scale, kmax, D, vmax):
    """Elementwise bound of a binary32 evaluation.  A score is a sum of D products (binary16 key times a query held to
    2^-22 at least): its error is at most (D/2 + 8) steps of 2^-24 of scale * sum|q||k|, taking half the steps for
    partial sums that grow evenly.  A weight's relative error is at most twice the largest score's error plus 2^-21
    (the exponential, the two sums); an output is a mean of values up to vmax."""
    s = scale * np.abs(q).reshape(q.shape[0], -1, D).sum(-1).max() * kmax
    return vmax * (2 * (D / 2 + 8) * 2.0 ** -24 * s + 2.0 ** -21)


class Case:
    def __init__(self, M, H, kvh, D, n, cap, origin, hm, window=0, n_sink=0, kind=CHAIN, sink_rows=0, gate=False, seed=0,
                 qscale=1.5, offset=0):
        rng = np.random.default_rng(seed * 1000 + M * 17 + n)
        self.M, self.H, self.kvh, self.D, self.hm = M, H, kvh, D, hm
        self.window, self.n_sink, self.scale, self.parent = window, n_sink, D ** -0.5, parents(kind, M)
        self.ring, self.key, self.value = plane(rng, cap, kvh, D, n, origin, hm)
        self.sink = None
        if sink_rows:
            r, sk, sv = plane(rng, sink_rows + 3, kvh, D, sink_rows, 0, not hm, physical=2)
            self.sink = (r, sk, sv, not hm)
        self.q = (qscale * rng.standard_normal((M, H * D))).astype(np.float32)
        self.k, self.v = (rng.standard_normal((M, kvh * D)).astype(np.float32) for _ in range(2))
        self.gate = rng.standard_normal((M, H * D)).astype(np.float32) if gate else None
        self.offset = offset

    def want(self):
        return oracle.tree_attention(self.ring, self.key, self.value, self.kvh * self.D, self.D, self.hm, self.q, self.k,
                                     self.v, self.H, self.scale, self.parent, self.window, self.n_sink, self.sink,
                                     self.gate)

    def to_device(self):
        o = self.offset

        def half(a):
            buf = torch.full((a.size + 8 + o,), 0x7E00, dtype=torch.int16, device="cuda")
            buf[o:o + a.size] = to_dev16(a)
            return buf[o:o + a.size]

        self.dkey, self.dvalue = half(self.key), half(self.value)
        self.plane = kv_plane(self.ring, self.dkey, self.dvalue, self.kvh, self.D, self.hm)
        self.dsink = None
        if self.sink:
            self.sk, self.sv = half(self.sink[1]), half(self.sink[2])
            self.dsink = kv_plane(self.sink[0], self.sk, self.sv, self.kvh, self.D, self.sink[3])
        self.dq, self.dk, self.dv = dev(self.q), dev(self.k), dev(self.v)
        self.dgate = None if self.gate is None else dev(self.gate)
        self.nbytes = mu.muser_kv_tree_attention_scratch_bytes(self.kvh * self.D, self.D, self.M, self.H)
        self.scratch = torch.zeros(self.nbytes // 4 + 4, device="cuda")
        self.scratch[self.nbytes // 4:] = 12345.0
        self.out = nan_like((self.M, self.H * self.D), 16)
        return self

    def call(self, stream=None):
        mu.muser_kv_tree_attention(self.plane, self.dq, self.dk, self.dv, self.M, self.H, self.out, self.scale,
                                   self.scratch, self.nbytes, self.parent, self.window, self.n_sink, self.dsink,
                                   self.dgate, stream)
        return self

    def check(self, want=None):
        n = self.M * self.H * self.D
        got, want = host(self.out)[:n].reshape(self.M, -1), self.want() if want is None else want
        check_canary(self.out, n)
        check_canary(self.scratch, self.nbytes // 4)
        vmax = 1.0
        for t in (self.value, None if self.sink is None else self.sink[2]):
            if t is not None:
                f = t.view(np.float16).astype(np.float32)
                vmax = max(vmax, np.abs(f[np.isfinite(f)]).max(initial=0))
        vmax = max(vmax, np.abs(self.v[np.isfinite(self.v)]).max())
        err = np.abs(got.astype(np.float64) - want)
        assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} outputs are not finite"
        assert err.max() <= attention_bound(self.q, self.scale, 5.0, self.D, vmax), err.max()
        rel = np.linalg.norm(err) / np.linalg.norm(want)
        assert rel <= 1e-5, rel   # binary32: outputs of random sign do not add their errors up
        return rel


SHAPES = [  # heads, K/V heads, head_dim
    (32, 2, 128), (4, 4, 64), (20, 5, 64), (6, 2, 80), (3, 1, 256), (6, 3, 5), (8, 1, 128), (2, 1, 72), (26, 1, 128),
]


@pytest.mark.parametrize("H,kvh,D", SHAPES)
@pytest.mark.parametrize("M,n", [(1, 0), (1, 1), (1, 37), (1, 700), (3, 16), (16, 0), (16, 1), (16, 333), (7, 129)])
@pytest.mark.parametrize("hm", [False, True])
def test_attention_shapes(H, kvh, D, M, n, hm):
    Case(M, H, kvh, D, n, n + 3, 0, hm, kind=BINARY if M == 7 else CHAIN, gate=M == 3).to_device().call().check()


@pytest.mark.parametrize("H,kvh,D", [(32, 2, 128), (6, 2, 80), (4, 2, 24)])
@pytest.mark.parametrize("M,n,cap,origin,window,n_sink,kind,sink_rows", [
    (1, 64, 64, 1000, 64, 0, CHAIN, 0),        # a full, turned ring as long as its window
    (16, 64, 64, 1000, 64, 4, TWO, 4),         # the same for a tree, first tokens kept apart
    (16, 64, 64, 1000, 5, 9, CHAIN, 6),        # the chain is deeper than the window
    (16, 200, 200, 33, 100, 40, BINARY, 20),   # first rows in the sink plane and in the ring's own start
    (16, 200, 256, 0, 64, 16, STAR, 0),        # first rows in the plane itself
    (9, 5, 256, 0, 3, 50, BINARY, 7),          # every row is a first row; the sink plane has nothing to add
    (16, 40, 64, 0, 1, 0, CHAIN, 0),           # a window of one: every row sees itself alone
    (5, 1000, 1024, 0, 999, 3, CHAIN, 0),
    (2, 300, 300, 299, 290, 2000, TWO, 5),     # more first tokens asked for than there are
])
def test_attention_windows_and_sinks(H, kvh, D, M, n, cap, origin, window, n_sink, kind, sink_rows):
    for hm in (False, True):
        Case(M, H, kvh, D, n, cap, origin, hm, window, n_sink, kind, sink_rows, gate=True, seed=2).to_device().call().check()


@pytest.mark.parametrize("sink_rows", [1, 4, 60, 127, 128, 131])
@pytest.mark.parametrize("M,n,H,kvh,D", [(1, 2048, 32, 2, 128), (5, 2048, 20, 5, 64), (16, 2048, 32, 2, 128), (16, 600, 32, 2, 128),
                                         (1, 130, 32, 2, 128), (3, 260, 6, 2, 80), (1, 20000, 32, 2, 128), (16, 20000, 32, 2, 128)])
def test_attention_short_runs_before_the_ring(sink_rows, M, n, H, kvh, D):
    """First rows kept in a plane that wraps (two short runs), then a full ring that wraps."""
    c = Case(M, H, kvh, D, n, n, 10 * n + 77, False, n, sink_rows, TWO, sink_rows, gate=True, seed=sink_rows)
    rng = np.random.default_rng(sink_rows)
    r, sk, sv = plane(rng, sink_rows + 3, kvh, D, sink_rows, 0, True, physical=sink_rows + 2)
    c.sink = (r, sk, sv, True)
    c.to_device().call().check()


@pytest.mark.parametrize("n", [1024, 4097, 33000])
@pytest.mark.parametrize("M,H,kvh,D", [(1, 32, 2, 128), (4, 32, 2, 128), (16, 32, 2, 128), (16, 16, 16, 64)])
def test_attention_long(n, M, H, kvh, D):
    c = Case(M, H, kvh, D, n, n + 5, 0, n != 4097, window=0 if n != 4097 else 4000, kind=TWO, seed=3)
    c.to_device().call().check()


@pytest.mark.parametrize("M,H,kvh,D,n", [(1, 3, 3, 5, 10), (1, 1, 1, 7, 0), (3, 9, 9, 33, 20), (5, 3, 1, 65, 700), (1, 1, 1, 1, 3),
                                         (7, 5, 5, 129, 333), (15, 21, 7, 255, 100)])
@pytest.mark.parametrize("gate", [False, True])
def test_attention_odd_rows_heads_and_head_sizes(M, H, kvh, D, n, gate):
    """An odd number of sums in the scratch: the maxima beside them are 8 bytes each."""
    Case(M, H, kvh, D, n, n + 1, 0, False, gate=gate, seed=21).to_device().call().check()


@pytest.mark.parametrize("M,H,kvh,D,n", [(16, 16, 1, 256, 130000), (16, 8, 2, 200, 40000), (16, 32, 2, 128, 130000), (1, 32, 2, 128, 130000),
                                         (16, 32, 4, 64, 60000), (2, 2, 1, 7, 130000)])
def test_attention_long_sums_do_not_drift(M, H, kvh, D, n):
    """Values of one sign, so that sums which lose their last bits downwards lose them together.  Against binary64, of the
    result's norm: sums of n / 16 terms to nearest lose 2^-25 of themselves at random each, sqrt(8192) 2^-25 = 2.7e-6 for
    the longest if no block shared it (a sixteenth of the rows or less a block: 7e-7); the products of 16 keys or of a
    tile lose 8 steps of 2^-24 at most (4.8e-7); queries and weights are held to 2^-22 and exponentials to 2^-22, at random
    (2.4e-7 each); the division 2^-23: 1.8e-6 in all.  4e-6 is twice that; one accumulator that truncates over 8,000 keys
    would lose 2e-5."""
    c = Case(M, H, kvh, D, 8, n, 0, True, seed=24)
    g = torch.Generator(device="cuda").manual_seed(D)
    key = torch.randn(kvh, n, D, generator=g, device="cuda").half()
    value = (1 + 0.25 * torch.rand(kvh, n, D, generator=g, device="cuda")).half()
    c.q *= 0.5
    c.v = 1 + np.abs(c.v) / 4
    c.to_device()
    c.plane = mu.KvPlane(key.data_ptr(), value.data_ptr(), n, n, 0, 0, kvh * D, D, 1, 0)
    got = host(c.call().out)[:M * H * D].reshape(M, H, D)
    group, want = H // kvh, np.empty((M, H, D))
    tk, tv = (t.half().double().view(M, kvh, D) for t in (c.dk, c.dv))
    for i in range(M):                       # a chain: row i sees the plane and rows 0..i
        for h in range(kvh):
            k, v = (torch.cat([a[h].double(), b[:i + 1, h]]) for a, b in ((key, tk), (value, tv)))
            q = c.dq.double().view(M, kvh, group, D)[i, h]
            want[i, h * group:(h + 1) * group] = (torch.softmax(c.scale * (q @ k.T), 1) @ v).cpu().numpy()
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 4e-6, rel


@pytest.mark.parametrize("offset", [1, 4])
def test_attention_planes_off_the_16_byte_grid(offset):
    Case(3, 4, 2, 64, 77, 80, 0, False, offset=offset).to_device().call().check()


@pytest.mark.parametrize("H,kvh,D", [(32, 2, 128), (4, 2, 24)])
def test_attention_large_queries_and_sharp_softmax(H, kvh, D):
    # scores of some hundreds: one row takes nearly all the weight; and queries beyond binary16's range
    Case(5, H, kvh, D, 500, 512, 0, True, qscale=60.0, seed=5).to_device().call().check()
    c = Case(2, H, kvh, D, 50, 64, 0, False, qscale=1e6, seed=6)
    c.scale = D ** -0.5 * 1e-6
    c.to_device().call().check()


@pytest.mark.parametrize("H,kvh,D", [(32, 2, 128), (5, 1, 64), (4, 2, 24), (4, 1, 256), (4, 1, 7)])
@pytest.mark.parametrize("M", [1, 2, 9])
@pytest.mark.parametrize("power", [-140, -110, 100, 117])
def test_attention_scores_at_the_ends_of_binary32(H, kvh, D, M, power):
    """scale = 2^power: finite scores of up to 2^117 (a sum of D products below 2^7 times log2(e): 2^126), whose largest
    takes all the weight, and vanishing ones, whose weights are alike."""
    c = Case(M, H, kvh, D, 300, 300, 0, False, seed=25)
    c.q = np.clip(c.q, -3, 3) / np.float32(D / 4)
    c.scale = 2.0 ** power
    c.to_device().call()
    n = M * H * D
    got, want = host(c.out)[:n].reshape(M, -1), c.want()
    assert np.isfinite(got).all()
    if power < 0:
        assert np.abs(got - want).max() <= 2.0 ** -18      # a mean of 300 values up to 5: 5 (300 / 32 + 8) 2^-24
    else:   # one row's value, unless two scores are within the binary32 sums' error, 2^-17 of themselves
        k = np.concatenate([c.key.view(np.float16).reshape(300, kvh, D), c.k.astype(np.float16).reshape(M, kvh, D)]).astype(np.float64)
        for i in range(M):
            for h in range(H):
                sc = np.sort(k[:301 + i, h // (H // kvh)] @ c.q.reshape(M, H, D)[i, h].astype(np.float64))
                if sc[-1] - sc[-2] > 2.0 ** -15 * np.abs(sc).max():
                    assert np.abs(got - want).reshape(M, H, D)[i, h].max() <= 2.0 ** -18, (i, h)


@pytest.mark.parametrize("H,kvh,D", [(32, 2, 128), (16, 2, 128), (5, 1, 64), (4, 2, 24), (4, 1, 256), (4, 1, 7)])
@pytest.mark.parametrize("M", [1, 2, 9])
@pytest.mark.parametrize("falling", [False, True])
def test_attention_scores_that_grow_along_the_cache(H, kvh, D, M, falling):
    """The running maximum moves in every tile (or is the first key's): scores run from 0 to 4 scale D, up to 45."""
    n = 3001
    c = Case(M, H, kvh, D, n, n, 0, False, seed=12)
    rng = np.random.default_rng(M)
    sign = rng.choice([-1.0, 1.0], (kvh, D))
    ramp = np.linspace(0, 4, n)[::-1 if falling else 1]
    k = (ramp[:, None, None] * sign + 0.1 * rng.standard_normal((n, kvh, D))).astype(np.float16)
    c.key[:] = np.ascontiguousarray(k.reshape(-1)).view(np.uint16)
    c.q = np.broadcast_to(sign[np.arange(H) // (H // kvh)].reshape(1, H * D), (M, H * D)).astype(np.float32) * \
        (0.5 + rng.random((M, H * D), np.float32))
    c.to_device().call().check()


@pytest.mark.parametrize("M,H,kvh,D,n", [(1, 64, 64, 64, 2100), (3, 40, 20, 128, 700), (16, 64, 8, 128, 2048), (2, 8, 2, 256, 9000),
                                         (13, 30, 2, 120, 5000), (1, 9, 9, 8, 300), (16, 512, 1, 64, 200)])
def test_attention_many_heads_and_odd_splits(M, H, kvh, D, n):
    Case(M, H, kvh, D, n, n + 1, 0, True, kind=BINARY, gate=True, seed=13).to_device().call().check()


@pytest.mark.parametrize("H,kvh,D", [(32, 2, 128), (6, 2, 80), (4, 2, 5)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_attention_what_is_not_seen_has_no_influence(H, kvh, D, bad):
    """Non-finite values in slots behind the rows, in rows outside some windows, and in a tree row that only its own
    branch sees."""
    M, n = 6, 150
    c = Case(M, H, kvh, D, n, 160, 0, False, window=100, kind=STAR, seed=7)
    want = c.want()
    c.k[3], c.v[3] = bad, bad   # row 3: a sibling of the others
    kk, vv = (t.reshape(160, kvh * D).view(np.float16) for t in (c.key, c.value))
    kk[:50], vv[:50] = bad, bad       # before position 50: in no window but the root's edge (150 - 100 + 1 = 51)
    c.to_device().call()
    n_out = M * H * D
    got = host(c.out)[:n_out].reshape(M, -1)
    keep = [0, 1, 2, 4, 5]
    assert np.isfinite(got[keep]).all()
    assert np.abs(got[keep] - want[keep]).max() <= attention_bound(c.q, c.scale, 5.0, D, 5.0)
    assert not np.isfinite(got[3]).any()
    # the row at the window's lower edge: seen by the root alone (51), not by the deeper ones
    c2 = Case(M, H, kvh, D, n, 160, 0, False, window=100, kind=STAR, seed=7)
    want = c2.want()
    kk, vv = (t.reshape(160, kvh * D).view(np.float16) for t in (c2.key, c2.value))
    kk[51], vv[51] = bad, bad
    c2.to_device().call()
    got = host(c2.out)[:n_out].reshape(M, -1)
    assert not np.isfinite(got[0]).any() and np.isfinite(got[1:]).all()
    assert np.abs(got[1:] - want[1:]).max() <= attention_bound(c2.q, c2.scale, 5.0, D, 5.0)


@pytest.mark.parametrize("M,H,kvh,D", [(1, 32, 2, 128), (2, 32, 2, 128), (9, 20, 5, 64), (16, 32, 2, 128), (16, 32, 1, 64), (1, 4, 1, 256),
                                       (9, 8, 2, 136), (1, 4, 2, 5), (9, 6, 2, 7)])
@pytest.mark.parametrize("where", ["cached", "first", "edge", "tree"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_one_infinite_key_element(M, H, kvh, D, where, sign):
    """A key with one infinite element.  Queries of that sign there: a score of +infinity, nothing finite.  Queries of
    the other sign: -infinity, which counts as weight 0 or makes the output NaN.  Rows that do not see it: no influence."""
    n, window = 700, 300
    if where == "edge" and M == 1:
        pytest.skip("one row has one window")
    c = Case(M, H, kvh, D, n, n, 0, False, window=window, kind=CHAIN, seed=23)
    element = D // 2
    c.q.reshape(M, H, D)[:, :, element] = 0.25 + np.abs(c.q.reshape(M, H, D)[:, :, element])
    seeing = np.ones(M, bool)
    if where == "tree":
        c.k.reshape(M, kvh, D)[M - 1, :, element] = sign * np.inf
        seeing[:M - 1] = False                  # the last row of a chain
    else:
        at = {"cached": n - 100, "first": n - window + M, "edge": n - window + 1}[where]
        c.key.reshape(n, kvh, D).view(np.float16)[at, :, element] = sign * np.inf
        if where == "edge":
            seeing[1:] = False                  # position 401: the root's alone
    want = c.want()                             # exp(-infinity) = 0 there
    got = host(c.to_device().call().out)[:M * H * D].reshape(M, -1)
    assert np.isfinite(want[~seeing]).all() and np.isfinite(got[~seeing]).all()
    bound = attention_bound(c.q, c.scale, 5.0, D, 5.0)
    if (~seeing).any():
        assert np.abs(got[~seeing] - want[~seeing]).max() <= bound
    if sign > 0:
        assert not np.isfinite(got[seeing]).any()
    else:
        ok = np.isnan(got[seeing]) | (np.abs(got[seeing] - want[seeing]) <= bound)
        assert np.isfinite(want[seeing]).all() and ok.all()


def test_attention_offsets_past_32_bits():
    """A head-major plane of 2^24 slots (2^32 elements a buffer): the second head's rows lie past 2^31 elements."""
    cap, kvh, D, n = 1 << 24, 2, 128, 300
    small = Case(16, 8, kvh, D, n, n, 0, True, kind=BINARY, seed=8)
    c = Case(16, 8, kvh, D, n, n, 0, True, kind=BINARY, seed=8).to_device()
    big = [torch.empty(cap * kvh * D, dtype=torch.int16, device="cuda") for _ in range(2)]
    at = cap - 100                        # wraps after 100 rows
    slots = (at + torch.arange(n, device="cuda")) % cap
    for b, src in zip(big, (c.dkey, c.dvalue)):
        b.view(kvh, cap, D)[:, slots] = src.view(kvh, n, D)
    c.plane = mu.KvPlane(big[0].data_ptr(), big[1].data_ptr(), cap, n, 0, at, kvh * D, D, 1, 0)
    c.call().check(small.want())


def test_attention_repeats_bit_for_bit_on_streams_and_in_graphs():
    c = Case(16, 32, 2, 128, 2048, 2048, 777, False, 2048, 4, TWO, 4, gate=True, seed=9).to_device()
    d = Case(1, 32, 2, 128, 1500, 2048, 0, False, 2048, 0, CHAIN, 0, seed=10).to_device()
    want = [t.call().check() for t in (c, d)] and [host(t.out).copy() for t in (c, d)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        c.call(s1)
        d.call(s2)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.out), want[0]) and np.array_equal(host(d.out), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
        d.call()
    c.out[:-16].fill_(float("nan"))
    c.dq.mul_(2.0)                       # a replay reads what the buffers hold then
    g.replay()
    c.q = c.q * 2
    c.check()
    c.dq.mul_(0.5)
    g.replay()
    g.replay()
    assert np.array_equal(host(c.out), want[0]) and np.array_equal(host(d.out), want[1])


def from_two_threads(*calls, times=3000):
    """Runs the calls at the same time, each again and again in a thread of its own; raises what one of them raised."""
    import threading
    errors, start = [], threading.Barrier(len(calls))

    def loop(call):
        try:
            start.wait()
            for _ in range(times):
                call()
                if errors:
                    break
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


def test_attention_of_two_head_sizes_from_two_threads():
    """Head sizes 256 and 136 off the 16-byte grid: one kernel, two amounts of shared memory."""
    cases = [Case(1, 2, 1, D, 5, 8, 0, False, offset=1, seed=22).to_device() for D in (256, 136)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    from_two_threads(*[lambda c=c, s=s: c.call(s) for c, s in zip(cases, streams)])
    for c in cases:
        c.check()


# --------------------------------------------------------------- verification
class Verify:
    def __init__(self, M, V, kind=CHAIN, T=1.0, draft=True, seed=0, close=0.6):
        rng = np.random.default_rng(seed * 31 + V + M)
        self.M, self.V, self.T, self.parent = M, V, T, parents(kind, M)
        self.target = logits(rng, M, V)
        d = (self.target + close * rng.standard_normal((M, V))).astype(np.float32)
        self.tokens = drafted(rng, d, self.parent, T or 0.2)
        self.draft = d if draft else None
        self.u = rng.random(M).astype(np.float32)
        self.u[self.u >= 1] = 0.5
        self.scratch = None

    def want(self):
        return oracle.tree_verify(self.target, self.tokens, self.T, self.u, self.draft, self.parent)

    def run(self, stream=None):
        t, d = dev(self.target), None if self.draft is None else dev(self.draft)
        x, u = dev(self.tokens), dev(self.u)
        r = torch.full((self.M + 2 + 4,), -77, dtype=torch.int32, device="cuda")
        n = mu.muser_tree_verify_scratch_bytes(self.V, self.M)
        if self.scratch is None:
            self.scratch = torch.zeros(n // 4, device="cuda")
        mu.muser_tree_verify(t, d, x, self.parent, self.M, self.V, self.T, u, r, self.scratch, n, stream)
        r = host(r)
        assert np.all(r[self.M + 2:] == -77)
        assert not host(self.scratch[:64]).any()
        return r[:self.M + 2]

    def resolved(self, row, taken):
        """Whether the decisions at `row`, up to its accepted child `taken` (None: to the next token), are above the
        library's resolution.  Its weights are off by at most 2^-37 of themselves and 2^-43 of the row's largest, so a
        drafted token of less than 2^-42 of the largest may have probability 0, and what rejected children leave, sum
        max(p - c q, 0) with c <= M, is known to (1 + M) 2^-37 + V 2^-43: below that nothing may be left.  (Tokens
        drawn from q do not get there: they have that probability, and a rejection has the chance that it leaves.)"""
        if self.draft is None or self.T == 0:
            return True
        p, q = (np.exp((t[row].astype(np.float64) - float(t[row].max())) / self.T) for t in (self.target, self.draft))
        least, p, q = 2.0 ** -42, p / p.sum(), q / q.sum()
        c, z = 0.0, 1.0
        for i in range(1, self.M):
            if self.parent[i] != row:
                continue
            x = int(self.tokens[i])
            if 0 <= x < self.V and (p[x] < least * p.max() or q[x] < least * q.max()):
                return False
            if i == taken:
                return True
            c += z
            z = np.maximum(p - c * q, 0).sum()
            if z < (1 + self.M) * 2.0 ** -37 + self.V * 2.0 ** -43:
                return False
        return True

    def check(self):
        want, got = self.want(), self.run()
        kept = want[2:2 + want[0]].tolist()
        for j, row in enumerate(kept):
            if want[1] >= 0 and not self.resolved(row, kept[j + 1] if j + 1 < len(kept) else None):
                assert np.array_equal(got[2:3 + j], want[2:3 + j]) and 0 <= got[1] < self.V, (got, want)
                return want
        assert np.array_equal(got, want), (got, want)
        return want


@pytest.mark.parametrize("V", [1, 2, 5, 1001, 4096, 50257, 202048])
@pytest.mark.parametrize("M,kind", [(1, CHAIN), (2, CHAIN), (16, CHAIN), (16, BINARY), (8, STAR), (16, TWO)])
@pytest.mark.parametrize("T,draft", [(1.0, True), (0.7, False), (0.0, True)])
def test_verify_against_the_oracle(V, M, kind, T, draft):
    for seed in range(3):
        Verify(M, V, kind, T, draft, seed).check()


def test_verify_takes_every_path():
    """Over many small trees: nothing accepted, all accepted, rejections behind acceptances, siblings after rejections."""
    seen, kept = set(), 0
    for seed in range(60):
        for kind in (CHAIN, STAR, BINARY):
            c = Verify(9, 3000, kind, (1.0, 0.5)[seed % 2], seed % 3 != 2, seed=100 + seed, close=(0.1, 1.5)[seed % 2])
            r = c.check()
            seen.add(int(r[0]))
            kept += r[0]
    assert {1, 2, 3}.issubset(seen) and max(seen) == 9


@pytest.mark.parametrize("u0", [0.0, 1e-30, 2.0 ** -24, 0.5, 1.0 - 2.0 ** -24])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_ends_of_the_unit_interval(u0, draft):
    for M, seed in ((1, 0), (4, 1), (4, 2)):
        c = Verify(M, 1234, STAR, 1.0, draft, seed)
        c.u[0] = u0
        c.u[1:] = 1.0 - 2.0 ** -24
        c.check()


def test_verify_equal_rows_accept_everything():
    c = Verify(16, 7001, CHAIN, 0.8, True, 3)
    c.draft = c.target.copy()
    c.u[1:] = 1.0 - 2.0 ** -24
    assert c.check()[0] == 16


def test_verify_duplicate_and_foreign_tokens():
    for draft in (True, False):
        for seed in range(6):
            c = Verify(8, 40, STAR, 1.0, draft, 50 + seed)
            c.tokens[2] = c.tokens[1]
            c.tokens[3], c.tokens[5] = 40, -3
            c.u[1:] = np.maximum(c.u[1:], 0.9)
            c.check()


@pytest.mark.parametrize("V", [200, 5001, 39999, 50257, 202048])
@pytest.mark.parametrize("rest", [0.6, 0.3, 1e-2, 1e-5, 3e-7])
@pytest.mark.parametrize("T", [1.0, 0.1])
def test_verify_siblings_after_a_nearly_certain_one(V, rest, T):
    """Drafts taken as certain: the first child has all but `rest` of the row and is rejected; its siblings are decided
    against what is left.  Their uniforms lie 2^-14 of the threshold p / left above it, then (one of them) below it; both
    are decided to about 2^-19."""
    M = 7
    rng = np.random.default_rng(V)
    for taken in (2, 3, 6):
        c = Verify(M, V, STAR, T, False, taken)
        c.tokens[1:] = rng.choice(V, M - 1, replace=False)
        if taken == 6:
            c.tokens[2] = min(c.tokens[1] ^ 1, V - 1)    # a neighbour: in the same share of the row
            c.tokens[4] = c.tokens[1]                    # the same again: nothing is left of it
            c.tokens[3] = (c.tokens[2] + V // 2) % V
            c.tokens[5], c.tokens[6] = (c.tokens[1] + V // 3) % V, (c.tokens[1] + V // 5) % V
        z = T * rng.standard_normal(V)
        z[c.tokens[2:]] = T * (4 + rng.random(M - 2))
        z[c.tokens[1]] = -np.inf
        z[c.tokens[1]] = T * (np.log(np.exp(z / T).sum()) + np.log((1 - rest) / rest))
        c.target[0] = z
        p = np.exp((c.target[0].astype(np.float64) - float(c.target[0].max())) / T)
        p /= p.sum()
        left = p.copy()
        c.u[1] = 1 - 2.0 ** -24
        for i in range(1, M):
            x = int(c.tokens[i])
            if i > 1 and left[x] > 0:
                c.u[i] = min(left[x] / left.sum() * (1 + (2.0 ** -14 if i < taken else -2.0 ** -14)), 1 - 2.0 ** -24)
            left[x] = 0.0
        want = c.check()
        assert want[:2].tolist()[0] == 2 and want[3] == taken, want


@pytest.mark.parametrize("V,blocks", [(39999, 16), (50257, 50), (3000, 16), (1000003, 152)])
@pytest.mark.parametrize("rest", [0.3, 1e-3, 2.4e-6, 7e-8])
def test_verify_next_token_after_a_nearly_certain_one(V, blocks, rest):
    """The next token of a row whose nearly certain token was drafted, taken as certain and rejected: the shares of the
    others are as fine as if that token had never been there.  uniform[0] points at the middle of a token's share, for
    tokens behind the rejected one in its block's share of the vocabulary and elsewhere.  (uniform[1] = 1 - 2^-24
    rejects p = 1 - rest; with 7e-8 left they are 1e-8 apart, acceptance is decided to 2^-19 = 1.9e-6: either is right.)"""
    rng = np.random.default_rng(V)
    c = Verify(2, V, CHAIN, 1.0, False, 1)
    z = 0.3 * rng.standard_normal(V)
    span = (V + blocks - 1) // blocks
    x = c.tokens[1] = span * 3 + 5
    z[x] = -np.inf
    z[x] = np.log(np.exp(z).sum()) + np.log((1 - rest) / rest)
    c.target[0] = z
    p = np.exp(c.target[0].astype(np.float64) - float(c.target[0].max()))
    p[x] = 0.0
    total, c.u[1] = np.cumsum(p), 1 - 2.0 ** -24
    for v in [0, V - 1, *rng.integers(x + 1, span * 4, 40).tolist(), *rng.integers(0, V, 10).tolist()]:
        if v != x:
            c.u[0] = (total[v] - p[v] / 2) / total[-1]
            if rest < 2.0 ** -19 and c.run()[0] == 2:
                continue
            assert c.check().tolist() == [1, v, 0, -1]


@pytest.mark.parametrize("V", [3000, 50257, 202048])
@pytest.mark.parametrize("noise", [1e-5, 1e-4, 1e-2])
def test_verify_next_token_where_the_rows_are_nearly_equal(V, noise):
    """A drafter whose logits differ by `noise` (the same model in other numerics): what a rejection leaves is that small,
    and uniform[0] points at the middle of a token's share of it.  A token's weight is off by 2^-37 of itself and 2^-43 of
    the row's largest (at most e^10 of it): 2^-37 / noise + 2^-28.5 / noise of its share, 3e-4 at most, and at random along
    the cumulative sum (450 steps at most for 202,048 tokens: 0.13 of a share)."""
    rng = np.random.default_rng(V)
    c = Verify(2, V, CHAIN, 1.0, True, 2)
    c.target[0] = np.clip(rng.standard_normal(V), -4, 4)
    c.draft[0] = c.target[0] + np.float32(noise) * rng.standard_normal(V).astype(np.float32)
    p, q = (np.exp(t[0].astype(np.float64)) for t in (c.target, c.draft))
    p, q = p / p.sum(), q / q.sum()
    c.tokens[1] = np.argmin(p / q)               # rejected: p / q is 1 - 3 noise, against u = 1 - 2^-24
    c.u[1] = 1 - 2.0 ** -24
    left = np.maximum(p - q, 0)
    total = np.cumsum(left)
    wrong = []
    for v in rng.choice(np.flatnonzero(left > 0.1 * noise / V), 40):
        c.u[0] = (total[v] - left[v] / 2) / total[-1]
        want, got = c.want(), c.run()
        assert want.tolist() == [1, v, 0, -1]
        wrong += [] if np.array_equal(got, want) else [(int(got[1]), int(v))]
    assert not wrong, wrong


@pytest.mark.parametrize("V", [3000, 50257])
@pytest.mark.parametrize("offset", [0.0, 100.0, 900.0])
def test_verify_next_token_where_the_rows_lie_apart(V, offset):
    """The draft's logits lie `offset` lower (the same distribution): at temperature 0.1 the binary32 sums of the rows then
    differ by up to 9,000 log2(e) 2^-25 = 4e-4 of themselves.  The rows differ by 0.02 in logit / temperature; weights are
    good to 2^-33 there, 2^-33 / 0.02 = 6e-9 of a token's share, and a share is at least 1e-6 of the sum."""
    rng = np.random.default_rng(V + 1)
    c = Verify(2, V, CHAIN, 0.1, True, 2)
    c.target[0] = 1000 + 0.1 * np.clip(rng.standard_normal(V), -4, 4)
    c.draft[0] = c.target[0] - offset + 0.002 * rng.standard_normal(V)
    p, q = (np.exp((t[0].astype(np.float64) - float(t[0].max())) / c.T) for t in (c.target, c.draft))
    p, q = p / p.sum(), q / q.sum()
    c.tokens[1] = np.argmin(p / q)
    c.u[1] = 1 - 2.0 ** -24
    left = np.maximum(p - q, 0)
    total = np.cumsum(left)
    wrong = []
    for v in rng.choice(np.flatnonzero(left > 0.1 * left.sum() / V), 40):
        c.u[0] = (total[v] - left[v] / 2) / total[-1]
        want, got = c.want(), c.run()
        assert want.tolist() == [1, v, 0, -1]
        wrong += [] if np.array_equal(got, want) else [(got.tolist(), int(v))]
    assert not wrong, wrong


def test_verify_masked_logits_and_sharp_rows():
    for T in (1.0, 0.05):
        for seed in range(4):
            c = Verify(6, 5000, BINARY, T, True, 70 + seed)
            c.target[:, ::3] = -np.inf
            c.draft[:, ::3] = -np.inf
            c.tokens = drafted(np.random.default_rng(seed), c.draft, c.parent, T)
            c.check()
            c.target *= 30.0
            c.draft *= 30.0
            c.check()
    c = Verify(4, 300, CHAIN, 1.0, True, 80)   # one token has all the mass
    c.target[:] = -np.inf
    c.target[:, 299] = 3.0
    c.draft = c.target.copy()
    c.tokens[:] = 299
    assert c.check().tolist() == [4, 299, 0, 1, 2, 3]


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_verify_rows_that_are_no_distribution(bad):
    for T, draft in ((1.0, True), (1.0, False), (0.0, False)):
        c = Verify(3, 1000, CHAIN, T, draft, 4)
        c.target[0, 998] = bad
        assert c.run().tolist() == [1, -1, 0, -1, -1]
        c = Verify(3, 1000, CHAIN, T, draft, 4)     # a row that the walk does not meet
        want = c.want()
        if want[0] < 3:
            c.target[2, 0] = bad
            assert np.array_equal(c.run(), want)
        c = Verify(1, 1000, CHAIN, T, draft, 4)
        c.target[:] = -np.inf
        assert c.run().tolist() == [1, -1, 0]
    c = Verify(3, 1000, CHAIN, 1.0, True, 4)
    c.draft[0, 5] = bad
    assert c.run().tolist() == [1, -1, 0, -1, -1]
    c = Verify(1, 1000, CHAIN, 1.0, False, 4)       # beyond the range of exponents
    c.target[0, 7] = 6e4
    assert c.run()[1] == -1


@pytest.mark.parametrize("V", [511, 513, 39999, 40000, 40001, 65536])
@pytest.mark.parametrize("kind,draft", [(CHAIN, True), (BINARY, True), (STAR, False)])
def test_verify_where_the_launch_changes(V, kind, draft):
    """Both sides of the sizes at which one cluster gives way to the whole grid, many siblings rejected."""
    for M in (2, 16):
        c = Verify(M, V, kind, 1.0, draft, 40 + M, close=1.5)
        c.check()
        c.u[1:] = np.maximum(c.u[1:], 0.95)
        c.check()


def test_verify_calls_of_all_kinds_share_scratch_in_a_stream():
    cases = [Verify(16, 202048, BINARY, 0.7, True, 6), Verify(5, 9999, STAR, 1.0, False, 7), Verify(1, 32768, CHAIN, 1.0, False, 8),
             Verify(9, 50257, CHAIN, 0.0, False, 9), Verify(16, 3000, STAR, 1.0, True, 10)]
    cases[0].check()
    for c in cases[1:]:
        c.scratch = cases[0].scratch
    wants = [c.want() for c in cases]
    for i in (0, 1, 2, 3, 4, 4, 0, 3, 1, 0, 2, 4, 2, 1, 3):
        assert np.array_equal(cases[i].run(), wants[i]), i


@pytest.mark.parametrize("T,M,draft", [(1e-3, 1, False), (1e6, 1, False), (1e6, 8, True), (1e30, 1, False), (1e30, 8, True),
                                       (1e30, 8, False)])
def test_verify_extreme_temperatures(T, M, draft):
    c = Verify(M, 5000, BINARY, T, draft, 30 + M)
    c.target *= 0.5                     # at T = 0.001 within the range of exponents
    c.target[:, 1::2] = -np.inf
    if draft:
        c.draft[:, 1::2] = -np.inf
    c.tokens = drafted(np.random.default_rng(M), c.draft if draft else c.target, c.parent, T)
    c.check()


def test_verify_of_two_vocabularies_from_two_threads():
    """2^20 and 500,000 tokens: one kernel, two amounts of shared memory."""
    cases, calls = [Verify(1, V, CHAIN, 1.0, False, 8) for V in (1 << 20, 500000)], []
    for c in cases:
        c.args = dev(c.target), dev(c.tokens), dev(c.u), torch.full((3,), -77, dtype=torch.int32, device="cuda")
        c.n = mu.muser_tree_verify_scratch_bytes(c.V, 1)
        c.scratch, s = torch.zeros(c.n // 4, device="cuda"), torch.cuda.Stream()
        calls.append(lambda c=c, s=s: mu.muser_tree_verify(c.args[0], None, c.args[1], None, 1, c.V, c.T, c.args[2],
                                                           c.args[3], c.scratch, c.n, s))
    torch.cuda.synchronize()
    from_two_threads(*calls)
    for c in cases:
        assert np.array_equal(host(c.args[3]), c.want())


def test_verify_greedy_ties_take_the_lowest_index():
    c = Verify(3, 202048, CHAIN, 0.0, False, 1)
    c.target[:, [5, 77, 150000, 202047]] = 50.0
    c.tokens[:] = [0, 5, 77]
    assert c.check().tolist() == [2, 5, 0, 1, -1]


def test_verify_scratch_streams_and_graphs():
    a, b = Verify(16, 202048, BINARY, 0.7, True, 6), Verify(5, 9999, STAR, 1.0, False, 7)
    wa, wb = a.check(), b.check()
    for _ in range(3):                       # the counters are back at zero after every call
        assert np.array_equal(a.run(), wa) and np.array_equal(b.run(), wb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t, d, x, u = dev(a.target), dev(a.draft), dev(a.tokens), dev(a.u)
    r = torch.full((18,), -77, dtype=torch.int32, device="cuda")
    n = mu.muser_tree_verify_scratch_bytes(a.V, a.M)
    torch.cuda.synchronize()
    mu.muser_tree_verify(t, d, x, a.parent, a.M, a.V, a.T, u, r, a.scratch, n, s)
    s.synchronize()
    assert np.array_equal(host(r), wa)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mu.muser_tree_verify(t, d, x, a.parent, a.M, a.V, a.T, u, r, a.scratch, n)
    u.copy_(torch.rand(16, device="cuda"))
    for _ in range(2):
        r.fill_(-77)
        g.replay()
        a.u = host(u)
        assert np.array_equal(host(r), a.want())
    assert mu.muser_device_status() == 0


# -------------------------------------------------------------------- commit
@pytest.mark.parametrize("kvh,D,offset", [(2, 128, 0), (3, 5, 0), (2, 40, 0), (1, 64, 1)])
@pytest.mark.parametrize("M,path", [(1, [0]), (16, [0, 3, 4, 9, 15]), (16, list(range(16))), (6, [5]), (4, [])])
def test_commit_is_bit_exact(kvh, D, offset, M, path):
    rng = np.random.default_rng(M + len(path))
    kv, position = kvh * D, 37
    planes, rings, bufs, ks, vs = [], [], [], [], []
    for cap, hm in ((64, False), (37, True), (5, False), (40, True), (1, False)):
        n = min(cap, position)
        ring, key, value = plane(rng, cap, kvh, D, n, position - n, hm)
        kbuf, vbuf = (torch.full((offset + t.size + 24,), 0x7777, dtype=torch.int16, device="cuda") for t in (key, value))
        kbuf[offset:offset + key.size] = to_dev16(key)
        vbuf[offset:offset + key.size] = to_dev16(value)
        planes.append(kv_plane(ring, kbuf[offset:], vbuf[offset:], kvh, D, hm))
        rings.append(ring)
        bufs.append((kbuf, vbuf, key, value, hm))
        k, v = ((100 * rng.standard_normal((M, kv))).astype(np.float32) for _ in range(2))
        k[:, 0], v[:, -1] = 1e6, -1e6                  # beyond binary16: infinities
        ks.append(k)
        vs.append(v)
    dk, dv = [dev(k) for k in ks], [dev(v) for v in vs]
    mu.muser_kv_tree_commit(planes, dk, dv, M, path, position)
    for p, ring, (kbuf, vbuf, key, value, hm), k, v in zip(planes, rings, bufs, ks, vs):
        for j, i in enumerate(path):
            assert oracle.kv_write(ring, key, value, kv, D, hm, k[i:i + 1], v[i:i + 1], position + j)[0] == 0
        assert (p.len, p.origin_logical, p.origin_physical) == (ring.len, ring.origin_logical, ring.origin_physical)
        for buf, want in ((kbuf, key), (vbuf, value)):
            got = host(buf).view(np.uint16)
            assert np.array_equal(got[offset:offset + want.size], want)
            assert np.all(got[:offset] == 0x7777) and np.all(got[offset + want.size:] == 0x7777)


def test_commit_of_128_planes_continues_the_rings():
    rng = np.random.default_rng(1)
    kv, cap, L = 256, 48, 128
    key, value = (torch.zeros(L, cap, kv, dtype=torch.int16, device="cuda") for _ in range(2))
    planes = (mu.KvPlane * L)(*[mu.KvPlane(key[l].data_ptr(), value[l].data_ptr(), cap, 0, 0, 0, kv, 128, 0, 0)
                                for l in range(L)])
    ring = oracle.Ring(cap, 0, 0, 0)
    okey, oval = np.zeros(cap * kv, np.uint16), np.zeros(cap * kv, np.uint16)
    position = 0
    for step in range(20):
        M = int(rng.integers(1, 17))
        path = sorted(rng.choice(M, int(rng.integers(1, M + 1)), replace=False).tolist())
        k, v = synth.kv_rows(M, kv, seed=5, step=step)
        dk, dv = dev(k), dev(v)
        mu.muser_kv_tree_commit(planes, [dk] * L, [dv] * L, M, path, position)
        assert oracle.kv_write(ring, okey, oval, kv, 128, False, k[path], v[path], position)[0] == 0
        position += len(path)
    for l in (0, 77, 127):
        assert (planes[l].len, planes[l].origin_logical) == (ring.len, ring.origin_logical)
        assert np.array_equal(host(key[l]).reshape(-1).view(np.uint16), okey)
        assert np.array_equal(host(value[l]).reshape(-1).view(np.uint16), oval)


# ------------------------------------------------------------- the whole step
class Model:
    """Two attention-only layers over 512 tokens: one sliding-window ring with a kept first token, one growing plane."""
    H, KVH, D, HID, VOCAB, WINDOW, SINKS, CAP = 4, 2, 128, 512, 512, 24, 1, 24

    def __init__(self, seed=0):
        self.emb = torch.randn(self.VOCAB, self.HID, generator=torch.Generator().manual_seed(seed)).cuda()
        rows = (self.H * self.D, self.KVH * self.D, self.KVH * self.D, self.H * self.D)
        self.rows = rows
        self.w = [[dev(synth.q4k_matrix(r, self.HID, seed=seed, workload=9, layer=l, tensor=synth.T_WQ + i))
                   for i, r in enumerate(rows)] for l in range(2)]
        self.wo = [dev(synth.q4k_matrix(self.HID, self.H * self.D, seed=seed, workload=9, layer=l, tensor=synth.T_WO))
                   for l in range(2)]
        self.lm = dev(synth.q4k_matrix(self.VOCAB, self.HID, seed=seed, workload=9, layer=3, tensor=synth.T_WQ))
        self.ones = torch.ones(self.HID, device="cuda")
        kv = self.KVH * self.D
        self.buf = [torch.full((c * kv,), 0x7E00, dtype=torch.int16, device="cuda")
                    for c in (self.CAP, self.CAP, 256, 256, self.SINKS, self.SINKS)]
        b = [t.data_ptr() for t in self.buf]
        self.planes = (mu.KvPlane * 2)(mu.KvPlane(b[0], b[1], self.CAP, 0, 0, 0, kv, self.D, 0, 0),
                                       mu.KvPlane(b[2], b[3], 256, 0, 0, 0, kv, self.D, 1, 0))
        self.sink = mu.KvPlane(b[4], b[5], self.SINKS, 0, 0, 0, kv, self.D, 0, 0)
        n = max(mu.muser_kv_tree_attention_scratch_bytes(kv, self.D, M, self.H) for M in range(1, 17))
        self.ascr, self.an = torch.zeros(n // 4, device="cuda"), n
        n = mu.muser_tree_verify_scratch_bytes(self.VOCAB, 16)
        self.vscr, self.vn = torch.zeros(n // 4, device="cuda"), n
        self.position = 0

    def step(self, tokens, parent, T=0.0, uniform=None, draft=None):
        """One pass over the rows `tokens`; returns the kept rows' tokens and the next one."""
        M = len(tokens)
        resid = self.emb[torch.tensor(tokens, device="cuda")].contiguous()
        x = torch.empty(M, self.HID, device="cuda")
        mu.muser_rms_norm(resid, self.ones, x, self.HID, M, 1e-5)
        ks, vs = [], []
        for l in range(2):
            q, k, v, gate = (torch.empty(M, r, device="cuda") for r in self.rows)
            mu.muser_qmatvec_group("q4_k", self.w[l], self.rows, self.HID, x, M, [q, k, v, gate])
            q, k, v, gate = (t / t.pow(2).mean(1, keepdim=True).sqrt() for t in (q, k, v, gate))
            a = torch.empty(M, self.H * self.D, device="cuda")
            mu.muser_kv_tree_attention(self.planes[l], q, k, v, M, self.H, a, self.D ** -0.5, self.ascr, self.an, parent,
                                       self.WINDOW if l == 0 else 0, self.SINKS if l == 0 else 0,
                                       self.sink if l == 0 else None, gate)
            proj, nx = torch.empty(M, self.HID, device="cuda"), torch.empty(M, self.HID, device="cuda")
            mu.muser_qmatvec("q4_k", self.wo[l], self.HID, self.H * self.D, a, M, proj)
            mu.muser_fused_residual_dual_rmsnorm(resid, proj, nx, self.ones, self.ones, self.HID, M, 1e-8, 1e-5)
            x = nx - nx.mean(1, keepdim=True)   # the weights' mean is positive: without it all logits are alike
            ks.append(k)
            vs.append(v)
        logit = torch.empty(M, self.VOCAB, device="cuda")
        mu.muser_lm_head("q4_k", self.lm, self.VOCAB, self.HID, x, M, logit, 0.1, 20.0)
        self.logits = logit
        r = torch.empty(M + 2, dtype=torch.int32, device="cuda")
        mu.muser_tree_verify(logit, draft, torch.tensor(tokens, dtype=torch.int32, device="cuda"), parent, M, self.VOCAB, T,
                             torch.zeros(M, device="cuda") if uniform is None else uniform, r, self.vscr, self.vn)
        r = r.tolist()
        path = r[2:2 + r[0]]
        if self.position < self.SINKS:
            mu.muser_kv_ring_write(self.sink, ks[0][:1].contiguous(), vs[0][:1].contiguous(), self.position, 1)
        mu.muser_kv_tree_commit(self.planes, ks, vs, M, path, self.position)
        self.position += len(path)
        return [tokens[i] for i in path], r[1]


def test_speculative_greedy_decoding_gives_the_tokens_of_plain_decoding():
    plain, want, t = Model(), [], 17
    for _ in range(60):
        kept, t = plain.step([t], None)
        top = plain.logits[0].topk(2).values
        assert float(top[0] - top[1]) > 2e-4, "the tokens are too close to be compared over two kernels"
        want.append(t)
    rng = np.random.default_rng(0)
    spec, got, t = Model(), [], 17
    sizes = []
    while len(got) < 60:
        M = int(rng.integers(1, 17))
        parent = parents((CHAIN, BINARY, TWO)[len(sizes) % 3], M)
        depth = [0] * M
        for i in range(1, M):
            depth[i] = depth[parent[i]] + 1
        # drafts: mostly the tokens that will come, some others
        tokens = [t] + [want[len(got) + depth[i] - 1] if len(got) + depth[i] <= 60 and rng.random() < 0.8
                        else int(rng.integers(0, 512)) for i in range(1, M)]
        kept, t = spec.step(tokens, parent)
        got += kept[1:] + [t]
        sizes.append(len(kept))
    assert got[:60] == want
    assert max(sizes) > 2 and spec.position == sum(sizes)
