"""Several sequences at once on the GPU against the fp64 oracle: page tables, copies and stores of pages, attention over
a paged cache, beam selection, and all of them together."""
import ctypes

import numpy as np
import pytest

from oracle import paged
from tests.gpu_util import check_canary, dev, host, nan_like
from tests.paged_util import NAN16, Cache, attention_bound, tables

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import quantized_weight_streaming_q4_gb300 as mu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mu.build()
    mu.lib()
    torch.cuda.init()


def ints(a):
    return dev(np.asarray(a, np.int32))


def to_dev16(a):
    return dev(a.view(np.int16))


# --------------------------------------------------------------- page tables
def run_tables(table, length, parent, add, pages, R, window=0, n_sink=0, max_new=4096, copies=True, in_place=False, lists=True):
    n = len(parent) if parent is not None else len(length)
    stride = table.shape[1]
    d = dict(table=ints(table), length=ints(length))
    if in_place:
        tout, lout = d["table"], d["length"]
    else:
        tout = torch.full((n, stride), -7, dtype=torch.int32, device="cuda")
        lout = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    o = {x: torch.full((m + 4,), -7, dtype=torch.int32, device="cuda")
         for x, m in (("last", n), ("first", n + 1), ("slots", max_new), ("position", max_new), ("sequence", max_new),
                      ("copies", 3 * n), ("result", 8))}
    names = ("slots", "position", "sequence") if lists else ()
    mu.muser_kv_page_tables(d["table"], d["length"], n, pages, R, tout, lout, o["result"],
                            parent=None if parent is None else ints(parent), add=None if add is None else ints(add),
                            window=window, n_sink=n_sink, last=o["last"], first=o["first"], max_new=max_new,
                            copies=o["copies"] if copies else None, **{x: o[x] for x in names})
    want = paged.page_tables(table, length, parent, add, pages, R, window, n_sink, max_new if lists else None, copies)
    got = {x: host(t) for x, t in o.items()}
    assert list(got["result"]) == want["result"] + [-7] * 4
    t = host(tout)
    for i in range(n):
        for k in range(stride):
            e = want["table"][i][k]
            assert t[i, k] == ((table[i, k] if in_place else -7) if e is None else e), (i, k)
    assert list(host(lout)) == want["length"]
    assert list(got["last"][:n]) == want["last"] and list(got["first"][:n + 1]) == want["first"]
    for x in names:
        assert list(got[x]) == want[x] + [-1] * (max_new - len(want[x])) + [-7] * 4, x
    flat = [y for c in want["copies"] for y in c]
    assert list(got["copies"]) == flat + [-7] * (3 * n + 4 - len(flat))
    return want


@pytest.mark.parametrize("seed", range(24))
def test_tables(seed):
    rng = np.random.default_rng(seed)
    n_old = int(rng.choice([1, 2, 5, 16, 33, 256]))
    R = int(rng.choice([1, 3, 16, 64]))
    stride = int(rng.integers(2, 40))
    length = rng.integers(0, stride * R // 2 + 1, n_old)
    pages = int((-(-length // R)).sum() + rng.integers(1, 2 * n_old + 40))
    table = tables(rng, length, R, pages, stride)
    parent = None
    if seed % 3:
        n = int(rng.choice([1, 7, 33, n_old]))
        parent = np.sort(rng.integers(-1, n_old, n)).astype(np.int32)
        if seed % 3 == 2:
            rng.shuffle(parent)
    n = n_old if parent is None else len(parent)
    add = None if seed % 4 == 0 else rng.integers(-R - 1, 2 * R + 2, n)
    window = int(rng.choice([0, 0, 1, R + 1, 3 * R]))
    run_tables(table, length, parent, add, pages, R, window, int(rng.choice([0, 1, R])) if window else 0,
               in_place=parent is None and seed % 2 == 0, copies=True)


@pytest.mark.parametrize("kw", [
    dict(add=[500, 0]), dict(add=[5, 5], max_new=9), dict(add=[60, 60]), dict(parent=[0, 0], add=[1, 2147483647]),
    dict(parent=[1, 1, 0, -1, 9], add=[1, 1, -3, 2, -5]), dict(add=[-2147483648, 2]), dict(parent=[-1, -1], add=[0, 0]),
    dict(add=[4, 4], lists=False, max_new=0),
])
def test_tables_edges(kw):
    table = np.array([[3, 1, -1, -1, -1, -1, -1, -1], [0, 2, 4, -1, -1, -1, -1, -1]], np.int32)
    run_tables(table, [6, 10], kw.pop("parent", None), kw.pop("add"), 12, 4, **kw)


def test_tables_without_copies_refuse_a_shared_page():
    table = np.array([[3, 1, -1], [3, 1, -1]], np.int32)  # two sequences in one partly filled page, no parents
    want = run_tables(table, [6, 6], None, None, 6, 4, copies=False)
    assert want["result"][0] == 4
    assert run_tables(table, [6, 6], None, None, 6, 4)["copies"] == [(1, 0, 2)]


def test_tables_entries_outside_the_cache_hold_nothing():
    table = np.array([[3, 77, -5, -1], [0, 2, 1, -1]], np.int32)
    run_tables(table, [10, 9], None, [2, 2], 6, 4)     # sequence 0 goes on in a page that is not there: a new one
    run_tables(table, [10, 9], [0, 1, 0], [0, -1, 5], 12, 4)


def test_tables_of_many_rows_on_a_cluster():
    rng = np.random.default_rng(1)
    R, stride, n = 16, 400, 48
    length = rng.integers(0, 4000, n)
    pages = 40000
    table = tables(rng, length, R, pages, stride)
    run_tables(table, length, None, rng.integers(1, 2000, n), pages, R, max_new=100000)
    run_tables(table, length, np.sort(rng.integers(0, n, n)), None, pages, R, max_new=20000)
    run_tables(table, length, None, None, pages, R, lists=False, max_new=0, in_place=True)
    run_tables(table, length, None, rng.integers(1, 2000, n), pages, R, max_new=10000)  # too many


def test_tables_of_the_most_pages():
    R, pages = 1, 1 << 20
    table = np.full((2, 8), -1, np.int32)
    table[0, :2] = pages - 1, 0
    run_tables(table, [2, 0], None, [3, 6], pages, R)


# ---------------------------------------------------------------- copy, write
@pytest.mark.parametrize("G,D,R", [(2, 128, 64), (5, 64, 16), (3, 5, 7), (2, 40, 8), (1, 1, 1)])
@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("layers", [1, 3, 70])
def test_copy(G, D, R, hm, layers):
    rng = np.random.default_rng(G * D + R)
    pages = 12
    bufs = rng.integers(0, 1 << 16, (2 * layers, pages * R * G * D)).astype(np.uint16)
    d = to_dev16(bufs)
    row = d[0].numel() * 2
    caches = [mu.KvPages(d.data_ptr() + l * row, d.data_ptr() + (layers + l) * row, pages, R, G * D, D, int(hm), 0) for l in range(layers)]
    copies = [(0, 5, R), (0, 6, 1), (3, 7, max(1, R // 2)), (1, 99, R), (-1, 8, R), (2, 9, 0), (2, 10, -4), (4, 11, R + 9), (1, 2, 1)]
    mu.muser_kv_page_copy(caches, ints(np.array(copies)), ints([8]), len(copies))  # the last one is behind the count
    want = bufs.reshape(2 * layers, pages, *((G, R, D) if hm else (1, R, G * D))).copy()
    for s, t, m in copies[:8]:
        if 0 <= s < pages and 0 <= t < pages and m > 0:
            want[:, t, :, :m] = want[:, s, :, :m]
    assert np.array_equal(host(d).view(np.uint16), want.reshape(2 * layers, -1))
    mu.muser_kv_page_copy(caches, ints(np.array([(5, 0, R)] * 2)), ints([-3]), 2)  # no copies
    mu.muser_kv_page_copy(caches, ints(np.array([(5, 1, R)])), ints([9]), 1)       # no more than max_copies
    want[:, 1] = want[:, 5]
    assert np.array_equal(host(d).view(np.uint16), want.reshape(2 * layers, -1))


@pytest.mark.parametrize("G,D,R,offset", [(2, 128, 64, 0), (5, 64, 16, 0), (3, 5, 7, 0), (2, 40, 8, 1), (2, 128, 64, 1), (1, 8, 1, 0)])
@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("rows", [1, 17, 300])
def test_write(G, D, R, offset, hm, rows):
    rng = np.random.default_rng(rows + D)
    pages = rows // R + 4
    slots = rng.permutation(pages * R)[:rows].astype(np.int32)
    slots[rng.random(rows) < 0.1] = -1
    slots[rng.random(rows) < 0.05] = pages * R
    k, v = (rng.standard_normal((rows, G * D)).astype(np.float32) for _ in range(2))
    k[0, 0], v[0, 0], k[0, -1] = 1e6, float("nan"), 2.0 ** -25  # overflow, NaN, a tie at the smallest number
    cache = Cache(rng, np.zeros((1, 1), np.int32), [0], pages, R, G, D, hm, 0x1234)
    pad = np.zeros(offset, np.float32)
    dk, dv = (dev(np.concatenate([pad, x.reshape(-1)]))[offset:] for x in (k, v))
    key, value = (to_dev16(b) for b in cache.bufs)
    mu.muser_kv_page_write(mu.KvPages(key.data_ptr(), value.data_ptr(), pages, R, G * D, D, int(hm), 0), dk, dv, ints(slots), rows)
    with np.errstate(over="ignore"):
        want = cache.with_rows([(s // R, s % R) if 0 <= s < pages * R else None for s in slots], k, v)
    for got, w in zip((key, value), want):
        g, w = host(got).view(np.float16), w.view(np.float16)
        assert np.array_equal(g[~np.isnan(w)], w[~np.isnan(w)]) and np.isnan(g[np.isnan(w)]).all()


# ------------------------------------------------------------------ attention
class Case:
    def __init__(self, lengths, H, G, D, R, hm, window=0, n_sink=0, gate=False, own=True, sequence=None, seed=0, qscale=1.5,
                 fill=NAN16, offset=0, stride=None):
        rng = np.random.default_rng(seed * 1000 + len(lengths) * 17 + H + D + R)
        self.H, self.G, self.D, self.R, self.hm, self.window, self.n_sink = H, G, D, R, hm, window, n_sink
        self.scale, self.own, self.offset = D ** -0.5, own, offset
        self.position = np.array(lengths, np.int32)     # rows before the token's own
        rows = [max(0, t + 1) for t in lengths]
        if sequence is not None:                        # several rows of a sequence: its pages hold the longest one's
            self.sequence = np.array(sequence, np.int32)
            n_tables = max(1, int(self.sequence.max()) + 1)
            rows = [max([r for r, s in zip(rows, sequence) if s == i], default=0) for i in range(n_tables)]
        else:
            self.sequence = None
        held = sum(-(-r // R) for r in rows)
        self.pages = held + 3
        stride = max(-(-r // R) for r in rows) + 1 if stride is None else stride
        self.table = tables(rng, rows, R, self.pages, stride)
        filled = [r - 1 if own and r else r for r in rows]  # the slot of a row that is given holds nothing yet
        self.cache = Cache(rng, self.table, filled, self.pages, R, G, D, hm, fill)
        n = len(lengths)
        self.n = n
        self.q = (qscale * rng.standard_normal((n, H * D))).astype(np.float32)
        self.k, self.v = (rng.standard_normal((n, G * D)).astype(np.float32) if own else None for _ in range(2))
        self.gate = rng.standard_normal((n, H * D)).astype(np.float32) if gate else None

    def to_device(self):
        o = self.offset
        self.dbufs = []
        for b in self.cache.bufs:
            t = torch.zeros(b.size + 8, dtype=torch.int16, device="cuda")[o:o + b.size]
            t.copy_(to_dev16(b))
            self.dbufs.append(t)
        self.handle = mu.KvPages(self.dbufs[0].data_ptr(), self.dbufs[1].data_ptr(), self.pages, self.R, self.G * self.D, self.D,
                                 int(self.hm), 0)
        self.dq = dev(self.q)
        self.dk, self.dv, self.dgate = (None if x is None else dev(x) for x in (self.k, self.v, self.gate))
        self.dtable, self.dposition = ints(self.table), ints(self.position)
        self.dsequence = None if self.sequence is None else ints(self.sequence)
        self.nbytes = mu.muser_kv_paged_attention_scratch_bytes(self.G * self.D, self.D, self.n, self.H)
        self.scratch = torch.zeros(self.nbytes // 4 + 4, device="cuda")
        self.scratch[self.nbytes // 4:] = 12345.0
        self.out = nan_like((self.n, self.H * self.D), 16)
        return self

    def call(self, stream=None):
        mu.muser_kv_paged_attention(self.handle, self.dtable, self.dposition, self.dq, self.n, self.H, self.out, self.scale,
                                    self.scratch, self.nbytes, k=self.dk, v=self.dv, gate=self.dgate, sequence=self.dsequence,
                                    window=self.window, n_sink=self.n_sink, stream=stream)
        return self

    def want(self):
        return paged.paged_attention(self.cache.key, self.cache.value, self.pages, self.R, self.G, self.D, self.hm, self.table,
                                     self.position, self.q, self.H, self.scale, self.k, self.v, self.gate, self.sequence,
                                     self.window, self.n_sink)

    def check(self, kmax=5.0):
        size = self.n * self.H * self.D
        got = host(self.out)[:size].reshape(self.n, -1)
        check_canary(self.out, size)
        check_canary(self.scratch, self.nbytes // 4)
        assert not host(self.scratch)[:512].any(), "the tickets are left zero"
        want, stored = self.want()
        vmax = np.abs(self.v).max() if self.own else 0
        f = self.cache.value.astype(np.float32)
        vmax = max(1.0, vmax, np.abs(f[np.isfinite(f)]).max(initial=0))
        bound = attention_bound(self.q, self.scale, kmax, self.D, vmax)
        for i, w in enumerate(want):
            if w is None:
                assert np.isnan(got[i]).all(), f"row {i} was written"
                continue
            assert np.isfinite(got[i]).all(), f"row {i}: {(~np.isfinite(got[i])).sum()} outputs are not finite"
            err = np.abs(got[i].astype(np.float64) - w)
            assert err.max() <= bound, (i, err.max(), bound)
            # binary32: outputs of random sign do not add their errors up
            assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(w) + 1e-30, (i, np.linalg.norm(err) / np.linalg.norm(w))
        for d, w in zip(self.dbufs, self.cache.with_rows(stored, self.k, self.v)):
            assert np.array_equal(host(d).view(np.uint16), w)
        assert mu.muser_device_status() == 0


SHAPES = [  # heads, K/V heads, head_dim
    (32, 2, 128), (4, 4, 64), (20, 5, 64), (6, 2, 80), (3, 1, 256), (8, 2, 136), (6, 3, 5), (9, 1, 8), (2, 1, 72), (26, 1, 128),
    (40, 1, 200), (20, 2, 32),
]


@pytest.mark.parametrize("H,G,D", SHAPES)
@pytest.mark.parametrize("lengths", [[0], [1], [37], [127, 128, 129], [700], [5, 0, 300, -1, 64, 63], list(range(0, 170, 10))],
                         ids=lambda x: str(len(x)) + "x" + str(max(x)))
@pytest.mark.parametrize("hm", [False, True])
def test_attention(H, G, D, lengths, hm):
    Case(lengths, H, G, D, 16 if hm else 64, hm, gate=len(lengths) % 2 == 0).to_device().call().check()


@pytest.mark.parametrize("R", [1, 3, 8, 16, 32, 48, 128, 256, 1024])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_page_sizes(R, own, D):
    Case([0, 130, 517, 255, 256], 8, 2, D, R, own, own=own).to_device().call().check()


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (40, 0), (128, 4), (129, 130), (300, 16), (1000, 700), (5000, 7), (0, 9)])
@pytest.mark.parametrize("R,H,G,D", [(16, 32, 2, 128), (64, 20, 5, 64), (7, 4, 2, 24), (256, 8, 2, 256)])
def test_attention_windows(window, n_sink, R, H, G, D):
    for own in (True, False):
        Case([0, 39, 40, 700, 1500, 128], H, G, D, R, R == 16, window, n_sink, own=own).to_device().call().check()


@pytest.mark.parametrize("lengths", [[20000], [20000, 3, 9000], [4000] * 16, [130, 131] * 40, list(range(1, 257))],
                         ids=["one", "three", "even", "many", "256"])
@pytest.mark.parametrize("H,G,D,R", [(16, 1, 128, 64), (2, 1, 64, 16), (4, 2, 40, 32), (2, 1, 20, 64), (2, 1, 256, 128)])
def test_attention_splits(lengths, H, G, D, R):
    Case(lengths, H, G, D, R, False).to_device().call().check()


@pytest.mark.parametrize("D", [128, 64, 256, 12])
def test_attention_rows_of_one_sequence_in_one_call(D):
    """A prompt's rows, stored first: row i sees rows 0..i of its sequence."""
    seq = [0] * 20 + [1] * 7 + [3] * 3 + [-1, 4, 9]
    lengths = list(range(100, 120)) + list(range(7)) + [300, 299, 298] + [5, 6, 7]
    c = Case(lengths, 4, 2, D, 16, True, own=False, sequence=seq)
    c.table = c.table[:5]
    c.to_device().call().check()


@pytest.mark.parametrize("fill", [0x7E00, 0x7C00, 0xFC00, 0x7BFF])
@pytest.mark.parametrize("D", [128, 64, 256, 12])
def test_attention_unseen_slots_have_no_influence(fill, D):
    Case([5, 300, 0, 129], 8, 2, D, 64, False, window=100, n_sink=3, fill=fill).to_device().call().check()
    c = Case([5, 300, 0, 700], 8, 2, D, 16, True, window=100, n_sink=3, fill=fill)
    table = c.table.copy()
    view = [b.reshape(c.pages, -1) for b in c.cache.bufs]
    for i, t in enumerate(c.position):                 # pages before the window are others', or gone
        for k in range(t // 16):
            if (k + 1) * 16 <= t - 99 and k * 16 >= 3:
                for b in view:
                    b[table[i, k]] = fill
                table[i, k] = (-1, 1 << 30, -2147483648)[k % 3]
    c.table = table
    c.to_device().call().check()


@pytest.mark.parametrize("D", [128, 12])
def test_attention_pages_that_are_not_there(D):
    c = Case([200, 40, 90, 10], 4, 2, D, 16, False)
    c.table[0, 3] = -1                    # rows 48..63 are not seen
    c.table[1, :3] = (-1, 99999, -1)      # nothing but itself, and it is not stored
    c.table[2, 5] = 1 << 30               # the new row's page
    c.to_device().call().check()
    c = Case([200, 40, 90, 10], 4, 2, D, 16, False, own=False)
    c.table[1, :3] = -1                   # sees nothing: zeros
    c.to_device().call().check()
    assert not host(c.out)[:c.n * 4 * D].reshape(4, -1)[1].any()
    c = Case([200, 40, 90, 10], 4, 2, D, 16, False, stride=13)
    c.table = np.ascontiguousarray(c.table[:, :4])  # positions beyond the table's stride
    c.to_device().call().check()


@pytest.mark.parametrize("window", [(1 << 30) - 30, 1 << 30, (1 << 30) + 7, (1 << 31) - 40, (1 << 31) - 1, 1 << 31, 1 << 40, 0])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("D", [128, 12])
def test_attention_positions_far_behind_the_table(D, own, window):
    """Up to the largest int32: which of the table's rows the window reaches goes by the position itself."""
    far = [64, (1 << 30) - 31, (1 << 30) - 2, (1 << 30) - 1, 1 << 30, (1 << 30) + 20, (1 << 31) - 41, (1 << 31) - 2, (1 << 31) - 1]
    c = Case([64] * len(far), 4, 2, D, 16, False, window, 5 if window else 0, own=own)
    c.table = np.ascontiguousarray(c.table[:, :4])  # 64 rows
    c.position = np.array(far, np.int32)
    c.to_device().call().check()


@pytest.mark.parametrize("D", [128, 12])
@pytest.mark.parametrize("what", [0x7C00, 0xFC00, 0x7E00])
def test_attention_rows_that_are_seen_and_not_finite(D, what):
    """An infinite or NaN value makes its outputs not finite, and no others."""
    c = Case([200, 40], 4, 2, D, 16, False)
    c.cache.bufs[1].reshape(c.pages, 16, 2, D)[c.table[0, 5], 3, 1, 2] = what  # V of row 83, head 1, element 2
    c.to_device().call()
    got = host(c.out)[:2 * 4 * D].reshape(2, 4, D)
    assert not np.isfinite(got[0, 2:, 2]).any()
    got[0, 2:, 2] = 0
    assert np.isfinite(got).all()
    c = Case([200, 40], 4, 2, D, 16, False)
    c.k[1, :] = np.inf if what == 0x7C00 else np.nan                            # the token's own key
    if what != 0xFC00:
        c.to_device().call()
        got = host(c.out)[:2 * 4 * D].reshape(2, 4, D)
        assert not np.isfinite(got[1]).any() and np.isfinite(got[0]).all()


@pytest.mark.parametrize("H,G,D,R", [(32, 2, 128, 64), (20, 5, 64, 16), (4, 2, 20, 5), (8, 2, 256, 32)])
def test_attention_large_and_growing_scores(H, G, D, R):
    """References move: keys grow along the sequence, so that every tile raises the maximum."""
    c = Case([900, 300], H, G, D, R, False, qscale=6.0)
    f = c.cache.key.reshape(c.pages, R, G * D)
    for i, t in enumerate(c.position):
        for p in range(t):
            row = f[c.table[i, p // R], p % R]
            row[:] = (row * (0.2 + 3.0 * p / t)).astype(np.float16)
    c.to_device().call().check(kmax=16.0)


@pytest.mark.parametrize("D", [128, 12])
def test_attention_without_any_work(D):
    Case([-1, -1, -5], 4, 2, D, 16, False).to_device().call().check()


def test_attention_same_positions_same_bits():
    c = Case([5000, 77, 1300, 9000], 32, 2, 128, 64, False).to_device().call()
    first = host(c.out).copy()
    for _ in range(5):
        c.out.fill_(float("nan"))
        c.out[c.n * 32 * 128:] = 12345.0
        c.call()
        assert np.array_equal(host(c.out), first)


def test_attention_other_streams_and_unaligned_caches():
    s = torch.cuda.Stream()
    c = Case([300, 2, 90], 32, 2, 128, 64, False).to_device()
    s.wait_stream(torch.cuda.current_stream())
    c.call(stream=s)
    s.synchronize()
    c.check()
    Case([300, 2, 90], 32, 2, 128, 64, False, offset=1).to_device().call().check()  # 2-byte aligned buffers
    Case([300, 2, 90], 32, 2, 128, 64, True, offset=4).to_device().call().check()


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("D", [128, 20])
def test_offsets_beyond_32_bits(hm, D):
    """A cache of 2^32 bytes and more: the last pages are written, copied and read."""
    G, H, R = 2, 8, 64
    pages = (1 << 32) // (R * G * D * 2) + 9
    rng = np.random.default_rng(7)
    n = 150
    key, value = (torch.empty(pages * R * G * D, dtype=torch.int16, device="cuda") for _ in range(2))
    handle = mu.KvPages(key.data_ptr(), value.data_ptr(), pages, R, G * D, D, int(hm), 0)
    table = np.array([[pages - 1, pages - 4, pages - 6]], np.int32)
    slots = ints([table[0, p // R] * R + p % R for p in range(n)])
    k, v = (rng.standard_normal((n, G * D)).astype(np.float32) for _ in range(2))
    mu.muser_kv_page_write(handle, dev(k), dev(v), slots, n)
    mu.muser_kv_page_copy([handle], ints([[pages - 6, pages - 2, n - 2 * R]]), ints([1]), 1)
    table[0, 2] = pages - 2
    q = rng.standard_normal((1, H * D)).astype(np.float32)
    nk, nv = (rng.standard_normal((1, G * D)).astype(np.float32) for _ in range(2))
    nb = mu.muser_kv_paged_attention_scratch_bytes(G * D, D, 1, H)
    out = torch.empty(H * D, device="cuda")
    mu.muser_kv_paged_attention(handle, ints(table), ints([n]), dev(q), 1, H, out, 0.3, torch.zeros(nb // 4, device="cuda"), nb,
                                k=dev(nk), v=dev(nv))
    small = np.zeros((3, R, G, D), np.float16), np.zeros((3, R, G, D), np.float16)
    for dst, src in zip(small, (k, v)):
        dst.reshape(-1, G * D)[:n] = src.astype(np.float16)
    want, _ = paged.paged_attention(small[0], small[1], 3, R, G, D, False, [[0, 1, 2]], [n], q, H, 0.3, nk, nv)
    assert np.linalg.norm(host(out) - want[0]) <= 1e-5 * np.linalg.norm(want[0])
    page = value.view(pages, -1)[pages - 2].clone().view(torch.float16).cpu().numpy()
    row = page.reshape(G, R, D)[:, n % R] if hm else page.reshape(R, G, D)[n % R]
    assert np.array_equal(row.reshape(-1), nv[0].astype(np.float16))


def test_attention_of_more_tiles_than_units():
    """2^24 tiles: the split counts in fours.  All of a sequence's 65,536 table entries name one page, so each of its 64
    rows is seen 65,536 times and the result is the softmax over 64 rows.  A thread adds up to 32,768 tiles, each
    addition off by half a step of 2^-24 of the sum at most: 2^-10 of the sums, once for the outputs and once for the
    weights' total."""
    rng = np.random.default_rng(11)
    n, H, G, D, R, entries = 256, 2, 2, 8, 64, 65536
    key, value = (rng.standard_normal((1, R, G, D)).astype(np.float16) for _ in range(2))
    dk, dv = dev(key), dev(value)
    q = rng.standard_normal((n, H * D)).astype(np.float32)
    out = nan_like((n, H * D), 16)
    nb = mu.muser_kv_paged_attention_scratch_bytes(G * D, D, n, H)
    mu.muser_kv_paged_attention(mu.KvPages(dk.data_ptr(), dv.data_ptr(), 1, R, G * D, D, 0, 0), ints(np.zeros((1, entries))),
                                ints([entries * R - 1] * n), dev(q), n, H, out, 0.3, torch.zeros(nb // 4, device="cuda"), nb,
                                sequence=ints([0] * n))
    got = host(out)[:n * H * D].reshape(n, -1)
    check_canary(out, n * H * D)
    want, _ = paged.paged_attention(key, value, 1, R, G, D, False, [[0]], [R - 1] * n, q, H, 0.3, sequence=[0] * n)
    assert np.abs(got - np.stack(want)).max() <= 2 * 2.0 ** -10 * np.abs(value.astype(np.float32)).max()
    assert mu.muser_device_status() == 0


@pytest.mark.parametrize("G", [2, 3])
def test_attention_units_of_several_tiles(G):
    """More than 2^23 tiles (units of two tiles for G = 2, of four for G = 3), each of which is seen in the result.  A
    sequence's 60,000 to 65,536 table entries name 31 pages at random; a few more pages, each named once, have a key that
    weighs about as much as a tenth of all other rows: at the first tile, the last one, two drawn ones and those on both
    sides of each place where a block's share ends.  The expected result is the softmax weighted by the pages' counts.
    A thread adds up to 32,768 tiles, each addition off by half a step of 2^-24 of a sum that only grows: 2^-9 of the
    sums, once for the outputs and once for the weights' total; leaving out or doubling one of the few pages must show
    at four times that."""
    n, R, D, entries, ordinary, special, H = 256, 64, 8, 65536, 31, 12, G
    rng = np.random.default_rng(100 + G)
    pages = ordinary + special
    key = rng.standard_normal((pages, R, G, D)).astype(np.float16)
    value = np.clip(rng.standard_normal((pages, R, G, D)), -4, 4).astype(np.float16)
    key[..., 0] = 0
    key[ordinary:, 0] = 0
    key[ordinary:, 0, :, 0] = 45.0  # 0.3 * 45 above what the other rows' scores lie around
    value[ordinary:, 0] = rng.choice([-4.0, 4.0], (special, G, D))
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    q[..., 0] = 1.0
    t = np.sort(rng.integers(60000 * R, entries * R, n)).astype(np.int64)
    table = rng.integers(0, ordinary, (n, entries)).astype(np.int32)
    tiles = t // 128 + 1
    assert (tiles % 4 != 0).any() and tiles.sum() * G > 1 << 23
    # the split: an item's units are its tiles in twos or fours and two more, the blocks' shares of all units are equal
    shift = int(tiles.sum() * G >> 23).bit_length()
    units = -(-tiles // (1 << shift)) + 2
    before = np.concatenate([[0], np.cumsum(units)]) * G
    blocks = min(160, torch.cuda.get_device_properties(0).multi_processor_count)
    places = [[0, int(x) - 1, *rng.integers(1, x - 1, 2)] for x in tiles]
    for b in range(1, blocks):
        at = int(before[-1]) * b // blocks
        i = int(np.searchsorted(before, at, side="right")) - 1
        first = max((at - int(before[i])) % int(units[i]) - 2, 0) << shift
        places[i] += [x for x in (first - 1, first) if 0 <= x < tiles[i]]
    for i in range(n):
        places[i] = sorted(set(int(x) for x in places[i]))
        assert len(places[i]) <= special
        for j, x in enumerate(places[i]):
            table[i, min(2 * x + int(rng.integers(0, 2)), t[i] // R)] = ordinary + j
    dk, dv = dev(key), dev(value)
    out = nan_like((n, H * D), 16)
    nb = mu.muser_kv_paged_attention_scratch_bytes(G * D, D, n, H)
    mu.muser_kv_paged_attention(mu.KvPages(dk.data_ptr(), dv.data_ptr(), pages, R, G * D, D, 0, 0), ints(table), ints(t), dev(q), n,
                                H, out, 0.3, torch.zeros(nb // 4, device="cuda"), nb)
    got = host(out)[:n * H * D].reshape(n, H, D)
    check_canary(out, n * H * D)
    assert mu.muser_device_status() == 0
    bound = 2 * 2.0 ** -9 * 4.0
    for i in range(n):
        full, rest = divmod(int(t[i]) + 1, R)
        count = np.repeat(np.bincount(table[i, :full], minlength=pages)[:, None], R, 1)
        if rest:
            count[table[i, full], :rest] += 1
        w = np.exp(0.3 * np.einsum("prhd,hd->hpr", key.astype(np.float64), q[i].astype(np.float64))) * count
        o = np.einsum("hpr,prhd->hpd", w, value.astype(np.float64))
        w = w.sum(2)
        want = o.sum(1) / w.sum(1)[:, None]
        assert np.abs(got[i] - want).max() <= bound, i
        for j in range(ordinary, ordinary + len(places[i])):
            for c in (-1, 1):
                other = (o.sum(1) + c * o[:, j]) / (w.sum(1) + c * w[:, j])[:, None]
                assert (np.abs(other - want).max(1) > 4 * bound).all(), "the page would not be missed"


def test_attention_agrees_with_the_ring():
    """One token over one sequence: the tree attention over a plane gives the same to rounding."""
    c = Case([1000], 32, 2, 128, 64, False).to_device()
    rows = np.stack([paged.cache_row(c.cache.bufs[0], c.pages, 64, 2, 128, False, c.table[0, p // 64], p % 64) for p in range(1000)])
    vals = np.stack([paged.cache_row(c.cache.bufs[1], c.pages, 64, 2, 128, False, c.table[0, p // 64], p % 64) for p in range(1000)])
    key, value = to_dev16(rows), to_dev16(vals)
    plane = mu.KvPlane(key.data_ptr(), value.data_ptr(), 1000, 1000, 0, 0, 256, 128, 0, 0)
    nb = mu.muser_kv_tree_attention_scratch_bytes(256, 128, 1, 32)
    out = torch.empty(32 * 128, device="cuda")
    mu.muser_kv_tree_attention(plane, c.dq, c.dk, c.dv, 1, 32, out, c.scale, torch.zeros(nb // 4, device="cuda"), nb)
    c.call().check()
    a, b = host(out), host(c.out)[:32 * 128]
    assert np.linalg.norm(a - b) <= 2e-6 * np.linalg.norm(a)


# -------------------------------------------------------------- beam selection
def run_select(x, score, groups, beams, n, ended=None, end_token=-1, in_place=False, offset=0):
    V = x.shape[1]
    nb = mu.muser_beam_select_scratch_bytes(groups, beams, V, n)
    scratch = torch.zeros(nb // 4 + 4, device="cuda")
    scratch[nb // 4:] = 12345.0
    d = dict(logits=dev(x), score=dev(score), ended=None if ended is None else ints(ended))
    o = {y: torch.full((groups * n + 2,), -7, dtype=torch.int32, device="cuda") for y in ("parent", "token", "ended_out", "add")}
    so = torch.full((groups * n + 2,), -7.0, device="cuda")
    if in_place:
        so, o["ended_out"] = d["score"], d["ended"]
    for _ in range(1 if in_place else 2):  # twice on one scratch
        mu.muser_beam_select(d["logits"], d["score"], groups, beams, V, n, o["parent"], o["token"], so, scratch, nb,
                             ended=d["ended"], end_token=end_token, ended_out=o["ended_out"], add=o["add"])
    p, t, s, e = paged.beam_select(x, score, groups, beams, n, ended, end_token)
    got = {y: host(z) for y, z in o.items()}
    m = groups * n
    assert list(got["parent"][:m]) == list(p) and list(got["token"][:m]) == list(t)
    if got["ended_out"] is not None:
        assert list(got["ended_out"][:m]) == list(e)
    assert list(got["add"][:m]) == [1 - y for y in e]
    gs = host(so)
    ok = np.isfinite(s)
    # a rounding to binary32, and the log-sum's error of 2^-24
    assert (np.abs(gs[:m][ok] - s[ok]) <= 2.0 ** -24 * np.abs(s[ok]) + 2.0 ** -22).all() and np.isneginf(gs[:m][~ok]).all()
    if not in_place:
        for y in got.values():
            assert list(y[m:]) == [-7, -7]
    check_canary(scratch, nb // 4)
    assert not host(scratch)[:256].any()


@pytest.mark.parametrize("groups,beams,n", [(1, 1, 1), (1, 4, 4), (4, 4, 8), (1, 16, 16), (3, 5, 10), (2, 32, 64), (16, 1, 3), (256, 1, 1)])
@pytest.mark.parametrize("V", [65, 1003, 20000])
def test_select(groups, beams, n, V):
    rng = np.random.default_rng(groups * 100 + beams + V)
    x = (2.0 * rng.standard_normal((groups * beams, V))).astype(np.float32)
    score = (-20 + 2 * rng.standard_normal(groups * beams)).astype(np.float32)
    run_select(x, score, groups, beams, n)
    ended = (rng.random(groups * beams) < 0.3).astype(np.int32)
    run_select(x, score, groups, beams, n, ended, int(rng.integers(0, V)))
    if n == beams:
        run_select(x, score, groups, beams, n, ended, 3, in_place=True)


@pytest.mark.parametrize("V", [202048, 202049, 1 << 20])
def test_select_large_vocabularies(V):
    rng = np.random.default_rng(V)
    x = rng.standard_normal((3, V)).astype(np.float32)
    run_select(x, np.array([-1.0, -1.5, -1.2], np.float32), 1, 3, 6)


@pytest.mark.parametrize("V", [2, 40, 1500, 5000, 40000])
@pytest.mark.parametrize("n", [1, 4, 64])
def test_select_equal_logits(V, n):
    """Ties go to the lowest beam, then the lowest token; thousands of equal values do not fit the list."""
    if n > 2 * V:
        n = 2 * V
    x = np.zeros((2, V), np.float32)
    run_select(x, np.array([-3.0, -3.0], np.float32), 1, 2, n)
    x[:, 1::2] = -0.0
    x[1, V // 2:] = 1.0
    run_select(x, np.array([-3.0, -3.0], np.float32), 1, 2, n)
    x[0, 0] = np.inf
    run_select(x, np.array([-3.0, -3.0], np.float32), 1, 2, min(n, V))


@pytest.mark.parametrize("groups,beams,n,V", [(1, 1, 16, 202048), (1, 16, 32, 20000), (1, 32, 64, 50000), (1, 32, 64, 2000),
                                              (1, 1, 64, 1500), (1, 3, 64, 1100), (2, 16, 16, 16000), (2, 1, 64, 2047)])
@pytest.mark.parametrize("spread", [0.0, 2.0, 50.0])
def test_select_few_parts_and_far_scores(groups, beams, n, V, spread):
    """Fewer parts than what bounds the n largest has groups, parts with empty groups, and beams of which some have no
    part in the result."""
    rng = np.random.default_rng(V + n)
    x = (2.0 * rng.standard_normal((groups * beams, V))).astype(np.float32)
    run_select(x, (-20.0 - spread * rng.random(groups * beams)).astype(np.float32), groups, beams, n)


def select_time(x, score, n):
    """The least of ten measurements of twenty selections."""
    beams, V = x.shape
    nb = mu.muser_beam_select_scratch_bytes(1, beams, V, n)
    x, score, scratch, so = dev(x), dev(score), torch.zeros(nb // 4, device="cuda"), torch.zeros(n, device="cuda")
    o = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2)]
    times = []
    for _ in range(10):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda.synchronize()
        e[0].record()
        for _ in range(20):
            mu.muser_beam_select(x, score, 1, beams, V, n, *o, so, scratch, nb)
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]))
    return min(times)


@pytest.mark.parametrize("beams,n,V", [(16, 32, 20000), (32, 64, 50000), (32, 64, 2000), (1, 64, 1500)])
def test_select_of_untied_logits_takes_no_turns(beams, n, V):
    """The n largest of untied logits are not taken one by one, which costs 15 to 90 times what the largest one does (the
    list: 1.3 to 7 times)."""
    rng = np.random.default_rng(V)
    x, score = (2.0 * rng.standard_normal((beams, V))).astype(np.float32), (-20.0 - rng.random(beams)).astype(np.float32)
    assert select_time(x, score, n) < 10 * select_time(x, score, 1)


@pytest.mark.parametrize("V", [1100, 1500, 2000])
def test_select_of_tied_logits_is_not_ranked(V):
    """More equal logits than are worth a ranking (quadratic: 25 times the time of untied ones) are taken one by one
    (twice)."""
    x = np.random.default_rng(V).standard_normal((1, V)).astype(np.float32)
    assert select_time(np.zeros_like(x), np.zeros(1, np.float32), 4) < 10 * select_time(x, np.zeros(1, np.float32), 4)


def test_select_rows_that_are_not_finite():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((8, 3000)).astype(np.float32)
    x[0, 77] = np.nan
    x[1, 78] = np.inf
    x[2, :] = -np.inf
    x[3, 5:] = -np.inf
    x[4, :] = np.nan
    score = np.full(8, -1.0, np.float32)
    score[5] = -np.inf
    score[6] = np.nan
    run_select(x, score, 1, 8, 20)
    run_select(x, score, 8, 1, 7)
    run_select(x, score, 2, 4, 6)
    x[3, :] = -np.inf
    run_select(x[:4], score[:4], 1, 4, 4)  # no way on at all


@pytest.mark.parametrize("mask", [-1e9, float(np.finfo(np.float32).min), -np.inf])
def test_select_masked_tokens(mask):
    """Tokens masked by large negative numbers: whole parts of a row, all but one token, and rows that are all masked."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 30000)).astype(np.float32)
    x[0, 100:] = mask
    x[1, :29990] = mask
    x[2, 1:] = mask
    x[3, ::2] = mask
    run_select(x, np.arange(6, dtype=np.float32), 1, 6, 16)
    run_select(x, np.arange(6, dtype=np.float32), 6, 1, 2)
    x[5, :] = mask
    nothing = x[4:].copy()
    nothing[1] = -np.inf  # no way on from a row whose largest logit is beyond -2^20
    got = []
    for y in (x[4:], nothing):
        o = [torch.zeros(8, dtype=torch.int32, device="cuda") for _ in range(2)]
        so, nb = torch.zeros(8, device="cuda"), mu.muser_beam_select_scratch_bytes(1, 2, 30000, 8)
        mu.muser_beam_select(dev(y), dev(np.array([-9.0, 0.0], np.float32)), 1, 2, 30000, 8, o[0], o[1], so,
                             torch.zeros(nb // 4, device="cuda"), nb)
        got.append([host(t).copy() for t in (*o, so)])
    assert all(np.array_equal(a, b) for a, b in zip(*got)) and set(got[0][0]) == {0}


def test_select_first_step():
    """All beams begin alike: only the first one counts (scores 0, -infinity, ...)."""
    rng = np.random.default_rng(2)
    x = np.repeat(rng.standard_normal((1, 5000)).astype(np.float32), 6, 0)
    run_select(x, np.array([0.0] + [-np.inf] * 5, np.float32), 1, 6, 6)
    run_select(x, np.zeros(6, np.float32), 1, 6, 12)  # equal rows: every token six times, by beam


@pytest.mark.parametrize("groups,beams,V", [(1, 16, 202048), (4, 4, 3000), (16, 1, 500)])
def test_select_steps_in_place(groups, beams, V):
    """Steps one behind the other on one stream: scores and flags in place, so that each reads what the one before wrote;
    no other kernel between them.  Scores of untied logits differ by more than the steps' errors together."""
    steps, n, end = 6, groups * beams, 5
    rng = np.random.default_rng(V)
    x = (2.0 * rng.standard_normal((steps, n, V))).astype(np.float32)
    for s in range(steps):  # beams end in the first steps, one after another
        x[s, rng.choice(n, max(1, n // 5), replace=False), end] = 30.0
    dx = [dev(y) for y in x]
    nb = mu.muser_beam_select_scratch_bytes(groups, beams, V, beams)
    scratch = torch.zeros(nb // 4, device="cuda")
    first = (-3.0 * rng.random(n)).astype(np.float32)
    want, score, ended = [], first.astype(np.float64), np.zeros(n, np.int32)
    for s in range(steps):
        p, t, score, e = paged.beam_select(x[s], score, groups, beams, beams, ended, end)
        ended = e.astype(np.int32)
        want.append((p, t, score, ended))
    assert 0 < want[0][3].sum() < want[-1][3].sum()
    for _ in range(20):
        dscore, dended = dev(first), ints([0] * n)
        o = [[torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(3)] for _ in range(steps)]
        torch.cuda.synchronize()
        for s in range(steps):
            mu.muser_beam_select(dx[s], dscore, groups, beams, V, beams, o[s][0], o[s][1], dscore, scratch, nb, ended=dended,
                                 end_token=end, ended_out=dended, add=o[s][2])
        for s in range(steps):
            assert list(host(o[s][0])) == list(want[s][0]) and list(host(o[s][1])) == list(want[s][1]), s
            assert list(host(o[s][2])) == [1 - y for y in want[s][3]], s
        assert list(host(dended)) == list(want[-1][3])
        # a step adds a rounding of the score and the log-sum's error
        assert (np.abs(host(dscore) - want[-1][2]) <= steps * (2.0 ** -24 * np.abs(want[-1][2]) + 2.0 ** -22)).all()


# ------------------------------------------------------------------ together
class Search:
    """A beam search over a made-up one-layer model: q, k, v of a token and its position from tables, logits from the
    attention's output.  The model itself is numpy; what the library does is compared step by step."""

    def __init__(self, groups, beams, V, H, G, D, seed):
        rng = np.random.default_rng(seed)
        self.emb = rng.standard_normal((V, H * D + 2 * G * D)).astype(np.float32)
        self.head = (rng.standard_normal((H * D, V)) * 3 / np.sqrt(H * D)).astype(np.float32)
        self.groups, self.beams, self.V, self.H, self.G, self.D = groups, beams, V, H, G, D

    def rows(self, tokens):
        e = self.emb[np.maximum(tokens, 0)]
        a, b = self.H * self.D, self.G * self.D
        return e[:, :a].copy(), e[:, a:a + b].copy(), e[:, a + b:].copy()


@pytest.mark.parametrize("R,graph", [(4, False), (16, True)])
def test_beam_search(R, graph):
    G_, B, V, H, G, D = 2, 4, 300, 4, 2, 32
    m = Search(G_, B, V, H, G, D, 9)
    n, pages, stride, layers, end = G_ * B, 120, 12, 2, 7
    scale = 0.5
    caches = [[torch.full((pages * R * G * D,), NAN16, dtype=torch.int16, device="cuda") for _ in range(2)] for _ in range(layers)]
    handles = [mu.KvPages(c[0].data_ptr(), c[1].data_ptr(), pages, R, G * D, D, 0, 0) for c in caches]
    prompt = [3, 11, 200, 42, 5]
    # the prompts: one sequence a request, its rows stored in one go
    table = [torch.full((n, stride), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    length = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2)]
    result, copies = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(3 * n, dtype=torch.int32, device="cuda")
    last = torch.zeros(n, dtype=torch.int32, device="cuda")
    P = len(prompt)
    slots, position, sequence = (torch.zeros(G_ * P, dtype=torch.int32, device="cuda") for _ in range(3))
    mu.muser_kv_page_tables(table[0], length[0], n, pages, R, table[1], length[1], result,
                            add=ints([P if i % B == 0 else 0 for i in range(n)]), slots=slots, position=position,
                            sequence=sequence, max_new=G_ * P)
    assert list(host(result))[:2] == [0, G_ * P]
    q, k, v = m.rows(np.array(prompt * G_))
    dq, dk, dv = dev(q), dev(k), dev(v)
    for h in handles:
        mu.muser_kv_page_write(h, dk, dv, slots, G_ * P)
    nb = mu.muser_kv_paged_attention_scratch_bytes(G * D, D, n, H)
    nb = max(nb, mu.muser_kv_paged_attention_scratch_bytes(G * D, D, G_ * P, H))
    scratch = torch.zeros(nb // 4, device="cuda")
    out = torch.zeros(G_ * P, H * D, device="cuda")
    mu.muser_kv_paged_attention(handles[0], table[1], position, dq, G_ * P, H, out, scale, scratch, nb, sequence=sequence)
    got = host(out)[P - 1::P]

    def attend(q, past):  # past: (k, v) rows as binary16
        K, W = (np.stack([p[i] for p in past]).astype(np.float16).astype(np.float64).reshape(-1, G, D) for i in range(2))
        o = np.zeros((H, D))
        for h in range(H):
            z = scale * K[:, h * G // H] @ q.reshape(H, D)[h].astype(np.float64)
            a = np.exp(z - z.max())
            o[h] = a @ W[:, h * G // H] / a.sum()
        return o.reshape(-1)

    past = [[(k[j], v[j]) for j in range(P)] for _ in range(n)]
    want = attend(q[P - 1], past[0])
    assert np.abs(got - want).max() < 1e-4
    # every beam of a request goes on from the prompt's sequence; the first step takes n different tokens of one beam
    score = np.where(np.arange(n) % B == 0, 0.0, -np.inf).astype(np.float32)
    dscore, dended = dev(score), ints([0] * n)
    logits = torch.zeros(n, V, device="cuda")
    head = dev(m.head)
    parent, token, add = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3))
    sb = mu.muser_beam_select_scratch_bytes(G_, B, V, B)
    sscratch = torch.zeros(sb // 4, device="cuda")
    demb = dev(m.emb)
    out = torch.zeros(n, H * D, device="cuda")
    # the rows of a request's beams but the first have no sequence yet: logits of the first one for all
    logits.copy_(dev(np.repeat((got @ m.head), B, 0).astype(np.float32)))

    def step(src):
        """Selection, the next tables, copies, and the new tokens through the layers: all on the device."""
        mu.muser_beam_select(logits, dscore, G_, B, V, B, parent, token, dscore, sscratch, sb, ended=dended, end_token=end,
                             ended_out=dended, add=add)
        mu.muser_kv_page_tables(table[src], length[src], n, pages, R, table[1 - src], length[1 - src], result, parent=parent,
                                add=add, last=last, copies=copies)
        mu.muser_kv_page_copy(handles, copies, result.data_ptr() + 8, n)
        e = demb[token.long().clamp_min(0)]
        a, b = H * D, G * D
        q, k, v = e[:, :a].contiguous(), e[:, a:a + b].contiguous(), e[:, a + b:].contiguous()
        for h in handles:
            mu.muser_kv_paged_attention(h, table[1 - src], last, q, n, H, out, scale, scratch, nb, k=k, v=v)
        logits.copy_(out @ head)

    graphs = [None, None]
    if graph:
        keep = [t.clone() for t in (*table, *length, dscore, dended, logits, out, last)]
        bufs = [c.clone() for pair in caches for c in pair]
        for src in (1, 0):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(src)  # warm-up
            torch.cuda.current_stream().wait_stream(side)
            graphs[src] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[src]):
                step(src)
        for t, c in zip((*table, *length, dscore, dended, logits, out, last), keep):
            t.copy_(c)
        for c, b in zip((c for pair in caches for c in pair), bufs):
            c.copy_(b)
    src = 1
    ended = np.zeros(n, np.int32)
    for it in range(20):
        x = host(logits).copy()
        if graph:
            graphs[src].replay()
        else:
            step(src)
        p, t, s, e = paged.beam_select(x, score, G_, B, B, ended, end)
        assert list(host(parent)) == list(p) and list(host(token)) == list(t) and list(host(dended)) == list(e)
        score, ended = host(dscore).copy(), e.astype(np.int32)
        assert host(result)[0] == 0
        grows = [1 - y for y in e]
        before = [past[r] for r in p] if it else [past[r // B * B] for r in p]
        _, k, v = m.rows(np.asarray(t))
        past = [list(b) + ([(k[i], v[i])] if grows[i] else []) for i, b in enumerate(before)]
        assert list(host(length[1 - src])) == [len(b) for b in past]
        tab = host(table[1 - src])
        got = host(out)
        for i in range(n):
            if grows[i]:
                assert np.abs(got[i] - attend(m.rows(np.asarray(t))[0][i], past[i])).max() < 1e-4
            for layer in caches:  # the cache holds exactly this beam's past
                for which in range(2):
                    buf = host(layer[which]).view(np.float16).reshape(pages, R, G * D)
                    rows = np.stack([buf[tab[i, j // R], j % R] for j in range(len(past[i]))])
                    assert np.array_equal(rows, np.stack([y[which] for y in past[i]]).astype(np.float16))
        # no beam grows in a page that another one holds
        tails = [tab[i, (len(past[i]) - 1) // R] for i in range(n) if grows[i] and len(past[i]) % R]
        assert len(set(tails)) == len(tails)
        src = 1 - src
    assert mu.muser_device_status() == 0
