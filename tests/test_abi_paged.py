"""Host-side checks of the calls on several sequences (no GPU): every refusal comes before any launch."""
import ctypes
import os
import shutil

import pytest

import quantized_weight_streaming_q4_gb300 as mu
from tests.test_abi_tree import host_program

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
F = 1 << 24  # aligned, never-dereferenced pointer values are multiples of it


@pytest.fixture(scope="module")
def L():
    mu.build()
    return mu.lib()


def cache(key=F, value=F * 2, pages=64, page_rows=64, kv_dim=256, head_dim=128, head_major=0):
    return mu.KvPages(key, value, pages, page_rows, kv_dim, head_dim, head_major)


TABLES = dict(table=F, length=F * 2, n_old=4, parent=None, add=None, n=4, stride=8, pages=64, page_rows=16, window=0,
              n_sink=0, table_out=F * 3, length_out=F * 4, last=F * 5, first=F * 6, slots=F * 7, position=F * 8,
              sequence=F * 9, max_new=100, copies=F * 10, result=F * 11)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), -1), (dict(n=257), -1), (dict(n_old=0), -1), (dict(n_old=257), -1), (dict(n=3), -1),
    (dict(pages=0), -1), (dict(page_rows=0), -1), (dict(pages=(1 << 20) + 1), -2), (dict(pages=1 << 20, page_rows=1 << 11), -2),
    (dict(stride=0), -1), (dict(stride=1 << 24), -2), (dict(stride=1 << 40), -2), (dict(window=-1), -1), (dict(n_sink=-1), -1),
    (dict(max_new=-1), -1), (dict(max_new=1 << 31), -1),
    (dict(table=None), -1), (dict(length=None), -1), (dict(table_out=None), -1), (dict(length_out=None), -1),
    (dict(result=None), -1), (dict(parent=F * 12, copies=None), -1),
    (dict(table=F + 2), -3), (dict(parent=F * 12 + 1), -3), (dict(add=F * 12 + 2), -3), (dict(slots=F * 7 + 2), -3),
    (dict(first=F * 6 + 1), -3), (dict(result=F * 11 + 2), -3),
    (dict(table_out=F + 16), -1), (dict(length_out=F * 2 + 4), -1),            # neither in place nor apart
    (dict(parent=F * 12, table_out=F), -1), (dict(parent=F * 12, length_out=F * 2), -1),  # in place with parents
    (dict(last=F * 4), -1), (dict(slots=F * 8 - 396), -1), (dict(copies=F * 11 - 12), -1), (dict(add=F * 5), -1),
])
def test_tables_refusals(L, kw, status):
    a = dict(TABLES, **kw)
    assert L.muser_kv_page_tables(*a.values(), None) == status
    assert mu.muser_last_error().startswith("muser_kv_page_tables")


BAD_CACHES = [(dict(key=None), -1), (dict(value=None), -1), (dict(key=F + 1), -3), (dict(pages=0), -1),
              (dict(page_rows=0), -1), (dict(kv_dim=0), -1), (dict(head_dim=96), -1), (dict(head_dim=0), -1),
              (dict(pages=(1 << 20) + 1), -2), (dict(pages=1 << 20, page_rows=1 << 11), -2),
              (dict(page_rows=1 << 24, pages=1), -2)]


def copy(L, layers=None, n_layers=None, copies=F * 10, count=F * 11, most=4):
    layers = [cache(), cache(F * 3, F * 4)] if layers is None else layers
    arr = (mu.KvPages * len(layers))(*layers)
    return L.muser_kv_page_copy(arr, len(layers) if n_layers is None else n_layers, copies, count, most, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_layers=0), -1), (dict(n_layers=129), -1), (dict(most=-1), -1), (dict(copies=None), -1), (dict(count=None), -1),
    (dict(copies=F * 10 + 2), -3), (dict(count=F * 11 + 1), -3),
    (dict(layers=[cache(), cache()]), -1), (dict(layers=[cache(value=F + 1024)]), -1),
    (dict(layers=[cache(), cache(F * 3, F * 4, pages=32)]), -1), (dict(layers=[cache(), cache(F * 3, F * 4, head_major=1)]), -1),
    (dict(copies=F + 64), -1), (dict(count=F * 2 + 64), -1),
] + [(dict(layers=[cache(**c)]), s) for c, s in BAD_CACHES])
def test_copy_refusals(L, kw, status):
    assert copy(L, **kw) == status
    assert mu.muser_last_error().startswith("muser_kv_page_copy")


def test_no_copies_launch_nothing(L):
    assert copy(L, most=0) == 0
    assert L.muser_kv_page_write(ctypes.byref(cache()), None, None, None, 0, None) == 0


def write(L, c=None, k=F * 5, v=F * 6, slots=F * 7, rows=10):
    return L.muser_kv_page_write(ctypes.byref(cache() if c is None else c), k, v, slots, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1),
    (dict(k=F * 5 + 2), -3), (dict(slots=F * 7 + 2), -3), (dict(k=F + 64), -1), (dict(slots=F * 2 + 4), -1),
    (dict(c=cache(value=F + 64)), -1)] + [(dict(c=cache(**c)), s) for c, s in BAD_CACHES])
def test_write_refusals(L, kw, status):
    assert write(L, **kw) == status
    assert mu.muser_last_error().startswith("muser_kv_page_write")


def attend(L, c=None, table=F * 5, stride=8, n_tables=4, position=F * 6, sequence=None, q=F * 7, k=F * 8, v=F * 9, gate=None,
           n=4, H=32, window=0, n_sink=0, scale=0.1, out=F * 11, scratch=F * 12, nbytes=1 << 23):
    return L.muser_kv_paged_attention(ctypes.byref(cache() if c is None else c), table, stride, n_tables, position, sequence,
                                      q, k, v, gate, n, H, window, n_sink, scale, out, scratch, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), -1), (dict(n=257), -1), (dict(H=0), -1), (dict(H=33), -1), (dict(H=2048), -2), (dict(stride=0), -1),
    (dict(stride=1 << 22), -2), (dict(n_tables=0), -1), (dict(window=-1), -1), (dict(n_sink=-1), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=3e38), -1),
    (dict(table=None), -1), (dict(position=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(out=None), -1), (dict(scratch=None), -1), (dict(table=F * 5 + 2), -3), (dict(position=F * 6 + 1), -3),
    (dict(sequence=F * 10 + 2), -3), (dict(q=F * 7 + 4), -3), (dict(k=F * 8 + 8), -3), (dict(gate=F * 10 + 4), -3),
    (dict(out=F * 11 + 8), -3), (dict(scratch=F * 12 + 4), -3), (dict(nbytes=1024), -1),
    (dict(out=F * 7), -1), (dict(out=F * 12 + 4096), -1), (dict(out=F + 4096), -1), (dict(scratch=F * 6 - 4096), -1),
    (dict(q=F * 2 + 64), -1), (dict(table=F * 2 + 64), -1), (dict(gate=F * 11), -1), (dict(c=cache(value=F + 64)), -1),
    (dict(c=cache(kv_dim=512, head_dim=512)), -2)] + [(dict(c=cache(**c)), s) for c, s in BAD_CACHES])
def test_attention_refusals(L, kw, status):
    assert attend(L, **kw) == status
    assert mu.muser_last_error().startswith("muser_kv_paged_attention")


def test_attention_scratch(L):
    n = mu.muser_kv_paged_attention_scratch_bytes(256, 128, 16, 32)
    assert 0 < n < 1 << 23 and n % 16 == 0
    for bad in ((256, 96, 1, 32), (256, 128, 0, 32), (256, 128, 257, 32), (256, 128, 1, 31), (0, 128, 1, 32), (512, 512, 1, 1)):
        assert mu.muser_kv_paged_attention_scratch_bytes(*bad) == 0


SELECT = dict(logits=F * 16, score=F, ended=None, groups=2, beams=4, vocab=1000, n=4, end_token=-1, parent=F * 2, token=F * 3,
              score_out=F * 4, ended_out=F * 5, add=F * 6, scratch=F * 8, nbytes=1 << 22)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), -1), (dict(beams=0), -1), (dict(n=0), -1), (dict(vocab=0), -1), (dict(beams=33), -2), (dict(groups=65), -2),
    (dict(n=65), -2), (dict(vocab=(1 << 20) + 1), -2), (dict(beams=1, vocab=3), -1), (dict(end_token=-2), -1),
    (dict(end_token=1000), -1), (dict(ended=F * 7), -1),
    (dict(logits=None), -1), (dict(score=None), -1), (dict(parent=None), -1), (dict(token=None), -1), (dict(score_out=None), -1),
    (dict(scratch=None), -1), (dict(logits=F * 16 + 4), -3), (dict(score=F + 2), -3), (dict(parent=F * 2 + 1), -3),
    (dict(ended=F * 7 + 2, end_token=1), -3), (dict(scratch=F * 8 + 8), -3), (dict(nbytes=512), -1),
    (dict(parent=F * 3), -1), (dict(score_out=F + 4), -1), (dict(n=8, score_out=F), -1),
    (dict(ended=F * 5, end_token=1, n=8), -1), (dict(token=F * 16 + 400), -1), (dict(scratch=F * 16 - 64), -1),
])
def test_select_refusals(L, kw, status):
    a = dict(SELECT, **kw)
    assert L.muser_beam_select(*a.values(), None) == status
    assert mu.muser_last_error().startswith("muser_beam_select")


def test_select_scratch(L):
    assert mu.muser_beam_select_scratch_bytes(1, 16, 202048, 16) > 1024
    for bad in ((0, 1, 10, 1), (1, 33, 10, 1), (1, 1, 10, 11), (1, 1, 1 << 21, 1), (300, 1, 10, 1), (1, 2, 100, 65)):
        assert mu.muser_beam_select_scratch_bytes(*bad) == 0


@pytest.mark.parametrize("name", ["beam.cu", "paged_attn.cu", "paged_tc.cu", "paged.cuh", "pages.cu", "pages.cuh"])
def test_programmatically_launched_kernels_load_nothing_on_the_read_only_path(name):
    """What the kernel before wrote, or what this one writes in place, is loaded past the read-only path: such a load may
    move above the wait for the kernel before, or meet an old line of an SM's cache."""
    from quantized_weight_streaming_q4_gb300 import buildlib
    with open(os.path.join(buildlib.CSRC, name)) as f:
        text = f.read()
    for load in ("ldg(", "ldg_", "global.nc"):
        assert load not in text, (name, load)


def _tables_call(table, out, **kw):
    z = 1 << 30  # never read: pages is 0, which the library refuses
    mu.muser_kv_page_tables(table, z, 4, 0, 16, out, z + 4096, z + 8192, stream=0, **kw)


def _attend_call(table, **kw):
    z = 1 << 30
    mu.muser_kv_paged_attention(cache(pages=0), table, z, z, 4, 32, z, 0.1, z, 0, stream=0, **kw)


def test_binding_refuses_tables_that_are_not_rows_of_int32(L):
    """A table's sizes come from its tensor, whose rows the library takes to lie one behind the other: a part of a wider
    tensor, a tensor of another type or of other dimensions would be read as something else, an expanded one beyond its
    end."""
    torch = pytest.importorskip("torch")
    good = torch.zeros(4, 8, dtype=torch.int32)
    wide = torch.zeros(4, 10, dtype=torch.int32)
    bad = [wide[:, :8], wide.t(), torch.zeros(1, 8, dtype=torch.int32).expand(4, 8), torch.zeros(4, 8, dtype=torch.int64),
           torch.zeros(4, 8, dtype=torch.int16), torch.zeros(4, 8), torch.zeros(32, dtype=torch.int32),
           torch.zeros(1, 4, 8, dtype=torch.int32)]
    for t in bad:
        for kw in ({}, dict(n_old=4), dict(width=8)):
            with pytest.raises(ValueError, match="table"):
                _tables_call(t, good, **kw)
        for kw in ({}, dict(n_tables=4), dict(width=8)):
            with pytest.raises(ValueError, match="table"):
                _attend_call(t, **kw)
    # the new tables have as many entries a row
    for t in (wide[:, :8], torch.zeros(4, 7, dtype=torch.int32), torch.zeros(3, 8, dtype=torch.int32),
              torch.zeros(4, 8, dtype=torch.int64), torch.zeros(4, 8)):
        with pytest.raises(ValueError, match="table_out"):
            _tables_call(good, t)
    # what goes through to the library: tables as they should be, buffers of any form whose sizes are given, addresses
    for call in (lambda: _tables_call(good, torch.zeros_like(good)), lambda: _tables_call(good, torch.zeros(9, 8, dtype=torch.int32)),
                 lambda: _tables_call(good, torch.zeros(32, dtype=torch.int32)), lambda: _tables_call(good, 1 << 29),
                 lambda: _tables_call(good.view(-1), torch.zeros_like(good), n_old=4, width=8),
                 lambda: _tables_call(1 << 29, 1 << 28, n_old=4, width=8),
                 lambda: _attend_call(good), lambda: _attend_call(wide[:, :8], n_tables=4, width=10), lambda: _attend_call(1 << 29, n_tables=4, width=8)):
        with pytest.raises(mu.MuserError, match="pages and page_rows must be positive"):
            call()


def test_tables_take_the_clusters_that_the_device_can_place(L, tmp_path):
    """Sixteen blocks are more than a device has to offer: fewer free SMs in its clusters' groups, and smaller clusters,
    down to one block, do the same work."""
    out = host_program(tmp_path, r"""
#include <cstdio>
#include "pages.cuh"
int main() {
    for (int most : {16, 15, 8, 7, 2, 1, 0}) {
        const int c = muser::largest_cluster([&](int size) { return size <= most; });
        std::printf("%d ", c);
    }
}
""")
    assert out == ["16", "8", "8", "4", "2", "1", "1"]
