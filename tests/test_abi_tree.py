"""Host-side checks of the speculative-step calls (no GPU): every refusal comes before any launch and changes nothing."""
import ctypes
import os
import shutil

import pytest

import quantized_weight_streaming_q4_gb300 as mu

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
FAKE = 1 << 20  # an aligned, never-dereferenced pointer value
Q, K, V, OUT, SCR = FAKE * 4, FAKE * 8, FAKE * 9, FAKE * 12, FAKE * 64


@pytest.fixture(scope="module")
def L():
    mu.build()
    return mu.lib()


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def attend(L, plane=None, sink=None, q=Q, k=K, v=V, gate=None, M=2, H=32, parent=None, window=0, n_sink=0, scale=0.1,
           out=OUT, scratch=SCR, nbytes=1 << 24):
    plane = mu.KvPlane(FAKE, FAKE * 2, 2048, 100, 0, 0, 256, 128, 0, 0) if plane is None else plane
    return L.muser_kv_tree_attention(ctypes.byref(plane), sink and ctypes.byref(sink), q, k, v, gate, M, H, parent,
                                     window, n_sink, scale, out, scratch, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), -1), (dict(M=17), -1), (dict(H=0), -1), (dict(H=33), -1),      # rows, heads not a multiple of 2
    (dict(H=2048), -2),
    (dict(parent=ints(0, 0)), -1), (dict(parent=ints(-1, 1)), -1), (dict(parent=ints(-1, -1)), -1),
    (dict(window=-1), -1), (dict(n_sink=-1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(scratch=None), -1),
    (dict(q=Q + 4), -3), (dict(k=K + 8), -3), (dict(gate=FAKE * 3 + 4), -3), (dict(out=OUT + 4), -3),
    (dict(scratch=SCR + 8), -3), (dict(nbytes=1024), -1),
    (dict(out=Q), -1), (dict(out=K + 16), -1), (dict(out=V), -1), (dict(gate=OUT), -1),   # overlaps
    (dict(scratch=Q - 1024), -1), (dict(out=SCR + 4096), -1),
    (dict(out=FAKE + 4096), -1), (dict(scratch=FAKE * 3 - 64), -1),                       # the planes
    (dict(sink=mu.KvPlane(OUT + 16, FAKE * 2, 4, 4, 0, 0, 256, 128, 0, 0)), -1),
    (dict(plane=mu.KvPlane(FAKE, FAKE * 2, 2048, 2049, 0, 0, 256, 128, 0, 0)), -1),
    (dict(plane=mu.KvPlane(FAKE, None, 2048, 0, 0, 0, 256, 128, 0, 0)), -1),
    (dict(plane=mu.KvPlane(FAKE, FAKE * 2, 2048, 0, 0, 0, 256, 0, 0, 0)), -1),      # head_dim is needed in both layouts
    (dict(plane=mu.KvPlane(FAKE, FAKE * 2, 2048, 0, 0, 0, 256, 96, 0, 0)), -1),
    (dict(plane=mu.KvPlane(FAKE, FAKE * 2, 2048, 0, 0, 0, 512, 512, 0, 0)), -2),
    (dict(plane=mu.KvPlane(FAKE, FAKE * 2, 1 << 40, 1 << 31, 0, 0, 256, 128, 0, 0)), -2),
    (dict(sink=mu.KvPlane(FAKE, FAKE * 2, 4, 4, 0, 0, 128, 128, 0, 0)), -1),
    (dict(sink=mu.KvPlane(FAKE, FAKE * 2, 4, 5, 0, 0, 256, 128, 0, 0)), -1),
    (dict(sink=mu.KvPlane(FAKE, FAKE * 2, 4, 4, 0, 0, 256, 64, 1, 0)), -1),
])
def test_attention_refusals(L, kw, status):
    assert attend(L, **kw) == status
    assert mu.muser_last_error().startswith("muser_kv_tree_attention")


def test_attention_scratch_does_not_depend_on_the_length(L):
    n = mu.muser_kv_tree_attention_scratch_bytes(256, 128, 16, 32)
    assert n > 0 and n % 16 == 0
    for bad in ((256, 96, 1, 32), (256, 128, 0, 32), (256, 128, 17, 32), (256, 128, 1, 31), (0, 128, 1, 32),
                (512, 512, 1, 1)):
        assert mu.muser_kv_tree_attention_scratch_bytes(*bad) == 0


def verify(L, target=FAKE * 16, draft=None, tokens=FAKE, parent=None, M=3, vocab=1000, T=1.0, u=FAKE * 2,
           result=FAKE * 3, scratch=SCR, nbytes=1 << 20):
    return L.muser_tree_verify(target, draft, tokens, parent, M, vocab, T, u, result, scratch, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), -1), (dict(M=17), -1), (dict(vocab=0), -1), (dict(vocab=(1 << 20) + 1), -2),
    (dict(T=-1.0), -1), (dict(T=float("nan")), -1), (dict(T=float("inf")), -1), (dict(T=1e-4), -1),
    (dict(parent=ints(-1, 0, 2)), -1), (dict(parent=ints(0, 0, 0)), -1),
    (dict(target=None), -1), (dict(target=FAKE + 4), -3), (dict(draft=FAKE * 20 + 4), -3), (dict(u=None), -1),
    (dict(u=FAKE + 2), -3), (dict(tokens=None), -1), (dict(tokens=FAKE + 1), -3), (dict(result=None), -1),
    (dict(result=FAKE * 3 + 2), -3), (dict(scratch=None), -1), (dict(scratch=SCR + 4), -3), (dict(nbytes=100), -1),
    (dict(result=FAKE), -1), (dict(result=FAKE * 2 + 8), -1), (dict(result=FAKE * 16 + 4 * 2999), -1),
    (dict(scratch=FAKE * 16 - 64), -1), (dict(result=SCR + 16), -1),
])
def test_verify_refusals(L, kw, status):
    assert verify(L, **kw) == status
    assert mu.muser_last_error().startswith("muser_tree_verify")


def test_verify_scratch_sizes(L):
    assert mu.muser_tree_verify_scratch_bytes(202048, 16) > 0
    for bad in ((0, 1), ((1 << 20) + 1, 1), (100, 0), (100, 17)):
        assert mu.muser_tree_verify_scratch_bytes(*bad) == 0


def commit(L, planes, k=None, v=None, M=4, path=ints(0, 2), n=2, position=100):
    P = ctypes.c_void_p * len(planes)
    arr = (mu.KvPlane * len(planes))(*planes)
    rc = L.muser_kv_tree_commit(arr, len(planes), P(*(k or [K] * len(planes))), P(*(v or [V] * len(planes))), M, path, n,
                                position, None)
    return rc, [(p.len, p.origin_logical, p.origin_physical) for p in arr]


def test_commit_refusals_change_no_plane(L):
    def plane(i, n=100, origin=0, **kw):
        return mu.KvPlane(FAKE * (16 + 4 * i), FAKE * (18 + 4 * i), 128, n, origin, 0, kw.get("kv", 256), 128, 0, 0)

    two = [plane(0), plane(1)]
    before = [(100, 0, 0)] * 2
    for kw, status in ((dict(M=0), -1), (dict(M=17), -1), (dict(n=3, M=2, path=ints(0, 1, 2)), -1), (dict(n=-1), -1),
                       (dict(path=ints(0, 4)), -1), (dict(path=ints(-1, 0)), -1), (dict(path=ints(1, 1)), -1),
                       (dict(path=ints(2, 0)), -1), (dict(path=None), -1), (dict(position=99), -4),
                       (dict(k=[K, None]), -1), (dict(v=[V, V + 2]), -3)):
        assert commit(L, two, **kw) == (status, before), kw
    assert commit(L, [plane(0), plane(1, n=99)])[0] == -4
    assert commit(L, [plane(0), plane(0)])[0] == -1 and "share memory" in mu.muser_last_error()
    near = plane(1)
    near.value = FAKE * 16 + 16
    assert commit(L, [plane(0), near])[0] == -1
    assert commit(L, [plane(0), mu.KvPlane(FAKE, FAKE * 2, 32, 40, 60, 0, 256, 128, 0, 0)])[0] == -1
    assert commit(L, two, n=0) == (0, before)
    arr = (mu.KvPlane * 1)(plane(0))
    assert L.muser_kv_tree_commit(arr, 0, None, None, 1, None, 0, 100, None) == -1
    assert L.muser_kv_tree_commit(arr, 129, None, None, 1, None, 0, 100, None) == -1


def test_binding_checks_lengths(L):
    plane = mu.KvPlane(FAKE, FAKE * 2, 2048, 100, 0, 0, 256, 128, 0, 0)
    with pytest.raises(ValueError, match="parent"):
        mu.muser_kv_tree_attention(plane, Q, K, V, 3, 32, OUT, 0.1, SCR, 1 << 24, parent=[-1, 0], stream=0)
    with pytest.raises(ValueError, match="parent"):
        mu.muser_tree_verify(FAKE * 16, None, FAKE, [-1], 2, 10, 1.0, FAKE * 2, FAKE * 3, SCR, 1 << 20, stream=0)
    with pytest.raises(ValueError, match="per plane"):
        mu.muser_kv_tree_commit([plane], [K, K], [V], 2, [0], 100, stream=0)
    with pytest.raises(mu.MuserError, match="discontinuity"):
        mu.muser_kv_tree_commit([plane], [K], [V], 2, [0], 101, stream=0)
    assert (plane.len, plane.origin_logical) == (100, 0)


def test_commit_finds_planes_that_share_memory_in_any_order(L):
    def plane(key, value):
        return mu.KvPlane(key, value, 128, 100, 0, 0, 256, 128, 0, 0)   # 65,536 bytes each

    S, B = 65536, FAKE * 16
    for order in ([0, 1, 2], [2, 0, 1], [1, 2, 0]):
        apart = [plane(B + 2 * S * i, B + 2 * S * i + S) for i in range(3)]
        for bad in (plane(B + S * 2 + 16, B + S * 9), plane(B + S * 9, B + S * 3 - 16), plane(B + S * 9, B + S * 10 - 16)):
            planes = [apart[i] for i in order] + [bad]
            assert commit(L, planes)[0] == -1 and "share memory" in mu.muser_last_error(), (order, bad.key - B, bad.value - B)
            assert commit(L, planes[::-1])[0] == -1


def test_sizes_beyond_the_kernels_indexes_are_refused(L):
    far = mu.KvPlane(FAKE, FAKE * 2, 2048, 100, (1 << 62) + 1, 0, 256, 128, 0, 0)
    ring = mu.KvPlane(FAKE, FAKE * 2, 2048, 100, 0, 0, 256, 128, 0, 0)
    assert attend(L, plane=far) == -2 and attend(L, plane=ring, sink=far) == -2
    assert commit(L, [far], position=(1 << 62) + 101)[0] == -2
    wide = mu.KvPlane(FAKE * 16, FAKE * 4096, 2, 1, 0, 0, (1 << 26) + 1, 1, 0, 0)
    assert commit(L, [wide], position=1)[0] == -2 and "kv_dim" in mu.muser_last_error()
    assert verify(L, T=1e31) == -1 and verify(L, T=5e-324) == -1


def test_a_scale_that_overflows_in_base_2_is_refused(L):
    """The kernels' exponentials are of base 2: the scale times log2(e) is held in binary32 as well."""
    assert attend(L, scale=2.4e38) == -1 and "scale" in mu.muser_last_error()
    assert attend(L, scale=-2.4e38) == -1
    assert attend(L, scale=2.3e38, nbytes=1024) == -1 and "scratch_bytes" in mu.muser_last_error()


def test_binding_converts_arrays_of_other_types(L):
    """A c_int64 or numpy array is converted, not read as if it held 32-bit integers."""
    import numpy as np
    plane = mu.KvPlane(FAKE, FAKE * 2, 2048, 100, 0, 0, 256, 128, 0, 0)
    for path in ((ctypes.c_int64 * 2)(1, 1), np.array([1, 1]), np.array([1, 1], dtype=np.int8)):
        with pytest.raises(mu.MuserError, match=r"path\[1\] = 1"):
            mu.muser_kv_tree_commit([plane], [K], [V], 4, path, 100, stream=0)
    with pytest.raises(mu.MuserError, match=r"path\[1\] = 1"):
        mu.muser_kv_tree_commit([plane], (ctypes.c_int64 * 1)(K), [V], 4, [1, 1], 100, stream=0)


def host_program(tmp_path, source):
    """Runs a C++ program (no GPU) against the library's headers; returns what it prints."""
    import subprocess
    from quantized_weight_streaming_q4_gb300 import buildlib
    (tmp_path / "p.cu").write_text(source)
    subprocess.run([buildlib._nvcc(), *buildlib.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", buildlib.INCLUDE, "-I",
                    buildlib.CSRC, str(tmp_path / "p.cu"), "-o", str(tmp_path / "p")], check=True, capture_output=True)
    return subprocess.run([str(tmp_path / "p")], check=True, capture_output=True, text=True).stdout.split()


def test_attention_parts_are_aligned_in_the_scratch(L, tmp_path):
    """The (maximum, sum) pairs are read and written 8 bytes at a time, the sums 16 (head sizes that are multiples of 4),
    whatever the parity of parts, rows and head size; neither reaches into the other nor past the scratch bytes."""
    out = host_program(tmp_path, r"""
#include <cstdio>
#include "attn.cuh"
int main() {
    int bad = 0, n = 0;
    for (long long parts : {1, 2, 3, 11, 101, 304})
        for (long long rows : {1, 3, 9, 27, 32, 48, 16384})
            for (long long D : {1, 3, 5, 7, 33, 65, 128, 136, 255, 256}) {
                const muser::AttnPartLayout l = muser::attn_part_layout(parts, rows, D);
                const size_t pairs = parts * rows * 8, sums = parts * rows * D * 4;
                bad += l.o % 16 != 0 || l.o < pairs || l.bytes < l.o + sums || l.bytes % 16 != 0;
                ++n;
            }
    std::printf("%d %d\n", bad, n);
}
""")
    assert out == ["0", "420"]
    for M, H, kvh, D in ((1, 3, 3, 5), (1, 1, 1, 7), (3, 9, 9, 33), (5, 3, 1, 65), (16, 32, 2, 128)):
        n = mu.muser_kv_tree_attention_scratch_bytes(kvh * D, D, M, H)
        assert n % 16 == 0 and n >= M * H * (8 + 4 * D)


def test_programmatically_launched_kernels_load_nothing_on_the_read_only_path():
    """A non-coherent load may move above the wait for the kernel before, whose output it then misses.  attn.cu's
    CUDA-core kernel has no such wait (an ordinary launch)."""
    from quantized_weight_streaming_q4_gb300 import buildlib
    for name in ("verify.cu", "attn_few.cu", "attn_tc.cu", "attn_mma.cu", "attn_parts.cuh", "tc.cuh"):
        with open(os.path.join(buildlib.CSRC, name)) as f:
            text = f.read()
        for load in ("ldg(", "ldg_", "global.nc", "attn_ragged("):
            assert load not in text, (name, load)
