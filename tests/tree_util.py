"""Inputs of the speculative-step tests (test-only): trees, planes and logits."""
import numpy as np

import oracle

CHAIN, BINARY, STAR, TWO = "chain", "binary", "star", "two"


def parents(kind, M):
    f = {CHAIN: lambda i: i - 1, BINARY: lambda i: (i - 1) // 2, STAR: lambda i: 0, TWO: lambda i: max(0, i - 2)}[kind]
    return [-1] + [f(i) for i in range(1, M)]


def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def plane(rng, cap, kv_heads, head_dim, n, origin, head_major, fill=0x7E00, physical=None):
    """(Ring, key, value): n live rows from logical position `origin`; every
    other slot holds `fill` (a NaN by default)."""
    kv = kv_heads * head_dim
    ring = oracle.Ring(cap, n, origin, origin % cap if physical is None else physical)
    bufs = []
    for _ in range(2):
        rows = rng.standard_normal((n, kv)).astype(np.float16).view(np.uint16)
        buf = np.full((kv_heads, cap, head_dim) if head_major else (cap, kv), fill, np.uint16)
        slots = (ring.origin_physical + np.arange(n)) % cap
        if head_major:
            buf[:, slots] = rows.reshape(n, kv_heads, head_dim).transpose(1, 0, 2)
        else:
            buf[slots] = rows
        bufs.append(np.ascontiguousarray(buf.reshape(-1)))
    return ring, bufs[0], bufs[1]


def logits(rng, M, V, spread=1.6, peaks=8):
    x = spread * rng.standard_normal((M, V))
    for i in range(M):
        x[i, rng.integers(0, V, peaks)] += 6 + 2 * rng.standard_normal(peaks)
    return x.astype(np.float32)


def drafted(rng, draft, parent, temperature):
    """Tokens drawn from each row's parent's draft distribution."""
    M, V = draft.shape
    out = np.zeros(M, np.int32)
    for i in range(1, M):
        z = draft[parent[i]].astype(np.float64) / temperature
        p = np.exp(z - z.max())
        out[i] = min(int(np.searchsorted(np.cumsum(p) / p.sum(), rng.random(), side="right")), V - 1)
    return out
