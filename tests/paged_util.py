"""Inputs of the tests of several sequences (test-only): page tables and caches."""
import numpy as np

NAN16 = 0x7E00


def tables(rng, lengths, page_rows, pages, stride, spare=0):
    """Tables of sequences whose pages lie anywhere in the cache; entries behind their ends are -1."""
    ids = rng.permutation(pages)
    table = np.full((len(lengths), stride), -1, np.int32)
    at = 0
    for i, n in enumerate(lengths):
        held = -(-n // page_rows)
        table[i, :held] = ids[at:at + held]
        at += held
    assert at + spare <= pages
    return table


class Cache:
    """A paged cache whose rows 0..length-1 of every sequence hold numbers and all other slots hold `fill`."""

    def __init__(self, rng, table, lengths, pages, page_rows, kv_heads, head_dim, head_major, fill=NAN16):
        self.pages, self.R, self.G, self.D, self.hm = pages, page_rows, kv_heads, head_dim, head_major
        live = np.zeros((pages, page_rows), bool)
        for i, n in enumerate(lengths):
            for p in range(n):
                e = table[i, p // page_rows]
                if 0 <= e < pages:
                    live[e, p % page_rows] = True
        self.bufs = []
        for _ in range(2):
            rows = rng.standard_normal((pages, page_rows, kv_heads, head_dim)).astype(np.float16).view(np.uint16)
            rows[~live] = fill
            self.bufs.append(np.ascontiguousarray(rows.transpose(0, 2, 1, 3) if head_major else rows).reshape(-1))

    @property
    def key(self):
        return self.bufs[0].view(np.float16)

    @property
    def value(self):
        return self.bufs[1].view(np.float16)

    def with_rows(self, stored, k, v):
        """The buffers' bits after row i of k and v went to (page, row) stored[i] (None: nowhere)."""
        out = []
        for buf, new in zip(self.bufs, (k, v)):
            buf = buf.copy()
            shape = (self.pages, self.G, self.R, self.D) if self.hm else (self.pages, self.R, self.G, self.D)
            view = buf.reshape(shape)
            for i, where in enumerate(stored):
                if where is not None:
                    row = new[i].astype(np.float16).view(np.uint16).reshape(self.G, self.D)
                    if self.hm:
                        view[where[0], :, where[1]] = row
                    else:
                        view[where[0], where[1]] = row
            out.append(buf)
        return out


def attention_bound(q, scale, kmax, D, vmax):
    """Elementwise bound of a binary32 evaluation.  A score is a sum of D products (binary16 key times a query held to
    2^-22 at least): its error is at most (D/2 + 8) steps of 2^-24 of scale * sum|q||k|, taking half the steps for
    partial sums that grow evenly.  A weight's relative error is at most twice the largest score's error plus 2^-21
    (the exponential, the two sums); an output is a mean of values up to vmax."""
    s = abs(scale) * np.abs(q).reshape(q.shape[0], -1, D).sum(-1).max() * kmax
    return vmax * (2 * (D / 2 + 8) * 2.0 ** -24 * s + 2.0 ** -21)
