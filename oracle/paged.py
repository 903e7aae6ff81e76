"""Page tables, attention over a paged K/V cache and beam selection from their definitions, in numpy: one row after
another, 64 bits, no code of the CUDA path."""
from __future__ import annotations

import numpy as np


def live(k: int, page_rows: int, keep: int, window: int, n_sink: int) -> bool:
    """Whether page k of a sequence of `keep` rows holds a row that its next token can see."""
    return window == 0 or k * page_rows < n_sink or (k + 1) * page_rows > keep - window + 1


def page_tables(table, length, parent, add, pages, page_rows, window=0, n_sink=0, max_new=None, copies_given=True):
    """dict of the outputs of muser_kv_page_tables.  `table` (out): the new rows' entries, None where an entry is not
    written; `slots`, `position`, `sequence` are lists of the new rows alone."""
    table = np.asarray(table)
    n = len(parent) if parent is not None else len(length)
    stride, R = table.shape[1], page_rows
    parent = list(range(n)) if parent is None else [p if 0 <= p < len(length) else -1 for p in parent]
    add = [1] * n if add is None else [int(a) for a in add]
    most = stride * R
    old = [0 if p < 0 else min(max(0, int(length[p])), most) for p in parent]
    rows = [max(0, o + a) for o, a in zip(old, add)]
    keep = [min(o, r) for o, r in zip(old, rows)]
    entry = [[None] * stride for _ in range(n)]
    held, own = set(), [None] * n
    for i in range(n):
        for k in range(-(-keep[i] // R)):
            e = int(table[parent[i], k])
            if not live(k, R, keep[i], window, n_sink):
                entry[i][k] = -1
                continue
            entry[i][k] = e
            if rows[i] > keep[i] and keep[i] % R and k == keep[i] // R:
                own[i] = e  # the row goes on in it
            elif 0 <= e < pages:
                held.add(e)
    copy, taken_by = [False] * n, set()
    for i in range(n):
        if own[i] is None:
            continue
        if not 0 <= own[i] < pages or own[i] in held or own[i] in taken_by:
            copy[i] = True
        else:
            taken_by.add(own[i])
    held |= taken_by
    free = [p for p in range(pages) if p not in held]
    need = [int(c) + -(-r // R) - -(-k // R) for c, r, k in zip(copy, rows, keep)]
    new = sum(r - k for r, k in zip(rows, keep))
    listed = [i for i in range(n) if copy[i] and 0 <= own[i] < pages]
    status = 0
    if any(r > most for r in rows):
        status = 2
    elif listed and not copies_given:
        status = 4
    elif max_new is not None and new > max_new:
        status = 3
    elif sum(need) > len(free):
        status = 1
    if status:
        return dict(table=entry, length=keep, last=[-1] * n, first=[0] * (n + 1), slots=[], position=[], sequence=[],
                    copies=[], result=[status, 0, 0, 0, len(free), 0, 0, 0])
    give, copies, first = iter(free), [], [0]
    slots, position, sequence = [], [], []
    for i in range(n):
        if copy[i]:
            page, k = next(give), keep[i] // R
            if 0 <= own[i] < pages:
                copies.append((own[i], page, keep[i] % R))
            entry[i][k] = page
        for k in range(-(-keep[i] // R), -(-rows[i] // R)):
            entry[i][k] = next(give)
        for t in range(keep[i], rows[i]):
            slots.append(entry[i][t // R] * R + t % R)
            position.append(t)
            sequence.append(i)
        first.append(len(slots))
    return dict(table=entry, length=rows, last=[r - 1 if r > k else -1 for r, k in zip(rows, keep)], first=first,
                slots=slots, position=position, sequence=sequence, copies=copies,
                result=[0, new, len(copies), sum(need), len(free) - sum(need), 0, 0, 0])


def cache_row(buf, pages, page_rows, kv_heads, head_dim, head_major, page, row):
    """[kv_heads][head_dim] view of a row of a cache buffer."""
    if head_major:
        return buf.reshape(pages, kv_heads, page_rows, head_dim)[page, :, row]
    return buf.reshape(pages, page_rows, kv_heads, head_dim)[page, row]


def paged_attention(key, value, pages, page_rows, kv_heads, head_dim, head_major, table, position, q, n_heads, scale,
                    k=None, v=None, gate=None, sequence=None, window=0, n_sink=0):
    """(out, stored): out[i] None for a row that is left as it was; stored: (page, row) that row i's K and V go to, or
    None.  key, value: float16 arrays, not changed."""
    n, D, g = len(position), head_dim, n_heads // kv_heads
    table = np.asarray(table)
    out, stored = [], []
    f64 = np.float64
    for i in range(n):
        t, s = int(position[i]), int(sequence[i]) if sequence is not None else i
        if t < 0 or not 0 <= s < len(table):
            out.append(None)
            stored.append(None)
            continue
        ks, vs = [], []
        for p in range(min(t + (k is None), table.shape[1] * page_rows)):
            if window and not (t - p < window or p < n_sink):
                continue
            page = int(table[s, p // page_rows])
            if 0 <= page < pages:
                ks.append(cache_row(key, pages, page_rows, kv_heads, D, head_major, page, p % page_rows))
                vs.append(cache_row(value, pages, page_rows, kv_heads, D, head_major, page, p % page_rows))
        where = None
        if k is not None:
            ks.append(k[i].astype(np.float16).reshape(kv_heads, D))
            vs.append(v[i].astype(np.float16).reshape(kv_heads, D))
            if t < table.shape[1] * page_rows and 0 <= int(table[s, t // page_rows]) < pages:
                where = (int(table[s, t // page_rows]), t % page_rows)
        stored.append(where)
        o = np.zeros((n_heads, D))
        if ks:
            K, V = np.stack(ks).astype(f64), np.stack(vs).astype(f64)
            for h in range(n_heads):
                z = scale * (K[:, h // g] @ q[i].astype(f64).reshape(n_heads, D)[h])
                with np.errstate(over="ignore", invalid="ignore"):
                    a = np.exp(z - z.max())
                    o[h] = (a @ V[:, h // g]) / a.sum()
        o = o.reshape(-1)
        if gate is not None:
            o = o / (1.0 + np.exp(-gate[i].astype(f64)))
        out.append(o)
    return out, stored


def beam_select(logits, score, groups, beams, n, ended=None, end_token=-1):
    """(parent, token, score, ended): per request the n largest sums of score and log-probability, the sums in 64 bits."""
    V = logits.shape[1]
    outs = ([], [], [], [])
    for g in range(groups):
        best = []
        for r in range(g * beams, (g + 1) * beams):
            s = float(score[r])
            if ended is not None and ended[r]:
                best.append((s, r, end_token))
                continue
            x = logits[r].astype(np.float64)
            with np.errstate(all="ignore"):
                m = x.max()
                total = s + x - (m + np.log(np.exp(x - m).sum()))
            ok = np.flatnonzero(total > -np.inf)
            keep = ok[np.argsort(-total[ok], kind="stable")[:n]]
            best += [(float(total[t]), r, int(t)) for t in keep]
        best = [b for b in best if b[0] > -np.inf]
        best.sort(key=lambda b: (-b[0], b[1], b[2]))
        best = best[:n] + [(-np.inf, -1, -1)] * (n - len(best[:n]))
        for s, r, t in best:
            outs[0].append(r)
            outs[1].append(t)
            outs[2].append(s)
            outs[3].append(1 if r < 0 or t == end_token or (ended is not None and ended[r]) else 0)
    return tuple(np.array(o) for o in outs)
