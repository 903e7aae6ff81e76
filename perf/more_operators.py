"""Measured cases of decoding several sequences, or beams, at once: block tables and slot maps from the sequences'
lengths, attention of one new token over a paged K/V cache, the store of prompt rows into pages, beam search's selection
over beams and vocabulary, and the copy of pages that beams no longer share.

Sizes are those of the decode model whose weights this library streams (32 query heads and 2 K/V heads of 128, windows of
2,048 rows, sessions up to 131,072 rows, 52 layers, 202,048 tokens, 16 rows a pass), and generic ones beside them.
"""
import numpy as np
import torch

own = False
mu = None


def _lib():
    """The library; asked for only where its own calls are measured."""
    global mu
    if mu is None:
        import quantized_weight_streaming_q4_gb300 as library
        mu = library
    return mu


# --------------------------------------------------------------------- cases
# "shortest", "longest": the sequences' lengths are spread between them by _lengths().
def listed():
    return [
        # 16 requests in their first sentences: one step of a batch, one layer
        dict(name="16 sequences, 9 to 190 rows", op="attention", n=16, heads=32, kv_heads=2, head_dim=128, shortest=9,
             longest=190, page_rows=64, head_major=False, window=0, sinks=0, gate=True),
        # one session at its longest in a full-attention layer
        dict(name="1 sequence, 130,815 rows", op="attention", n=1, heads=32, kv_heads=2, head_dim=128, shortest=130815,
             longest=130815, page_rows=64, head_major=True, window=0, sinks=0, gate=True),
        # 16 requests of very different lengths in a full-attention layer
        dict(name="16 sequences, 500 to 40,000 rows", op="attention", n=16, heads=32, kv_heads=2, head_dim=128,
             shortest=500, longest=40000, page_rows=64, head_major=False, window=0, sinks=0, gate=True),
        # another model's heads, more requests than one pass of the weights takes, small pages, a window with sinks
        dict(name="48 sequences, 64-wide heads, window", op="attention", n=48, heads=20, kv_heads=5, head_dim=64,
             shortest=30, longest=5000, page_rows=16, head_major=False, window=1500, sinks=4, gate=False),
        # the tables of the next step of 16 beams, which share the pages of their common past
        dict(name="tables of 16 beams", op="tables", n=16, shortest=500, longest=8000, grow=1, page_rows=64, pages=8192,
             beams=True, window=0, sinks=0),
        # 48 prompts, or parts of prompts, arrive at once
        dict(name="tables of 48 prompts", op="tables", n=48, shortest=30, longest=5000, grow=2000, page_rows=16,
             pages=65536, beams=False, window=0, sinks=0),
        # a beam search of four beams for each of four requests, small vocabulary
        dict(name="4 x 4 beams of 32,768", op="select", groups=4, beams=4, n=4, vocab=32768, ended=False),
        # 16 beams of one request against the model's vocabulary, some of them at their end
        dict(name="16 beams of 202,048", op="select", groups=1, beams=16, n=16, vocab=202048, ended=True),
        # two beams part inside a page, one layer
        dict(name="copy 1 page, 1 layer", op="copy", n=1, layers=1, kv_heads=2, head_dim=128, page_rows=64, pages=256,
             head_major=False),
        # all beams go on from one: 15 pages in every layer
        dict(name="copy 15 pages, 52 layers", op="copy", n=15, layers=52, kv_heads=2, head_dim=128, page_rows=64,
             pages=64, head_major=False),
        # 16 prompt rows, one pass of the weights, one layer
        dict(name="write 16 rows", op="write", rows=16, kv_heads=2, head_dim=128, page_rows=64, pages=256,
             head_major=False),
        # a whole prompt's rows of one layer
        dict(name="write 40,007 rows", op="write", rows=40007, kv_heads=2, head_dim=128, page_rows=64, pages=2048,
             head_major=True),
    ]


HEADS = ((32, 2, 128), (32, 2, 128), (16, 16, 64), (20, 5, 64), (8, 1, 128), (12, 4, 80), (8, 2, 256), (28, 4, 128))


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("attention",) * 5 + ("tables", "tables", "select", "select", "copy", "write"))
    if op == "attention":
        heads, kv_heads, head_dim = rng.choice(HEADS)
        n = rng.choice((1, rng.randint(2, 16), 16, rng.randint(17, 64)))
        # as many rows in all as the largest listed case in bytes, at most
        most = max(2, min(130815, 140000 * 256 // (kv_heads * head_dim) // n))
        lo, hi = sorted((_log(rng, 1, most), _log(rng, 1, most)))
        window = rng.choice((0, 0, rng.randint(1, hi), 2048))
        return dict(op=op, n=n, heads=heads, kv_heads=kv_heads, head_dim=head_dim, shortest=lo, longest=hi,
                    page_rows=rng.choice((16, 32, 64, 64, 128, 256)), head_major=rng.random() < 0.4, window=window,
                    sinks=rng.choice((0, rng.randint(1, 64))) if window else 0, gate=rng.random() < 0.5)
    if op == "tables":
        n, page_rows = rng.randint(1, 48), rng.choice((8, 16, 64, 128))
        beams = rng.random() < 0.5
        lo, hi = sorted((_log(rng, 1, 5000), _log(rng, 1, 5000)))
        grow = 1 if beams else rng.choice((1, 16, _log(rng, 2, 2000)))
        need = n * (hi // page_rows + grow // page_rows + 3)
        window = rng.choice((0, 0, rng.randint(1, 3000)))
        return dict(op=op, n=n, shortest=lo, longest=hi, grow=grow, page_rows=page_rows,
                    pages=min(65536, need + rng.randint(0, need)), beams=beams, window=window,
                    sinks=rng.choice((0, rng.randint(1, 64))) if window else 0)
    if op == "select":
        groups, beams = rng.choice(((1, rng.randint(1, 16)), (2, rng.randint(1, 8)), (4, 4), (16, 1), (3, 5)))
        ended = rng.random() < 0.5
        return dict(op=op, groups=groups, beams=beams, n=beams if ended else beams * rng.choice((1, 2)),
                    vocab=_log(rng, 1000, 202048), ended=ended)
    kv_heads, head_dim = rng.choice(((2, 128), (2, 128), (5, 64), (4, 80), (3, 40)))
    page_rows, head_major = rng.choice((16, 64, 128)), rng.random() < 0.4
    if op == "copy":
        layers = rng.randint(1, 52)
        n = rng.randint(1, 15)
        if layers * page_rows * kv_heads * head_dim > 52 * 64 * 256:
            layers = max(1, 52 * 64 * 256 // (page_rows * kv_heads * head_dim))
        return dict(op=op, n=n, layers=layers, kv_heads=kv_heads, head_dim=head_dim, page_rows=page_rows, pages=64,
                    head_major=head_major)
    rows = _log(rng, 1, 30000)
    return dict(op=op, rows=rows, kv_heads=kv_heads, head_dim=head_dim, page_rows=page_rows,
                pages=rows // page_rows + rng.randint(2, 100), head_major=head_major)


def _lengths(case):
    """The sequences' rows: from the shortest to the longest in even steps of their logarithm, in a mixed order."""
    n, lo, hi = case["n"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    step = next(s for s in (7, 5, 11, 13, 3, 1) if np.gcd(s, n) == 1)
    return [int(round(lo * (hi / lo) ** ((i * step % n) / (n - 1)))) for i in range(n)]


def _growth(case):
    """New rows of every sequence: one a step, else ragged up to `grow`."""
    return [1 if case["grow"] == 1 else 1 + (i * 7919 + 13) % case["grow"] for i in range(case["n"])]


def _parents(case, rng):
    """The sequences that 'n' rows go on from: themselves, or drawn beams."""
    return sorted(rng.randint(0, case["n"], case["n"]).tolist()) if case["beams"] else list(range(case["n"]))


def _live(rows, page_rows, window, sinks):
    """Table entries of a sequence that has `rows` rows and a next one to come, as truth values."""
    k = np.arange(-(-rows // page_rows))
    return (k * page_rows < sinks) | ((k + 1) * page_rows > rows - window + 1) if window else np.ones(len(k), bool)


# -------------------------------------------------------------------- inputs
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda"), \
        lambda *shape: torch.rand(*shape, generator=g, device="cuda"), np.random.RandomState(seed % (2 ** 32))


def prepare(case, seed):
    return {"attention": _prepare_attention, "tables": _prepare_tables, "select": _prepare_select, "copy": _prepare_copy,
            "write": _prepare_write}[case["op"]](case, seed)


def _cuda_ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cache(case, key, value, pages):
    m = _lib()
    return m.KvPages(key.data_ptr(), value.data_ptr(), pages, case["page_rows"], case["kv_heads"] * case["head_dim"],
                     case["head_dim"], int(case["head_major"]), 0)


def _prepare_attention(case, seed):
    normal, _, rng = _rand(seed)
    n, H, G, D, R = case["n"], case["heads"], case["kv_heads"], case["head_dim"], case["page_rows"]
    lens = _lengths(case)
    width = max(lens) // R + 1
    table = np.full((n, width), -1, np.int32)
    live = [np.flatnonzero(_live(t + 1, R, case["window"] + 1 if case["window"] else 0, case["sinks"])) for t in lens]
    pages = sum(len(x) for x in live) + 8
    ids = rng.permutation(pages)
    for i, x in enumerate(live):  # the pages lie anywhere in the cache; those before a window are gone
        table[i, x] = ids[:len(x)]
        ids = ids[len(x):]
    s = dict(case=case, lens=lens, host_table=table, table=_cuda_ints(table), position=_cuda_ints(lens), scale=D ** -0.5,
             q=1.7 * normal(n, H * D), k=normal(n, G * D), v=normal(n, G * D),
             gate=normal(n, H * D) if case["gate"] else None, key=normal(pages * R * G * D).half(),
             value=normal(pages * R * G * D).half(), out=torch.empty(n, H * D, device="cuda"))
    if own:
        m = _lib()
        s["cache"] = _cache(case, s["key"], s["value"], pages)
        s["scratch_bytes"] = m.muser_kv_paged_attention_scratch_bytes(G * D, D, n, H)
        s["scratch"] = torch.zeros(s["scratch_bytes"] // 4, device="cuda")
    return s


def _prepare_tables(case, seed):
    _, _, rng = _rand(seed)
    n, R = case["n"], case["page_rows"]
    lens, grow = _lengths(case), _growth(case)
    parent = _parents(case, rng)
    width = max(lens) // R + max(grow) // R + 2
    table = np.full((n, width), -1, np.int32)
    ids = rng.permutation(case["pages"]).tolist()
    shared = [ids.pop() for _ in range(min(lens) // R // 2)] if case["beams"] else []  # the beams' common past
    for i, rows in enumerate(lens):
        for k in np.flatnonzero(_live(rows, R, case["window"], case["sinks"])):
            table[i, k] = shared[k] if k < len(shared) else ids.pop()
    new = sum(grow)
    s = dict(case=case, host_table=table, host_parent=parent, lens=lens, grow=grow, width=width, new=new,
             table=_cuda_ints(table), length=_cuda_ints(lens), add=_cuda_ints(grow),
             parent=_cuda_ints(parent) if case["beams"] else None,
             table_out=torch.full((n, width), -1, dtype=torch.int32, device="cuda"))
    for name, size in (("length_out", n), ("last", n), ("first", n + 1), ("slots", new), ("position", new),
                       ("sequence", new), ("copies", 3 * n), ("result", 8)):
        s[name] = torch.full((size,), -1, dtype=torch.int32, device="cuda")
    if own:
        _lib()
    return s


def _prepare_select(case, seed):
    normal, uniform, rng = _rand(seed)
    rows, V = case["groups"] * case["beams"], case["vocab"]
    # capped logits as the LM head leaves them: a wide floor and a few likely tokens
    base = 1.6 * normal(rows, V)
    likely = (uniform(rows, 24) * V).long()
    base.scatter_add_(1, likely, 9.0 + 2.0 * normal(rows, 24))
    s = dict(case=case, logits=20.0 * torch.tanh(base / 20.0), score=-20.0 - 2.0 * normal(rows).abs(),
             ended=_cuda_ints(rng.rand(rows) < 0.2) if case["ended"] else None)
    for name, dtype in (("parent", torch.int32), ("token", torch.int32), ("score_out", torch.float32),
                        ("ended_out", torch.int32), ("add", torch.int32)):
        s[name] = torch.empty(case["groups"] * case["n"], dtype=dtype, device="cuda")
    if own:
        m = _lib()
        s["scratch_bytes"] = m.muser_beam_select_scratch_bytes(case["groups"], case["beams"], V, case["n"])
        s["scratch"] = torch.zeros(s["scratch_bytes"] // 4, device="cuda")
    return s


def _prepare_copy(case, seed):
    normal, _, rng = _rand(seed)
    L, R, kv = case["layers"], case["page_rows"], case["kv_heads"] * case["head_dim"]
    ids = rng.permutation(case["pages"])
    copies = [(int(rng.choice(ids[:8])), int(ids[8 + j]), int(rng.randint(1, R + 1))) for j in range(case["n"])]
    s = dict(case=case, host_copies=copies, copies=_cuda_ints(copies), count=_cuda_ints([case["n"]]),
             key=normal(L, case["pages"] * R * kv).half(), value=normal(L, case["pages"] * R * kv).half())
    if own:
        m = _lib()
        s["caches"] = (m.KvPages * L)(*[_cache(case, s["key"][l], s["value"][l], case["pages"]) for l in range(L)])
    return s


def _prepare_write(case, seed):
    normal, _, rng = _rand(seed)
    R, kv, rows, pages = case["page_rows"], case["kv_heads"] * case["head_dim"], case["rows"], case["pages"]
    first = rng.randint(0, min(R, pages * R - rows + 1))
    ids = rng.permutation(pages)
    at = first + np.arange(rows)
    s = dict(case=case, slots=_cuda_ints(ids[at // R] * R + at % R), k=normal(rows, kv), v=normal(rows, kv),
             key=normal(pages * R * kv).half(), value=normal(pages * R * kv).half())
    if own:
        s["cache"] = _cache(case, s["key"], s["value"], pages)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"attention": _plain_attention, "tables": _plain_tables, "select": _plain_select, "copy": _plain_copy,
            "write": _plain_write}[op](s)


TABLES = ("table_out", "length_out", "last", "first", "slots", "position", "sequence", "copies", "result")
SELECT = ("parent", "token", "score_out", "ended_out", "add")


def _own(op, s):
    case = s["case"]
    if op == "attention":
        mu.muser_kv_paged_attention(s["cache"], s["table"], s["position"], s["q"], case["n"], case["heads"], s["out"],
                                    scale=s["scale"], scratch=s["scratch"], scratch_bytes=s["scratch_bytes"], k=s["k"],
                                    v=s["v"], gate=s["gate"], window=case["window"], n_sink=case["sinks"])
        return s["out"], s["key"], s["value"]
    if op == "tables":
        mu.muser_kv_page_tables(s["table"], s["length"], case["n"], case["pages"], case["page_rows"], s["table_out"],
                                s["length_out"], s["result"], parent=s["parent"], add=s["add"], window=case["window"],
                                n_sink=case["sinks"], last=s["last"], first=s["first"], slots=s["slots"],
                                position=s["position"], sequence=s["sequence"], max_new=s["new"], copies=s["copies"])
        return tuple(s[x] for x in TABLES)
    if op == "select":
        mu.muser_beam_select(s["logits"], s["score"], case["groups"], case["beams"], case["vocab"], case["n"], s["parent"],
                             s["token"], s["score_out"], s["scratch"], s["scratch_bytes"], ended=s["ended"], end_token=2,
                             ended_out=s["ended_out"], add=s["add"])
        return tuple(s[x] for x in SELECT)
    if op == "copy":
        mu.muser_kv_page_copy(s["caches"], s["copies"], s["count"], case["n"])
    else:
        mu.muser_kv_page_write(s["cache"], s["k"], s["v"], s["slots"], case["rows"])
    return s["key"], s["value"]


def _pages(buf, case):
    """[pages][page rows][K/V heads][head size] of a cache, whatever its layout."""
    G, D, R = case["kv_heads"], case["head_dim"], case["page_rows"]
    if case["head_major"]:
        return buf.view(-1, G, R, D).transpose(1, 2)
    return buf.view(-1, R, G, D)


def _plain_attention(s):
    case = s["case"]
    n, H, G, D, R = case["n"], case["heads"], case["kv_heads"], case["head_dim"], case["page_rows"]
    w = case["window"]
    key, value = _pages(s["key"], case), _pages(s["value"], case)
    at = s["position"].long()
    page = s["table"].gather(1, (at // R)[:, None])[:, 0].long()
    key[page, at % R] = s["k"].view(n, G, D).half()  # the new rows first: then all that is seen lies in the cache
    value[page, at % R] = s["v"].view(n, G, D).half()
    out = []
    for i, t in enumerate(s["lens"]):
        low = max(0, t - w + 1) if w else 0
        p = torch.arange(t + 1, device="cuda")
        if low:
            p = torch.cat([p[:min(case["sinks"], low)], p[low:]])
        page = s["table"][i, p // R].long()
        keys = key[page, p % R].float().permute(1, 2, 0)
        values = value[page, p % R].float().transpose(0, 1)
        scores = torch.bmm(s["q"][i].view(G, H // G, D), keys) * s["scale"]
        weights = torch.exp(scores - scores.amax(-1, keepdim=True))
        out.append((torch.bmm(weights, values) / weights.sum(-1, keepdim=True)).reshape(H * D))
    out = torch.stack(out)
    return out if s["gate"] is None else out / (1.0 + torch.exp(-s["gate"])), s["key"], s["value"]


def _plain_tables(s):
    case = s["case"]
    n, R, pages, w, sinks, width = case["n"], case["page_rows"], case["pages"], case["window"], case["sinks"], s["width"]
    dev = "cuda"
    row, k = torch.arange(n, device=dev), torch.arange(width, device=dev)
    parent = row if s["parent"] is None else s["parent"].long()
    old = s["length"].long()[parent]
    length = old + s["add"].long()
    h0, h1 = (old + R - 1) // R, (length + R - 1) // R
    live = k[None] < h0[:, None]
    if w:
        live &= (k * R < sinks)[None] | ((k + 1)[None] * R > (old - w + 1)[:, None])
    entry = torch.where(live, s["table"].long()[parent], -1)
    # held pages, but for the partly filled ones that their row goes on in
    partial = (old % R != 0)[:, None] & (k[None] == h0[:, None] - 1)
    held = torch.zeros(pages + 1, dtype=torch.int64, device=dev)
    held.scatter_(0, torch.where(live & ~partial & (entry >= 0), entry, pages).reshape(-1), 1)
    held[pages] = 0
    mine = torch.where(old % R != 0, entry.gather(1, (h0 - 1).clamp_min(0)[:, None])[:, 0], pages)
    same = (mine[:, None] == mine[None]) & (row[None] < row[:, None])
    copy = (mine < pages) & ((held[mine] > 0) | same.any(1))
    held.scatter_(0, torch.where(copy, pages, mine), 1)
    free = torch.where(held[:pages] > 0, pages, torch.arange(pages, device=dev)).sort().values
    need = copy.long() + h1 - h0
    start = torch.cumsum(need, 0) - need
    fresh = start[:, None] + copy.long()[:, None] + k[None] - h0[:, None]
    new = (k[None] >= h0[:, None]) & (k[None] < h1[:, None])
    entry = torch.where(new, free[fresh.clamp(0, pages - 1)], entry)
    entry = torch.where(partial & copy[:, None], free[start.clamp_max(pages - 1)][:, None], entry)
    s["table_out"].copy_(torch.where((k[None] < h1[:, None]), entry, s["table_out"].long()))
    s["length_out"].copy_(length)
    s["last"].copy_(length - 1)
    end = torch.cumsum(length - old, 0)
    s["first"].copy_(torch.cat([torch.zeros_like(end[:1]), end]))
    j = torch.arange(s["new"], device=dev)
    owner = (end[None] <= j[:, None]).sum(1)
    position = j - (end - (length - old))[owner] + old[owner]
    s["slots"].copy_(entry[owner, position // R] * R + position % R)
    s["position"].copy_(position)
    s["sequence"].copy_(owner)
    triple = torch.stack([mine, free[start.clamp_max(pages - 1)], old % R], 1)
    order = torch.where(copy, row, n + row).sort().indices
    count = copy.sum()
    s["copies"].copy_(torch.where((row < count)[:, None], triple[order], s["copies"].view(n, 3).long()).view(-1))
    zero = torch.zeros_like(count)
    left = (held[:pages] == 0).sum() - need.sum()
    s["result"].copy_(torch.stack([zero, end[-1], count, need.sum(), left, zero, zero, zero]))
    return tuple(s[x] for x in TABLES)


def _plain_select(s):
    case = s["case"]
    groups, B, V, n = case["groups"], case["beams"], case["vocab"], case["n"]
    l = s["logits"].double()
    top = l.amax(1, keepdim=True)
    total = s["score"].double()[:, None] + l - (top + torch.log(torch.exp(l - top).sum(1, keepdim=True)))
    if s["ended"] is not None:  # a beam at its end has one way on: the same again
        stay = torch.full_like(total, float("-inf"))
        stay[:, 2] = s["score"].double()
        total = torch.where(s["ended"][:, None] > 0, stay, total)
    value, index = total.view(groups, B * V).sort(dim=1, descending=True, stable=True)
    value, index = value[:, :n].reshape(-1), index[:, :n]
    parent = (index // V + B * torch.arange(groups, device="cuda")[:, None]).reshape(-1)
    token = (index % V).reshape(-1)
    ended = token == 2
    if s["ended"] is not None:
        ended = ended | (s["ended"][parent] > 0)
    return (parent.int(), token.int(), value.float(), ended.int(), 1 - ended.int())


def _plain_copy(s):
    case = s["case"]
    R, kv = case["page_rows"], case["kv_heads"] * case["head_dim"]
    c = s["copies"].view(-1, 3).long()
    row = torch.arange(R, device="cuda")
    for buf in (s["key"], s["value"]):
        if case["head_major"]:
            p = buf.view(case["layers"], -1, case["kv_heads"], R, case["head_dim"])
            keep = (row[None] < c[:, 2:])[None, :, None, :, None]
        else:
            p = buf.view(case["layers"], -1, R, kv)
            keep = (row[None] < c[:, 2:])[None, :, :, None]
        p[:, c[:, 1]] = torch.where(keep, p[:, c[:, 0]], p[:, c[:, 1]])
    return s["key"], s["value"]


def _plain_write(s):
    case = s["case"]
    R, slot = case["page_rows"], s["slots"].long()
    for buf, rows in ((s["key"], s["k"]), (s["value"], s["v"])):
        _pages(buf, case)[slot // R, slot % R] = rows.view(-1, case["kv_heads"], case["head_dim"]).half()
    return s["key"], s["value"]


# -------------------------------------------------------- what has to be done
def work(case):
    if case["op"] == "attention":
        n, H, G, D, w = case["n"], case["heads"], case["kv_heads"], case["head_dim"], case["window"]
        seen = 0
        for t in _lengths(case):
            low = max(0, t - w + 1) if w else 0
            seen += t - low + min(case["sinks"], low)
        rows = 4 * n * (H * D * (2 + case["gate"]) + 2 * G * D) + 4 * n * G * D  # q, out and the gate; k and v, and stored
        return {"bytes": 4 * seen * G * D + rows, "flops": 4 * D * H * (seen + n)}
    if case["op"] == "tables":
        R = case["page_rows"]
        before = sum(int(_live(t, R, case["window"], case["sinks"]).sum()) for t in _lengths(case))
        grow = _growth(case)
        return {"bytes": 4 * (2 * before + sum(g // R for g in grow) + 3 * sum(grow) + 8 * case["n"]),
                "flops": before + 3 * sum(grow)}
    if case["op"] == "select":
        rows = case["groups"] * case["beams"]
        return {"bytes": 4 * rows * case["vocab"] + 20 * case["groups"] * case["n"], "flops": 4 * rows * case["vocab"]}
    kv = case["kv_heads"] * case["head_dim"]
    if case["op"] == "copy":
        rows = case["n"] * (case["page_rows"] + 1) // 2  # a copied page is half full in the mean
        return {"bytes": 8 * case["layers"] * rows * kv, "flops": 2 * case["layers"] * rows * kv}
    return {"bytes": 12 * case["rows"] * kv, "flops": 2 * case["rows"] * kv}


# ----------------------------------------------------------- the definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "tables": _exact_tables, "select": _exact_select, "copy": _exact_copy,
            "write": _exact_write}[case["op"]](case, s)


def _exact_attention(case, s):
    """Sequence by sequence and head by head: the rows that the token sees are listed, then a softmax in 64 bits."""
    n, H, G, D, R, w = (case[x] for x in ("n", "heads", "kv_heads", "head_dim", "page_rows", "window"))
    key, value, f64 = s["key"].clone(), s["value"].clone(), torch.float64
    out = torch.empty(n, H, D, dtype=f64, device="cuda")
    g = H // G

    def rows(buf, i, c, seen):
        slot = s["table"][i].long().index_select(0, seen // R) * R + seen % R
        if case["head_major"]:
            return buf.view(-1, D).index_select(0, (slot // R * G + c) * R + slot % R)
        return buf.view(-1, G * D).index_select(0, slot)[:, c * D:(c + 1) * D]

    for i in range(n):
        t = s["lens"][i]
        seen = [p for p in range(t) if not w or t - p < w or p < case["sinks"]]
        seen = torch.tensor(seen, dtype=torch.long, device="cuda")
        for c in range(G):
            k = torch.cat([rows(s["key"], i, c, seen), s["k"][i:i + 1, c * D:(c + 1) * D].half()]).to(f64)
            v = torch.cat([rows(s["value"], i, c, seen), s["v"][i:i + 1, c * D:(c + 1) * D].half()]).to(f64)
            a = torch.softmax(s["scale"] * (s["q"][i].view(H, D)[c * g:(c + 1) * g].to(f64) @ k.T), 1)
            out[i, c * g:(c + 1) * g] = a @ v
        page, r = int(s["host_table"][i, t // R]), t % R
        for buf, new in ((key, s["k"]), (value, s["v"])):
            row = new[i].half()
            if case["head_major"]:
                buf.view(-1, G, R, D)[page, :, r] = row.view(G, D)
            else:
                buf.view(-1, R, G * D)[page, r] = row
    out = out.view(n, H * D)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].to(f64))
    return out, key, value


def _exact_tables(case, s):
    """One row after another, as the tables are defined, in plain Python."""
    n, R, pages, width = case["n"], case["page_rows"], case["pages"], s["width"]
    table = np.full((n, width), -1, np.int64)
    lens, held, writer = [], set(), {}
    for i, p in enumerate(s["host_parent"]):
        rows = s["lens"][p]
        lens.append(rows)
        for k in np.flatnonzero(_live(rows, R, case["window"], case["sinks"])):
            table[i, k] = s["host_table"][p, k]
            if (k + 1) * R <= rows:
                held.add(int(table[i, k]))
    copied = []
    for i in range(n):
        if lens[i] % R:
            page = int(table[i, lens[i] // R])
            if page in held or page in writer:
                copied.append(i)
            else:
                writer[page] = i
    free = iter([p for p in range(pages) if p not in held and p not in writer])
    taken, copies, slots, position, sequence, first = 0, [], [], [], [], [0]
    for i in range(n):
        if i in copied:
            k, page = lens[i] // R, next(free)
            taken += 1
            copies += [int(table[i, k]), page, lens[i] % R]
            table[i, k] = page
        for t in range(lens[i], lens[i] + s["grow"][i]):
            if t % R == 0:
                table[i, t // R] = next(free)
                taken += 1
            slots.append(table[i, t // R] * R + t % R)
            position.append(t)
            sequence.append(i)
        first.append(len(slots))
    left = sum(1 for _ in free)
    result = [0, len(slots), len(copied), taken, left, 0, 0, 0]
    length = [a + b for a, b in zip(lens, s["grow"])]
    copies += [-1] * (3 * n - len(copies))
    return tuple(torch.tensor(np.asarray(x), dtype=torch.int32)
                 for x in (table, length, [x - 1 for x in length], first, slots, position, sequence, copies, result))


def _exact_select(case, s):
    """A heap's work done by numpy: the rows' candidates in 64 bits, the best one taken again and again."""
    groups, B, V, n = case["groups"], case["beams"], case["vocab"], case["n"]
    logits, score = s["logits"].cpu().numpy(), s["score"].cpu().numpy().astype(np.float64)
    ended = np.zeros(groups * B, bool) if s["ended"] is None else s["ended"].cpu().numpy() > 0
    parent, token, total = [], [], []
    for g in range(groups):
        best = []
        for r in range(g * B, (g + 1) * B):
            if ended[r]:
                best.append((-score[r], r, 2))
                continue
            x = logits[r].astype(np.float64)
            lse = np.logaddexp.reduce(x) if V < 5000 else x.max() + np.log(np.exp(x - x.max()).sum())
            floor = np.partition(x, V - n)[V - n]
            for v in np.flatnonzero(x >= floor):
                best.append((-(score[r] + x[v] - lse), r, int(v)))
        for t, r, v in sorted(best)[:n]:
            parent.append(r)
            token.append(v)
            total.append(-t)
    end = [int(ended[r] or v == 2) for r, v in zip(parent, token)]
    ints = [torch.tensor(x, dtype=torch.int32) for x in (parent, token, end, [1 - e for e in end])]
    return ints[0], ints[1], torch.tensor(total, dtype=torch.float64), ints[2], ints[3]


def _exact_copy(case, s):
    G, D, R = case["kv_heads"], case["head_dim"], case["page_rows"]
    both = []
    for buf in (s["key"], s["value"]):
        new = buf.clone()
        for src, dst, rows in s["host_copies"]:
            for l in range(case["layers"]):
                shape = (-1, G, R, D) if case["head_major"] else (-1, 1, R, G * D)
                new[l].view(shape)[dst, :, :rows] = buf[l].view(shape)[src, :, :rows]
        both.append(new)
    return tuple(both)


def _exact_write(case, s):
    G, D, R = case["kv_heads"], case["head_dim"], case["page_rows"]
    slots = s["slots"].cpu().numpy()
    both = []
    for buf, rows in ((s["key"], s["k"]), (s["value"], s["v"])):
        new = buf.cpu().numpy().copy()
        rows = rows.cpu().numpy().astype(np.float64).astype(np.float16)
        if case["head_major"]:
            new.reshape(-1, G, R, D)[slots // R, :, slots % R] = rows.reshape(-1, G, D)
        else:
            new.reshape(-1, G * D)[slots] = rows
        both.append(torch.from_numpy(new))
    return tuple(both)
