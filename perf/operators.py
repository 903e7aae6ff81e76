"""Measured cases of the speculative decode step: attention of drafted rows over the K/V ring, verification of the
drafts against the target's probabilities, and the append of the accepted rows to every layer's ring.

Sizes are those of the decode model whose weights this library streams (32 query heads and 2 K/V heads of 128, rings
of 2,048 rows, growing planes up to 131,072 rows, 52 layers, 202,048 tokens, at most 16 rows), and generic ones
beside them.
"""
import ctypes

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
# "tree": drafted rows hang on row max(0, i - tree); 1 is a chain, 0 the binary tree (parent (i - 1) // 2).
def listed():
    return [
        # the first tokens of an answer: 37 rows in a sliding-window layer's ring
        dict(name="token, 37 rows", op="attention", M=1, heads=32, kv_heads=2, head_dim=128, len=37, capacity=2048,
             origin=0, head_major=False, window=2048, sinks=0, tree=1, gate=True),
        # one token of a sliding-window layer deep in a session: the ring is full and turned, four first tokens kept
        dict(name="token, full ring, sinks", op="attention", M=1, heads=32, kv_heads=2, head_dim=128, len=2048,
             capacity=2048, origin=10347, head_major=False, window=2048, sinks=4, tree=1, gate=True),
        # one token of a full-attention layer at the end of the longest session
        dict(name="token, 130,815 rows", op="attention", M=1, heads=32, kv_heads=2, head_dim=128, len=130815,
             capacity=131072, origin=0, head_major=True, window=0, sinks=0, tree=1, gate=True),
        # a whole drafted block with three branches in a sliding-window layer
        dict(name="16 rows, full ring, sinks", op="attention", M=16, heads=32, kv_heads=2, head_dim=128, len=2048,
             capacity=2048, origin=10347, head_major=False, window=2048, sinks=4, tree=3, gate=True),
        # a whole drafted chain in a full-attention layer at the end of the longest session
        dict(name="16 rows, 130,815 rows", op="attention", M=16, heads=32, kv_heads=2, head_dim=128, len=130815,
             capacity=131072, origin=0, head_major=True, window=0, sinks=0, tree=1, gate=True),
        # another model's heads: groups of four, 64 wide, five rows in a binary tree, a window with sinks in one plane
        dict(name="5 rows, 64-wide heads, window", op="attention", M=5, heads=20, kv_heads=5, head_dim=64, len=7001,
             capacity=8192, origin=0, head_major=False, window=4097, sinks=16, tree=0, gate=False),
        # plain sampling of one token from a small vocabulary
        dict(name="sample, 32,768 tokens", op="verify", M=1, vocab=32768, tree=1, temperature=0.8, drafted=False),
        # a drafted chain of fifteen against the model's vocabulary
        dict(name="chain of 15, 202,048 tokens", op="verify", M=16, vocab=202048, tree=1, temperature=1.0, drafted=True),
        # fifteen drafts in a binary tree: siblings are tried in turn on what the rejected ones left
        dict(name="tree of 15, 202,048 tokens", op="verify", M=16, vocab=202048, tree=0, temperature=0.7, drafted=True),
        # greedy decoding with eight drafts
        dict(name="greedy, 8 drafts", op="verify", M=9, vocab=202048, tree=2, temperature=0.0, drafted=False),
        # one accepted row in one ring
        dict(name="append 1 row, 1 ring", op="commit", M=1, n=1, planes=1, kv_heads=2, head_dim=128, capacity=2048,
             position=900, head_major=False),
        # five accepted of sixteen drafted rows in the rings of all layers
        dict(name="append 5 of 16, 52 rings", op="commit", M=16, n=5, planes=52, kv_heads=2, head_dim=128,
             capacity=2048, position=12345, head_major=False),
    ]


HEADS = ((32, 2, 128), (32, 2, 128), (16, 16, 64), (20, 5, 64), (8, 1, 128), (12, 4, 80), (8, 2, 256), (28, 4, 128))


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "verify", "verify", "commit"))
    if op == "attention":
        heads, kv_heads, head_dim = rng.choice(HEADS)
        ring = rng.random() < 0.5
        M = rng.choice((1, 1, rng.randint(2, 7), rng.randint(8, 16), 16))
        # wide caches stay as long as the largest listed one is in bytes
        most = min(130815, 130815 * 256 // (kv_heads * head_dim))
        if M * heads * head_dim > 32 * 128 * 16 or head_dim > 128:
            most = min(most, 30000)
        if ring:
            capacity = rng.choice((512, 1000, 2048, 4096))
            n = rng.choice((capacity, rng.randint(1, capacity)))
            origin = rng.randint(1, 100000) if n == capacity else 0
            window = rng.choice((capacity, capacity, rng.randint(1, capacity)))
        else:
            n = _log(rng, 1, most)
            capacity, origin = n + rng.randint(0, 500), 0
            window = rng.choice((0, 0, rng.randint(1, n)))
        return dict(op=op, M=M, heads=heads, kv_heads=kv_heads, head_dim=head_dim, len=n, capacity=capacity,
                    origin=origin, head_major=not ring and rng.random() < 0.7, window=window,
                    sinks=rng.choice((0, rng.randint(1, 64))) if window else 0, tree=rng.choice((0, 1, 1, 2, 3, 5)),
                    gate=rng.random() < 0.5)
    if op == "verify":
        M = rng.choice((1, rng.randint(2, 8), rng.randint(9, 16)))
        return dict(op=op, M=M, vocab=_log(rng, 1000, 202048), tree=rng.choice((0, 1, 1, 2, 3, 15)),
                    temperature=rng.choice((0.0, 1.0, round(rng.uniform(0.3, 1.5), 3))), drafted=rng.random() < 0.7)
    M = rng.randint(1, 16)
    kv_heads, head_dim = rng.choice(((2, 128), (2, 128), (5, 64), (4, 80), (3, 40)))
    return dict(op=op, M=M, n=rng.randint(1, M), planes=rng.randint(1, 52), kv_heads=kv_heads, head_dim=head_dim,
                capacity=rng.choice((256, 1000, 2048)), position=rng.randint(0, 50000), head_major=rng.random() < 0.3)


def _parents(case):
    M, w = case["M"], case["tree"]
    return [-1] + [(i - 1) // 2 if w == 0 else max(0, i - w) for i in range(1, M)]


def _ancestors(parents):
    """[M][M] truth values: column j is row i or one of its ancestors."""
    M = len(parents)
    anc = np.eye(M, dtype=bool)
    for i in range(1, M):
        anc[i] |= anc[parents[i]]
    return anc


def _sink_rows(case):
    """First tokens that the ring itself no longer holds and that are kept in a plane of their own."""
    return min(case["sinks"], case["origin"])


# -------------------------------------------------------------------- inputs
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda"), \
        lambda *shape: torch.rand(*shape, generator=g, device="cuda")


def prepare(case, seed):
    return {"attention": _prepare_attention, "verify": _prepare_verify, "commit": _prepare_commit}[case["op"]](case, seed)


def _prepare_attention(case, seed):
    normal, _ = _rand(seed)
    M, H, G, D, cap = case["M"], case["heads"], case["kv_heads"], case["head_dim"], case["capacity"]
    s = dict(case=case, scale=D ** -0.5, parents=_parents(case))
    anc = _ancestors(s["parents"])
    s["ancestors"] = torch.from_numpy(anc).cuda()
    s["depth"] = torch.from_numpy(anc.sum(1) - 1).cuda()
    # normalised keys and queries: scores of a few units, so that some rows of the cache matter more than others
    s["q"] = 1.7 * normal(M, H * D)
    s["k"], s["v"] = normal(M, G * D), normal(M, G * D)
    s["gate"] = normal(M, H * D) if case["gate"] else None
    s["key"], s["value"] = normal(cap * G * D).half(), normal(cap * G * D).half()
    ns = _sink_rows(case)
    s["sink_key"] = normal(ns * G * D).half() if ns else None
    s["sink_value"] = normal(ns * G * D).half() if ns else None
    s["out"] = torch.empty(M, H * D, device="cuda")
    if own:
        m = _lib()
        s["plane"] = m.KvPlane(s["key"].data_ptr(), s["value"].data_ptr(), cap, case["len"], case["origin"],
                               case["origin"] % cap, G * D, D, int(case["head_major"]), 0)
        s["sink"] = m.KvPlane(s["sink_key"].data_ptr(), s["sink_value"].data_ptr(), ns, ns, 0, 0, G * D, D, 0, 0) \
            if ns else None
        s["parent"] = (ctypes.c_int32 * M)(*s["parents"])
        s["scratch_bytes"] = m.muser_kv_tree_attention_scratch_bytes(G * D, D, M, H)
        s["scratch"] = torch.zeros(s["scratch_bytes"] // 4, device="cuda")
    return s


def _prepare_verify(case, seed):
    normal, uniform = _rand(seed)
    M, V, T = case["M"], case["vocab"], case["temperature"]
    parents = _parents(case)
    # capped logits as the LM head leaves them: a wide floor and a few likely tokens; the drafter is a noisy copy
    base = 1.6 * normal(M, V)
    likely = (uniform(M, 24) * V).long()
    base.scatter_add_(1, likely, 9.0 + 2.0 * normal(M, 24))
    target = 20.0 * torch.tanh(base / 20.0)
    draft = 20.0 * torch.tanh((base + 0.6 * normal(M, V)) / 20.0)
    t = T if T > 0 else 0.2
    noise = -torch.log(-torch.log(uniform(M, V).clamp_(1e-12, 1.0 - 1e-7)))
    up = torch.tensor([max(p, 0) for p in parents], device="cuda")
    tokens = (draft[up] / t + noise).argmax(1).to(torch.int32)  # each drafted token is drawn from its parent's row
    del noise, base
    s = dict(case=case, target=target, tokens=tokens, parents=parents, uniform=uniform(M),
             draft=draft if case["drafted"] and T > 0 else None,
             ancestors=torch.from_numpy(_ancestors(parents)).cuda(), up=up,
             result=torch.empty(M + 2, dtype=torch.int32, device="cuda"))
    rank = [sum(parents[j] == parents[i] for j in range(1, i)) for i in range(M)]
    s["rank"] = torch.tensor(rank, device="cuda")
    s["ranks"] = max(rank[1:], default=-1) + 1
    # siblings[i][j]: j is an earlier child of i's parent
    s["siblings"] = torch.tensor([[0 < j < i and parents[j] == parents[i] for j in range(M)] for i in range(M)]).cuda()
    s["children"] = torch.tensor([[parents[j] == i for j in range(M)] for i in range(M)]).cuda()
    if own:
        m = _lib()
        s["parent"] = (ctypes.c_int32 * M)(*parents)
        s["scratch_bytes"] = m.muser_tree_verify_scratch_bytes(V, M)
        s["scratch"] = torch.zeros(max(1, s["scratch_bytes"] // 4), device="cuda")
    return s


def _prepare_commit(case, seed):
    normal, _ = _rand(seed)
    L, M, n, G, D, cap = case["planes"], case["M"], case["n"], case["kv_heads"], case["head_dim"], case["capacity"]
    rng = np.random.RandomState(seed % (2 ** 32))
    path = [0] + sorted(int(i) for i in rng.choice(np.arange(1, M), n - 1, replace=False)) if n > 1 else [0]
    rows = min(case["position"], cap)
    s = dict(case=case, path=path, key=normal(L, cap * G * D).half(), value=normal(L, cap * G * D).half(),
             k=normal(L, M, G * D), v=normal(L, M, G * D),
             paths=torch.tensor(path, device="cuda"))
    if own:
        m = _lib()
        origin = case["position"] - rows
        step = cap * G * D * 2
        s["planes"] = (m.KvPlane * L)(*[m.KvPlane(s["key"].data_ptr() + l * step, s["value"].data_ptr() + l * step, cap,
                                                  rows, origin, origin % cap, G * D, D, int(case["head_major"]), 0)
                                        for l in range(L)])
        s["before"] = bytes(s["planes"])
        row = M * G * D * 4
        s["ks"] = (ctypes.c_void_p * L)(*[s["k"].data_ptr() + l * row for l in range(L)])
        s["vs"] = (ctypes.c_void_p * L)(*[s["v"].data_ptr() + l * row for l in range(L)])
        s["rows"] = (ctypes.c_int32 * n)(*path)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"attention": _plain_attention, "verify": _plain_verify, "commit": _plain_commit}[op](s)


def _own(op, s):
    case = s["case"]
    if op == "attention":
        mu.muser_kv_tree_attention(s["plane"], s["q"], s["k"], s["v"], case["M"], case["heads"], s["out"],
                                   scale=s["scale"], scratch=s["scratch"], scratch_bytes=s["scratch_bytes"],
                                   parent=s["parent"], window=case["window"], n_sink=case["sinks"], sink=s["sink"],
                                   gate=s["gate"])
        return s["out"]
    if op == "verify":
        mu.muser_tree_verify(s["target"], s["draft"], s["tokens"], s["parent"], case["M"], case["vocab"],
                             case["temperature"], s["uniform"], s["result"], s["scratch"], s["scratch_bytes"])
        return s["result"]
    ctypes.memmove(s["planes"], s["before"], len(s["before"]))  # the planes' lengths as before the append
    mu.muser_kv_tree_commit(s["planes"], s["ks"], s["vs"], case["M"], s["rows"], case["position"])
    return s["key"], s["value"]


def _rows(buf, case, slots):
    """[K/V heads][rows][head_dim] in 32 bits of the plane's rows in these slots."""
    G, D = case["kv_heads"], case["head_dim"]
    if case["head_major"]:
        return buf.view(G, -1, D)[:, slots].float()
    return buf.view(-1, G, D)[slots].float().transpose(0, 1)


def _plain_attention(s):
    case = s["case"]
    M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["head_dim"]
    o, n, cap, w, sinks = case["origin"], case["len"], case["capacity"], case["window"], case["sinks"]
    logical = o + torch.arange(n, device="cuda")
    slots = logical % cap
    keys = [_rows(s["key"], case, slots), s["k"].half().float().view(M, G, D).transpose(0, 1)]
    values = [_rows(s["value"], case, slots), s["v"].half().float().view(M, G, D).transpose(0, 1)]
    at = o + n + s["depth"]
    position, allowed = [logical, at], [torch.ones(M, n, dtype=torch.bool, device="cuda"), s["ancestors"]]
    if s["sink_key"] is not None:
        ns = _sink_rows(case)
        keys.insert(0, s["sink_key"].view(ns, G, D).float().transpose(0, 1))
        values.insert(0, s["sink_value"].view(ns, G, D).float().transpose(0, 1))
        position.insert(0, torch.arange(ns, device="cuda"))
        allowed.insert(0, torch.ones(M, ns, dtype=torch.bool, device="cuda"))
    keys, values, position, allowed = torch.cat(keys, 1), torch.cat(values, 1), torch.cat(position), torch.cat(allowed, 1)
    if w:
        allowed = allowed & ((at[:, None] - position[None] < w) | (position[None] < sinks))
    q = s["q"].view(M, G, H // G, D).permute(1, 0, 2, 3).reshape(G, M * (H // G), D)
    scores = (torch.bmm(q, keys.transpose(1, 2)) * s["scale"]).view(G, M, H // G, -1)
    scores = torch.where(allowed[None, :, None], scores, float("-inf"))
    weights = torch.exp(scores - scores.amax(-1, keepdim=True))
    total = weights.sum(-1, keepdim=True)
    out = (torch.bmm(weights.view(G, M * (H // G), -1), values).view(G, M, H // G, D) / total)
    out = out.permute(1, 0, 2, 3).reshape(M, H * D)
    return out if s["gate"] is None else out / (1.0 + torch.exp(-s["gate"]))


def _plain_verify(s):
    case = s["case"]
    M, V, T = case["M"], case["vocab"], case["temperature"]
    token = s["tokens"].long()
    row = torch.arange(M, device="cuda")
    if T == 0:
        best = s["target"].argmax(1)
        accepted = token == best[s["up"]]
    else:
        z = s["target"].double() / T
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        px = p[s["up"], token]
        if s["draft"] is not None:
            z = s["draft"].double() / T
            q = torch.exp(z - z.amax(1, keepdim=True))
            q = q / q.sum(1, keepdim=True)
            qx = q[s["up"], token]
            c, left = torch.zeros(M, 1, device="cuda", dtype=torch.float64), torch.ones(M, 1, device="cuda", dtype=torch.float64)
            cs, lefts = [c], [left]
            for _ in range(s["ranks"]):  # what is left of each row's target after its k-th rejected child
                c = c + left
                left = (p - c * q).clamp_min(0).sum(1, keepdim=True)
                cs.append(c)
                lefts.append(left)
            cs, lefts = torch.cat(cs, 1), torch.cat(lefts, 1)
            c, left = cs[s["up"], s["rank"]], lefts[s["up"], s["rank"]]
            accepted = s["uniform"].double() * left * qx < (px - c * qx).clamp_min(0)
        else:
            same = s["siblings"] & (token[:, None] == token[None])
            first = ~same.any(1)
            earlier = s["siblings"] & first[None]
            left = 1.0 - (earlier * px[None]).sum(1)
            accepted = first & (s["uniform"].double() * left < px)
    accepted = accepted & ~(s["siblings"] & accepted[None]).any(1)  # the first accepted child is taken
    accepted = accepted | (row == 0)
    kept = (accepted[None] | ~s["ancestors"]).all(1)
    count = kept.sum()
    last = torch.where(kept, row, -1).amax()
    if T == 0:
        following = best[last]
    else:
        w = p[last]
        tried = s["children"][last]
        if s["draft"] is not None:
            k = tried.sum()
            w = (w - cs[last, k] * q[last]).clamp_min(0)
        else:
            w = torch.where(torch.zeros_like(w).scatter_add(0, token, tried.double()) > 0, 0.0, w)
        w = torch.where(w.sum() > 0, w, p[last])
        cumulated = torch.cumsum(w, 0)
        following = (cumulated <= s["uniform"][0].double() * cumulated[-1]).sum().clamp_max(V - 1)
    order = torch.where(kept, row, M + row).sort().values
    rows = torch.where(order < M, order, -1)
    return torch.cat([count[None], following[None], rows]).to(torch.int32)


def _plain_commit(s):
    case = s["case"]
    L, n, G, D, cap = case["planes"], case["n"], case["kv_heads"], case["head_dim"], case["capacity"]
    slots = (case["position"] + torch.arange(n, device="cuda")) % cap
    k, v = s["k"][:, s["paths"]].half(), s["v"][:, s["paths"]].half()
    if case["head_major"]:
        s["key"].view(L, G, cap, D)[:, :, slots] = k.view(L, n, G, D).transpose(1, 2)
        s["value"].view(L, G, cap, D)[:, :, slots] = v.view(L, n, G, D).transpose(1, 2)
    else:
        s["key"].view(L, cap, G * D)[:, slots] = k
        s["value"].view(L, cap, G * D)[:, slots] = v
    return s["key"], s["value"]


# -------------------------------------------------------- what has to be done
def work(case):
    if case["op"] == "attention":
        M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["head_dim"]
        anc = _ancestors(_parents(case))
        depth = anc.sum(1) - 1
        o, n, w, sinks = case["origin"], case["len"], case["window"], case["sinks"]
        ns = _sink_rows(case)
        seen, union = 0, 0
        for i in range(M):
            low = max(o, o + n + int(depth[i]) - w + 1) if w else o
            low = min(low, o + n)
            cached = o + n - low + min(max(0, min(sinks, o + n) - o), low - o)
            tree = int(anc[i].sum()) if not w else int((anc[i] & (depth[i] - depth < w)).sum())
            seen += ns + cached + tree
            union = max(union, ns + cached)
        rows = 4 * M * (H * D * (2 + case["gate"]) + 2 * G * D)  # q, out and the gate; k and v
        return {"bytes": 4 * union * G * D + rows, "flops": 4 * D * H * seen}
    if case["op"] == "verify":
        parents = _parents(case)
        rows = case["M"] + (len(set(parents[1:])) if case["drafted"] and case["temperature"] > 0 else 0)
        return {"bytes": rows * case["vocab"] * 4, "flops": rows * case["vocab"] * (1 if case["temperature"] == 0 else 5)}
    elements = 2 * case["planes"] * case["n"] * case["kv_heads"] * case["head_dim"]
    return {"bytes": 6 * elements, "flops": elements}


# ----------------------------------------------------------- the definition
def exact(case, seed):
    s = {"attention": _prepare_attention, "verify": _prepare_verify, "commit": _prepare_commit}[case["op"]](case, seed)
    return {"attention": _exact_attention, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](case, s)


def _exact_attention(case, s):
    """Row by row: the rows that a query sees are listed one after another, then a softmax in 64 bits."""
    M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["head_dim"]
    o, n, cap, w, sinks = case["origin"], case["len"], case["capacity"], case["window"], case["sinks"]
    parents, g, f64 = s["parents"], H // G, torch.float64
    depth = [0] * M
    for i in range(1, M):
        depth[i] = depth[parents[i]] + 1
    out = torch.empty(M, H, D, dtype=f64, device="cuda")
    key = s["key"].view(G, cap, D) if case["head_major"] else s["key"].view(cap, G, D).permute(1, 0, 2)
    value = s["value"].view(G, cap, D) if case["head_major"] else s["value"].view(cap, G, D).permute(1, 0, 2)
    for i in range(M):
        t = o + n + depth[i]
        low = max(o, t - w + 1) if w else o
        cached = list(range(o, min(sinks, low, o + n))) + list(range(low, o + n)) if w else list(range(o, o + n))
        cached = torch.tensor(cached, dtype=torch.long, device="cuda") % cap
        line, j = [], i
        while j >= 0:
            if not w or depth[i] - depth[j] < w or o + n + depth[j] < sinks:
                line.append(j)
            j = parents[j]
        line = torch.tensor(line, dtype=torch.long, device="cuda")
        for c in range(G):
            K = [key[c].index_select(0, cached).to(f64), s["k"][line, c * D:(c + 1) * D].half().to(f64)]
            V = [value[c].index_select(0, cached).to(f64), s["v"][line, c * D:(c + 1) * D].half().to(f64)]
            if s["sink_key"] is not None:
                K.append(s["sink_key"].view(-1, G, D)[:, c].to(f64))
                V.append(s["sink_value"].view(-1, G, D)[:, c].to(f64))
            K, V = torch.cat(K), torch.cat(V)
            a = torch.softmax(s["scale"] * (s["q"][i].view(H, D)[c * g:(c + 1) * g].to(f64) @ K.T), 1)
            out[i, c * g:(c + 1) * g] = a @ V
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].to(f64)).view(M, H, D)
    return out.reshape(M, H * D)


def _exact_verify(case, s):
    """The walk as it is defined, one drafted row after another, in numpy."""
    M, V, T = case["M"], case["vocab"], case["temperature"]
    target, tokens, u = s["target"].cpu().numpy(), s["tokens"].cpu().numpy(), s["uniform"].cpu().numpy().astype(np.float64)
    draft = None if s["draft"] is None else s["draft"].cpu().numpy()

    def softmax(x):
        e = np.exp((x.astype(np.float64) - float(x.max())) / T)
        return e / e.sum()

    kept, cur = [0], 0
    while True:
        row = target[cur]
        children = [i for i in range(1, M) if s["parents"][i] == cur]
        taken = None
        if T == 0:
            best = int(row.argmax())
            taken = next((i for i in children if tokens[i] == best), None)
        else:
            p = softmax(row)
            r, q = p.copy(), None if draft is None else softmax(draft[cur])
            for i in children:
                x = int(tokens[i])
                if q is None:
                    if u[i] * r.sum() < r[x]:
                        taken = i
                        break
                    r[x] = 0.0
                else:
                    if u[i] * q[x] < r[x]:
                        taken = i
                        break
                    r = np.maximum(r - q, 0.0)
                    if r.sum() > 0:
                        r /= r.sum()
        if taken is None:
            break
        kept.append(taken)
        cur = taken
    if T == 0:
        following = best
    else:
        r = r if r.sum() > 0 else p
        total = np.cumsum(r)
        following = min(int(np.searchsorted(total, u[0] * total[-1], side="right")), V - 1)
    return torch.tensor([len(kept), following] + kept + [-1] * (M - len(kept)), dtype=torch.int32)


def _exact_commit(case, s):
    L, G, D, cap = case["planes"], case["kv_heads"], case["head_dim"], case["capacity"]
    both = []
    for plane, rows in ((s["key"], s["k"]), (s["value"], s["v"])):
        plane, rows = plane.cpu().numpy().copy(), rows.cpu().numpy()
        for j, i in enumerate(s["path"]):
            slot = (case["position"] + j) % cap
            new = rows[:, i].astype(np.float64).astype(np.float16)
            if case["head_major"]:
                plane.reshape(L, G, cap, D)[:, :, slot] = new.reshape(L, G, D)
            else:
                plane.reshape(L, cap, G * D)[:, slot] = new
        both.append(torch.from_numpy(plane))
    return tuple(both)
