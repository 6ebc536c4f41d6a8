"""Measured cases of the drafted-tree and paged-cache operators.

``listed()`` names the cases, ``prepare`` makes a case's inputs on the GPU,
``run`` makes one pass: the plain form in elementary torch operations, or
(``own``) the calls a user makes of this package.  ``exact`` gives the
operators' values from their definitions in 64 bits.

Four operations:

* ``attend``: attention of a tree of drafted tokens (or a chain, or a single
  token) over a paged key/value cache and the tree itself;
* ``verify``: greedy verification of a drafted tree, the longest path from
  the root that follows the target's choices;
* ``commit``: the accepted path's keys and values appended to the paged
  caches of all layers (new pages, shared last pages copied first), then the
  sequences taken back to their lengths before (pages given up);
* ``step``: a beam step on paged caches, every slot takes its parent's pages
  (shared), appends one token (its last page copied first where it is shared),
  and gives the token up again.
"""

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _attend(name, B, N, Hq, Hkv, D, length, page, dtype, tree, ragged):
    return {"name": name, "op": "attend", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "length": length,
            "page": page, "dtype": dtype, "tree": tree, "ragged": ragged}


def listed():
    return [
        # one interactive request, one token at a time: latency
        _attend("attend one token", 1, 1, 32, 8, 128, 777, 16, "bf16", False, False),
        # one interactive request, a tree of drafts after a document
        _attend("attend one tree", 1, 60, 32, 8, 128, 8191, 16, "bf16", True, False),
        # a small batch of mixed requests: short and long, some idle, seven heads to a group, pages that end inside a tile
        _attend("attend odd batch", 9, 13, 28, 4, 80, 3001, 24, "f16", True, True),
        # two very long contexts, a chain of five drafts
        _attend("attend long contexts", 2, 6, 32, 8, 128, 100000, 64, "bf16", False, False),
        # a full serving batch with trees
        _attend("attend batch", 64, 32, 64, 8, 128, 4096, 64, "bf16", True, True),
        # one request's tree: latency
        {"name": "verify one tree", "op": "verify", "B": 1, "N": 16, "V": 32000, "dtype": "f32", "pad": 0, "ragged": False},
        # a small batch, odd vocabulary, ragged trees, rows padded to a stride
        {"name": "verify odd trees", "op": "verify", "B": 5, "N": 31, "V": 129281, "dtype": "f16", "pad": 3, "ragged": True},
        # a full batch
        {"name": "verify batch", "op": "verify", "B": 64, "N": 32, "V": 128256, "dtype": "bf16", "pad": 0, "ragged": False},
        # one request's accepted path into 24 layers: latency
        {"name": "commit one path", "op": "commit", "B": 1, "N": 16, "layers": 24, "Hkv": 8, "D": 128, "length": 777,
         "page": 16, "dtype": "bf16"},
        # a full batch, long paths
        {"name": "commit batch", "op": "commit", "B": 64, "N": 32, "layers": 16, "Hkv": 8, "D": 128, "length": 600,
         "page": 64, "dtype": "bf16"},
        # beams of one request
        {"name": "step one request", "op": "step", "B": 1, "W": 4, "layers": 8, "Hkv": 8, "D": 128, "length": 1000,
         "page": 16, "dtype": "bf16"},
        # a batch of wide beams, head size and pages odd
        {"name": "step batch", "op": "step", "B": 24, "W": 8, "layers": 12, "Hkv": 4, "D": 80, "length": 2000, "page": 24,
         "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "commit", "step"])
    if op == "attend":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 7, 8])
        c = {"op": op, "B": _log_int(rng, 1, 64), "N": _log_int(rng, 1, 64), "Hq": Hkv * G, "Hkv": Hkv,
             "D": rng.choice([64, 80, 96, 128]), "length": _log_int(rng, 1, 120000),
             "page": rng.choice([8, 16, 24, 32, 64, 128]), "dtype": rng.choice(["bf16", "f16"]),
             "tree": rng.random() < 0.7, "ragged": rng.random() < 0.5}
        while c["B"] * c["length"] * Hkv > 64 * 4096 * 8:
            c["B"], c["length"] = max(1, c["B"] // 2), max(1, c["length"] * 2 // 3)
        while c["B"] * c["length"] * c["Hq"] * c["N"] > 64 * 4096 * 64 * 32:
            c["N"] = max(1, c["N"] // 2)
        return c
    if op == "verify":
        dtype = rng.choice(["f32", "bf16", "f16"])
        V, N = _log_int(rng, 1000, 160000), _log_int(rng, 1, 64)
        most = 64 * 32 * 128256 * 2 // (N * V * _BYTES[dtype])
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most))), "N": N, "V": V, "dtype": dtype,
                "pad": rng.choice([0, 0, 1, 64]), "ragged": rng.random() < 0.5}
    dtype, Hkv, D = rng.choice(["bf16", "f16", "f32"]), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128])
    page, layers, length = rng.choice([8, 16, 24, 64]), rng.randint(1, 24), _log_int(rng, 1, 2000)
    c = {"op": op, "B": _log_int(rng, 1, 64), "layers": layers, "Hkv": Hkv, "D": D, "length": length, "page": page,
         "dtype": dtype}
    c.update({"N": _log_int(rng, 1, 32)} if op == "commit" else {"W": rng.randint(1, 12)})
    # (pools of at most some 3 GB)
    while c["B"] * c.get("W", 1) * (c["length"] + 2 * page + c.get("N", 1)) * Hkv * D * _BYTES[dtype] * 2 * c["layers"] > 3e9:
        c["B"], c["layers"] = max(1, c["B"] // 2), max(1, c["layers"] * 2 // 3)
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tree(rng, n, tree):
    """Parents of n nodes, -1 for the root: each node under an earlier one (a
    random recursive tree), or a chain."""
    return [-1] + [rng.randrange(i) if tree else i - 1 for i in range(1, n)] if n else []


def _nodes(rng, case):
    """Nodes of each sequence; where they are ragged, every tenth sequence
    idles.  Their total is the case's."""
    B, N = case["B"], case["N"]
    if not case.get("ragged"):
        return [N] * B
    n = [N] + [0 if b % 10 == 5 else 1 + 7 * b % N for b in range(1, B)]
    rng.shuffle(n)
    return n


def _lengths(rng, case):
    B, L = case["B"], case["length"]
    return [L] + [rng.randint(L // 2, L) for _ in range(B - 1)]


def _pages(rng, lengths, page, shared=None):
    """Page tables of the sequences, pages spread over the pool, with room to
    grow; ``shared``: sequence b's first pages are those of shared[b] = (other,
    count).  Returns the table's rows."""
    rows, n = [], 0
    for b, length in enumerate(lengths):
        used = -(-length // page)
        row = []
        if shared is not None and shared[b] is not None:
            other, count = shared[b]
            row = rows[other][:count]
        while len(row) < used:
            row.append(n)
            n += 1
        rows.append(row)
    return rows


def _pool(g, rows, P, width, page, H, D, dtype, tensors, rng):
    at = list(range(P))
    rng.shuffle(at)
    table = torch.full((len(rows), width), 0, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    for b, row in enumerate(rows):
        if row:
            ids = torch.tensor([at[p] for p in row], dtype=torch.int32)
            table[b, :len(row)] = ids
            refs.index_add_(0, ids, torch.ones_like(ids))
    pools = [torch.randn(P, page, H, D, generator=g, device="cuda", dtype=dtype) for _ in range(tensors)]
    return pools, table.cuda(), refs.cuda()


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("attend", "verify"):
        n = _nodes(rng, case)
        trees = [_tree(rng, k, case.get("tree", True)) for k in n]
        total = sum(n)
        s["n"], s["total"] = n, total
        s["cu"] = _int([sum(n[:b]) for b in range(case["B"] + 1)]) if case["ragged"] else None
        s["parents"] = _int([p for t in trees for p in t]) if case.get("tree", True) else None
    if op == "attend":
        dt, Hq, Hkv, D, page = _DTYPES[case["dtype"]], case["Hq"], case["Hkv"], case["D"], case["page"]
        lengths = _lengths(rng, case)
        rows = _pages(rng, lengths, page)
        # queries a little longer than unit variance, as trained ones: some keys stand out
        s["q"] = (2.0 * torch.randn(total, Hq, D, generator=g, device="cuda")).to(dt)
        s["k"] = torch.randn(total, Hkv, D, generator=g, device="cuda", dtype=dt)
        s["v"] = torch.randn(total, Hkv, D, generator=g, device="cuda", dtype=dt)
        width = max(1, -(-(case["length"] + case["N"]) // page))
        (s["keys"], s["values"]), s["table"], _ = _pool(g, rows, len(rows) * width + 8, width, page, Hkv, D, dt, 2, rng)
        s["lengths"] = _int(lengths)
        return s
    if op == "verify":
        V, dt = case["V"], _DTYPES[case["dtype"]]
        tokens = [rng.randrange(V) for _ in range(total)]
        # the target's choice after every node: three times in four one of its children
        choice = []
        at = 0
        for t in trees:
            kids = [[] for _ in t]
            for i, p in enumerate(t):
                if p >= 0:
                    kids[p].append(i)
            for k in kids:
                choice.append(tokens[at + rng.choice(k)] if k and rng.random() < 0.75 else rng.randrange(V))
            at += len(t)
        rows = torch.empty(total, V + case["pad"], dtype=dt, device="cuda")
        step = max(1, (1 << 26) // V)
        for r in range(0, total, step):
            rows[r:r + step] = 3.0 * torch.randn(min(step, total - r), V + case["pad"], generator=g, device="cuda")
        rows.scatter_(1, _int(choice).long()[:, None], 30.0)
        s["target"], s["tokens"] = rows[:, :V], _int(tokens)
        return s
    dt, H, D, page, layers, B = _DTYPES[case["dtype"]], case["Hkv"], case["D"], case["page"], case["layers"], case["B"]
    if op == "commit":
        N = case["N"]
        lengths = _lengths(rng, case)
        # every fourth sequence shares its prefix with the one before (a system prompt), its last, partly filled page too
        shared = [None] * B
        for b in range(1, B):
            if b % 4 == 1:
                lengths[b] = lengths[b - 1]
                shared[b] = (b - 1, -(-lengths[b] // page))
        grow = -(-N // page) + 1
        trees = [_tree(rng, N, True) for _ in range(B)]
        path, counts = [], []
        for t in trees:  # an accepted path: from the root some way down
            kids = [[i for i, p in enumerate(t) if p == j] for j in range(N)]
            way = [0]
            while kids[way[-1]] and rng.random() < 0.75:
                way.append(rng.choice(kids[way[-1]]))
            counts.append(len(way))
            path.append(way + [-1] * (N - len(way)))
        s["path"], s["counts"] = _int(path), _int(counts)
        new = B * N
    else:
        W = case["W"]
        base = _lengths(rng, case)
        lengths = [base[b] for b in range(B) for _ in range(W)]
        # beams share their prompt, three quarters of what they hold
        shared = [None if i % W == 0 else (i - i % W, base[i // W] * 3 // 4 // page) for i in range(B * W)]
        grow = 2
        s["parents"] = _int([[int(W * rng.random() ** 1.5) for _ in range(W)] for _ in range(B)])
        new = B * W
    rows = _pages(rng, lengths, page, shared)
    width = -(-case["length"] // page) + grow
    P = len(rows) * (width + grow)
    pools, s["table"], s["refs"] = _pool(g, rows, P, width, page, H, D, dt, 2 * layers, rng)
    s["keys"], s["values"] = pools[:layers], pools[layers:]
    s["lengths"] = _int(lengths)
    s["back"] = s["lengths"].clone()  # what the sequences are taken back to
    s["new_keys"] = [torch.randn(new, H, D, generator=g, device="cuda", dtype=dt) for _ in range(layers)]
    s["new_values"] = [torch.randn(new, H, D, generator=g, device="cuda", dtype=dt) for _ in range(layers)]
    if op == "step":
        s["table"] = s["table"].view(B, W, width)
        s["lengths"], s["back"] = s["lengths"].view(B, W), s["back"].view(B, W)
    return s


# ------------------------------------------------------------------ one pass

def _rows_of(s):
    """Row of node i of sequence b, [B, N], and whether there is one."""
    c = s["case"]
    i = torch.arange(c["N"], device="cuda")[None, :]
    if s["cu"] is None:
        return torch.arange(c["B"], device="cuda")[:, None] * c["N"] + i, torch.ones(c["B"], c["N"], dtype=torch.bool, device="cuda")
    first, end = s["cu"][:-1, None].long(), s["cu"][1:, None].long()
    return (first + i).clamp_(max=max(s["total"] - 1, 0)), first + i < end


def _ancestors(s, rows, there):
    """[B, N, N]: whether node j is node i or one of its ancestors."""
    c = s["case"]
    B, N = c["B"], c["N"]
    i = torch.arange(N, device="cuda")
    if s["parents"] is None:
        return (i[None, :] <= i[:, None]).expand(B, N, N)
    up = torch.where(there, s["parents"][rows], -1)
    at = i.expand(B, N).clone()
    seen = torch.zeros(B, N, N + 1, dtype=torch.bool, device="cuda")
    for _ in range(N):  # one generation up at a time
        seen.scatter_(2, at[:, :, None], True)
        at = torch.where(at == N, N, up.gather(1, at.clamp(max=N - 1)).long())
        at = torch.where(at < 0, N, at)
    return seen[:, :, :N]


def _plain_attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D, L, page = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "length", "page"))
    G = Hq // Hkv
    rows, there = _rows_of(s)
    seen = _ancestors(s, rows, there)
    out = torch.zeros(s["total"], Hq, D, device="cuda")
    lse = torch.zeros(s["total"], Hq, device="cuda")
    at = torch.arange(L, device="cuda")
    step = max(1, (1 << 29) // (Hq * N * (L + N)))
    for b0 in range(0, B, step):
        b = slice(b0, min(B, b0 + step))
        r, n = rows[b], rows[b].shape[0]
        place = s["table"][b].long()[:, at // page]
        k = torch.cat((s["keys"][place, at % page], s["k"][r]), 1).float()  # [n, L + N, Hkv, D]
        v = torch.cat((s["values"][place, at % page], s["v"][r]), 1).float()
        q = s["q"][r].float().view(n, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * N, D)
        ok = torch.cat(((at < s["lengths"][b, None])[:, None, :].expand(n, N, L), seen[b]), 2)  # [n, N, L + N]
        x = (q @ k.permute(0, 2, 3, 1)).view(n, Hkv, G, N, L + N) * (1.0 / math.sqrt(D))
        x = torch.where(ok[:, None, None], x, -math.inf)
        m = x.amax(4, keepdim=True)
        x = (x - m).exp()
        z = x.sum(4, keepdim=True)
        o = (x / z).view(n, Hkv, G * N, L + N) @ v.permute(0, 2, 1, 3)
        o = o.view(n, Hkv, G, N, D).permute(0, 3, 1, 2, 4).reshape(n, N, Hq, D)
        e = (m + z.log())[..., 0].permute(0, 3, 1, 2).reshape(n, N, Hq)
        if s["cu"] is None:
            out[r.reshape(-1)], lse[r.reshape(-1)] = o.flatten(0, 1), e.flatten(0, 1)
        else:
            out[r[there[b]]], lse[r[there[b]]] = o[there[b]], e[there[b]]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_verify(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    x = s["target"]
    index = torch.arange(V, device="cuda", dtype=torch.int32)
    best = torch.where(x == x.amax(1, keepdim=True), index, V).amin(1)  # the lowest index of a row's largest
    rows, there = _rows_of(s)
    token = torch.where(there, s["tokens"][rows], -1)
    up = torch.where(there, s["parents"][rows], -2)
    best = best[rows]
    i = torch.arange(N, device="cuda")
    at = torch.zeros(B, 1, dtype=torch.int64, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path[:, :1] = 0
    n = torch.zeros(B, 1, dtype=torch.int64, device="cuda")
    for j in range(1, N):  # a path is no longer than the tree
        fits = (up == at) & (token == best.gather(1, at))
        child = torch.where(fits, i, N).amin(1, keepdim=True)
        go = (child < N) & (n == j - 1)
        at = torch.where(go, child, at)
        path[:, j:j + 1] = torch.where(go, child, -1).int()
        n = n + go
    any_ = there[:, :1]
    return {"n_accepted": n[:, 0].int(), "next_token": torch.where(any_, best.gather(1, at), -1)[:, 0].int(),
            "path": torch.where(any_, path, -1)}


def _plain_append(s, table, lengths, counts, path, N):
    """Appends to the caches, the sequences one after another; ``table``
    [S, pages], ``lengths`` [S].  (In these cases every sequence appends, and
    the pools never run out of pages.)"""
    page, S = s["keys"][0].shape[1], table.shape[0]
    refs = s["refs"]
    b = torch.arange(S, device="cuda")
    length, count = lengths.long(), counts.long()
    part = length % page
    last = table[b, length // page].long()
    # a partly filled last page that others hold too is copied, but not by the last that still holds it
    before = ((last[:, None] == last[None, :]) & (part > 0)[None, :] & (b[None, :] < b[:, None])).sum(1)
    copy = (part > 0) & (refs[last] - before > 1)
    first = (length + page - 1) // page - copy.long()
    need = (length + count + page - 1) // page - first
    offset = need.cumsum(0) - need
    free = (refs != 0).to(torch.int8).argsort(stable=True)  # free pages first, lowest first
    for j in range(-(-N // page) + 1):
        take = j < need
        slot = torch.where(take, first + j, 0)
        new = free[torch.where(take, offset + j, 0)]
        table[b, slot] = torch.where(take, new.int(), table[b, slot])
        refs.index_add_(0, new, take.int())
    refs.index_add_(0, last, -copy.int())
    # the shared last pages' tokens; a sequence without a copy repeats the first one
    i = torch.arange(page, device="cuda")
    one = torch.where(copy, b, copy.int().argmax())
    last, to = last[one], table[b, length // page].long()[one]
    moved = (copy[:, None] & (i[None, :] < part[:, None]))[one][:, :, None, None]
    # the new tokens: an entry past the end of a path repeats its first one
    j = torch.arange(N, device="cuda")[None, :]
    live = j < count[:, None]
    at = torch.where(live, length[:, None] + j, length[:, None])
    page_of = table.gather(1, at // page).long()
    row = b[:, None] * N + (torch.where(live, path.long(), path[:, :1].long()) if path is not None else 0 * at)
    for pools, new in ((s["keys"], s["new_keys"]), (s["values"], s["new_values"])):
        for pool, x in zip(pools, new):
            pool[to] = torch.where(moved, pool[last], pool[to])
            pool[page_of, at % page] = x[row]
    lengths += counts


def _plain_give_up(s, table, lengths, to):
    """The sequences back to lengths ``to``."""
    page = s["keys"][0].shape[1]
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    gone = (j >= ((to + page - 1) // page)[:, None]) & (j < ((lengths + page - 1) // page)[:, None])
    s["refs"].index_add_(0, table.reshape(-1), -gone.reshape(-1).int())
    lengths.copy_(to)


def _plain_fork(s):
    page = s["keys"][0].shape[1]
    table, lengths, refs = s["table"], s["lengths"], s["refs"]
    b = torch.arange(table.shape[0], device="cuda")[:, None]
    p = s["parents"].long()
    j = torch.arange(table.shape[2], device="cuda")
    used = j < ((lengths + page - 1) // page)[:, :, None]
    refs.index_add_(0, table.reshape(-1), -used.reshape(-1).int())
    used = used[b, p]
    table.copy_(torch.where(used, table[b, p], table))
    refs.index_add_(0, table.reshape(-1), used.reshape(-1).int())
    lengths.copy_(lengths[b, p])


def _state(s):
    return {k: s[k] for k in ("keys", "values", "table", "lengths", "refs")}


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import speculative_decoding_verification_decode_gb300 as sv
        if op == "attend":
            r = sv.tree_attention(s["q"], s["k"], s["v"], s["keys"], s["values"], s["table"], s["lengths"],
                                  parents=s["parents"], cu_nodes=s["cu"], n=c["N"])
            return {"out": r.out, "lse": r.lse}
        if op == "verify":
            r = sv.verify_tree_greedy(s["target"], s["tokens"], s["parents"], cu_nodes=s["cu"], n=c["N"])
            return {"n_accepted": r.n_accepted, "next_token": r.next_token, "path": r.path}
        cache = sv.PagedCache(s["keys"], s["values"], s["table"], s["lengths"], s["refs"])
        if op == "commit":
            sv.cache_append(cache, s["new_keys"], s["new_values"], counts=s["counts"], path=s["path"])
        else:
            sv.cache_fork(cache, s["parents"])
            sv.cache_append(cache, s["new_keys"], s["new_values"])
        sv.cache_truncate(cache, s["back"])
        return _state(s)
    if op == "attend":
        return _plain_attend(s)
    if op == "verify":
        return _plain_verify(s)
    if op == "commit":
        table, lengths, counts, path, N = s["table"], s["lengths"], s["counts"], s["path"], c["N"]
    else:
        _plain_fork(s)
        table, lengths = s["table"].flatten(0, 1), s["lengths"].flatten()
        counts, path, N = torch.ones_like(lengths), None, 1
    _plain_append(s, table, lengths, counts, path, N)
    _plain_give_up(s, table, lengths, s["back"].flatten())
    return _state(s)


# ------------------------------------------------------------------ what a pass cannot do without

def _mean_path(N):
    """Mean number of nodes on the accepted path of a random tree."""
    rng, total = random.Random(1), 0
    for _ in range(200):
        t = _tree(rng, N, True)
        at = 0
        while True:
            total += 1
            kids = [i for i, p in enumerate(t) if p == at]
            if not kids or rng.random() >= 0.75:
                break
            at = rng.choice(kids)
    return total / 200


def work(case):
    op, B = case["op"], case["B"]
    e = _BYTES[case["dtype"]]
    if op == "attend":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        nodes = case["N"] + (B - 1) * (0.9 * (case["N"] + 1) / 2 if case["ragged"] else case["N"])
        cached = case["length"] * (1 + 0.75 * (B - 1))
        per_row = cached / B + case["N"] / 2
        return {"bytes": e * (2 * cached * Hkv * D + 2 * nodes * Hkv * D + 2 * nodes * Hq * D) + 4 * nodes * Hq
                + 4 * cached / case["page"], "flops": 4.0 * nodes * Hq * per_row * D}
    if op == "verify":
        n = case["N"]
        path = _mean_path(n)
        if case["ragged"]:
            path += (B - 1) * sum(_mean_path(k) for k in range(1, n + 1)) / n * 0.9
        else:
            path *= B
        return {"bytes": path * case["V"] * e, "flops": path * case["V"]}
    H, D, page = case["Hkv"], case["D"], case["page"]
    token = 2 * case["layers"] * H * D * e  # keys and values of all layers
    if op == "commit":
        # (a shared page is copied in a state's first pass only, so it is not counted)
        return {"bytes": 2 * token * B * _mean_path(case["N"]) + B * 4 * (case["N"] + 3), "flops": 0}
    W = case["W"]
    # of the slots that take one parent's pages all but one copy its last
    law = [((j + 1) / W) ** (2 / 3) - (j / W) ** (2 / 3) for j in range(W)]
    copied = W - sum(1 - (1 - p) ** W for p in law)
    tables = 2 * 4 * B * W * 0.75 * case["length"] / page
    return {"bytes": 2 * token * B * (W + copied * (page - 1) / 2) + tables, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attend(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["B"] * c["length"] * Hq * c["N"] * D > 5e12:
        return None
    out = torch.zeros(s["total"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], Hq, dtype=torch.float64, device="cuda")
    parents = None if s["parents"] is None else s["parents"].tolist()
    first = 0
    for b, n in enumerate(s["n"]):
        L = int(s["lengths"][b])
        ids = s["table"][b, :-(-L // page)].long()
        sees = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):  # node i sees what its parent sees, and itself
            p = i - 1 if parents is None else parents[first + i]
            if p >= 0:
                sees[i] = sees[p]
            sees[i, i] = True
        sees = sees.cuda()
        r = slice(first, first + n)
        for h in range(Hkv if n else 0):
            k = torch.cat((s["keys"][ids, :, h].flatten(0, 1)[:L], s["k"][r, h])).double()
            v = torch.cat((s["values"][ids, :, h].flatten(0, 1)[:L], s["v"][r, h])).double()
            for qh in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = s["q"][r, qh].double() @ k.T / math.sqrt(D)
                x[:, L:].masked_fill_(~sees, -math.inf)
                e = torch.logsumexp(x, 1)
                lse[r, qh] = e
                out[r, qh] = (x - e[:, None]).exp() @ v
        first += n
    return {"out": out, "lse": lse}


def _exact_verify(s):
    n_acc, nxt, path = [], [], []
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    first = 0
    for n in s["n"]:
        way, pick = [], -1
        at = 0 if n else None
        while at is not None:
            way.append(at)
            row = s["target"][first + at].double()
            pick = int((row == row.max()).nonzero()[0])
            at = next((i for i in range(n) if parents[first + i] == at and tokens[first + i] == pick), None)
        n_acc.append(max(0, len(way) - 1))
        nxt.append(pick)
        path.append(way + [-1] * (s["case"]["N"] - len(way)))
        first += n
    return {"n_accepted": _int(n_acc), "next_token": _int(nxt), "path": _int(path)}


def _exact_pages(s):
    """One sequence after another, one token after another, on the host's page
    tables."""
    c = s["case"]
    page = c["page"]
    pools = s["keys"] + s["values"]
    new = s["new_keys"] + s["new_values"]
    shape = s["table"].shape
    table = [row for row in s["table"].reshape(-1, shape[-1]).tolist()]
    lengths, refs = s["lengths"].flatten().tolist(), s["refs"].tolist()
    back = list(lengths)
    if c["op"] == "step":
        W = c["W"]
        old, old_len = [list(r) for r in table], list(lengths)
        for b, line in enumerate(s["parents"].tolist()):
            for w, p in enumerate(line):
                i, j = b * W + w, b * W + p
                for x in range(-(-old_len[i] // page)):
                    refs[old[i][x]] -= 1
                for x in range(-(-old_len[j] // page)):
                    refs[old[j][x]] += 1
                    table[i][x] = old[j][x]
                lengths[i] = old_len[j]
        back = s["back"].flatten().tolist()
        ways = [[0]] * len(lengths)
        N = 1
    else:
        ways = [p[:k] for p, k in zip(s["path"].tolist(), s["counts"].tolist())]
        N = c["N"]
    free = iter([i for i, r in enumerate(refs) if r == 0])
    copies, writes = [], []
    for b, way in enumerate(ways):
        L = lengths[b]
        if way and L % page and refs[table[b][L // page]] > 1:
            p = next(free)
            copies.append((table[b][L // page], p, L % page))
            refs[table[b][L // page]] -= 1
            refs[p] += 1
            table[b][L // page] = p
        for node in way:
            if L % page == 0:
                p = next(free)
                refs[p] += 1
                table[b][L // page] = p
            writes.append((table[b][L // page], L % page, b * N + node))
            L += 1
        for x in range(-(-back[b] // page), -(-L // page)):
            refs[table[b][x]] -= 1
        lengths[b] = back[b]
    w = torch.tensor(writes).cuda()
    done = []
    for pool, x in zip(pools, new):
        made = pool.clone()
        for a, p, k in copies:
            made[p, :k] = pool[a, :k]
        made[w[:, 0], w[:, 1]] = x[w[:, 2]]
        done.append(made.double() if c["dtype"] == "f32" else made)
    n = c["layers"]
    return {"keys": done[:n], "values": done[n:], "table": _int(table).view(shape),
            "lengths": _int(lengths).view(s["lengths"].shape), "refs": _int(refs)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_attend(s) if op == "attend" else _exact_verify(s) if op == "verify" else _exact_pages(s)
