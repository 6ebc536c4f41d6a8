"""Measured cases of the beam-search and 4-bit LM-head operators.

``listed()`` names the cases, ``prepare`` makes a case's inputs on the GPU,
``run`` makes one pass: the plain form in elementary torch operations, or
(``own``) the calls a user makes of this package.  ``exact`` gives the
operators' values from their definitions in 64 bits.

Three operators:

* ``select``: the n best continuations of W beams over the vocabulary,
  ``score + log_softmax(logits)``, ties to the lowest (beam, token);
* ``reorder``: the beams' states (key/value caches, token histories,
  recurrent states) moved in place to the slots of the chosen parents;
* ``head``: logits of a few rows of hidden states through a vocabulary
  projection held in 4 bits with group scales.
"""

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "u8": torch.uint8,
           "i32": torch.int32}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2, "u8": 1, "i32": 4}


def listed():
    return [
        # one interactive request, four beams, a 32000-token vocabulary: latency
        {"name": "select one request", "op": "select", "B": 1, "W": 4, "n": 8, "V": 32000, "dtype": "f32",
         "pad": 0, "finished": False},
        # a small service batch; an odd vocabulary, so rows start at any 2-byte address
        {"name": "select odd rows", "op": "select", "B": 5, "W": 5, "n": 10, "V": 129281, "dtype": "bf16",
         "pad": 0, "finished": False},
        # wide beams late in the search: some beams have ended, rows padded to a stride
        {"name": "select wide", "op": "select", "B": 8, "W": 16, "n": 32, "V": 152064, "dtype": "f16",
         "pad": 64, "finished": True},
        # a full batch of offline translation / captioning
        {"name": "select batch", "op": "select", "B": 64, "W": 8, "n": 16, "V": 128256, "dtype": "bf16",
         "pad": 0, "finished": False},
        # token histories of one request: a few KB, latency
        {"name": "reorder tokens", "op": "reorder", "B": 4, "W": 4, "states": 1, "heads": 0, "T": 777, "D": 1,
         "dtype": "i32", "lengths": True},
        # recurrent states, every element in use, sequence and beam last dims odd
        {"name": "reorder recurrent", "op": "reorder", "B": 7, "W": 5, "states": 12, "heads": 0, "T": 1,
         "D": 65537, "dtype": "f32", "lengths": False},
        # key and value caches of eight layers in 16 bits
        {"name": "reorder caches", "op": "reorder", "B": 8, "W": 4, "states": 16, "heads": 8, "T": 1024, "D": 128,
         "dtype": "bf16", "lengths": True},
        # the same with wide beams and caches held in 8 bits
        {"name": "reorder 8-bit caches", "op": "reorder", "B": 3, "W": 16, "states": 8, "heads": 8, "T": 2049,
         "D": 128, "dtype": "u8", "lengths": True},
        # one token of one sequence: a matrix-vector product
        {"name": "head one row", "op": "head", "rows": 1, "V": 32000, "d": 4096, "group": 128, "dtype": "bf16",
         "scale": "bf16", "zeros": False},
        # verification of one sequence with K = 5: six target and five draft rows
        {"name": "head one sequence", "op": "head", "rows": 11, "V": 128256, "d": 4096, "group": 128,
         "dtype": "bf16", "scale": "bf16", "zeros": False},
        # beams of three sequences, small groups with zero points, a width that no group divides
        {"name": "head odd", "op": "head", "rows": 15, "V": 50257, "d": 2080, "group": 64, "dtype": "f16",
         "scale": "f16", "zeros": True},
        # verification of four sequences with K = 5
        {"name": "head batch", "op": "head", "rows": 44, "V": 152064, "d": 4096, "group": 32, "dtype": "bf16",
         "scale": "f16", "zeros": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "reorder", "head"])
    if op == "select":
        dtype = rng.choice(["f32", "bf16", "f16"])
        V, W = _log_int(rng, 1000, 160000), rng.randint(1, 16)
        most = 64 * 8 * 128256 * 2 // (W * V * _BYTES[dtype])
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most))), "W": W, "n": rng.randint(W, 2 * W), "V": V,
                "dtype": dtype, "pad": rng.choice([0, 0, 1, 64]), "finished": rng.random() < 0.5}
    if op == "reorder":
        kind = rng.choice(["cache", "cache", "tokens", "recurrent"])
        B, W = _log_int(rng, 1, 16), rng.randint(2, 16)
        if kind == "tokens":
            return {"op": op, "B": B, "W": W, "states": 1, "heads": 0, "T": _log_int(rng, 16, 8192), "D": 1,
                    "dtype": "i32", "lengths": True}
        if kind == "recurrent":
            return {"op": op, "B": B, "W": W, "states": rng.randint(1, 12), "heads": 0, "T": 1,
                    "D": _log_int(rng, 1000, 70000), "dtype": rng.choice(["f32", "bf16"]), "lengths": False}
        dtype, heads, D = rng.choice(["bf16", "f16", "u8"]), rng.choice([1, 2, 8]), rng.choice([64, 80, 128])
        T = _log_int(rng, 64, 4096)
        most = 16 * 8 * 4 * 8 * 1024 * 128 * 2 // (B * W * heads * T * D * _BYTES[dtype])
        return {"op": op, "B": B, "W": W, "states": max(1, min(rng.randint(2, 16), most)) if most else 1,
                "heads": heads, "T": T if most else 64, "D": D, "dtype": dtype, "lengths": rng.random() < 0.8}
    rows, V, d = _log_int(rng, 1, 64), _log_int(rng, 1000, 152064), 32 * _log_int(rng, 8, 256)
    while V * d > 152064 * 4096 or rows * V * d > 44 * 152064 * 4096:
        V, rows = max(1000, V // 2), max(1, rows // 2)
    return {"op": op, "rows": rows, "V": V, "d": d, "group": rng.choice([32, 64, 128]),
            "dtype": rng.choice(["bf16", "f16"]), "scale": rng.choice(["bf16", "f16", "f32"]),
            "zeros": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _parent_law(W):
    """Probability of each beam to be a slot's parent: better beams have more
    descendants (slot u^1.5 W for uniform u)."""
    return [((j + 1) / W) ** (2 / 3) - (j / W) ** (2 / 3) for j in range(W)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "select":
        B, W, V, n = case["B"], case["W"], case["V"], case["n"]
        # logits N(0, 3^2) with a few raised tokens per row, as peaked as a trained model's rows
        rows = torch.empty(B * W, V + case["pad"], dtype=_DTYPES[case["dtype"]], device="cuda")
        peaks = torch.randint(0, V, (B * W, 20), generator=g, device="cuda")
        step = max(1, (1 << 25) // V)
        at = 0
        while at < B * W:
            x = 3.0 * _randn(g, min(step, B * W - at), V)
            x.scatter_add_(1, peaks[at:at + step], torch.full_like(peaks[at:at + step], 8, dtype=torch.float32))
            rows[at:at + step, :V] = x.to(rows.dtype)
            at += step
        s["logits"] = rows[:, :V].unflatten(0, (B, W))
        # running scores of a search some thirty tokens long, best beam first
        s["scores"] = (-40.0 - 20.0 * _rand(g, B, 1) - torch.cumsum(0.8 * _rand(g, B, W), 1)).contiguous()
        s["finished"] = (_rand(g, B, W) < 0.25) if case["finished"] else None
        s["eos"] = 2 if case["finished"] else -1
        return s
    if op == "reorder":
        B, W, T, D, H = case["B"], case["W"], case["T"], case["D"], case["heads"]
        dt = _DTYPES[case["dtype"]]
        shape = (B, W, H, T, D) if H else ((B, W, T) if D == 1 else (B, W, D))
        s["states"] = []
        while len(s["states"]) < case["states"]:
            if dt == torch.int32:
                s["states"].append(torch.randint(0, 128256, shape, generator=g, device="cuda", dtype=dt))
            elif dt == torch.uint8:
                s["states"].append(torch.randint(0, 256, shape, generator=g, device="cuda", dtype=dt))
            else:
                s["states"].append(torch.randn(*shape, generator=g, device="cuda", dtype=dt))
        s["time_dim"] = (3 if H else 2) if case["lengths"] else None
        s["parents"] = (W * _rand(g, B, W).pow(1.5)).to(torch.int32).clamp_(max=W - 1)
        s["lengths"] = None
        if case["lengths"]:
            s["lengths"] = (T // 2 + (T - T // 2) * _rand(g, B)).to(torch.int32).clamp_(max=T)
        return s
    rows, V, d, group = case["rows"], case["V"], case["d"], case["group"]
    G = -(-d // group)
    s["states"] = _randn(g, rows, d).to(_DTYPES[case["dtype"]])
    s["packed"] = torch.randint(0, 256, (V, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    # groups of N(0, 1/d) weights spread over 15 steps
    s["scales"] = ((0.6 + 0.8 * _rand(g, V, G)) * (3.0 / (7.0 * math.sqrt(d)))).to(_DTYPES[case["scale"]])
    s["zeros"] = torch.randint(5, 11, (V, G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    return s


# ------------------------------------------------------------------ one pass

def _plain_select(s):
    logits, scores, finished, eos, n = s["logits"], s["scores"], s["finished"], s["eos"], s["case"]["n"]
    B, W, V = logits.shape
    # candidates of different beams are ordered by sums that differ in the last bits of 32-bit arithmetic: 64 bits
    x = logits.double()
    m = x.amax(2, keepdim=True)
    lse = m + (x - m).exp().sum(2, keepdim=True).log()
    x = scores.double()[:, :, None] + (x - lse)
    if finished is not None:
        x = torch.where(finished[:, :, None], -math.inf, x)
        x[:, :, eos] = torch.where(finished, scores.double(), x[:, :, eos])
    x = x.reshape(B, W * V)
    # the n best, equal scores by the lowest index: all above the n-th, then the first of those equal to it
    last = x.topk(n, dim=1).values[:, -1:]
    above, equal = x > last, x == last
    room = n - above.sum(1, keepdim=True)
    chosen = above | (equal & (equal.cumsum(1, dtype=torch.int32) <= room))
    index = torch.arange(W * V, 0, -1, device=x.device, dtype=torch.int32)
    at = W * V - (chosen * index).topk(n, dim=1).values.long()  # ascending indices of the chosen
    best, order = x.gather(1, at).sort(dim=1, descending=True, stable=True)
    at = at.gather(1, order)
    none = best == -math.inf
    return {"scores": best.float(), "parents": torch.where(none, -1, at // V).int(),
            "tokens": torch.where(none, -1, at % V).int()}


def _plain_reorder(s):
    b = torch.arange(s["parents"].shape[0], device="cuda")[:, None]
    p = s["parents"].long()
    for t in s["states"]:
        moved = t[b, p]
        if s["lengths"] is not None:
            T = t.shape[s["time_dim"]]
            live = torch.arange(T, device="cuda")[None, :] < s["lengths"][:, None]
            live = live.reshape([live.shape[0]] + [1] * (s["time_dim"] - 1) + [T] + [1] * (t.dim() - s["time_dim"] - 1))
            moved = torch.where(live, moved, t)
        t.copy_(moved)
    return s["states"]


def _plain_head(s):
    group, d = s["case"]["group"], s["case"]["d"]
    q = torch.stack((s["packed"] & 15, s["packed"] >> 4), 2).flatten(1).float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(group, 1)[:, :d]
    w = (q - z) * s["scales"].float().repeat_interleave(group, 1)[:, :d]
    return s["states"].float() @ w.T


def run(s):
    op = s["case"]["op"]
    if own:
        import speculative_decoding_verification_decode_gb300 as sv
        if op == "select":
            r = sv.beam_select(s["logits"], s["scores"], n=s["case"]["n"], finished=s["finished"], eos=s["eos"])
            return {"scores": r.scores, "parents": r.parents, "tokens": r.tokens}
        if op == "reorder":
            sv.beam_reorder(s["states"], s["parents"], lengths=s["lengths"], time_dim=s["time_dim"])
            return s["states"]
        return sv.lm_head_logits(s["states"], sv.Q4Projection(s["packed"], s["scales"], s["zeros"], s["case"]["group"]))
    return _plain_select(s) if op == "select" else _plain_reorder(s) if op == "reorder" else _plain_head(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "select":
        B, W, V, n = case["B"], case["W"], case["V"], case["n"]
        live = B * W * (0.75 if case["finished"] else 1.0)  # ended beams' rows are not needed
        return {"bytes": live * V * _BYTES[case["dtype"]] + B * W * 4 + B * n * 12, "flops": live * V * 5}
    if op == "reorder":
        B, W = case["B"], case["W"]
        law = _parent_law(W)
        written = W - 1.0  # slots whose parent is another, on average
        read = sum(1 - (1 - p) ** (W - 1) for p in law)  # distinct parents of moved slots, on average
        kept = 0.75 if case["lengths"] else 1.0  # mean length over T
        beam = max(1, case["heads"]) * case["T"] * case["D"] * _BYTES[case["dtype"]] * kept
        return {"bytes": case["states"] * B * beam * (written + read) + B * W * 4, "flops": 0}
    rows, V, d = case["rows"], case["V"], case["d"]
    G = -(-d // case["group"])
    per_row = d / 2 + G * (_BYTES[case["scale"]] + (1 if case["zeros"] else 0))
    return {"bytes": V * per_row + rows * d * 2 + rows * V * 4, "flops": 2.0 * rows * V * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        B, W, V, n = case["B"], case["W"], case["V"], case["n"]
        scores, parents, tokens = [], [], []
        for b in range(B):  # one sequence at a time: every beam's own best, then the best of those
            found = []
            for w in range(W):
                c = float(s["scores"][b, w])
                if s["finished"] is not None and bool(s["finished"][b, w]):
                    found.append((-c, w, s["eos"]))
                    continue
                x = s["logits"][b, w].double()
                lse = float(torch.logsumexp(x, 0))
                v, i = x.sort(descending=True, stable=True)
                v, i = v[:n].tolist(), i[:n].tolist()
                found += [(-(c + (a - lse)), w, j) for a, j in zip(v, i) if a > -math.inf]
            found = sorted(found)[:n]
            found += [(math.inf, -1, -1)] * (n - len(found))
            scores.append([-f[0] for f in found])
            parents.append([f[1] for f in found])
            tokens.append([f[2] for f in found])
        return {"scores": torch.tensor(scores, dtype=torch.float64), "parents": torch.tensor(parents, dtype=torch.int32),
                "tokens": torch.tensor(tokens, dtype=torch.int32)}
    if op == "reorder":
        out = []
        for t in s["states"]:
            old, new = t, t.clone()
            for b, line in enumerate(s["parents"].tolist()):
                end = None if s["lengths"] is None else int(s["lengths"][b])
                for w, p in enumerate(line):
                    if end is None:
                        new[b, w] = old[b, p]
                    else:
                        axis = s["time_dim"] - 2
                        new[b, w].narrow(axis, 0, end).copy_(old[b, p].narrow(axis, 0, end))
            out.append(new if new.dtype in (torch.int32, torch.uint8) else new.double())
        return out
    group, d = case["group"], case["d"]
    h = s["states"].double()
    out = torch.zeros(case["rows"], case["V"], dtype=torch.float64, device="cuda")
    for k0 in range(0, d, group):  # group by group: the integers' products, then their scale
        k1 = min(d, k0 + group)
        p = s["packed"][:, k0 // 2:k1 // 2].to(torch.int16)
        q = torch.empty(case["V"], k1 - k0, dtype=torch.float64, device="cuda")
        q[:, 0::2] = (p % 16).double()
        q[:, 1::2] = (p // 16).double()
        q -= 8 if s["zeros"] is None else s["zeros"][:, k0 // group, None].double()
        out += (h[:, k0:k1] @ q.T) * s["scales"][:, k0 // group].double()
    return out
