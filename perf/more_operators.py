"""What a block and a head on looked-up rows are measured on.

A model over an embedding lookup ends in blocks whose two projections gate
each other, and in a head that scores its rows against every row of a
vocabulary (the items that can follow).  The operators:

* ``gated``    every row through its group's two projections, one gating the
               other: y = act(z) u, and the gradients;
* ``loss``     softmax cross entropy of rows against a whole vocabulary, and
               the gradients of the rows and of the vocabulary;
* ``distill``  the same head learning a teacher's top logits.

``run`` computes them in their plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
UNSEEN = 0.05                             # of the rows have no target (padding)
MOST = {"bf16": 1 << 41, "f32": 1 << 37}  # products of one score pass, of the largest cases


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token through one block, as a serving step has it: the weights' bytes, and latency
        {"name": "gated-token", "op": "gated", "rows": 1, "groups": 1, "layout": "experts", "k": 2048, "n": 4096,
         "dtype": "bf16", "act": "silu", "step": False, "keep": False},
        # a serving step of 64 tokens over 16 experts
        {"name": "gated-tokens", "op": "gated", "rows": 64, "groups": 16, "layout": "experts", "k": 2048, "n": 4096,
         "dtype": "bf16", "act": "silu", "step": False, "keep": False},
        # a training step of each feature table's block, sample-major rows, projections kept
        {"name": "gated-tables", "op": "gated", "rows": 26 * 16384, "groups": 26, "layout": "tables", "k": 128, "n": 256,
         "dtype": "bf16", "act": "sigmoid", "step": True, "keep": True},
        # a training step of experts with ragged shares of the tokens, projections computed again
        {"name": "gated-experts", "op": "gated", "rows": 16384, "groups": 16, "layout": "experts", "k": 2048, "n": 4096,
         "dtype": "bf16", "act": "silu", "step": True, "keep": False},
        # fp32 rows of odd lengths
        {"name": "gated-odd", "op": "gated", "rows": 5001, "groups": 3, "layout": "sorted", "k": 513, "n": 777,
         "dtype": "f32", "act": "silu", "step": True, "keep": False},
        # the likelihood of one request's next items, narrow rows: latency
        {"name": "loss-request", "op": "loss", "rows": 8, "vocab": 65536, "k": 128, "dtype": "bf16", "heat": 1.0,
         "step": False},
        # a training step over a vocabulary and rows of odd lengths
        {"name": "loss-odd", "op": "loss", "rows": 1000, "vocab": 100003, "k": 250, "dtype": "bf16", "heat": 1.0,
         "step": True},
        # a training step of fp32 embedding rows against each other's items, at a temperature
        {"name": "loss-items", "op": "loss", "rows": 16384, "vocab": 65536, "k": 128, "dtype": "f32", "heat": 0.5,
         "step": True},
        # a training step of wide rows over a large vocabulary
        {"name": "loss-large", "op": "loss", "rows": 8192, "vocab": 131072, "k": 2048, "dtype": "bf16", "heat": 1.0,
         "step": True},
        # how far a few rows are from the teacher
        {"name": "distill-request", "op": "distill", "rows": 16, "vocab": 65536, "k": 1024, "top": 16, "dtype": "bf16",
         "heat": 2.0, "step": False},
        # fp32, long lists, odd sizes
        {"name": "distill-odd", "op": "distill", "rows": 777, "vocab": 30011, "k": 96, "top": 100, "dtype": "f32",
         "heat": 1.0, "step": True},
        # a training step of wide rows, a teacher's 64 top logits each
        {"name": "distill-large", "op": "distill", "rows": 4096, "vocab": 131072, "k": 2048, "top": 64, "dtype": "bf16",
         "heat": 2.0, "step": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, hi):
    """Widths in eights mostly, as weights are laid out; any now and then."""
    return _log_int(rng, 16, hi) if rng.random() < 0.25 else 8 * _log_int(rng, 2, hi // 8)


def draw(rng):
    op = rng.choice(["gated", "loss", "distill"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    step = rng.random() < 0.65
    k = _width(rng, 4096)
    if op == "gated":
        n = _width(rng, 8192)
        groups = _log_int(rng, 1, max(1, min(64, (1 << 27) // (k * n))))
        most = min(MOST[dtype] // 4 // (2 * n * k), (1 << 28) // (k + 2 * n))
        return {"op": op, "rows": _log_int(rng, 1, max(1, min(1 << 19, most))), "groups": groups,
                "layout": rng.choice(["experts", "tables", "sorted"]), "k": k, "n": n, "dtype": dtype,
                "act": rng.choice(["silu", "silu", "sigmoid", "none"]), "step": step, "keep": rng.random() < 0.5}
    vocab = _log_int(rng, 2, min(1 << 18, (1 << 28) // k))
    most = min(1 << 15, MOST[dtype] // (vocab * k), (1 << 30) // vocab)
    case = {"op": op, "rows": _log_int(rng, 1, max(1, most)), "vocab": vocab, "k": k, "dtype": dtype,
            "heat": rng.choice([0.5, 1.0, 1.0, 2.0]), "step": step}
    return case if op == "loss" else {**case, "top": _log_int(rng, 1, min(128, vocab))}


# ----------------------------------------------------------------- inputs --
def _acts(gen, rows, dim, dtype):
    """Activations: N(0,1), a few channels larger."""
    x = torch.randn(rows, dim, device="cuda", generator=gen)
    x *= 1.0 + 3.0 * (torch.rand(dim, device="cuda", generator=gen) < 0.02)
    return x.to(TORCH[dtype])


def _plan(case, gen):
    """Each row's group, rows group by group, and where each group starts."""
    m, g = case["rows"], case["groups"]
    if case["layout"] == "tables":        # sample-major: row i is table i mod G's
        ids = (torch.arange(m, device="cuda") % g).to(torch.int32)
    else:                                 # skewed shares
        share = torch.empty(g, device="cuda").exponential_(generator=gen) ** 2 + 1e-6
        ids = torch.multinomial(share, m, replacement=True, generator=gen).to(torch.int32)
        if case["layout"] == "sorted":
            ids = torch.sort(ids).values
    if g > 1:                             # one row in a hundred belongs to no group (a dropped token)
        ids[torch.rand(m, device="cuda", generator=gen) < 0.01] = -1
    key = torch.where(ids < 0, g, ids.long())
    offsets = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(key, minlength=g + 1)[:g].cumsum(0)
    return ids, torch.sort(key, stable=True).indices.to(torch.int32), offsets


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, k, dt = case["op"], case["rows"], case["k"], TORCH[case["dtype"]]
    s = {"case": case, "x": _acts(gen, m, k, case["dtype"])}
    if op == "gated":
        g, n = case["groups"], case["n"]
        s["ids"], s["order"], s["offsets"] = _plan(case, gen)
        s["ends"] = s["offsets"].tolist()  # a program that loops over groups has them on the host
        s["w"] = (torch.randn(g, 2 * n, k, device="cuda", generator=gen) / math.sqrt(k)).to(dt)
        if case["step"]:
            s["dy"] = torch.randn(m, n, device="cuda", generator=gen).to(dt)
        return s
    v = case["vocab"]
    # rows whose scores spread by two or so, as a head in training has them
    s["w"] = (torch.randn(v, k, device="cuda", generator=gen) * (2.0 / math.sqrt(k))).to(dt)
    # frequent items first; one row in twenty is padding
    first = (v * torch.rand(m, device="cuda", generator=gen) ** 3).long().clamp(max=v - 1)
    unseen = torch.rand(m, device="cuda", generator=gen) < UNSEEN
    if op == "loss":
        s["targets"] = torch.where(unseen, -100, first).to(torch.int32)
    else:
        t = case["top"]
        beside = torch.multinomial(torch.ones(min(v, 1 << 16), device="cuda"), t, generator=gen)
        top = (first[:, None] + beside) % v                       # t distinct items a row
        logits = 12.0 - torch.empty(m, t, device="cuda").exponential_(generator=gen).mul_(8.0 / t).cumsum(1)
        listed_ = torch.randint(1, t + 1, (m, 1), device="cuda", generator=gen)
        whole = torch.rand(m, 1, device="cuda", generator=gen) < 0.9
        gone = unseen[:, None] | (~whole & (torch.arange(t, device="cuda") >= listed_))
        s["top"] = torch.where(gone, -1, top).to(torch.int32)     # a shorter list ends in -1
        s["top_logits"] = logits
    if case["step"]:                      # of a mean over rows, with weights
        s["dloss"] = (0.5 + torch.rand(m, device="cuda", generator=gen)) / m
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import hash_table_lookup_amd as htl
    c = s["case"]
    if c["op"] == "gated":
        groups = htl.RowGroups(s["ids"], s["order"], s["offsets"], c["groups"])
        y, kept = htl.gated_mm(s["x"], s["w"], groups, act=c["act"], keep=c["keep"])
        if not c["step"]:
            return {"y": y, "kept": kept} if c["keep"] else {"y": y}
        dx, dw = htl.gated_mm_backward(s["dy"], s["x"], s["w"], kept, groups, act=c["act"])
        return {"y": y, "dx": dx, "dw": dw}
    if c["op"] == "loss":
        loss, lse = htl.softmax_loss(s["x"], s["w"], s["targets"], temperature=c["heat"])
        if not c["step"]:
            return {"loss": loss, "lse": lse}
        dx, dw = htl.softmax_loss_backward(s["dloss"], s["x"], s["w"], s["targets"], lse, temperature=c["heat"])
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    loss, kept = htl.distill_loss(s["x"], s["w"], s["top"], s["top_logits"], temperature=c["heat"])
    if not c["step"]:
        return {"loss": loss, "lse": kept[0]}
    dx, dw = htl.distill_loss_backward(s["dloss"], s["x"], s["w"], s["top"], s["top_logits"], kept, temperature=c["heat"])
    return {"loss": loss, "lse": kept[0], "dx": dx, "dw": dw}


# ------------------------------------------------------------- plain form --
def _act(z, kind):
    """(act(z), its slope) in fp32."""
    if kind == "none":
        return z, torch.ones_like(z)
    sig = torch.sigmoid(z)
    return (sig, sig * (1 - sig)) if kind == "sigmoid" else (z * sig, sig * (1 + z * (1 - sig)))


def _plain_gated(s):
    c, dt, n = s["case"], s["x"].dtype, s["case"]["n"]
    x, w = s["x"].float(), s["w"].float()
    out = {"y": torch.zeros(c["rows"], n, device="cuda", dtype=dt)}
    if c["step"]:
        dy = s["dy"].float()
        out["dx"] = torch.zeros(c["rows"], c["k"], device="cuda", dtype=dt)
        out["dw"] = torch.zeros(c["groups"], 2 * n, c["k"], device="cuda", dtype=dt)
    elif c["keep"]:
        out["kept"] = torch.zeros(c["rows"], 2 * n, device="cuda", dtype=dt)
    for i in range(c["groups"]):
        rows = s["order"][s["ends"][i]:s["ends"][i + 1]].long()
        if not len(rows):
            continue
        xg = x.index_select(0, rows)
        both = xg @ w[i].t()
        z, u = both[:, :n], both[:, n:]
        a, da = _act(z, c["act"])
        out["y"][rows] = (a * u).to(dt)
        if c["step"]:
            d = dy.index_select(0, rows)
            d = torch.cat([d * u * da, d * a], 1)
            out["dx"][rows] = (d @ w[i]).to(dt)
            out["dw"][i] = (d.t() @ xg).to(dt)
        elif c["keep"]:
            out["kept"][rows] = both.to(dt)
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "gated":
        return _plain_gated(s)
    dt, heat = s["x"].dtype, c["heat"]
    x, w = s["x"].float(), s["w"].float()
    scores = (x @ w.t()).div_(heat)
    most = scores.amax(1, keepdim=True)
    lse = (most + (scores - most).exp_().sum(1, keepdim=True).log_()).squeeze(1)
    if c["op"] == "loss":
        on = s["targets"] >= 0
        at = s["targets"].long().clamp(min=0)[:, None]
        share = on.float()[:, None]
        loss = lse - scores.gather(1, at).squeeze(1)
    else:
        listed_ = s["top"] >= 0
        on = listed_.any(1)
        at = s["top"].long().clamp(min=0)
        taught = torch.where(listed_, s["top_logits"] / heat, -torch.inf)
        taught = taught - torch.where(on, taught.amax(1), 0.0)[:, None]
        taught = taught - torch.where(on, taught.exp().sum(1), 1.0).log()[:, None]   # log of the teacher's shares
        share = taught.exp()
        loss = torch.where(listed_, share * (taught - scores.gather(1, at) + lse[:, None]), 0.0).sum(1)
    out = {"loss": torch.where(on, loss, 0.0), "lse": torch.where(on, lse, 0.0)}
    if not c["step"]:
        return out
    d = scores.sub_(lse[:, None]).exp_()
    d.scatter_add_(1, at, -share)
    d.mul_(torch.where(on, s["dloss"] / heat, 0.0)[:, None])
    return {**out, "dx": (d @ w).to(dt), "dw": (d.t() @ x).to(dt)}


# ---------------------------------------------------------- in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    m, k = case["rows"], case["k"]
    f8 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "gated":
        n, g = case["n"], case["groups"]
        res = {"y": torch.zeros(m, n, **f8)}
        if case["step"]:
            res |= {"dx": torch.zeros(m, k, **f8), "dw": torch.zeros(g, 2 * n, k, **f8)}
        elif case["keep"]:
            res["kept"] = torch.zeros(m, 2 * n, **f8)
        for i in range(g):
            rows = torch.nonzero(s["ids"] == i).flatten()
            if not len(rows):
                continue
            x, wz, wu = s["x"][rows].double(), s["w"][i, :n].double(), s["w"][i, n:].double()
            z, u = torch.mm(x, wz.t().contiguous()), torch.mm(x, wu.t().contiguous())
            e = torch.exp(-z)
            act = {"none": z, "sigmoid": 1 / (1 + e), "silu": z / (1 + e)}[case["act"]]
            res["y"][rows] = act * u
            if case["step"]:
                slope = {"none": torch.ones_like(e), "sigmoid": e / (1 + e) ** 2,
                         "silu": (1 + e + z * e) / (1 + e) ** 2}[case["act"]]
                d = s["dy"][rows].double()
                dz, du = d * u * slope, d * act
                res["dx"][rows] = torch.mm(dz, wz) + torch.mm(du, wu)
                res["dw"][i, :n] = torch.mm(dz.t().contiguous(), x)
                res["dw"][i, n:] = torch.mm(du.t().contiguous(), x)
            elif case["keep"]:
                res["kept"][rows, :n], res["kept"][rows, n:] = z, u
        return res
    # -sum p log(q / p) over the rows that have p: q the softmax of x w / heat, p the target's or the teacher's
    t = s["targets"][:, None] if case["op"] == "loss" else s["top"]
    rows = torch.nonzero((t >= 0).any(1)).flatten()
    t = t[rows].long()
    x, w = s["x"][rows].double(), s["w"].double()
    q = torch.mm(x, w.t().contiguous()) / case["heat"]
    lse = torch.logsumexp(q, 1)
    logp = torch.zeros(t.shape, **f8)
    if case["op"] == "distill":
        a = s["top_logits"][rows].double() / case["heat"]
        a[t < 0] = -math.inf
        logp = a - torch.logsumexp(a, 1, keepdim=True)
    p = torch.exp(logp) * (t >= 0)
    q -= lse[:, None]                     # log q
    terms = p * (logp.nan_to_num(neginf=0.0) - torch.gather(q, 1, t.clamp(min=0)))
    res = {"loss": torch.zeros(m, **f8), "lse": torch.zeros(m, **f8)}
    res["loss"][rows], res["lse"][rows] = terms.sum(1), lse
    if case["step"]:
        q = q.exp_()
        for j in range(t.shape[1]):       # items of a list are distinct, but for -1, whose p is 0
            q[torch.arange(len(rows), device="cuda"), t[:, j].clamp(min=0)] -= p[:, j]
        q *= s["dloss"][rows].double()[:, None] / case["heat"]
        res["dx"] = torch.zeros(m, k, **f8)
        res["dx"][rows] = torch.mm(q, w)
        res["dw"] = torch.mm(q.t().contiguous(), x)
    return res


# ------------------------------------------------------------------- work --
def work(case):
    b, m, k, three = SIZE[case["dtype"]], case["rows"], case["k"], 3 if case["step"] else 1
    if case["op"] == "gated":
        n, g = case["n"], case["groups"]
        # no more groups than rows have their weights read
        size = b * (m * k + min(g, m) * 2 * n * k + m * n) + (4 * m if g > 1 else 0)
        if case["step"]:                  # dy in, dx and dw out
            size += b * (m * n + m * k + g * 2 * n * k)
        elif case["keep"]:
            size += b * 2 * m * n
        return {"bytes": size, "flops": 4 * m * n * k * three}
    v, on = case["vocab"], m if m == 1 else m * (1 - UNSEEN)      # rows with a target
    size = b * (on * k + v * k) + 8 * m + (4 if case["op"] == "loss" else 8 * case["top"]) * m
    if case["step"]:                      # dloss in, dx and dw out
        size += 4 * m + b * (m * k + v * k)
    return {"bytes": size, "flops": 2 * on * v * k * three}
