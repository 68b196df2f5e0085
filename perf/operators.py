"""What the dense operators beside the embedding lookup are measured on.

A lookup hands over rows that belong to groups (the feature table of each
row, or the expert that a router chose for it).  The operators that follow:

* ``groups``   which rows belong to which group, in a stable order;
* ``norm``     a per-group norm before a block, with the input kept in 8 bits
               for the backward pass;
* ``product``  every row times its group's matrix, and the gradients;
* ``gate``     a per-group norm after a block, its gate, and the residual sum;
* ``rows8``    rows kept in 8 bits and read back.

``run`` computes them in their plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
BLOCK = 32                                # elements that share one 8-bit scale
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
MERGED = 26 * 65536                       # the merged-tables batch: 65,536 samples of 26 feature tables


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one serving step's tokens sorted by expert: latency
        {"name": "groups-step", "op": "groups", "rows": 1000, "groups": 26, "layout": "experts"},
        # the merged-tables batch, sample-major, sorted by feature table
        {"name": "groups-merged", "op": "groups", "rows": MERGED, "groups": 26, "layout": "tables"},
        # a few rows of odd width kept in 8 bits and read back: latency
        {"name": "rows8-odd", "op": "rows8", "rows": 333, "dim": 77, "dtype": "f32", "save": "i8"},
        # a layer's activations on the merged-tables batch
        {"name": "rows8-merged", "op": "rows8", "rows": MERGED, "dim": 128, "dtype": "bf16", "save": "e4m3"},
        # one request: a sample's 26 feature rows from an fp32 table, normed to bf16
        {"name": "norm-request", "op": "norm", "rows": 26, "dim": 128, "groups": 26, "layout": "tables",
         "dtype": "f32", "inner": "bf16", "kind": "layer", "bias": True, "step": False, "save": "none"},
        # a training step of the norm on the merged-tables batch, input kept in 8 bits
        {"name": "norm-merged", "op": "norm", "rows": MERGED, "dim": 128, "groups": 26, "layout": "tables",
         "dtype": "bf16", "inner": "bf16", "kind": "layer", "bias": True, "step": True, "save": "i8"},
        # a training step after a wide block: one group, nothing quantised
        {"name": "gate-wide", "op": "gate", "rows": 16384, "dim": 4096, "groups": 1, "layout": "experts",
         "dtype": "bf16", "inner": "bf16", "kind": "rms", "bias": False, "act": "silu", "step": True, "save": "none"},
        # a training step after each feature table's projection, fp32 residual, block outputs kept in 8 bits
        {"name": "gate-merged", "op": "gate", "rows": MERGED // 4, "dim": 128, "groups": 26, "layout": "tables",
         "dtype": "f32", "inner": "bf16", "kind": "layer", "bias": True, "act": "sigmoid", "step": True,
         "save": "e4m3"},
        # one request through each table's projection in fp32: latency
        {"name": "product-request", "op": "product", "rows": 26, "groups": 26, "layout": "tables",
         "k": 128, "n": 256, "dtype": "f32", "step": False},
        # a serving step of 64 tokens over 16 experts: the weights' bytes count
        {"name": "product-tokens", "op": "product", "rows": 64, "groups": 16, "layout": "experts",
         "k": 2048, "n": 4096, "dtype": "bf16", "step": False},
        # a training step of each feature table's projection on the merged-tables batch
        {"name": "product-merged", "op": "product", "rows": MERGED, "groups": 26, "layout": "tables",
         "k": 128, "n": 256, "dtype": "bf16", "step": True},
        # a training step of experts with ragged shares of the tokens
        {"name": "product-experts", "op": "product", "rows": 16384, "groups": 16, "layout": "experts",
         "k": 2048, "n": 4096, "dtype": "bf16", "step": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["groups", "rows8", "norm", "gate", "product", "product"])
    layout = rng.choice(["experts", "tables", "sorted"])
    if op == "groups":
        return {"op": op, "rows": _log_int(rng, 1, MERGED), "groups": _log_int(rng, 1, 1000), "layout": layout}
    if op == "product":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # widths in eights mostly, as weights are laid out; odd ones now and then
        k = _log_int(rng, 16, 4096) if rng.random() < 0.2 else 8 * _log_int(rng, 2, 512)
        n = _log_int(rng, 16, 4096) if rng.random() < 0.2 else 8 * _log_int(rng, 2, 512)
        most = min((1 << 37) // (k * n), (1 << 28) // (k + n))
        groups = _log_int(rng, 1, max(1, min(64, (1 << 27) // (k * n))))
        return {"op": op, "rows": _log_int(rng, 1, max(1, most if dtype == "bf16" else most // 8)), "groups": groups,
                "layout": layout, "k": k, "n": n, "dtype": dtype, "step": rng.random() < 0.6}
    dim = _log_int(rng, 1, 8192) if rng.random() < 0.3 else 8 * _log_int(rng, 1, 1024)
    rows = _log_int(rng, 1, min(MERGED, (1 << 26) // dim))
    case = {"op": op, "rows": rows, "dim": dim, "dtype": rng.choice(["f32", "bf16"])}
    if op == "rows8":
        return {**case, "save": rng.choice(["i8", "e4m3"])}
    case |= {"groups": rng.choice([1, 1, _log_int(rng, 2, 100)]), "layout": layout, "inner": rng.choice(["bf16", "bf16", "f32"]),
             "kind": rng.choice(["rms", "layer"]), "bias": rng.random() < 0.5, "step": rng.random() < 0.7,
             "save": rng.choice(["none", "i8", "e4m3"])}
    return case if op == "norm" else {**case, "act": rng.choice(["silu", "sigmoid", "none"])}


# ----------------------------------------------------------------- inputs --
def _ids(case, gen):
    m, g = case["rows"], case["groups"]
    if case["layout"] == "tables":        # sample-major: row i is table i mod G's
        ids = (torch.arange(m, device="cuda") % g).to(torch.int32)
    else:                                 # skewed shares
        share = torch.empty(g, device="cuda").exponential_(generator=gen) ** 2 + 1e-6
        ids = torch.multinomial(share, m, replacement=True, generator=gen).to(torch.int32)
        if case["layout"] == "sorted":
            ids = torch.sort(ids).values
    if g > 1:                             # one row in a hundred belongs to no group (a missing feature, a dropped token)
        ids[torch.rand(m, device="cuda", generator=gen) < 0.01] = -1
    return ids


def _acts(gen, rows, dim, dtype):
    """Activations: N(0,1), a few channels far larger."""
    x = torch.randn(rows, dim, device="cuda", generator=gen)
    x *= 1.0 + 7.0 * (torch.rand(dim, device="cuda", generator=gen) < 0.02)
    return x.to(TORCH[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op != "rows8":
        ids = s["ids"] = _ids(case, gen)
        g = case["groups"]
        if op != "groups":                # the plan of rows per group, which a program keeps per batch
            if own:
                import hash_table_lookup_amd as htl
                s["groups"] = htl.group_rows(ids, g)
            else:
                key = torch.where(ids < 0, g, ids.long())
                s["order"] = torch.sort(key, stable=True).indices
                s["ends"] = torch.bincount(key, minlength=g + 1)[:g].cumsum(0).tolist()
    if op == "rows8":
        s["x"] = _acts(gen, case["rows"], case["dim"], case["dtype"])
    elif op == "product":
        dt = TORCH[case["dtype"]]
        s["x"] = _acts(gen, case["rows"], case["k"], case["dtype"])
        s["w"] = (torch.randn(g, case["n"], case["k"], device="cuda", generator=gen) / math.sqrt(case["k"])).to(dt)
        if case["step"]:
            s["dy"] = torch.randn(case["rows"], case["n"], device="cuda", generator=gen).to(dt)
    elif op in ("norm", "gate"):
        rows, dim = case["rows"], case["dim"]
        s["weight"] = 1.0 + 0.1 * torch.randn(g, dim, device="cuda", generator=gen)
        s["bias"] = 0.1 * torch.randn(g, dim, device="cuda", generator=gen) if case["bias"] else None
        s["x"] = _acts(gen, rows, dim, case["dtype"])
        if op == "gate":
            s["z"] = _acts(gen, rows, dim, case["inner"])
            s["gate"] = torch.randn(rows, dim, device="cuda", generator=gen).to(TORCH[case["inner"]])
        if case["step"]:
            s["dy"] = torch.randn(rows, dim, device="cuda", generator=gen).to(TORCH[case["inner" if op == "norm" else "dtype"]])
            if op == "norm":
                s["dres"] = torch.randn(rows, dim, device="cuda", generator=gen).to(TORCH[case["dtype"]])
    return s


SCALE = 0.5                               # of the block's output in the residual sum


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import hash_table_lookup_amd as htl
    c = s["case"]
    op = c["op"]
    if op == "groups":
        plan = htl.group_rows(s["ids"], c["groups"])
        return {"order": plan.order, "offsets": plan.offsets}
    save = None if c.get("save", "none") == "none" else c["save"]
    if op == "rows8":
        return {"values": htl.load_rows8(htl.save_rows8(s["x"], save))}
    if op == "product":
        out = {"y": htl.grouped_mm(s["x"], s["w"], s["groups"])}
        if c["step"]:
            out["dx"], out["dw"] = htl.grouped_mm_backward(s["dy"], s["x"], s["w"], s["groups"])
        return out
    if op == "norm":
        y, kept = htl.norm_rows(s["x"], s["weight"], s["bias"], groups=s["groups"], kind=c["kind"], eps=EPS,
                                out_dtype=c["inner"], save=save)
        if not c["step"]:
            return {"y": y} if save is None else {"y": y, "kept": htl.load_rows8(kept)}
        dx, dw, db = htl.norm_rows_backward(s["dy"], kept, s["weight"], groups=s["groups"], kind=c["kind"], eps=EPS,
                                            bias=c["bias"], dresidual=s["dres"])
        out = {"y": y, "dx": dx, "dweight": dw}
        return out if db is None else {**out, "dbias": db}
    out, kept_z, kept_gate = htl.norm_gate(s["x"], s["z"], s["gate"], s["weight"], s["bias"], groups=s["groups"],
                                           kind=c["kind"], eps=EPS, act=c["act"], scale=SCALE, save=save)
    if not c["step"]:
        return {"out": out} if save is None else {"out": out, "z": htl.load_rows8(kept_z), "gate": htl.load_rows8(kept_gate)}
    dz, dgate, dw, db = htl.norm_gate_backward(s["dy"], kept_z, kept_gate, s["weight"], s["bias"], groups=s["groups"],
                                               kind=c["kind"], eps=EPS, act=c["act"], scale=SCALE)
    res = {"out": out, "dz": dz, "dgate": dgate, "dweight": dw}
    return res if db is None else {**res, "dbias": db}


# ------------------------------------------------------------- plain form --
def _rows8(x, fmt):
    """x (fp32) after 8 bits: per block of 32 a power of two, then an integer or an e4m3 number."""
    rows, dim = x.shape
    pad = -dim % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).view(rows, -1, BLOCK)
    top, most = b.abs().amax(-1, keepdim=True), 127.0 if fmt == "i8" else 448.0
    lead = 6 if fmt == "i8" else 8        # most = 1.98 * 2^6 or 1.75 * 2^8
    frac, e = torch.frexp(top)            # top = 2 frac * 2^(e - 1), 2 frac in [1, 2)
    e = e - 1 - lead + (2.0 * frac > most / 2.0 ** lead)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    q = torch.ldexp(b, -e)
    q = torch.round(q) if fmt == "i8" else q.to(torch.float8_e4m3fn).to(x.dtype)
    v = torch.ldexp(q, e)
    v = torch.where(torch.isfinite(b).all(-1, keepdim=True), v, float("nan"))
    return v.view(rows, dim + pad)[:, :dim]


def _norm(x, kind):
    """(x's normed rows, 1 / deviation) in fp32."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_back(dn, n, r, kind):
    """The gradient of the norm's input from that of its output."""
    d = dn - n * (dn * n).mean(-1, keepdim=True)
    return (d - dn.mean(-1, keepdim=True) if kind == "layer" else d) * r


def _per_group(t, s):
    """Sums of rows by group, fp32 [G, dim]."""
    out = torch.zeros(s["case"]["groups"], t.shape[1], device=t.device, dtype=t.dtype)
    at = 0
    for i, end in enumerate(s["ends"]):
        if end > at:
            out[i] = t.index_select(0, s["order"][at:end]).sum(0)
        at = end
    return out


def _param(p, ids):
    return p.index_select(0, ids.clamp(min=0))


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "groups":
        key = torch.where(s["ids"] < 0, c["groups"], s["ids"].long())
        offsets = torch.zeros(c["groups"] + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.bincount(key, minlength=c["groups"] + 1)[:c["groups"]].cumsum(0)
        return {"order": torch.sort(key, stable=True).indices.to(torch.int32), "offsets": offsets}
    if op == "rows8":
        return {"values": _rows8(s["x"].float(), c["save"]).to(s["x"].dtype)}
    if op == "product":
        x, w, dt = s["x"].float(), s["w"].float(), s["x"].dtype
        out = {"y": torch.zeros(c["rows"], c["n"], device="cuda", dtype=dt)}
        if c["step"]:
            dy = s["dy"].float()
            out["dx"] = torch.zeros(c["rows"], c["k"], device="cuda", dtype=dt)
            out["dw"] = torch.zeros(c["groups"], c["n"], c["k"], device="cuda")
        at = 0
        for i, end in enumerate(s["ends"]):
            rows, at = s["order"][at:end], end
            if not len(rows):
                continue
            xg = x.index_select(0, rows)
            out["y"][rows] = (xg @ w[i].t()).to(dt)
            if c["step"]:
                dg = dy.index_select(0, rows)
                out["dx"][rows] = (dg @ w[i]).to(dt)
                out["dw"][i] = dg.t() @ xg
        return out
    ids, xd, inner = s["ids"].long(), s["x"].dtype, TORCH[c["inner"]]
    on = (ids >= 0).unsqueeze(1)          # a row of no group: the block adds nothing, and gets no gradient
    weight = _param(s["weight"], ids)
    bias = _param(s["bias"], ids) if c["bias"] else 0.0
    if op == "norm":
        n, _ = _norm(s["x"].float(), c["kind"])
        out = {"y": torch.where(on, n * weight + bias, 0.0).to(inner)}
        kept = s["x"].float() if c["save"] == "none" else _rows8(s["x"].float(), c["save"])
        if not c["step"]:
            return out if c["save"] == "none" else {**out, "kept": kept.to(xd)}
        n, r = _norm(kept, c["kind"])
        dy = torch.where(on, s["dy"].float(), 0.0)
        out["dx"] = (torch.where(on, _norm_back(dy * weight, n, r, c["kind"]), 0.0) + s["dres"].float()).to(xd)
        out["dweight"] = _per_group(dy * n, s)
        return {**out, "dbias": _per_group(dy, s)} if c["bias"] else out

    def act(u):
        sig = torch.sigmoid(u)
        if c["act"] == "none":
            return u, torch.ones_like(u)
        return (sig, sig * (1 - sig)) if c["act"] == "sigmoid" else (u * sig, sig * (1 + u * (1 - sig)))

    z, u = s["z"].float(), s["gate"].float()
    n, _ = _norm(z, c["kind"])
    out = {"out": (s["x"].float() + torch.where(on, SCALE * act(u)[0] * (n * weight + bias), 0.0)).to(xd)}
    if c["save"] != "none":
        z, u = _rows8(z, c["save"]), _rows8(u, c["save"])
    if not c["step"]:
        return out if c["save"] == "none" else {**out, "z": z.to(inner), "gate": u.to(inner)}
    n, r = _norm(z, c["kind"])
    a, da = act(u)
    d = torch.where(on, SCALE * s["dy"].float(), 0.0)
    out["dz"] = _norm_back(d * a * weight, n, r, c["kind"]).to(inner)
    out["dgate"] = (d * da * (n * weight + bias)).to(inner)
    out["dweight"] = _per_group(d * a * n, s)
    return {**out, "dbias": _per_group(d * a, s)} if c["bias"] else out


# ---------------------------------------------------------- in 64 bits --
def _exact8(x, fmt):
    """The 8-bit value of every element of x (fp64), from the definition: with 2^e the least power of two,
    e >= -126, that brings a block's largest magnitude to 127 (or 448), the nearest multiple of 2^e
    (or the nearest e4m3 number times 2^e), ties to even."""
    rows, dim = x.shape
    out = torch.empty_like(x)
    most = 127.0 if fmt == "i8" else 448.0
    for a in range(0, dim, BLOCK):
        b = x[:, a:a + BLOCK]
        top = b.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / most))
        e = torch.where(torch.exp2(e - 1) * most >= top, e - 1, torch.where(torch.exp2(e) * most < top, e + 1, e))
        unit = torch.exp2(e.clamp(min=-126.0))
        q = b / unit
        if fmt == "e4m3":                 # spacing 2^(k - 3) in [2^k, 2^(k + 1)), at least 2^-9
            k = torch.frexp(q.abs()).exponent - 1
            step = torch.exp2(torch.where(q != 0, k, -6).clamp(min=-6).double() - 3)
            q = torch.round(q / step) * step
        else:
            q = torch.round(q)
        out[:, a:a + BLOCK] = q * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, ids, g = case["op"], s.get("ids"), case.get("groups", 1)
    members = [torch.nonzero(ids == i).flatten() for i in range(g)] if op != "rows8" else []
    if op == "groups":
        ends = torch.tensor([0] + [len(m) for m in members]).cumsum(0).to(torch.int32)
        return {"order": torch.cat(members + [torch.nonzero(ids < 0).flatten()]).to(torch.int32), "offsets": ends}
    if op == "rows8":
        return {"values": _exact8(s["x"].double(), case["save"])}
    if op == "product":
        out = {"y": torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")}
        if case["step"]:
            out["dx"] = torch.zeros(case["rows"], case["k"], dtype=torch.float64, device="cuda")
            out["dw"] = torch.zeros(g, case["n"], case["k"], dtype=torch.float64, device="cuda")
        for i, m in enumerate(members):
            if not len(m):
                continue
            x, w = s["x"][m].double(), s["w"][i].double()
            out["y"][m] = torch.mm(x, w.t().contiguous())
            if case["step"]:
                d = s["dy"][m].double()
                out["dx"][m] = torch.mm(d, w)
                out["dw"][i] = torch.mm(d.t().contiguous(), x)
        return out

    def stats(t):                         # (x - mean) / sqrt(var + eps), and 1 / sqrt(var + eps)
        mid = t.sum(1, keepdim=True) / t.shape[1] if case["kind"] == "layer" else torch.zeros_like(t[:, :1])
        inv = 1.0 / torch.sqrt(((t - mid) ** 2).sum(1, keepdim=True) / t.shape[1] + EPS)
        return (t - mid) * inv, inv

    def dstats(d, t):                     # inv (d - [mean d] - n mean(d n))
        n, inv = stats(t)
        mid = d.sum(1, keepdim=True) / d.shape[1] if case["kind"] == "layer" else 0.0
        return inv * (d - mid - n * ((d * n).sum(1, keepdim=True) / d.shape[1]))

    step, save = case["step"], case["save"]
    src = s["x"].double() if op == "norm" else s["z"].double()
    kept = _exact8(src, save) if save != "none" else src
    res = {("y" if op == "norm" else "out"): torch.zeros_like(src) if op == "norm" else s["x"].double()}
    if op == "gate":
        u = s["gate"].double()
        kept_u = _exact8(u, save) if save != "none" else u
    if not step:
        if save != "none":
            res |= {"kept": kept} if op == "norm" else {"z": kept, "gate": kept_u}
    elif op == "norm":
        res |= {"dx": s["dres"].double(), "dweight": torch.zeros(g, case["dim"], dtype=torch.float64, device="cuda")}
    else:
        res |= {"dz": torch.zeros_like(src), "dgate": torch.zeros_like(src),
                "dweight": torch.zeros(g, case["dim"], dtype=torch.float64, device="cuda")}
    if step and case["bias"]:
        res["dbias"] = torch.zeros(g, case["dim"], dtype=torch.float64, device="cuda")
    a_of = {"none": lambda v: v, "sigmoid": lambda v: 1.0 / (1.0 + torch.exp(-v)), "silu": lambda v: v / (1.0 + torch.exp(-v))}
    for i, m in enumerate(members):
        if not len(m):
            continue
        w = s["weight"][i].double()
        b = s["bias"][i].double() if case["bias"] else torch.zeros_like(w)
        v = stats(src[m])[0] * w + b
        if op == "norm":
            res["y"][m] = v
        else:
            act = a_of[case["act"]]
            res["out"][m] += SCALE * act(u[m]) * v
        if not step:
            continue
        n = stats(kept[m])[0]
        d = s["dy"][m].double()
        if op == "gate":
            e = torch.exp(-kept_u[m])
            slope = {"none": torch.ones_like(e), "sigmoid": e / (1 + e) ** 2,
                     "silu": 1 / (1 + e) + kept_u[m] * e / (1 + e) ** 2}[case["act"]]
            res["dgate"][m] = SCALE * d * slope * (n * w + b)
            d = SCALE * d * act(kept_u[m])
            res["dz"][m] = dstats(d * w, kept[m])
        else:
            res["dx"][m] += dstats(d * w, kept[m])
        res["dweight"][i] = (d * n).sum(0)
        if case["bias"]:
            res["dbias"][i] = d.sum(0)
    return res


# ------------------------------------------------------------------- work --
def work(case):
    op, m = case["op"], case["rows"]
    if op == "groups":                    # ids once, order and offsets once
        return {"bytes": 8 * m + 4 * (case["groups"] + 1), "flops": 0}
    if op == "product":
        b, k, n, g = SIZE[case["dtype"]], case["k"], case["n"], case["groups"]
        # no more groups than rows have their weights read
        size, flops = b * (m * k + min(g, m) * n * k + m * n), 2 * m * k * n
        if case["step"]:                  # dy in, dx and dw out; x, dy and w counted once
            size += b * (m * n + m * k) + 4 * g * n * k
            flops *= 3
        return {"bytes": size, "flops": flops}
    d = case["dim"]
    b = SIZE[case["dtype"]]
    eight = 0 if case["save"] == "none" else m * (d + -(-d // BLOCK))
    if op == "rows8":                     # in, codes out and in, values out
        return {"bytes": 2 * b * m * d + 2 * eight, "flops": 4 * m * d}
    i = SIZE[case["inner"]]
    par = 4 * min(case["groups"], m) * d * (2 if case["bias"] else 1) + (4 * m if case["groups"] > 1 else 0)
    if op == "norm":
        size = (b + i) * m * d + par + eight
        if case["step"]:                  # dy and dres in, dx out, the kept rows read back
            size += (i + 2 * b) * m * d + 2 * par + eight
        elif eight:
            size += eight + b * m * d
        return {"bytes": size, "flops": (25 if case["step"] else 8) * m * d}
    size = (2 * b + 2 * i) * m * d + par + 2 * eight
    if case["step"]:                      # dout in, dz and dgate out, the kept rows read back
        size += (b + 2 * i) * m * d + 2 * par + 2 * eight
    elif eight:
        size += 2 * eight + 2 * i * m * d
    return {"bytes": size, "flops": (50 if case["step"] else 16) * m * d}
