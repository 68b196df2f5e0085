"""Dense operators on rows against plain 64-bit forms.

Tolerances are derived, not fitted: with u = 2^-24 the half step of fp32, a
sum of n terms in fp32 is off by at most n u times the sum of magnitudes in
any order, each further operation by u, and a bf16 result by half a step,
2^-8 of its value.  The bounds below add these up per element.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def _ids(rng, m, g, kind):
    if kind == "tables":
        ids = np.arange(m) % g
    elif kind == "none":
        ids = np.full(m, -1)
    elif kind == "one":                       # every row in one group, the others empty
        ids = np.full(m, g // 2)
    else:
        ids = np.minimum((rng.random(m) ** 2 * g).astype(np.int64), g - 1)
        if kind == "dropped" and m:
            ids[rng.random(m) < 0.2] = -1
            ids[rng.random(m) < 0.1] = g + 5
        if kind == "sorted":
            ids = np.sort(ids)
    return ids.astype(np.int32)


def _plan(htl, ids, g):
    return htl.group_rows(torch.from_numpy(ids).cuda(), g)


def _members(ids, g):
    return [np.flatnonzero(ids == i) for i in range(g)]


def _close(got, want, tol, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs()[bad].max()), float(tol[bad].min()))


# ---------------------------------------------------------------- groups --
@pytest.mark.parametrize("m", [0, 1, 2, 63, 64, 65, 1000, 16384, 16385, 70001, 1 << 20])
@pytest.mark.parametrize("g,kind", [(1, "one"), (26, "tables"), (26, "dropped"), (70, "sorted"), (300, "none"),
                                    (1023, "dropped"), (1024, "dropped"), (4095, "dropped")])
def test_group_rows(htl, m, g, kind):
    rng = np.random.default_rng(m + g)
    ids = _ids(rng, m, g, kind)
    plan = _plan(htl, ids, g)
    key = np.where((ids < 0) | (ids >= g), g, ids)
    assert np.array_equal(plan.order.cpu().numpy(), np.argsort(key, kind="stable"))
    want = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=g + 1)[:g])])
    assert np.array_equal(plan.offsets.cpu().numpy(), want)


# ----------------------------------------------------------------- rows8 --
def _rows8(x, fmt):
    """Values, scale bytes of 8-bit rows by their definition, in fp64."""
    x = x.double()
    m, dim = x.shape
    nb = (dim + 31) // 32
    most = 127.0 if fmt == "i8" else 448.0
    out, scales = torch.empty_like(x), torch.empty(m, nb, dtype=torch.uint8)
    for b in range(nb):
        v = x[:, 32 * b:32 * b + 32]
        top = v.abs().amax(1, keepdim=True)
        e = torch.full_like(top, -126.0)
        for k in range(-126, 122):
            e = torch.where(torch.ldexp(torch.tensor(most).double(), torch.tensor(k)) < top, float(k + 1), e)
        unit = torch.exp2(e)
        q = v / unit
        if fmt == "e4m3":
            k = (torch.frexp(q.abs()).exponent - 1).clamp(min=-6).double()
            step = torch.exp2(torch.where(q == 0, -6.0, k) - 3)
            q = torch.round(q / step) * step
        else:
            q = torch.round(q)
        fin = torch.isfinite(v).all(1, keepdim=True)
        out[:, 32 * b:32 * b + 32] = torch.where(fin, q * unit, float("nan"))
        scales[:, b] = torch.where(fin, e + 127, 255.0)[:, 0].to(torch.uint8)
    return out, scales


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,dim", [(0, 8), (1, 1), (3, 7), (5, 31), (4, 32), (9, 33), (17, 64), (33, 77), (300, 128),
                                   (2, 1000), (1, 65536)])
def test_rows8(htl, fmt, dtype, m, dim):
    gen = torch.Generator().manual_seed(m + dim)
    x = (torch.randn(m, dim, generator=gen) * torch.exp2(torch.randint(-20, 20, (m, 1), generator=gen).float())).to(dtype)
    if m > 2:
        x[0] = 0.0
        x[1, dim // 2] = float("inf") if fmt == "i8" else float("nan")
        x[2] = torch.tensor(3.0e38).to(dtype) * torch.sign(x[2].float()).to(dtype)
        x[-1] *= 2.0 ** -110                   # scales at their floor
    want, scales = _rows8(x, fmt)
    kept = htl.save_rows8(x.cuda(), fmt)
    assert torch.equal(kept.scales.cpu(), scales)
    for out in (torch.float32, torch.bfloat16):
        got = htl.load_rows8(kept, out).cpu()
        assert torch.equal(torch.nan_to_num(got.double(), nan=7.25), torch.nan_to_num(want.to(out).double(), nan=7.25))


def test_rows8_ties_and_edges(htl):
    # values half-way between codes, at the largest code, and just beyond it
    x = torch.zeros(4, 32)
    x[0, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    x[1, :4] = torch.tensor([127.0 + 2.0 ** -10, 1.0, 3.0, -1.0])    # the scale doubles
    x[2, :4] = torch.tensor([448.0, 17.0, 19.0, -2.0 ** -10])
    x[3, :4] = torch.tensor([449.0, 34.0, 38.0, 2.0 ** -8])
    for fmt in ("i8", "e4m3"):
        want, scales = _rows8(x, fmt)
        kept = htl.save_rows8(x.cuda(), fmt)
        assert torch.equal(kept.scales.cpu(), scales)
        assert torch.equal(htl.load_rows8(kept).cpu().double(), want)


# ----------------------------------------------------------------- norms --
class Norm:
    """n and r of rows in fp64, and how far fp32 statistics may put n off, per element (e_n)."""

    def __init__(self, x, kind):
        x = x.double()
        d = x.shape[1]
        mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
        c = x - mean
        self.r = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        self.n = c * self.r
        shift = (d + 4) * U * x.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
        self.e_n = self.r * shift * (1 + self.n.abs()) + (d + 16) * U * self.n.abs()
        self.kind, self.dim = kind, d

    def back(self, dn, e_dn):
        """Gradient from that of n (off by e_dn), and its bound before rounding."""
        d, n, r = self.dim, self.n, self.r
        c1 = dn.mean(1, keepdim=True) if self.kind == "layer" else torch.zeros_like(r)
        c2 = (dn * n).mean(1, keepdim=True)
        e1 = e_dn.mean(1, keepdim=True) + (d + 4) * U * dn.abs().mean(1, keepdim=True) if self.kind == "layer" else 0.0
        e2 = ((e_dn * n.abs() + dn.abs() * self.e_n).mean(1, keepdim=True)
              + (d + 8) * U * (dn * n).abs().mean(1, keepdim=True))
        mag = dn.abs() + c1.abs() + (n * c2).abs()
        err = e_dn + e1 + n.abs() * e2 + self.e_n * c2.abs() + 8 * U * mag
        return r * (dn - c1 - n * c2), r * (err + (d + 16) * U * mag)


def _param_of(p, ids, g):
    on = (ids >= 0) & (ids < g)
    out = p.double()[torch.from_numpy(np.where(on, ids, 0)).long()]
    return out, torch.from_numpy(on).unsqueeze(1)


def _sum_of(t, tol, ids, g):
    """Per-group sums of t's rows and their bound: each row's own, and the sum's."""
    s = torch.zeros(g, t.shape[1], dtype=torch.float64)
    e = torch.zeros_like(s)
    for i, rows in enumerate(_members(ids, g)):
        s[i] = t[rows].sum(0)
        e[i] = tol[rows].sum(0) + (len(rows) + 8) * U * t[rows].abs().sum(0)
    return s, e + 1e-30


SHAPES = [(1, 1), (2, 7), (70, 8), (33, 33), (65, 64), (129, 100), (1000, 128), (7, 200), (40, 256), (19, 512),
          (6, 1000), (9, 1024), (5, 2048), (3, 3000), (4, 4096), (3, 5001), (2, 8192), (3, 16384)]


def _inputs(m, dim, g, seed, kinds=("tables", "dropped", "sorted", "one", "none")):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    ids = _ids(rng, m, g, kinds[seed % len(kinds)])
    return gen, ids


@pytest.mark.parametrize("m,dim", SHAPES)
@pytest.mark.parametrize("xd,yd,kind,save,bias,g", [
    (torch.bfloat16, torch.bfloat16, "layer", "i8", True, 26), (torch.float32, torch.bfloat16, "rms", "e4m3", False, 3),
    (torch.float32, torch.float32, "layer", None, True, 70), (torch.bfloat16, torch.float32, "rms", None, True, 1)])
def test_norm_rows(htl, m, dim, xd, yd, kind, save, bias, g):
    gen, ids = _inputs(m, dim, g, m + dim + g)
    x = (torch.randn(m, dim, generator=gen) + 0.5).to(xd)
    weight = 1 + 0.1 * torch.randn(g, dim, generator=gen)
    b = 0.1 * torch.randn(g, dim, generator=gen) if bias else None
    plan = _plan(htl, ids, g)
    bc = None if b is None else b.cuda()
    kw = dict(groups=plan, kind=kind, eps=EPS)
    y, kept = htl.norm_rows(x.cuda(), weight.cuda(), bc, out_dtype=yd, save=save, **kw)
    w, on = _param_of(weight, ids, g)
    bw = _param_of(b, ids, g)[0] if bias else torch.zeros_like(w)

    def check_y(y, src):
        N = Norm(src, kind)
        want = torch.where(on, N.n * w + bw, 0.0)
        _close(y, want, w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs()) + HALF[yd] * want.abs() + 1e-37, "y")

    check_y(y, x)
    if save is None:
        src = x
    else:
        src = _rows8(x, save)[0]
        assert torch.equal(htl.load_rows8(kept, torch.float32).cpu().double(), src)
        again, _ = htl.norm_rows(kept, weight.cuda(), bc, out_dtype=yd, **kw)     # recomputed from the copy
        check_y(again, src)
    N = Norm(src, kind)
    dy = torch.randn(m, dim, generator=gen).to(yd)
    dres = torch.randn(m, dim, generator=gen).to(xd)
    for res in (dres, None):
        dx, dw, db = htl.norm_rows_backward(dy.cuda(), kept, weight.cuda(), bias=bias,
                                            dresidual=None if res is None else res.cuda(), **kw)
        dyd = torch.where(on, dy.double(), 0.0)
        gx, e = N.back(dyd * w, U * (dyd * w).abs())
        gx = torch.where(on, gx, 0.0)
        want = gx + (0.0 if res is None else res.double())
        _close(dx, want, e + U * want.abs() + HALF[xd] * want.abs() * 1.01 + 1e-37, "dx")
        s, t = _sum_of(dyd * N.n, dyd.abs() * N.e_n, ids, g)
        _close(dw, s, t, "dweight")
        if bias:
            s, t = _sum_of(dyd, torch.zeros_like(dyd), ids, g)
            _close(db, s, t, "dbias")
        else:
            assert db is None


def _act(u, act):
    s = torch.sigmoid(u)
    if act == "none":
        return u, torch.ones_like(u)
    return (s, s * (1 - s)) if act == "sigmoid" else (u * s, s * (1 + u * (1 - s)))


@pytest.mark.parametrize("m,dim", SHAPES)
@pytest.mark.parametrize("xd,zd,kind,act,save,bias,g", [
    (torch.float32, torch.bfloat16, "layer", "sigmoid", "e4m3", True, 26),
    (torch.bfloat16, torch.bfloat16, "rms", "silu", None, False, 1),
    (torch.bfloat16, torch.float32, "rms", "none", "i8", True, 3),
    (torch.float32, torch.float32, "layer", "silu", None, True, 70)])
def test_norm_gate(htl, m, dim, xd, zd, kind, act, save, bias, g):
    gen, ids = _inputs(m, dim, g, m + dim + g + 1)
    x = torch.randn(m, dim, generator=gen).to(xd)
    z = (2 * torch.randn(m, dim, generator=gen) - 0.3).to(zd)
    u = (2 * torch.randn(m, dim, generator=gen)).to(zd)
    weight = 1 + 0.1 * torch.randn(g, dim, generator=gen)
    b = 0.1 * torch.randn(g, dim, generator=gen) if bias else None
    bc = None if b is None else b.cuda()
    plan = _plan(htl, ids, g)
    kw = dict(groups=plan, kind=kind, eps=EPS, act=act, scale=0.75)
    out, kz, ku = htl.norm_gate(x.cuda(), z.cuda(), u.cuda(), weight.cuda(), bc, save=save, **kw)
    w, on = _param_of(weight, ids, g)
    bw = _param_of(b, ids, g)[0] if bias else torch.zeros_like(w)
    N = Norm(z, kind)
    v = N.n * w + bw
    e_v = w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs())
    a, _ = _act(u.double(), act)
    add = torch.where(on, 0.75 * a * v, 0.0)
    want = x.double() + add
    # the activation is a few operations and one exponential: 16 u
    _close(out, want, 0.75 * a.abs() * e_v + 20 * U * add.abs() + (U + HALF[xd]) * want.abs() + 1e-37, "out")
    zs, us = z, u
    if save is not None:
        zs, us = _rows8(z, save)[0], _rows8(u, save)[0]
        assert torch.equal(htl.load_rows8(kz, torch.float32).cpu().double(), zs)
        assert torch.equal(htl.load_rows8(ku, torch.float32).cpu().double(), us)
    dout = torch.randn(m, dim, generator=gen).to(xd)
    dz, du, dw, db = htl.norm_gate_backward(dout.cuda(), kz, ku, weight.cuda(), bc, **kw)
    N = Norm(zs, kind)
    v = N.n * w + bw
    e_v = w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs())
    uu = us.double()
    a, slope = _act(uu, act)
    D = torch.where(on, 0.75 * dout.double(), 0.0)
    s = torch.sigmoid(uu)
    mag = s * (1 + uu.abs() * (1 + s)) if act == "silu" else (s if act == "sigmoid" else torch.ones_like(uu))
    want = D * slope * v
    _close(du, want, D.abs() * (16 * U * mag * v.abs() + (slope.abs() + 16 * U * mag) * e_v)
           + (4 * U + HALF[zd]) * want.abs() + 1e-37, "dgate")
    e = D * a
    gz, err = N.back(e * w, 20 * U * (e * w).abs())
    gz = torch.where(on, gz, 0.0)
    _close(dz, gz, err + HALF[zd] * gz.abs() * 1.01 + 1e-37, "dz")
    sums, t = _sum_of(e * N.n, e.abs() * N.e_n + 20 * U * (e * N.n).abs(), ids, g)
    _close(dw, sums, t, "dweight")
    if bias:
        sums, t = _sum_of(e, 20 * U * e.abs(), ids, g)
        _close(db, sums, t, "dbias")


def test_norm_gradients_against_differences(htl):
    """The backward calls against central differences of the forward calls (fp32).

    f = sum(c * output) is differenced in single elements with h = 2^-6: the
    truncation is f''' h^2 / 6 (bounded here by 1 with unit-scale inputs,
    so 1e-4 of the scale of the derivative), and fp32 outputs off by u of
    their value give 2 u sum|c y| / (2 h)."""
    gen = torch.Generator().manual_seed(3)
    m, dim, g, h = 6, 40, 2, 2.0 ** -6
    ids = np.array([0, 1, 1, 0, -1, 1], np.int32)
    plan = _plan(htl, ids, g)
    x, z, u, c = (torch.randn(m, dim, generator=gen) for _ in range(4))
    w, b = 1 + 0.1 * torch.randn(g, dim, generator=gen), 0.1 * torch.randn(g, dim, generator=gen)
    kw = dict(groups=plan, kind="layer", eps=EPS)

    def f_norm(x, w, b):
        return htl.norm_rows(x.cuda(), w.cuda(), b.cuda(), **kw)[0].cpu().double().mul(c).sum()

    def f_gate(z, u, w, b):
        return htl.norm_gate(x.cuda(), z.cuda(), u.cuda(), w.cuda(), b.cuda(), scale=0.5, **kw)[0].cpu().double().mul(c).sum()

    got = htl.norm_rows_backward(c.cuda(), x.cuda(), w.cuda(), bias=True, **kw)
    dz, du, dw, db = htl.norm_gate_backward(c.cuda(), z.cuda(), u.cuda(), w.cuda(), b.cuda(), scale=0.5, **kw)
    tol = 20 * h * h + 2 * U * float(c.abs().sum()) * 4 / (2 * h)
    for f, args, grads in ((f_norm, [x, w, b], got), (f_gate, [z, u, w, b], (dz, du, dw, db))):
        for k, grad in enumerate(grads):
            for i, j in ((0, 0), (1, 17), (args[k].shape[0] - 1, dim - 1)):
                up, dn = [t.clone() for t in args], [t.clone() for t in args]
                up[k][i, j] += h
                dn[k][i, j] -= h
                want = float((f(*up) - f(*dn)) / (2 * h))
                assert abs(float(grad[i, j]) - want) <= tol, (f.__name__, k, i, j, float(grad[i, j]), want)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_leaves_other_rows_alone(htl, kind):
    """A row with a NaN, one of infinities, a constant row and a zero row: their neighbours, and rows of no
    group whatever they hold, come out as without them."""
    gen = torch.Generator().manual_seed(5)
    m, dim, g = 40, 96, 3
    ids = (np.arange(m) % (g + 1)).astype(np.int32)          # id 3: no group
    x = torch.randn(m, dim, generator=gen)
    w = torch.ones(g, dim)
    plan = _plan(htl, ids, g)
    kw = dict(groups=plan, kind=kind, eps=EPS)
    dy = torch.randn(m, dim, generator=gen)
    clean = htl.norm_rows(x.cuda(), w.cuda(), **kw)[0].cpu()
    clean_dx, clean_dw, _ = htl.norm_rows_backward(dy.cuda(), x.cuda(), w.cuda(), **kw)
    bad = x.clone()
    bad[3, 5], bad[7] = float("nan"), float("inf")            # both of no group
    got = htl.norm_rows(bad.cuda(), w.cuda(), **kw)[0].cpu()
    assert torch.equal(got, clean)
    dx, dw, _ = htl.norm_rows_backward(dy.cuda(), bad.cuda(), w.cuda(), **kw)
    assert torch.equal(dx, clean_dx) and torch.equal(dw, clean_dw)
    bad[0, 1], bad[4], bad[8], bad[12] = float("nan"), float("inf"), 0.0, 3.0
    got = htl.norm_rows(bad.cuda(), w.cuda(), **kw)[0].cpu()
    keep = [i for i in range(m) if i not in (0, 4, 8, 12)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[0]).all() and not torch.isfinite(got[4]).any()
    assert torch.equal(got[8], torch.zeros(dim))
    if kind == "layer":
        assert torch.equal(got[12], torch.zeros(dim))         # no deviation: eps alone under the root


def test_norm_without_groups_and_strided_rows(htl):
    gen = torch.Generator().manual_seed(6)
    wide = torch.randn(50, 3 * 136, generator=gen).cuda()
    w = (1 + 0.1 * torch.randn(128, generator=gen)).cuda()
    for off in (0, 8, 1, 3):                                  # aligned and unaligned rows inside wider ones
        x, z, u = wide[:, off:off + 128], wide[:, 136 + off:264 + off], wide[:, 272 + off:400 + off]
        y, kept = htl.norm_rows(x, w)
        yc, _ = htl.norm_rows(x.contiguous(), w)
        assert torch.equal(y, yc)
        assert kept.data_ptr() == x.data_ptr()
        a = htl.norm_rows_backward(u, x, w, dresidual=z)
        b = htl.norm_rows_backward(u.contiguous(), x.contiguous(), w, dresidual=z.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] is None and a[1].shape == (1, 128)
        a = htl.norm_gate(x, z, u, w)[0]
        b = htl.norm_gate(x.contiguous(), z.contiguous(), u.contiguous(), w)[0]
        assert torch.equal(a, b)
        a = htl.norm_gate_backward(x, z, u, w)
        b = htl.norm_gate_backward(x.contiguous(), z.contiguous(), u.contiguous(), w)
        assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))
    # a broadcast row, and transposed storage
    y, _ = htl.norm_rows(wide[:1, :128].expand(50, 128), w)
    assert torch.equal(y, y[:1].expand(50, 128))
    t = wide[:, :128].t().contiguous().t()
    assert torch.equal(htl.norm_rows(t, w)[0], htl.norm_rows(wide[:, :128], w)[0])


# -------------------------------------------------------------- products --
PRODUCTS = [(1, 1, 1, 1), (3, 2, 7, 5), (26, 26, 128, 256), (64, 16, 64, 64), (200, 3, 72, 40), (300, 5, 128, 128),
            (1000, 26, 64, 100), (999, 1, 33, 65), (70, 70, 136, 24), (513, 4, 256, 520), (2000, 3, 8, 8),
            (16, 2, 1032, 264), (5, 3, 2048, 16), (700, 2, 1, 9), (4100, 2, 64, 72), (1500, 2, 264, 520)]


def _product_check(htl, m, g, k, n, dtype, ids, seed, out=None):
    gen = torch.Generator().manual_seed(seed)
    out = out or dtype
    x = torch.randn(m, k, generator=gen).to(dtype)
    w = (torch.randn(g, n, k, generator=gen) / k ** 0.5).to(dtype)
    dy = torch.randn(m, n, generator=gen).to(dtype)
    plan = _plan(htl, ids, g)
    y = htl.grouped_mm(x.cuda(), w.cuda(), plan, out_dtype=out)
    dx, dw = htl.grouped_mm_backward(dy.cuda(), x.cuda(), w.cuda(), plan, dx_dtype=out)
    ry, ty = torch.zeros(m, n, dtype=torch.float64), torch.zeros(m, n, dtype=torch.float64)
    rx, tx = torch.zeros(m, k, dtype=torch.float64), torch.zeros(m, k, dtype=torch.float64)
    for i, rows in enumerate(_members(ids, g)):
        a, b, d = x[rows].double(), w[i].double(), dy[rows].double()
        ry[rows], ty[rows] = a @ b.t(), (k + 2) * U * (a.abs() @ b.abs().t())
        rx[rows], tx[rows] = d @ b, (n + 2) * U * (d.abs() @ b.abs())
        _close(dw[i], d.t() @ a, (len(rows) + 2) * U * (d.abs().t() @ a.abs()) + 1e-37, ("dw", i))
    _close(y, ry, ty + HALF[out] * (ry.abs() + ty) + 1e-37, "y")
    _close(dx, rx, tx + HALF[out] * (rx.abs() + tx) + 1e-37, "dx")
    return x, w, dy, plan, y, dx, dw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,g,k,n", PRODUCTS)
def test_grouped_mm(htl, m, g, k, n, dtype):
    rng = np.random.default_rng(m + k)
    kinds = ("dropped", "tables", "sorted", "one")
    ids = _ids(rng, m, g, kinds[(m + g) % 4])
    out = torch.float32 if (m + n) % 3 == 0 else dtype
    x, w, dy, plan, y, dx, dw = _product_check(htl, m, g, k, n, dtype, ids, m + n, out)
    # one gradient at a time
    only_x = htl.grouped_mm_backward(dy.cuda(), x.cuda(), w.cuda(), plan, dx_dtype=out, need_dw=False)
    only_w = htl.grouped_mm_backward(dy.cuda(), x.cuda(), w.cuda(), plan, need_dx=False)
    assert only_x[1] is None and torch.equal(only_x[0], dx)
    assert only_w[0] is None and torch.equal(only_w[1], dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_mm_no_rows_in_any_group(htl, dtype):
    for m in (0, 5, 300):
        _product_check(htl, m, 4, 64, 72, dtype, np.full(m, -1, np.int32), m)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_mm_keeps_nan_in_its_row(htl, dtype):
    """A NaN or an infinity in a row of no group reaches nothing; in a row of a
    group it reaches that row's products and that group's weight gradient."""
    m, g, k, n = 333, 3, 72, 136
    ids = (np.arange(m) % (g + 1)).astype(np.int32)
    x, w, dy, plan, y, dx, dw = _product_check(htl, m, g, k, n, dtype, ids, 1)
    bad, bdy = x.clone(), dy.clone()
    bad[3], bad[7, 2], bdy[11, 3], bdy[15] = float("inf"), float("nan"), float("nan"), float("inf")
    assert torch.equal(htl.grouped_mm(bad.cuda(), w.cuda(), plan), y)
    b_dx, b_dw = htl.grouped_mm_backward(bdy.cuda(), bad.cuda(), w.cuda(), plan)
    assert torch.equal(b_dx, dx) and torch.equal(b_dw, dw)
    bad[5, 1] = float("nan")                                   # row 5: group 1
    got = htl.grouped_mm(bad.cuda(), w.cuda(), plan)
    keep = [i for i in range(m) if i != 5]
    assert torch.equal(got[keep], y[keep]) and torch.isnan(got[5]).all()
    _, b_dw = htl.grouped_mm_backward(dy.cuda(), bad.cuda(), w.cuda(), plan)
    assert torch.equal(b_dw[0], dw[0]) and torch.equal(b_dw[2], dw[2]) and torch.isnan(b_dw[1][:, 1]).all()


def test_grouped_mm_strided_rows_and_no_plan(htl):
    gen = torch.Generator().manual_seed(8)
    wide = torch.randn(90, 400, generator=gen).bfloat16().cuda()
    w = torch.randn(136, 128, generator=gen).bfloat16().cuda()
    for off in (0, 8, 3):
        x, dy = wide[:, off:off + 128], wide[:, 200 + off:336 + off]
        assert torch.equal(htl.grouped_mm(x, w), htl.grouped_mm(x.contiguous(), w))
        a, b = htl.grouped_mm_backward(dy, x, w), htl.grouped_mm_backward(dy.contiguous(), x.contiguous(), w)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[1].shape == (1, 136, 128)
    # rows that lie group by group: offsets alone are the plan
    ids = np.sort(_ids(np.random.default_rng(1), 90, 4, "dropped") % 4).astype(np.int32)
    plan = _plan(htl, ids, 4)
    w4 = torch.randn(4, 136, 128, generator=gen).bfloat16().cuda()
    x = wide[:, :128]
    assert torch.equal(htl.grouped_mm(x, w4, plan), htl.grouped_mm(x, w4, plan._replace(order=None)))


@pytest.mark.parametrize("seed", range(3))
def test_broken_plans_stay_in_bounds(htl, seed):
    """Offsets out of range or decreasing, and order entries outside the rows, are clamped or skipped: rows
    around the tensors keep their bits."""
    rng = np.random.default_rng(seed)
    m, g, k, n = 500, 5, 64, 72
    off = rng.integers(-100, 700, g + 1).astype(np.int32)
    order = rng.integers(-300, 800, m).astype(np.int32)
    ids = torch.from_numpy(rng.integers(-2, 8, m).astype(np.int32)).cuda()
    plan = htl.RowGroups(ids, torch.from_numpy(order).cuda(), torch.from_numpy(off).cuda(), g)
    x = torch.randn(m, k, device="cuda").bfloat16()
    dy = torch.randn(m, n, device="cuda").bfloat16()
    w = torch.randn(g, n, k, device="cuda").bfloat16()
    p = torch.ones(g, k, device="cuda")
    y = htl.grouped_mm(x, w, plan)
    dx, dw = htl.grouped_mm_backward(dy, x, w, plan)
    a = htl.norm_rows(x, p, groups=plan)
    b = htl.norm_rows_backward(x, x, p, groups=plan)
    c = htl.norm_gate_backward(x, x, x, p, groups=plan)
    torch.cuda.synchronize()
    assert y.shape == (m, n) and dx.shape == (m, k) and dw.shape == (g, n, k) and a[0].shape == b[0].shape == c[0].shape


def test_calls_on_another_stream_and_in_a_graph(htl):
    gen = torch.Generator().manual_seed(9)
    m, g, k = 4000, 7, 64
    ids = torch.from_numpy(_ids(np.random.default_rng(2), m, g, "dropped")).cuda()
    x = torch.randn(m, k, generator=gen).cuda()
    w = torch.randn(g, k, k, generator=gen).bfloat16().cuda()
    p = torch.ones(g, k, device="cuda")

    def step():
        plan = htl.group_rows(ids, g)
        h, kept = htl.norm_rows(x, p, groups=plan, out_dtype="bf16", save="i8")
        z = htl.grouped_mm(h, w, plan)
        out, kz, ku = htl.norm_gate(x, z, h, p, groups=plan, save="e4m3")
        dz, du, dp2, _ = htl.norm_gate_backward(out, kz, ku, p, groups=plan)
        dh, dw = htl.grouped_mm_backward(dz, h, w, plan)
        dx, dp, _ = htl.norm_rows_backward(dh, kept, p, groups=plan, dresidual=out)
        return out, dx, dw, dp, dp2, du

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for i in range(4):
        x.add_(0.25 * i)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_rows_past_32_bits(htl):
    """More than 2^32 elements in a tensor: the last rows against the same rows alone."""
    m, dim = (1 << 25) + 65, 136
    x = torch.empty(m, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, m, 1 << 23):
        x[a:a + (1 << 23)].normal_()
    w = (1 + 0.1 * torch.randn(dim)).cuda()
    mat = torch.randn(dim, dim, device="cuda").bfloat16()
    tail = x[-1000:].clone()
    y, kept = htl.norm_rows(x, w, save="i8")
    ty, tkept = htl.norm_rows(tail, w, save="i8")
    assert torch.equal(y[-1000:], ty)
    assert torch.equal(kept.codes[-1000:], tkept.codes) and torch.equal(kept.scales[-1000:], tkept.scales)
    assert torch.equal(htl.load_rows8(kept)[-1000:], htl.load_rows8(tkept))
    dx, _, _ = htl.norm_rows_backward(y, kept, w)
    assert torch.equal(dx[-1000:], htl.norm_rows_backward(ty, tkept, w)[0])
    del dx, kept
    out = htl.grouped_mm(x, mat)
    assert torch.equal(out[-1000:], htl.grouped_mm(tail, mat))
    dx, dw = htl.grouped_mm_backward(x, y, mat)
    assert torch.equal(dx[-1000:], htl.grouped_mm_backward(tail, ty, mat)[0])
    assert torch.isfinite(dw).all()


# ------------------------------------------------- each kernel's own sizes --
@pytest.mark.parametrize("m", [4096, 4097, 5000, 131073, 300000])
@pytest.mark.parametrize("g,kind", [(5, "sorted"), (26, "tables"), (64, "dropped"), (127, "dropped"), (128, "one"),
                                    (500, "dropped")])
def test_group_rows_over_blocks(htl, m, g, kind):
    ids = _ids(np.random.default_rng(m * g), m, g, kind)
    plan = _plan(htl, ids, g)
    key = np.where((ids < 0) | (ids >= g), g, ids)
    assert np.array_equal(plan.order.cpu().numpy(), np.argsort(key, kind="stable"))
    want = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=g + 1)[:g])])
    assert np.array_equal(plan.offsets.cpu().numpy(), want)


# short reductions, tiles of 256 x 256 in the forward product and in the input gradient, long sums over rows
@pytest.mark.parametrize("m,g,k,n", [(1100, 2, 32, 1100), (1100, 2, 64, 600), (1100, 2, 128, 300), (1100, 2, 200, 136),
                                     (1100, 2, 31, 33), (1600, 3, 100, 50), (1200, 2, 250, 20), (8300, 3, 136, 4104),
                                     (8300, 3, 4104, 136), (9000, 2, 264, 264)])
@pytest.mark.parametrize("kind", ["tables", "dropped"])
def test_grouped_mm_kernels(htl, m, g, k, n, kind):
    ids = _ids(np.random.default_rng(m + k + n), m, g, kind)
    _product_check(htl, m, g, k, n, torch.bfloat16, ids, m + k)


@pytest.mark.parametrize("m,k,n", [(70001, 32, 1100), (70001, 64, 600), (70001, 128, 300), (70001, 31, 33),
                                   (70001, 100, 50), (1050000, 200, 136), (1050000, 136, 72)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_grouped_mm_many_rows(htl, m, k, n, out):
    """Products of many rows, whose matrices stay in LDS, against the same rows in slices, which take tiles: a
    row's product is summed in the same order, so the bits are the same."""
    g = 3
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    ids = torch.randint(-1, g, (m,), device="cuda", generator=gen).to(torch.int32)
    x = torch.randn(m, k, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(m, n, device="cuda", generator=gen).bfloat16()
    w = torch.randn(g, n, k, device="cuda", generator=gen).bfloat16()
    plan = htl.group_rows(ids, g)
    y = htl.grouped_mm(x, w, plan, out_dtype=out)
    dx, _ = htl.grouped_mm_backward(dy, x, w, plan, dx_dtype=out, need_dw=False)
    for a in (0, 30000, m - 3001):
        rows = slice(a, a + 3001)
        part = htl.group_rows(ids[rows], g)
        assert torch.equal(y[rows], htl.grouped_mm(x[rows], w, part, out_dtype=out))
        assert torch.equal(dx[rows], htl.grouped_mm_backward(dy[rows], x[rows], w, part, dx_dtype=out, need_dw=False)[0])
    assert torch.isfinite(y).all() and torch.isfinite(dx).all() and not y[ids < 0].any()


def test_grouped_mm_rows_far_apart(htl):
    """Operands that span more than 4 GiB take 64-bit addresses, with the same result to the bit."""
    m, k, n, ld = 66000, 264, 272, 33000
    gen = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.empty(m, ld, dtype=torch.bfloat16, device="cuda")
    x, dy = wide[:, 8:8 + k], wide[:, 1000:1000 + n]
    x.normal_(generator=gen)
    dy.normal_(generator=gen)
    ids = torch.randint(-1, 3, (m,), device="cuda", generator=gen).to(torch.int32)
    plan = htl.group_rows(ids, 3)
    w = torch.randn(3, n, k, device="cuda", generator=gen).bfloat16()
    xc, dyc = x.contiguous(), dy.contiguous()
    assert torch.equal(htl.grouped_mm(x, w, plan), htl.grouped_mm(xc, w, plan))
    a, b = htl.grouped_mm_backward(dy, x, w, plan), htl.grouped_mm_backward(dyc, xc, w, plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("m,dim,g", [(3000, 4104, 3), (1500, 9000, 1), (5000, 2048, 26), (20000, 20, 4), (9000, 600, 2)])
def test_norms_over_many_rows(htl, m, dim, g):
    """More rows than a launch has teams: every row of the outputs, and the sums over chunks."""
    gen, ids = _inputs(m, dim, g, 5 * m + 1)                  # ids with dropped rows
    x = torch.randn(m, dim, generator=gen)
    z, u = torch.randn(m, dim, generator=gen), torch.randn(m, dim, generator=gen)
    weight, b = 1 + 0.1 * torch.randn(g, dim, generator=gen), 0.1 * torch.randn(g, dim, generator=gen)
    plan = _plan(htl, ids, g)
    kw = dict(groups=plan, kind="layer", eps=EPS)
    w, on = _param_of(weight, ids, g)
    bw = _param_of(b, ids, g)[0]
    y, _ = htl.norm_rows(x.cuda(), weight.cuda(), b.cuda(), **kw)
    N = Norm(x, "layer")
    want = torch.where(on, N.n * w + bw, 0.0)
    _close(y, want, w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs()) + U * want.abs() + 1e-37, "y")
    dy = torch.randn(m, dim, generator=gen)
    dx, dw, db = htl.norm_rows_backward(dy.cuda(), x.cuda(), weight.cuda(), bias=True, **kw)
    d = torch.where(on, dy.double(), 0.0)
    gx, e = N.back(d * w, U * (d * w).abs())
    want = torch.where(on, gx, 0.0)
    _close(dx, want, e + 3 * U * want.abs() + 1e-37, "dx")
    _close(dw, *_sum_of(d * N.n, d.abs() * N.e_n, ids, g), "dweight")
    _close(db, *_sum_of(d, torch.zeros_like(d), ids, g), "dbias")
    del dx, y, want, gx, e
    out, _, _ = htl.norm_gate(x.cuda(), z.cuda(), u.cuda(), weight.cuda(), b.cuda(), act="sigmoid", **kw)
    N = Norm(z, "layer")
    v = N.n * w + bw
    e_v = w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs())
    a, slope = _act(u.double(), "sigmoid")
    add = torch.where(on, a * v, 0.0)
    want = x.double() + add
    _close(out, want, a * e_v + 20 * U * add.abs() + 2 * U * want.abs() + 1e-37, "out")
    dz, du, dw, db = htl.norm_gate_backward(dy.cuda(), z.cuda(), u.cuda(), weight.cuda(), b.cuda(), act="sigmoid", **kw)
    want = d * slope * v
    _close(du, want, d.abs() * (16 * U * a * v.abs() + (slope + 16 * U * a) * e_v) + 6 * U * want.abs() + 1e-37, "dgate")
    t = d * a
    gz, err = N.back(t * w, 20 * U * (t * w).abs())
    gz = torch.where(on, gz, 0.0)
    _close(dz, gz, err + 3 * U * gz.abs() + 1e-37, "dz")
    _close(dw, *_sum_of(t * N.n, t.abs() * N.e_n + 20 * U * (t * N.n).abs(), ids, g), "dweight")
    _close(db, *_sum_of(t, 20 * U * t.abs(), ids, g), "dbias")


def test_product_gradients_against_differences(htl):
    """f = sum(c y) is linear in each of x and w, so central differences are exact but for rounding: y is off by
    (k + 2) u of the products' magnitudes, twice, over 2 h; a gradient by its own sum's (rows or n, below 32 terms)."""
    m, k, n, g, h = 9, 24, 10, 2, 0.125
    gen = torch.Generator().manual_seed(7)
    ids = np.array([0, 1, 1, -1, 0, 1, 0, 5, 1], np.int32)
    plan = _plan(htl, ids, g)
    x, w, c = torch.randn(m, k, generator=gen), torch.randn(g, n, k, generator=gen), torch.randn(m, n, generator=gen)

    def f(x, w):
        return htl.grouped_mm(x.cuda(), w.cuda(), plan).cpu().double().mul(c).sum()

    dx, dw = htl.grouped_mm_backward(c.cuda(), x.cuda(), w.cuda(), plan)
    size = sum(float((c[r].double().abs() @ (w[int(i)].double().abs() + h) @ (x[r].double().abs() + h)))
               for r, i in enumerate(ids) if 0 <= i < g)
    tol = (k + 2) * U * size / h + 40 * U * size
    for arg, grad in ((0, dx), (1, dw)):
        base = (x, w)[arg]
        for flat in (0, 5, k + 3, 3 * k + 1, 7 * k, base.numel() - 1):
            at = np.unravel_index(flat, base.shape)
            up, dn = base.clone(), base.clone()
            up[at] += h
            dn[at] -= h
            args = [(up, w), (dn, w)] if arg == 0 else [(x, up), (x, dn)]
            want = float((f(*args[0]) - f(*args[1])) / ((up[at] - dn[at]).double()))
            assert abs(float(grad[at]) - want) <= tol, (arg, at, float(grad[at]), want, tol)


# ------------------------------------------------------- plans of one's own --
def test_plans_of_other_types_and_sizes_are_refused(htl):
    """What torch's own sorts and sums give (int64), and plans of other rows, are refused before a launch; strided
    int32 tensors are read as what they hold."""
    m, g, k = 90, 3, 16
    gen = torch.Generator().manual_seed(11)
    plan = _plan(htl, _ids(np.random.default_rng(3), m, g, "dropped"), g)
    x = torch.randn(m, k, generator=gen).cuda()
    w, p = torch.randn(g, k, k, generator=gen).cuda(), torch.ones(g, k, device="cuda")
    forward = (lambda q: htl.norm_rows(x, p, groups=q)[0], lambda q: htl.norm_gate(x, x, x, p, groups=q)[0])
    planned = (lambda q: htl.grouped_mm(x, w, q), lambda q: htl.grouped_mm_backward(x, x, w, q)[1],
               lambda q: htl.norm_rows_backward(x, x, p, groups=q)[1], lambda q: htl.norm_gate_backward(x, x, x, p, groups=q)[2])
    for f in forward:
        for bad in (plan.ids.long(), plan.ids[:-1], plan.ids.cpu()):
            with pytest.raises(ValueError, match="groups.ids"):
                f(plan._replace(ids=bad))
    for f in planned:
        for bad in (plan.order.long(), plan.order[:-1], plan.order.cpu()):
            with pytest.raises(ValueError, match="groups.order"):
                f(plan._replace(order=bad))
        for bad in (plan.offsets.long(), plan.offsets[:-1], plan.offsets.cpu()):
            with pytest.raises(ValueError, match="groups.offsets"):
                f(plan._replace(offsets=bad))

    def strided(t):
        return torch.stack([t, torch.full_like(t, -7)], 1)[:, 0]

    wide = htl.RowGroups(strided(plan.ids), strided(plan.order), strided(plan.offsets), g)
    assert not wide.order.is_contiguous()
    for f in forward + planned:
        assert torch.equal(f(wide), f(plan))


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows8_keeps_the_largest_values_finite(htl, fmt, dtype):
    """Up to the largest finite number: the nearest code, or the last one whose value is finite (63 * 2^122 in
    integers, 240 * 2^120 in e4m3), by saving alone and beside a norm."""
    most = torch.finfo(dtype).max
    top = torch.tensor([most, 3.39e38, 3.38e38, 3.377e38, 3.375e38, 3.35e38, 3.3e38, 3.29e38, 3.0e38, 2.98e38, 2.97e38,
                        1.7e38], dtype=torch.float64)
    gen = torch.Generator().manual_seed(12)
    x = torch.rand(2 * len(top), 70, generator=gen, dtype=torch.float64) * 2 - 1
    x *= torch.cat([top, top])[:, None]
    x[:len(top), 3], x[len(top):, 40] = top, -top
    x[0, 64:] = most
    x = x.clamp(-most, most).to(dtype)
    assert torch.isfinite(x).all()
    want, scales = _rows8(x, fmt)
    last = 63.0 * 2.0**122 if fmt == "i8" else 240.0 * 2.0**120
    big = scales.repeat_interleave(32, 1)[:, :70] == (249 if fmt == "i8" else 247)
    assert big.any() and (want[big].abs() > last).any()
    want = torch.where(big, want.clamp(-last, last), want)
    w = torch.ones(70).cuda()
    for kept in (htl.save_rows8(x.cuda(), fmt), htl.norm_rows(x.cuda(), w, save=fmt)[1],
                 htl.norm_gate(x.cuda(), x.cuda(), x.cuda(), w, save=fmt)[2]):
        assert torch.equal(kept.scales.cpu(), scales)
        for out in (torch.float32, torch.bfloat16):
            assert torch.equal(htl.load_rows8(kept, out).cpu().double(), want)


# ------------------------------------------------------ rows far from zero --
class FarNorm(Norm):
    """A layer norm whose mean is taken out in two steps, the second by the sum of what the first left.

    A lane adds up at most 16 elements, then 64 lanes in 6 steps, then 16 waves: no element goes through more than
    h = 40 additions, so a sum is off by h u of its magnitudes.  With A the row's mean magnitude, the first mean is off
    by at most s = (h + 4) u A, so what is summed then is of size C = s + |x - mean|, and the centre is off by (h + 5) u
    mean(C), an element by 3 u C beside.  The squares' mean, var + s^2 at most, is off by (h + 12) u of itself: e_r,
    relative, is how far 1 / deviation is off."""

    def __init__(self, x):
        super().__init__(x, "layer")
        x = x.double()
        h = min(x.shape[1], 40)
        dev = (x - x.mean(1, keepdim=True)).abs()
        var = (dev * dev).mean(1, keepdim=True)
        s = (h + 4) * U * x.abs().mean(1, keepdim=True)
        size = s + dev
        self.e_r = (h + 12) * U * (var + s * s) / (var + EPS) + 4 * U
        self.e_n = self.r * ((h + 5) * U * size.mean(1, keepdim=True) + 3 * U * size) + self.n.abs() * (self.e_r + 4 * U)

    def back(self, dn, e_dn):
        g, e = super().back(dn, e_dn)
        return g, e + self.e_r * g.abs()


@pytest.mark.parametrize("dim", [7, 77, 100, 128, 250, 500, 1000, 2000, 4100, 5001, 9000])
@pytest.mark.parametrize("save", [None, "i8"])
def test_layer_norm_far_from_zero(htl, dim, save):
    """Constant rows and rows of small deviation, far from zero: n is 0, or the deviation's own, not what the
    rounding of the mean leaves."""
    gen = torch.Generator().manual_seed(dim)
    far = torch.tensor([1000.1, 10000.1, 54321.7, -10000.1, 777777.7, 0.1])
    rows = [far[:, None].expand(6, dim)]
    rows += [far[:, None] + s * far[:, None].abs() * torch.randn(6, dim, generator=gen) for s in (1e-6, 1e-4, 1e-2)]
    x = torch.cat(rows)
    m, g = x.shape[0], 2
    ids = (np.arange(m) % g).astype(np.int32)
    plan = _plan(htl, ids, g)
    weight, b = 1 + 0.1 * torch.randn(g, dim, generator=gen), 0.1 * torch.randn(g, dim, generator=gen)
    w, bw = weight.double()[ids.astype(np.int64)], b.double()[ids.astype(np.int64)]
    dy = torch.randn(m, dim, generator=gen)
    kw = dict(groups=plan, kind="layer", eps=EPS)
    y, kept = htl.norm_rows(x.cuda(), weight.cuda(), b.cuda(), save=save, **kw)
    out, kz, ku = htl.norm_gate(dy.cuda(), x.cuda(), dy.cuda(), weight.cuda(), b.cuda(), act="none", save=save, **kw)
    N = FarNorm(x)
    e_v = w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs())
    v = N.n * w + bw
    _close(y, v, e_v + U * v.abs(), "y")
    assert float(N.e_n[:5].max()) < 0.05                       # what is told apart: they were off by up to 1
    d = dy.double()
    _close(out, d + d * v, d.abs() * e_v + 4 * U * (d * v).abs() + 2 * U * d.abs(), "out")
    src = x if save is None else _rows8(x, save)[0]
    us = dy if save is None else _rows8(dy, save)[0]
    N = FarNorm(src)
    dx, dw, db = htl.norm_rows_backward(dy.cuda(), kept, weight.cuda(), bias=True, **kw)
    gx, e = N.back(d * w, U * (d * w).abs())
    _close(dx, gx, e + 3 * U * gx.abs(), "dx")
    _close(dw, *_sum_of(d * N.n, d.abs() * N.e_n, ids, g), "dweight")
    dz, du, dw, db = htl.norm_gate_backward(dy.cuda(), kz, ku, weight.cuda(), b.cuda(), act="none", **kw)
    t = d * us.double()
    gz, e = N.back(t * w, 3 * U * (t * w).abs())
    _close(dz, gz, e + 3 * U * gz.abs(), "dz")
    v = N.n * w + bw
    e_v = w.abs() * N.e_n + 2 * U * ((N.n * w).abs() + bw.abs())
    _close(du, d * v, d.abs() * e_v + 4 * U * (d * v).abs(), "dgate")
    _close(dw, *_sum_of(t * N.n, t.abs() * N.e_n + 3 * U * (t * N.n).abs(), ids, g), "dweight")


# -------------------------------------------------- what lies around results --
class Guarded:
    """A tensor with margins of a byte pattern before and after it, itself of the pattern or of what it is given."""
    MARGIN = 1 << 17

    def __init__(self, *shape, dtype=torch.float32, pattern=0xA5, values=None):
        if values is not None:
            shape, dtype = values.shape, values.dtype
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.pattern = pattern
        self.raw = torch.full((n + 2 * self.MARGIN,), pattern, dtype=torch.uint8, device="cuda")
        self.t = self.raw[self.MARGIN:self.MARGIN + n].view(dtype).view(*shape)
        if values is not None:
            self.t.copy_(values)

    @property
    def ptr(self):
        return self.t.data_ptr()

    def intact(self):
        return all(bool((side == self.pattern).all()) for side in (self.raw[:self.MARGIN], self.raw[-self.MARGIN:]))


def _sizes_plan(htl, sizes, seed):
    """A plan of groups of the sizes given, rows shuffled, 37 of no group."""
    ids = np.repeat(np.arange(len(sizes)), sizes)
    ids = np.concatenate([ids, np.full(37, -1)]).astype(np.int32)
    np.random.default_rng(seed).shuffle(ids)
    return ids, _plan(htl, ids, len(sizes))


SPLIT = [[5000, 1, 0, 700, 300, 9000, 2, 256, 257], [1] * 70 + [6000] + [0] * 70 + [300] * 3 + [7000, 1], [20000]]


@pytest.mark.parametrize("sizes", SPLIT, ids=["mixed", "150 groups", "one"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(40, 72), (264, 520)])
def test_product_sums_of_split_and_whole_groups(htl, sizes, dtype, n, k):
    """Groups of one chunk, of several and of none side by side, in a workspace of exactly the size asked for."""
    ids, plan = _sizes_plan(htl, sizes, n)
    m, g, L = len(ids), len(sizes), htl.lib()
    gen = torch.Generator().manual_seed(n + g)
    x, dy = torch.randn(m, k, generator=gen).to(dtype), torch.randn(m, n, generator=gen).to(dtype)
    xc, dyc = x.cuda(), dy.cuda()
    nb = L.grouped_mm_backward_workspace_bytes(m, g, n, k)
    dw, ws = Guarded(g, n, k), Guarded(nb, dtype=torch.uint8)
    code = 0 if dtype == torch.float32 else 1
    assert L.grouped_mm_backward(dyc.data_ptr(), n, xc.data_ptr(), k, None, code, m, n, k, plan.order.data_ptr(),
                                 plan.offsets.data_ptr(), g, None, code, dw.ptr, ws.ptr, nb, 0) == 0
    torch.cuda.synchronize()
    assert dw.intact() and ws.intact()
    for i, rows in enumerate(_members(ids, g)):
        a, d = x[rows].double(), dy[rows].double()
        _close(dw.t[i], d.t() @ a, (len(rows) + 2) * U * (d.abs().t() @ a.abs()) + 1e-37, ("dw", i))


@pytest.mark.parametrize("sizes", SPLIT, ids=["mixed", "150 groups", "one"])
@pytest.mark.parametrize("dim", [24, 200, 1000, 4100])
def test_norm_sums_of_split_and_whole_groups(htl, sizes, dim):
    ids, plan = _sizes_plan(htl, sizes, dim)
    m, g, L = len(ids), len(sizes), htl.lib()
    gen = torch.Generator().manual_seed(dim + g)
    x, dy = torch.randn(m, dim, generator=gen), torch.randn(m, dim, generator=gen)
    w, xc, dyc = torch.ones(g, dim, device="cuda"), x.cuda(), dy.cuda()
    nb = L.norm_back_workspace_bytes(m, g, dim)
    N = Norm(x, "rms")
    d = dy.double()
    want = [_sum_of(d * N.n, d.abs() * N.e_n, ids, g), _sum_of(d, torch.zeros_like(d), ids, g)]
    order, offsets = plan.order.data_ptr(), plan.offsets.data_ptr()
    for gate in (False, True):
        dx, du, dw, db, ws = Guarded(m, dim), Guarded(m, dim), Guarded(g, dim), Guarded(g, dim), Guarded(nb, dtype=torch.uint8)
        if gate:                              # no activation, a gate of ones
            ones = torch.ones(m, dim, device="cuda")
            status = L.norm_gate_backward(dyc.data_ptr(), 0, dim, xc.data_ptr(), dim, None, ones.data_ptr(), dim, None, 0,
                                          0, m, dim, w.data_ptr(), None, order, offsets, g, 0, EPS, 0, 1.0, dx.ptr, du.ptr,
                                          dw.ptr, db.ptr, ws.ptr, nb, 0)
        else:
            status = L.norm_rows_backward(dyc.data_ptr(), 0, dim, xc.data_ptr(), 0, dim, None, 0, None, 0, m, dim,
                                          w.data_ptr(), order, offsets, g, 0, EPS, dx.ptr, dw.ptr, db.ptr, ws.ptr, nb, 0)
        torch.cuda.synchronize()
        assert status == 0 and all(t.intact() for t in (dx, du, dw, db, ws))
        for got, (s, e), what in zip((dw.t, db.t), want, ("dweight", "dbias")):
            _close(got, s, e + 2 * U * s.abs(), (what, gate))


# ---------------------------------------------------------- gates far open --
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("zd", [torch.float32, torch.bfloat16])
def test_gates_far_from_zero(htl, act, zd):
    """Gates up to the largest finite numbers: out, and the slope relative to itself.

    With e = exp(-|u|) the sigmoid is 1 / (1 + e) or e / (1 + e), its slope e / (1 + e)^2: an exponential and four
    operations of fp32, 16 u of their value at most.  silu's slope is s (1 + u t): 16 u of s (1 + |u| t).  Below 2^-126
    values may go to zero."""
    m, dim = 64, 40
    gen = torch.Generator().manual_seed(21)
    u = torch.randn(m, dim, generator=gen)
    top = float(torch.finfo(zd).max)
    for i, v in enumerate([8.0, 10.0, 12.0, 15.0, 17.0, 18.0, 20.0, 30.0, 50.0, 80.0, 87.0, 88.0, 89.0, 100.0, 1e4, 1e20, top]):
        u[2 * i], u[2 * i + 1] = v, -v
    u = u.to(zd)
    x, z = torch.zeros(m, dim), torch.randn(m, dim, generator=gen).to(zd)
    w, b = torch.ones(1, dim), 0.5 * torch.ones(1, dim)
    dout = (1 + torch.rand(m, dim, generator=gen)).to(torch.float32)
    scale = 2.0**-10                                           # out stays finite
    kw = dict(kind="rms", eps=EPS, act=act, scale=scale)
    out, _, _ = htl.norm_gate(x.cuda(), z.cuda(), u.cuda(), w.cuda(), b.cuda(), **kw)
    dz, du, dw, db = htl.norm_gate_backward(dout.cuda(), z.cuda(), u.cuda(), w.cuda(), b.cuda(), **kw)
    N = Norm(z, "rms")
    v, e_v = N.n + 0.5, N.e_n + 2 * U * (N.n.abs() + 0.5)
    uu = u.double()
    e = torch.exp(-uu.abs())
    s = torch.where(uu < 0, e / (1 + e), 1 / (1 + e))
    t = torch.where(uu < 0, 1 / (1 + e), e / (1 + e))
    a, slope, mag = (s, s * t, s * t) if act == "sigmoid" else (uu * s, s * (1 + uu * t), s * (1 + uu.abs() * t))
    D = scale * dout.double()
    small = 2.0**-126 * (1 + v.abs()) * 4 * (1 if act == "sigmoid" else 200.0)
    _close(out, scale * a * v, scale * (a.abs() * e_v + 20 * U * (a * v).abs()) + small, "out")
    want = D * slope * v
    _close(du, want, D * (16 * U * mag * v.abs() + (slope.abs() + 16 * U * mag) * e_v)
           + (4 * U + HALF[zd]) * want.abs() + small, "dgate")
    assert torch.isfinite(out).all() and torch.isfinite(du).all()
    ea = D * a
    keep = torch.isfinite(ea.float()).all(1) & (ea.abs().amax(1) < 1e18)       # (beyond, the sums of dz pass fp32)
    gz, err = N.back(ea, 20 * U * ea.abs())
    gz, err = gz[keep], err[keep]
    _close(dz[keep.cuda()], gz, err + HALF[zd] * gz.abs() * 1.01 + 1e-30, "dz")


def test_infinite_gates_stay_in_their_elements(htl):
    """A gate of +-infinity, or NaN, reaches its own element's output and gate gradient, its row's dz and the sums, and
    no other row; in a row of no group, nothing."""
    m, dim, g = 30, 48, 2
    gen = torch.Generator().manual_seed(22)
    ids = (np.arange(m) % 3).astype(np.int32)                  # id 2: no group
    plan = _plan(htl, ids, g)
    x, z, u, dout = (torch.randn(m, dim, generator=gen) for _ in range(4))
    w = torch.ones(g, dim).cuda()

    def both(u, act):
        kw = dict(groups=plan, act=act, eps=EPS)
        out = htl.norm_gate(x.cuda(), z.cuda(), u.cuda(), w, **kw)[0].cpu()
        return (out, *(t.cpu() for t in htl.norm_gate_backward(dout.cuda(), z.cuda(), u.cuda(), w, **kw)[:3]))

    inf, nan = float("inf"), float("nan")
    for act in ("none", "sigmoid", "silu"):
        clean = both(u, act)
        bad = u.clone()
        bad[2, 3], bad[5, 4], bad[8] = inf, -inf, nan
        assert all(torch.equal(a, b) for a, b in zip(both(bad, act), clean))
        bad[0, 1], bad[3, 2], bad[6, 7] = inf, -inf, nan       # rows of group 0
        out, dz, du, dw = both(bad, act)
        rows = [i for i in range(m) if i not in (0, 3, 6)]
        assert torch.equal(out[rows], clean[0][rows]) and torch.equal(dz[rows], clean[1][rows])
        assert torch.equal(du[rows], clean[2][rows]) and torch.equal(dw[1], clean[3][1])
        for r, c in ((0, 1), (3, 2), (6, 7)):
            cols = [j for j in range(dim) if j != c]
            assert torch.equal(out[r, cols], clean[0][r, cols]) and torch.equal(du[r, cols], clean[2][r, cols])
        assert torch.isnan(out[6, 7]) and torch.isnan(du[6, 7]).item() == (act != "none")
        if act == "sigmoid":                                   # limits: 1 and 0, slope 0
            assert torch.isfinite(out[0]).all() and out[3, 2] == x[3, 2] and du[0, 1] == 0 and du[3, 2] == 0


def _broken_plan(m, g, seed):
    """ids, order and offsets that break every rule: entries below and past the rows, offsets that decrease and overlap."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(-3, g + 3, m)
    order = rng.integers(-15, m + 15, m)
    offsets = rng.integers(-100, m + 200, g + 1)
    if seed % 2:
        ids[::7], order[::7], offsets[1] = 2**31 - 1, -2**31, 2**31 - 1
    else:
        ids[::7], order[::7], offsets[1] = -2**31, 2**31 - 1, -2**31
    return [Guarded(values=torch.from_numpy(t.astype(np.int32))) for t in (ids, order, offsets)]


def _nan_around(values):
    return Guarded(values=values, pattern=0xFF)              # 0xFF bytes: NaN in fp32 and bf16


# tiles of 32, 128 and 256 rows, matrices kept in LDS; lengths of whole and of odd pieces
@pytest.mark.parametrize("m,k,n", [(500, 64, 72), (700, 33, 77), (20000, 64, 136), (20000, 63, 135), (14600, 264, 1024),
                                   (14600, 1024, 264), (70000, 64, 72), (70000, 33, 50)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_of_broken_plans_keep_to_their_rows(htl, m, k, n, dtype):
    """Nothing is written outside the results and the workspace, and nothing read outside the operands: the NaN there
    would show in the results, or in rows that no entry names, which keep their finite pattern."""
    g, L = 5, htl.lib()
    gen = torch.Generator().manual_seed(m + k)
    code = 0 if dtype == torch.float32 else 1
    for seed in (m, m + 1):
        _, order, offsets = _broken_plan(m, g, seed)
        x, dy, w = (_nan_around(torch.randn(*s, generator=gen).to(dtype)) for s in ((m, k), (m, n), (g, n, k)))
        nb = L.grouped_mm_backward_workspace_bytes(m, g, n, k)
        y, dx = Guarded(m, n, dtype=dtype), Guarded(m, k, dtype=dtype)
        dw, ws = Guarded(g, n, k), Guarded(nb, dtype=torch.uint8)
        for o in (order.ptr, None):
            assert L.grouped_mm(x.ptr, k, w.ptr, code, m, n, k, o, offsets.ptr, g, y.ptr, code, 0) == 0
            assert L.grouped_mm_backward(dy.ptr, n, x.ptr, k, w.ptr, code, m, n, k, o, offsets.ptr, g, dx.ptr, code,
                                         dw.ptr, ws.ptr, nb, 0) == 0
            torch.cuda.synchronize()
            for name, t in dict(x=x, dy=dy, w=w, y=y, dx=dx, dw=dw, ws=ws, order=order, offsets=offsets).items():
                assert t.intact(), name
            assert all(torch.isfinite(t.t).all() for t in (y, dx, dw))


@pytest.mark.parametrize("m,dim", [(500, 24), (500, 77), (9000, 128), (700, 600), (300, 2000), (200, 5001), (100, 9001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_of_broken_plans_keep_to_their_rows(htl, m, dim, dtype):
    g, L = 5, htl.lib()
    gen = torch.Generator().manual_seed(m + dim)
    code = 0 if dtype == torch.float32 else 1
    blocks = (dim + 31) // 32
    for seed in (m, m + 1):
        ids, order, offsets = _broken_plan(m, g, seed)
        x, z, u, d = (_nan_around(torch.randn(m, dim, generator=gen).to(dtype)) for _ in range(4))
        w, b = (_nan_around(torch.randn(g, dim, generator=gen)) for _ in range(2))
        nb = L.norm_back_workspace_bytes(m, g, dim)
        rows = [Guarded(m, dim, dtype=dtype) for _ in range(5)]
        sums = [Guarded(g, dim) for _ in range(2)]
        codes = [Guarded(m, dim, dtype=torch.uint8) for _ in range(2)]
        scales = [Guarded(m, blocks, dtype=torch.uint8) for _ in range(2)]
        ws = Guarded(nb, dtype=torch.uint8)
        y, dx, out, dz, du = rows
        assert L.norm_rows(x.ptr, code, dim, None, 0, m, dim, w.ptr, b.ptr, ids.ptr, g, 1, EPS, y.ptr, code, codes[0].ptr,
                           scales[0].ptr, 0, 0) == 0
        assert L.norm_gate(x.ptr, code, dim, z.ptr, dim, u.ptr, dim, code, m, dim, w.ptr, b.ptr, ids.ptr, g, 1, EPS, 2, 1.0,
                           out.ptr, codes[0].ptr, scales[0].ptr, codes[1].ptr, scales[1].ptr, 1, 0) == 0
        torch.cuda.synchronize()
        assert all(torch.isfinite(t.t).all() for t in (y, out))
        for o in (order.ptr, None):
            assert L.norm_rows_backward(d.ptr, code, dim, x.ptr, code, dim, None, 0, u.ptr, dim, m, dim, w.ptr, o, offsets.ptr,
                                        g, 1, EPS, dx.ptr, sums[0].ptr, sums[1].ptr, ws.ptr, nb, 0) == 0
            torch.cuda.synchronize()
            assert all(t.intact() and torch.isfinite(t.t).all() for t in (dx, *sums))
            assert L.norm_gate_backward(d.ptr, code, dim, codes[0].ptr, dim, scales[0].ptr, codes[1].ptr, dim, scales[1].ptr,
                                        code, 1, m, dim, w.ptr, b.ptr, o, offsets.ptr, g, 1, EPS, 2, 1.0, dz.ptr, du.ptr,
                                        sums[0].ptr, sums[1].ptr, ws.ptr, nb, 0) == 0
            torch.cuda.synchronize()
            assert all(t.intact() and torch.isfinite(t.t).all() for t in (dz, du, *sums))
        for t in (ids, order, offsets, x, z, u, d, w, b, ws, *rows, *codes, *scales):
            assert t.intact()


def test_sums_past_32_bits(htl):
    """Gradients over more than 2^32 elements that come from the last rows alone: the incoming gradient is zero in all
    others, so that an address cut short reads zeros, or other rows."""
    m, dim, n = (1 << 25) + 65, 136, 1000
    x = torch.empty(m, dim, dtype=torch.bfloat16, device="cuda")
    for a in range(0, m, 1 << 23):
        x[a:a + (1 << 23)].normal_()
    dy = torch.zeros(m, dim, dtype=torch.bfloat16, device="cuda")
    dy[-n:].normal_()
    w = torch.ones(2, dim).cuda()
    mat = torch.zeros(2, dim, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.ones(m, dtype=torch.int32, device="cuda")
    ids[:1 << 24] = -1                                        # the rest is of group 1, group 0 is empty
    plan = htl.group_rows(ids, 2)
    a, d = x[-n:].cpu().double(), dy[-n:].cpu().double()
    N = Norm(a, "rms")
    whole = torch.ones(n, dtype=torch.int64).numpy()
    sums = _sum_of(d * N.n, d.abs() * N.e_n, whole, 2), _sum_of(d, torch.zeros_like(d), whole, 2)
    for groups, p in ((None, w[:1]), (plan, w)):
        _, dw, db = htl.norm_rows_backward(dy, x, p, groups=groups, eps=EPS, bias=True)
        _close(dw[-1:], sums[0][0][1:], sums[0][1][1:], "dweight")
        _close(db[-1:], sums[1][0][1:], sums[1][1][1:], "dbias")
        _, du, dw, _ = htl.norm_gate_backward(dy, x, dy, p, groups=groups, eps=EPS, act="none")
        s, t = _sum_of(d * d * N.n, d * d * N.e_n + 3 * U * (d * d * N.n).abs(), whole, 2)
        _close(dw[-1:], s[1:], t[1:], "gate's dweight")
        assert not du[:-n].any()
        _close(du[-n:], d * N.n, d.abs() * N.e_n + (3 * U + HALF[torch.bfloat16]) * (d * N.n).abs(), "dgate")
        del du
        _, dw = htl.grouped_mm_backward(dy, x, mat[:p.shape[0]], groups, need_dx=False)
        _close(dw[-1], d.t() @ a, (n + 2) * U * (d.abs().t() @ a.abs()), "dw")
        if groups is not None:
            assert not dw[0].any()


@pytest.mark.parametrize("g", [71, 1000, 4095])
def test_many_groups(htl, g):
    """As many groups as there may be, most of them of a few rows or none."""
    m = 9000
    ids = _ids(np.random.default_rng(g), m, g, "dropped")
    for dtype in (torch.bfloat16, torch.float32):
        _product_check(htl, m, g, 16, 24, dtype, ids, g)
    gen = torch.Generator().manual_seed(g)
    dim = 40
    x, dy = torch.randn(m, dim, generator=gen), torch.randn(m, dim, generator=gen)
    weight = 1 + 0.1 * torch.randn(g, dim, generator=gen)
    kw = dict(groups=_plan(htl, ids, g), kind="layer", eps=EPS)
    w, on = _param_of(weight, ids, g)
    N = Norm(x, "layer")
    want = torch.where(on, N.n * w, 0.0)
    _close(htl.norm_rows(x.cuda(), weight.cuda(), **kw)[0], want, w.abs() * N.e_n + 4 * U * want.abs() + 1e-37, "y")
    dx, dw, db = htl.norm_rows_backward(dy.cuda(), x.cuda(), weight.cuda(), bias=True, **kw)
    d = torch.where(on, dy.double(), 0.0)
    gx, e = N.back(d * w, U * (d * w).abs())
    want = torch.where(on, gx, 0.0)
    _close(dx, want, e + 3 * U * want.abs() + 1e-37, "dx")
    _close(dw, *_sum_of(d * N.n, d.abs() * N.e_n, ids, g), "dweight")
    _close(db, *_sum_of(d, torch.zeros_like(d), ids, g), "dbias")
