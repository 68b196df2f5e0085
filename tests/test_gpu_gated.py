"""Gated projections against plain 64-bit forms.

Tolerances are derived, not fitted: with u = 2^-24 the half step of fp32, a
sum of n products in fp32 is off by at most (n + 2) u times the sum of their
magnitudes in any order, each further operation by u, the activation and its
slope by 8 u of their values and, through their argument, by at most 1.1 and
0.5 of its error; a result, or an operand of a later product, kept in bf16 by
half a step, 2^-8 of its value.  The bounds below add these up per element.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
ACTS = ("none", "sigmoid", "silu")


def _act(z, kind):
    """(act, slope) in fp64 from exp(-|z|)."""
    if kind == "none":
        return z, torch.ones_like(z)
    s = torch.sigmoid(z)
    t = torch.sigmoid(-z)
    return (s, s * t) if kind == "sigmoid" else (z * s, s * (1 + z * t))


def _ids(rng, m, g, kind):
    ids = np.minimum((rng.random(m) ** 2 * g).astype(np.int64), g - 1)
    if kind == "dropped":
        ids[rng.random(m) < 0.2] = -1
        ids[rng.random(m) < 0.1] = g + 5
    if kind == "none":
        ids[:] = -1
    if kind == "one":
        ids[:] = g // 2
    return ids.astype(np.int32)


def _close(got, want, tol, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs()[bad].max()), float(tol[bad].min()))


class Want:
    """The formulas in fp64, with each value's bound."""

    def __init__(self, x, w, dy, ids, act, kept, out=None, dx=None):
        dt = x.dtype
        half = HALF[dt]
        m, k = x.shape
        g, n = w.shape[0], w.shape[1] // 2
        z8 = dict(dtype=torch.float64)
        self.y, self.ty = torch.zeros(m, n, **z8), torch.zeros(m, n, **z8)
        self.kept, self.tkept = torch.zeros(m, 2 * n, **z8), torch.zeros(m, 2 * n, **z8)
        self.dx, self.tdx = torch.zeros(m, k, **z8), torch.zeros(m, k, **z8)
        self.dw, self.tdw = torch.zeros(g, 2 * n, k, **z8), torch.zeros(g, 2 * n, k, **z8)
        oh, dh = HALF[out or dt], HALF[dx or dt]
        for i in range(g):
            rows = torch.from_numpy(np.flatnonzero(ids == i))
            if not len(rows):
                continue
            xg, wg, d = x[rows].double(), w[i].double(), dy[rows].double()
            both, e = xg @ wg.t(), (k + 2) * U * (xg.abs() @ wg.abs().t())
            self.kept[rows], self.tkept[rows] = both, e + half * (both.abs() + e)
            z, u, ez, eu = both[:, :n], both[:, n:], e[:, :n], e[:, n:]
            a, s = _act(z, act)
            ea = 1.1 * ez + 8 * U * a.abs()
            y = a * u
            ey = ea * (u.abs() + eu) + a.abs() * eu + U * y.abs()
            self.y[rows], self.ty[rows] = y, ey + oh * (y.abs() + ey)
            if kept:                              # the backward pass takes z and u as they were kept
                ez, eu = (t + half * (v.abs() + t) for t, v in ((ez, z), (eu, u)))
                ea = 1.1 * ez + 8 * U * a.abs()
            es = (0.0 if act == "none" else 0.5) * ez + 8 * U * (s.abs() + z.abs() * U + 2.0 ** -100)
            both = torch.cat([d * u * s, d * a], 1)
            e = torch.cat([d.abs() * (es * (u.abs() + eu) + s.abs() * eu + 2 * U * (u * s).abs()), d.abs() * (ea + U * a.abs())], 1)
            e = e + half * (both.abs() + e)
            v, ev = both @ wg, e @ wg.abs() + (2 * n + 2) * U * ((both.abs() + e) @ wg.abs())
            self.dx[rows], self.tdx[rows] = v, ev + dh * (v.abs() + ev)
            v, ev = both.t() @ xg, e.t() @ xg.abs() + (len(rows) + 2) * U * ((both.abs() + e).t() @ xg.abs())
            self.dw[i], self.tdw[i] = v, ev + half * (v.abs() + ev)


def _data(m, n, k, g, dtype, seed=0):
    gen = torch.Generator().manual_seed(1000 * m + 10 * n + k + seed)
    x = torch.randn(m, k, generator=gen).to(dtype)
    w = (torch.randn(g, 2 * n, k, generator=gen) * (2.0 / k ** 0.5)).to(dtype)
    return x, w, torch.randn(m, n, generator=gen).to(dtype)


SIZES = [(0, 8, 8, 1), (1, 1, 1, 1), (1, 64, 32, 1), (1, 8192, 64, 1), (2, 3, 5, 2), (17, 64, 96, 3), (33, 65, 40, 2),
         (65, 130, 31, 4), (128, 64, 64, 1), (150, 96, 257, 5), (300, 33, 72, 26), (513, 264, 136, 1), (700, 40, 520, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,g", SIZES)
def test_gated(htl, m, n, k, g, keep, dtype):
    act = ACTS[(m + n + keep) % 3]
    rng = np.random.default_rng(m + n)
    ids = _ids(rng, m, g, "dropped" if g > 1 else "one")
    x, w, dy = _data(m, n, k, g, dtype)
    want = Want(x, w, dy, ids, act, keep)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g) if g > 1 else None
    xc, wc, dc = x.cuda(), w.cuda(), dy.cuda()
    y, kept = htl.gated_mm(xc, wc, groups, act=act, keep=keep)
    assert y.dtype == dtype and (kept is None) == (not keep)
    _close(y, want.y, want.ty, "y")
    if keep:
        _close(kept, want.kept, want.tkept, "kept")
    dx, dw = htl.gated_mm_backward(dc, xc, wc, kept, groups, act=act)
    assert dx.dtype == dtype and dw.dtype == dtype
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("kind", ["none", "one"])
def test_groups_without_rows(htl, kind):
    ids = _ids(np.random.default_rng(0), 70, 6, kind)
    x, w, dy = _data(70, 40, 48, 6, torch.bfloat16)
    want = Want(x, w, dy, ids, "silu", False)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), 6)
    bad = torch.from_numpy((ids < 0) | (ids >= 6))
    x[bad], dy[bad] = float("nan"), float("inf")     # what no group has is not looked at
    y, kept = htl.gated_mm(x.cuda(), w.cuda(), groups, keep=True)
    _close(y, want.y, want.ty, "y")
    for from_ in (kept, None):
        want = Want(x.masked_fill(bad[:, None], 0), w, dy.masked_fill(bad[:, None], 0), ids, "silu", from_ is not None)
        dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), from_, groups)
        _close(dx, want.dx, want.tdx, "dx")
        _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("m,n,k,g", [(2048, 1024, 512, 3), (4096, 2048, 136, 1), (1500, 777, 250, 2)])
def test_large_tiles(htl, m, n, k, g):
    ids = _ids(np.random.default_rng(m), m, g, "dropped" if g > 1 else "one")
    x, w, dy = _data(m, n, k, g, torch.bfloat16)
    want = Want(x, w, dy, ids, "silu", False)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g)
    y, _ = htl.gated_mm(x.cuda(), w.cuda(), groups)
    _close(y, want.y, want.ty, "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), None, groups)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_types(htl, dtype):
    m, n, k = 90, 48, 56
    x, w, dy = _data(m, n, k, 1, dtype)
    ids = np.zeros(m, dtype=np.int32)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    want = Want(x, w, dy, ids, "silu", False, out=other, dx=other)
    wide, wide_d = torch.full((m, k + 9), float("nan"), dtype=dtype), torch.full((m, n + 3), float("nan"), dtype=dtype)
    wide[:, 1:k + 1], wide_d[:, 2:n + 2] = x, dy
    xs, ds = wide.cuda()[:, 1:k + 1], wide_d.cuda()[:, 2:n + 2]
    y, _ = htl.gated_mm(xs, w[0].cuda(), out_dtype=other)
    assert y.dtype == other
    _close(y, want.y, want.ty, "y")
    dx, dw = htl.gated_mm_backward(ds, xs, w[0].cuda(), dx_dtype=other)
    assert dx.dtype == other
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")
    only, none = htl.gated_mm_backward(ds, xs, w[0].cuda(), need_dw=False)
    assert none is None and only is not None
    none, only = htl.gated_mm_backward(ds, xs, w[0].cuda(), need_dx=False)
    assert none is None and torch.equal(only, dw)


def test_differences(htl):
    """The gradients against central differences of the fp32 forward."""
    m, n, k, step = 5, 6, 7, 2.0 ** -7
    x, w, dy = _data(m, n, k, 1, torch.float32)
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda())

    def f(x, w):
        return float((htl.gated_mm(x.cuda(), w.cuda())[0].cpu().double() * dy.double()).sum())
    # the third derivative of act(z) u along one coordinate is at most 6 |x|^3 (1 + |u|), the forward off by
    # (k + 16) u of terms that sum to at most 100 here: differences are off by step^2 * 100 + 200 * 32 u / step
    tol = step ** 2 * 100 + 200 * 32 * U / step
    for t, d in ((x, dx.cpu()), (w, dw.cpu())):
        for i in range(0, t.numel(), max(1, t.numel() // 20)):
            a, b = t.clone(), t.clone()
            a.view(-1)[i] += step
            b.view(-1)[i] -= step
            diff = (f(a, w) - f(b, w) if t is x else f(x, a) - f(x, b)) / (2 * step)
            assert abs(diff - float(d.view(-1)[i])) <= tol


def test_steep_gates(htl):
    """Gates far open and far shut, and infinities in a row: only that row and its sums have them."""
    x = torch.tensor([[60.0], [-60.0], [1e4], [-1e4], [float("inf")], [0.5]])
    w = torch.ones(1, 2, 1)
    ids = np.zeros(6, dtype=np.int32)
    dy = torch.ones(6, 1)
    want = Want(x[[0, 1, 2, 3, 5]], w, dy[:5], ids[:5], "silu", False)
    y, _ = htl.gated_mm(x.cuda(), w.cuda())
    _close(y[[0, 1, 2, 3, 5]], want.y, want.ty + 2.0 ** -120, "y")
    assert torch.isinf(y[4]).all()
    dx, _ = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda())
    _close(dx[[0, 1, 2, 3, 5]], want.dx, want.tdx + 2.0 ** -100, "dx")


def test_graph_and_streams(htl):
    """A forward and backward pass captured and replayed with new inputs, and calls on another stream."""
    m, n, k = 300, 64, 80
    x, w, dy = (t.cuda() for t in _data(m, n, k, 1, torch.bfloat16))
    htl.gated_mm_backward(dy, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = htl.gated_mm(x, w, keep=True)
        dx, dw = htl.gated_mm_backward(dy, x, w, kept)
    for seed in range(3):
        nx, nw, nd = _data(m, n, k, 1, torch.bfloat16, seed)
        x.copy_(nx), w.copy_(nw), dy.copy_(nd)
        graph.replay()
        e_y, e_kept = htl.gated_mm(x, w, keep=True)
        e_dx, e_dw = htl.gated_mm_backward(dy, x, w, e_kept)
        torch.cuda.synchronize()
        for a, b in ((y, e_y), (dx, e_dx), (dw, e_dw)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s_y, s_kept = htl.gated_mm(x, w, keep=True)
        s_dx, s_dw = htl.gated_mm_backward(dy, x, w, s_kept)
    side.synchronize()
    for a, b in ((s_y, e_y), (s_dx, e_dx), (s_dw, e_dw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,k,g", [(70000, 256, 128, 26), (66000, 40, 31, 3), (65536, 33, 64, 1), (68000, 72, 200, 5)])
def test_many_rows_of_small_blocks(htl, m, n, k, g):
    """Projections that stay in LDS: every 37th row against its own, and those of no group."""
    ids = _ids(np.random.default_rng(m), m, g, "dropped" if g > 1 else "one")
    x, w, dy = _data(m, n, k, g, torch.bfloat16)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g)
    y, kept = htl.gated_mm(x.cuda(), w.cuda(), groups, act="sigmoid", keep=True)
    some = torch.arange(0, m, 37)
    want = Want(x[some], w, dy[some], ids[some.numpy()], "sigmoid", False)
    _close(y[some], want.y, want.ty, "y")
    _close(kept[some], want.kept, want.tkept, "kept")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), kept, groups, act="sigmoid")
    want = Want(x[some], w, dy[some], ids[some.numpy()], "sigmoid", True)
    _close(dx[some], want.dx, want.tdx, "dx")


def test_wide_graph_and_repeats(htl):
    """Calls in the largest tiles: repeated, captured and replayed, the same to the bit."""
    m, n, k, g = 2100, 1040, 300, 3
    ids = _ids(np.random.default_rng(4), m, g, "dropped")
    x, w, dy = (t.cuda() for t in _data(m, n, k, g, torch.bfloat16))
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g)

    def step():
        y, kept = htl.gated_mm(x, w, groups, keep=True)
        return (y, kept, *htl.gated_mm_backward(dy, x, w, kept, groups), *htl.gated_mm_backward(dy, x, w, None, groups))
    first = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        for a, b in zip((x, w, dy), _data(m, n, k, g, torch.bfloat16, seed)):
            a.copy_(b)
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
        if seed == 0:
            assert all(torch.equal(a, b) for a, b in zip(first, eager))


@pytest.mark.parametrize("m,n,k", [(40, 16, 24), (2048, 1024, 304)])
@pytest.mark.parametrize("keep", [False, True])
def test_broken_plans(htl, m, n, k, keep):
    """A plan whose order names rows that are not there reads and writes nothing outside, and the others are right."""
    x, w, dy = _data(m, n, k, 1, torch.bfloat16)
    order = torch.arange(m, dtype=torch.int32)
    gone = torch.arange(m) % 7 == 3
    bad = order.clone()
    bad[gone] = torch.where(torch.arange(int(gone.sum())) % 2 == 0, -5, m + 9).to(torch.int32)
    plan = htl.RowGroups(torch.zeros(m, dtype=torch.int32).cuda(), bad.cuda(), torch.tensor([0, m], dtype=torch.int32).cuda(), 1)
    ids = np.where(gone.numpy(), -1, 0).astype(np.int32)
    want = Want(x, w, dy, ids, "silu", keep)
    xc, wc, dc = x.cuda(), w.cuda(), dy.cuda()
    y, kept = htl.gated_mm(xc, wc, plan, keep=keep)
    _close(y[~gone], want.y[~gone], want.ty[~gone], "y")
    dx, dw = htl.gated_mm_backward(dc, xc, wc, kept, plan)
    _close(dx[~gone], want.dx[~gone], want.tdx[~gone], "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("m,n,k", [(40, 24, 32), (300, 40, 48), (2100, 1024, 304)])
def test_matrix_at_any_alignment(htl, m, n, k):
    x, w, dy = _data(m, n, k, 1, torch.bfloat16)
    flat = torch.zeros(w.numel() + 1, dtype=torch.bfloat16)
    flat[1:] = w.view(-1)
    loose = flat.cuda()[1:].view(1, 2 * n, k)
    want = Want(x, w, dy, np.zeros(m, dtype=np.int32), "silu", False)
    y, _ = htl.gated_mm(x.cuda(), loose)
    _close(y, want.y, want.ty, "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), loose)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("m,n,k,g,dx_dtype", [(66000, 256, 128, 3, None), (65536, 33, 50, 1, torch.float32),
                                              (70000, 100, 72, 26, None), (65551, 32, 7, 2, None), (65600, 64, 128, 4, None),
                                              (66001, 128, 96, 5, torch.float32), (65536, 250, 128, 1, None)])
def test_gradients_of_small_blocks(htl, m, n, k, g, dx_dtype):
    """Backward passes of many rows through blocks that fit in LDS, from z and u: all of dx and dw, with rows of no group."""
    ids = _ids(np.random.default_rng(m), m, g, "dropped" if g > 1 else "one")
    x, w, dy = _data(m, n, k, g, torch.bfloat16)
    want = Want(x, w, dy, ids, "silu", True, dx=dx_dtype)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g) if g > 1 else None
    none = torch.from_numpy((ids < 0) | (ids >= g))
    x[none], dy[none] = float("nan"), float("inf")
    xc, wc, dc = x.cuda(), w.cuda(), dy.cuda()
    _, kept = htl.gated_mm(xc, wc, groups, keep=True)
    dx, dw = htl.gated_mm_backward(dc, xc, wc, kept, groups, dx_dtype=dx_dtype)
    assert dx.dtype == (dx_dtype or torch.bfloat16)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")
    only, none_ = htl.gated_mm_backward(dc, xc, wc, kept, groups, dx_dtype=dx_dtype, need_dw=False)
    assert none_ is None and torch.equal(only, dx)
    _, only = htl.gated_mm_backward(dc, xc, wc, kept, groups, need_dx=False)
    _close(only, want.dw, want.tdw, "dw alone")


def test_broken_plan_of_small_blocks(htl):
    m, n, k = 65600, 96, 40
    x, w, dy = _data(m, n, k, 1, torch.bfloat16)
    bad = torch.arange(m, dtype=torch.int32)
    gone = torch.arange(m) % 7 == 3
    bad[gone] = torch.where(torch.arange(int(gone.sum())) % 2 == 0, -5, m + 9).to(torch.int32)
    plan = htl.RowGroups(torch.zeros(m, dtype=torch.int32).cuda(), bad.cuda(), torch.tensor([0, m], dtype=torch.int32).cuda(), 1)
    want = Want(x, w, dy, np.where(gone.numpy(), -1, 0).astype(np.int32), "silu", True)
    y, kept = htl.gated_mm(x.cuda(), w.cuda(), plan, keep=True)
    _close(y[~gone], want.y[~gone], want.ty[~gone], "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), kept, plan)
    _close(dx[~gone], want.dx[~gone], want.tdx[~gone], "dx")
    _close(dw, want.dw, want.tdw, "dw")


def _backward_of_some(htl, x, w, dy, some, **kw):
    """dw of one group against the formulas, at `some` of its n outputs (all of x's rows count)."""
    n = w.shape[0] // 2
    rows = torch.cat([some, n + some])
    dx, dw = htl.gated_mm_backward(dy, x, w, **kw)
    want = Want(x.cpu(), w[rows].cpu()[None], dy[:, some].cpu(), np.zeros(x.shape[0], dtype=np.int32), "silu", False)
    _close(dw[0][rows], want.dw[0], want.tdw[0], "dw")
    return dx, dw


def test_rows_of_a_larger_matrix_past_4_gib(htl):
    """x's rows so far apart that they span more than 4 GiB: the same as of rows that lie together."""
    m, n, k = 65_600, 128, 256
    x, w, dy = (t.cuda() for t in _data(m, n, k, 1, torch.bfloat16))
    apart = torch.full((m, 32_768), float("nan"), dtype=torch.bfloat16, device="cuda")
    apart[:, 512:512 + k] = x
    dx, dw = _backward_of_some(htl, x, w[0], dy, torch.arange(n, device="cuda"))
    for got, want in zip(htl.gated_mm_backward(dy, apart[:, 512:512 + k], w[0]), (dx, dw)):
        assert torch.equal(got, want)


def test_slopes_past_4_gib(htl):
    """dz and du that take 4.3 GB together, in one chunk of sums if it went by the matrices alone."""
    m, n, k = 32_760, 32_768, 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(m, k, device="cuda", generator=gen).bfloat16()
    w = (torch.randn(2 * n, k, device="cuda", generator=gen) / 8.0).bfloat16()
    dy = torch.randn(m, n, device="cuda", generator=gen).bfloat16()
    some = torch.cat([torch.arange(0, n, 257, device="cuda"), torch.tensor([n - 1], device="cuda")])
    _backward_of_some(htl, x, w, dy, some, need_dx=False)


# Sizes of the tiles of 256 x 256 (tests/test_launches.py looks at the kernels that these calls take).
WIDE = [(4096, 2048, 264, 3), (3700, 2056, 300, 2), (4096, 2048, 304, 1), (8192, 1024, 256, 20), (7300, 1000, 2050, 5)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,g", WIDE)
def test_wide_tiles(htl, m, n, k, g, keep):
    """The largest tiles over several groups, some of few rows or none, with rows of no group that hold anything."""
    rng = np.random.default_rng(m + k)
    ids = _ids(rng, m, g, "dropped" if g > 1 else "one")
    if g > 3:
        ids[ids == 1] = 2                     # a group of no rows
    x, w, dy = _data(m, n, k, g, torch.bfloat16)
    want = Want(x, w, dy, ids, "silu", keep)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g) if g > 1 else None
    none = torch.from_numpy((ids < 0) | (ids >= g))
    x[none], dy[none] = float("nan"), float("inf")
    xc, wc, dc = x.cuda(), w.cuda(), dy.cuda()
    y, kept = htl.gated_mm(xc, wc, groups, keep=keep)
    _close(y, want.y, want.ty, "y")
    if keep:
        _close(kept, want.kept, want.tkept, "kept")
    dx, dw = htl.gated_mm_backward(dc, xc, wc, kept, groups)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")
    # rows of larger matrices, and results one at a time, are the same to the bit
    apart = torch.full((m, k + 13), float("nan"), dtype=torch.bfloat16, device="cuda")
    apart[:, 5:5 + k] = xc
    d_apart = torch.full((m, n + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    d_apart[:, 1:1 + n] = dc
    a, _ = htl.gated_mm_backward(d_apart[:, 1:1 + n], apart[:, 5:5 + k], wc, kept, groups, need_dw=False)
    _, b = htl.gated_mm_backward(d_apart[:, 1:1 + n], apart[:, 5:5 + k], wc, kept, groups, need_dx=False)
    assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("keep", [False, True])
def test_broken_plan_of_wide_tiles(htl, keep):
    m, n, k, _ = WIDE[2]
    x, w, dy = _data(m, n, k, 1, torch.bfloat16)
    bad = torch.arange(m, dtype=torch.int32).flip(0).contiguous()
    gone = torch.arange(m) % 7 == 3
    there = torch.ones(m, dtype=torch.bool)
    there[bad[gone].long()] = False
    bad[gone] = torch.where(torch.arange(int(gone.sum())) % 2 == 0, -5, m + 9).to(torch.int32)
    plan = htl.RowGroups(torch.zeros(m, dtype=torch.int32).cuda(), bad.cuda(), torch.tensor([0, m], dtype=torch.int32).cuda(), 1)
    want = Want(x, w, dy, np.where(there.numpy(), 0, -1).astype(np.int32), "silu", keep)
    y, kept = htl.gated_mm(x.cuda(), w.cuda(), plan, keep=keep)
    _close(y[there.cuda()], want.y[there], want.ty[there], "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), kept, plan)
    _close(dx[there.cuda()], want.dx[there], want.tdx[there], "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,g", [(68000, 72, 200, 5), (66000, 300, 64, 3), (65536, 520, 24, 1), (60000, 100, 264, 2)])
def test_all_of_many_rows(htl, m, n, k, g, keep):
    """Many rows through small blocks whose backward pass does not fit in LDS, or whose z and u are not kept: all results."""
    ids = _ids(np.random.default_rng(m + n), m, g, "dropped" if g > 1 else "one")
    x, w, dy = _data(m, n, k, g, torch.bfloat16)
    want = Want(x, w, dy, ids, "sigmoid", keep)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g) if g > 1 else None
    y, kept = htl.gated_mm(x.cuda(), w.cuda(), groups, act="sigmoid", keep=keep)
    _close(y, want.y, want.ty, "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), kept, groups, act="sigmoid")
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_group_has_most_rows(htl, dtype):
    """Eight rows a group on average, 300 of them in one group and none in some."""
    m, n, k, g = 512, 72, 136, 64
    ids = (np.arange(m) * 7 % g).astype(np.int32)
    ids[100:400] = 5
    ids[ids % 9 == 8] = 3
    x, w, dy = _data(m, n, k, g, dtype)
    want = Want(x, w, dy, ids, "silu", False)
    groups = htl.group_rows(torch.from_numpy(ids).cuda(), g)
    y, _ = htl.gated_mm(x.cuda(), w.cuda(), groups)
    _close(y, want.y, want.ty, "y")
    dx, dw = htl.gated_mm_backward(dy.cuda(), x.cuda(), w.cuda(), None, groups)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")
