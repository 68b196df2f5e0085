"""Losses over a vocabulary against plain 64-bit forms.

Tolerances are derived, not fitted.  With u = 2^-24, a score of k products is
off by at most e = (k + 6) u times the sum of their magnitudes / T (scaling and
the change to base 2 among it).  An exponential of it is off by e and by the
rounding of its argument, 4 u of the largest score, relative; a sum of V such
by (V + 64) u more.  So lse is off by r = max e + 8 u max |s| + (V + 64) u + 2 u
|lse|, the shares q = exp(s - lse) by 2 r relative (r small), d = (q - p) g by
|g| (2 r q + 8 u p (1 + the teacher's logits' size)) + 2 u |d|, and where d is
kept in bf16 by half a step, 2^-8 |d|; products with d add theirs as above.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _close(got, want, tol, what):
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs()[bad].max()), float(tol[bad].min()))


class Want:
    """Losses and gradients in fp64 with their bounds: items [m, t] and the log shares [m, t] of each row."""

    def __init__(self, x, w, items, logp, heat, dloss=None, size=0.0, dx=None):
        m, v, dt = x.shape[0], w.shape[0], x.dtype
        k, half, dh = x.shape[1], HALF[dt], HALF[dx or dt]
        here = (items >= 0) & (items < v) & (logp > -math.inf)
        on = here.any(1)
        p = torch.where(here, torch.exp(logp), 0.0)
        x, w = x.double(), w.double()
        x = torch.where(on[:, None], x, 0.0)
        s, e = x @ w.t() / heat, (k + 6) * U * (x.abs() @ w.abs().t()) / heat
        lse = torch.logsumexp(s, 1)
        r = e.amax(1) + (8 * s.abs().amax(1) + v + 64 + 2 * lse.abs()) * U
        at = items.clamp(0, v - 1).long()
        terms = torch.where(here, p * (torch.where(here, logp, 0.0) - s.gather(1, at) + lse[:, None]), 0.0)
        each = e.gather(1, at) + r[:, None] + 8 * U * (size + logp.abs().nan_to_num(posinf=0.0) + s.gather(1, at).abs() + lse.abs()[:, None])
        rel = (items.shape[1] + 8 + 8 * size) * U
        self.loss = torch.where(on, terms.sum(1), 0.0)
        self.tloss = torch.where(on, (p * each).sum(1) + rel * terms.abs().sum(1), 0.0)
        self.lse, self.tlse = torch.where(on, lse, 0.0), torch.where(on, r, 0.0)
        if dloss is None:
            return
        g = torch.where(on, dloss.double() / heat, 0.0)[:, None]
        q = torch.exp(s - lse[:, None])
        share = torch.zeros_like(q).scatter_add_(1, at, p)
        d = (q - share) * g
        ed = g.abs() * (2 * r[:, None] * q + (16 + 8 * size) * U * share) + 2 * U * d.abs()
        ed = ed + half * (d.abs() + ed)
        self.dx = d @ w
        t = ed @ w.abs() + (v + 2) * U * ((d.abs() + ed) @ w.abs())
        self.tdx = t + dh * (self.dx.abs() + t)
        self.dw = d.t() @ x
        t = ed.t() @ x.abs() + (m + 2) * U * ((d.abs() + ed).t() @ x.abs())
        self.tdw = t + half * (self.dw.abs() + t)


def _data(m, v, k, dtype, seed=0, spread=2.0):
    gen = torch.Generator().manual_seed(1000 * m + 10 * v + k + seed)
    x = torch.randn(m, k, generator=gen).to(dtype)
    w = (torch.randn(v, k, generator=gen) * (spread / k ** 0.5)).to(dtype)
    targets = torch.randint(0, v, (m,), generator=gen)
    targets[torch.rand(m, generator=gen) < 0.15] = -100
    targets[torch.rand(m, generator=gen) < 0.05] = v
    dloss = (torch.rand(m, generator=gen) - 0.3) / max(m, 1)
    return x, w, targets, dloss


def _teacher(m, v, t, seed=0):
    gen = torch.Generator().manual_seed(77 * m + v + t + seed)
    items = torch.stack([torch.randperm(v, generator=gen)[:t] for _ in range(m)]) if m else torch.zeros(0, t, dtype=torch.int64)
    logits = torch.randn(m, t, generator=gen) * 3.0
    items[torch.rand(m, t, generator=gen) < 0.1] = -1
    logits[torch.rand(m, t, generator=gen) < 0.05] = -math.inf
    if m > 3:
        items[1] = -1                           # no entry at all
        logits[2] = -math.inf                   # entries of no share
        items[3, :] = items[3, 0].clamp(min=0)  # one item, listed over and over
    return items, logits


def _log_shares(items, logits, v, heat):
    a = torch.where((items >= 0) & (items < v), logits.double() / heat, -math.inf)
    top = a.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    return a - top - torch.exp(a - top).sum(1, keepdim=True).log()


SIZES = [(0, 5, 8), (1, 1, 1), (1, 70, 16), (3, 2, 7), (7, 1000, 40), (48, 129, 64), (49, 257, 24), (130, 640, 72),
         (200, 1023, 31), (257, 2049, 130), (600, 300, 256), (64, 20000, 96)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,v,k", SIZES)
def test_softmax(htl, m, v, k, dtype):
    heat = (1.0, 0.5, 2.0)[(m + v) % 3]
    x, w, targets, dloss = _data(m, v, k, dtype)
    if m % 2:
        targets = targets.to(torch.int32)
    items = targets.long()[:, None]
    want = Want(x, w, items, torch.zeros(m, 1).double(), heat, dloss)
    xc, wc, tc = x.cuda(), w.cuda(), targets.cuda()
    loss, lse = htl.softmax_loss(xc, wc, tc, temperature=heat)
    _close(lse, want.lse, want.tlse, "lse")
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), xc, wc, tc, lse, temperature=heat)
    assert dx.dtype == dtype and dw.dtype == dtype
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,v,k,t", [(0, 5, 8, 2), (1, 1, 1, 1), (5, 33, 16, 33), (40, 500, 24, 7), (60, 700, 40, 64),
                                     (130, 640, 72, 65), (257, 2049, 130, 100), (20, 3000, 64, 1024)])
def test_distill(htl, m, v, k, t, dtype):
    heat = (1.0, 2.0)[(m + v) % 2]
    x, w, _, dloss = _data(m, v, k, dtype)
    items, logits = _teacher(m, v, t)
    if m % 2:
        items = items.to(torch.int32)
    if v % 2:
        logits = logits.bfloat16()
    size = float(logits.float()[logits > -math.inf].abs().max()) / heat if (logits > -math.inf).any() else 0.0
    want = Want(x, w, items.long(), _log_shares(items, logits, v, heat), heat, dloss, size)
    xc, wc, ic, lc = x.cuda(), w.cuda(), items.cuda(), logits.cuda()
    loss, kept = htl.distill_loss(xc, wc, ic, lc, temperature=heat)
    _close(kept[0], want.lse, want.tlse, "lse")
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.distill_loss_backward(dloss.cuda(), xc, wc, ic, lc, kept, temperature=heat)
    assert dx.dtype == dtype and dw.dtype == dtype
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("m,v,k", [(1100, 20000, 256), (3000, 5000, 264), (1030, 7001, 130)])
def test_large_tiles(htl, m, v, k):
    x, w, targets, dloss = _data(m, v, k, torch.bfloat16)
    want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), 1.0, dloss)
    loss, lse = htl.softmax_loss(x.cuda(), w.cuda(), targets.cuda())
    _close(lse, want.lse, want.tlse, "lse")
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_a_target(htl, dtype):
    """They may hold anything: nothing of it reaches a result."""
    m, v, k = 150, 300, 40
    x, w, targets, dloss = _data(m, v, k, dtype)
    off = (targets < 0) | (targets >= v)
    want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), 1.0, dloss)
    x[off], dloss[off] = float("nan"), float("inf")
    loss, lse = htl.softmax_loss(x.cuda(), w.cuda(), targets.cuda())
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")
    items = torch.where(off, -1, targets)[:, None].repeat(1, 2)
    logits = torch.full((m, 2), float("nan"))
    logits[~off] = 0.5
    loss, kept = htl.distill_loss(x.cuda(), w.cuda(), items.cuda(), logits.cuda())
    # one item listed twice with a half each: the loss is less by log 2, off by 64 u for the halves' logarithms
    _close(loss, torch.where(off, 0.0, want.loss - math.log(2.0)), want.tloss + 64 * U, "loss of halves")
    dx2, dw2 = htl.distill_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), items.cuda(), logits.cuda(), kept)
    _close(dx2, want.dx, want.tdx, "dx")
    _close(dw2, want.dw, want.tdw, "dw")


def test_no_row_has_a_target(htl):
    x, w, targets, dloss = _data(30, 100, 24, torch.bfloat16)
    targets[:] = -100
    loss, lse = htl.softmax_loss(x.cuda(), w.cuda(), targets.cuda())
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    for t in (loss, lse, dx, dw):
        assert not t.any()


def test_nan_stays_in_its_row(htl):
    m, v, k = 70, 200, 32
    x, w, targets, dloss = _data(m, v, k, torch.float32)
    targets[:] = 3
    want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), 1.0, dloss)
    x[11, 5] = float("nan")
    loss, lse = htl.softmax_loss(x.cuda(), w.cuda(), targets.cuda())
    rest = torch.arange(m) != 11
    assert torch.isnan(loss[11]) and torch.isnan(lse[11])
    _close(loss[rest], want.loss[rest], want.tloss[rest], "loss")
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    assert torch.isnan(dx[11]).all() and torch.isnan(dw).all()
    _close(dx[rest], want.dx[rest], want.tdx[rest], "dx")


def test_scores_of_any_size(htl):
    """Scores in the thousands, one far above the others, and a temperature near zero: nothing overflows."""
    m, v, k = 40, 500, 16
    x, w, targets, dloss = _data(m, v, k, torch.float32, spread=400.0)
    for heat in (1.0, 0.01):
        want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), heat, dloss)
        loss, lse = htl.softmax_loss(x.cuda(), w.cuda(), targets.cuda(), temperature=heat)
        assert torch.isfinite(loss).all()
        _close(lse, want.lse, want.tlse, "lse")
        _close(loss, want.loss, want.tloss, "loss")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_types(htl, dtype):
    m, v, k = 90, 333, 56
    x, w, targets, dloss = _data(m, v, k, dtype)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), 1.0, dloss, dx=other)
    for pad, first in ((9, 1), (8, 0)):
        wide, wide_w = torch.full((m, k + pad), float("nan"), dtype=dtype), torch.full((v, k + pad), float("nan"), dtype=dtype)
        wide[:, first:k + first], wide_w[:, first:k + first] = x, w
        xs, ws = wide.cuda()[:, first:k + first], wide_w.cuda()[:, first:k + first]
        loss, lse = htl.softmax_loss(xs, ws, targets.cuda())
        _close(loss, want.loss, want.tloss, "loss")
        dx, dw = htl.softmax_loss_backward(dloss.cuda(), xs, ws, targets.cuda(), lse, dx_dtype=other)
        assert dx.dtype == other
        _close(dx, want.dx, want.tdx, "dx")
        _close(dw, want.dw, want.tdw, "dw")
    a, none = htl.softmax_loss_backward(dloss.cuda(), xs, ws, targets.cuda(), lse, dx_dtype=other, need_dw=False)
    assert none is None and torch.equal(a, dx)
    none, b = htl.softmax_loss_backward(dloss.cuda(), xs, ws, targets.cuda(), lse, need_dx=False)
    assert none is None and torch.equal(b, dw)


def test_teacher_with_one_item_is_cross_entropy(htl):
    m, v, k = 120, 700, 64
    x, w, targets, dloss = _data(m, v, k, torch.float32)
    xc, wc, tc, dc = x.cuda(), w.cuda(), targets.cuda(), dloss.cuda()
    want = Want(x, w, targets[:, None], torch.zeros(m, 1).double(), 1.0, dloss)
    loss, kept = htl.distill_loss(xc, wc, tc[:, None], torch.full((m, 1), 3.0, device="cuda"))
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.distill_loss_backward(dc, xc, wc, tc[:, None], torch.full((m, 1), 3.0, device="cuda"), kept)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


def test_differences(htl):
    """The gradients against central differences of the losses."""
    m, v, k, step = 6, 50, 9, 2.0 ** -6
    x, w, targets, _ = _data(m, v, k, torch.float32)
    items, logits = _teacher(m, v, 5)
    ones = torch.ones(m).cuda()
    heads = (lambda a, b: htl.softmax_loss(a.cuda(), b.cuda(), targets.cuda()),
             lambda a, b: htl.distill_loss(a.cuda(), b.cuda(), items.cuda(), logits.cuda()))
    backs = (lambda kept: htl.softmax_loss_backward(ones, x.cuda(), w.cuda(), targets.cuda(), kept),
             lambda kept: htl.distill_loss_backward(ones, x.cuda(), w.cuda(), items.cuda(), logits.cuda(), kept))
    # along one coordinate a loss has a third derivative of at most |x|^3 (or |w|^3) < 64 a row, m rows, and is off by
    # 200 u: differences are off by step^2 / 6 * 64 m + 200 m u / step
    tol = step ** 2 / 6 * 64 * m + 200 * m * U / step
    for head, back in zip(heads, backs):
        dx, dw = (t.cpu() for t in back(head(x, w)[1]))
        for t, d in ((x, dx), (w, dw)):
            for i in range(0, t.numel(), max(1, t.numel() // 25)):
                a, b = t.clone(), t.clone()
                a.view(-1)[i] += step
                b.view(-1)[i] -= step
                up, down = (head(a, w)[0], head(b, w)[0]) if t is x else (head(x, a)[0], head(x, b)[0])
                diff = float((up.cpu().double() - down.cpu().double()).sum()) / (2 * step)
                assert abs(diff - float(d.view(-1)[i])) <= tol


def test_repeats_are_equal(htl):
    x, w, targets, dloss = (t.cuda() for t in _data(700, 3000, 136, torch.bfloat16))
    first = None
    for _ in range(3):
        loss, lse = htl.softmax_loss(x, w, targets)
        got = (loss, lse, *htl.softmax_loss_backward(dloss, x, w, targets, lse))
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_graph_and_streams(htl):
    """Both losses' steps captured and replayed with new inputs, beside eager calls, and on another stream."""
    m, v, k, t = 200, 900, 72, 6
    x, w, targets, dloss = (a.cuda() for a in _data(m, v, k, torch.bfloat16))
    items, logits = (a.cuda() for a in _teacher(m, v, t))

    def step():
        loss, lse = htl.softmax_loss(x, w, targets)
        l2, kept = htl.distill_loss(x, w, items, logits)
        return (loss, lse, *htl.softmax_loss_backward(dloss, x, w, targets, lse), l2,
                *htl.distill_loss_backward(dloss, x, w, items, logits, kept))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        for a, b in zip((x, w, targets, dloss), _data(m, v, k, torch.bfloat16, seed)):
            a.copy_(b)
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_block_and_head(htl):
    """Looked-up rows through a gated block and the head, forward and backward, as a model runs them."""
    from_, v, k, n, m = 512, 600, 64, 96, 300
    table = htl.Table(12, k, "f32", init_seed=3)
    rng = np.random.default_rng(5)
    keys = torch.from_numpy(rng.integers(0, from_, m)).cuda()
    x = htl.lookup(table, keys)[0].bfloat16() * 200.0
    gen = torch.Generator().manual_seed(9)
    wg = (torch.randn(2 * n, k, generator=gen) / k ** 0.5).bfloat16()
    wo = (torch.randn(1, k, n, generator=gen) / n ** 0.5).bfloat16()
    w = (torch.randn(v, k, generator=gen) / k ** 0.5).bfloat16()
    targets = torch.randint(0, v, (m,), generator=gen)
    y, kept = htl.gated_mm(x, wg.cuda(), keep=True)
    h = htl.grouped_mm(y, wo.cuda())
    loss, lse = htl.softmax_loss(h, w.cuda(), targets.cuda())
    dloss = torch.full((m,), 1.0 / m, device="cuda")
    dh, dw = htl.softmax_loss_backward(dloss, h, w.cuda(), targets.cuda(), lse)
    dy, dwo = htl.grouped_mm_backward(dh, y, wo.cuda())
    dx, dwg = htl.gated_mm_backward(dy, x, wg.cuda(), kept)
    # autograd's in fp64 on the CPU; each of the chain's seven roundings to bf16 is off by 2^-8 of values of the
    # result's own size, so norms are off by at most 8 * 2^-8
    a = [t.double().requires_grad_() for t in (x.cpu(), wg, wo, w)]
    z = a[0] @ a[1].t()
    hh = (torch.nn.functional.silu(z[:, :n]) * z[:, n:]) @ a[2][0].t()
    want = torch.nn.functional.cross_entropy(hh @ a[3].t(), targets)
    want.backward()
    assert abs(float(loss.double().mean()) - want.item()) <= 8 * 2.0 ** -8 * (1 + want.item())
    for got, p in zip((dx, dwg, dwo, dw), a):
        got = got.cpu().double().reshape(p.grad.shape)
        assert float((got - p.grad).norm()) <= 8 * 2.0 ** -8 * float(p.grad.norm())


def test_wide_graph_and_repeats(htl):
    """Both losses in the largest tiles, dx in parts: repeated, captured and replayed, the same to the bit."""
    m, v, k, t = 1030, 16400, 520, 9
    x, w, targets, dloss = (a.cuda() for a in _data(m, v, k, torch.bfloat16))
    gen = torch.Generator().manual_seed(1)
    items, logits = torch.randint(0, v, (m, t), generator=gen).cuda(), torch.randn(m, t, generator=gen).cuda()

    def step():
        loss, lse = htl.softmax_loss(x, w, targets)
        l2, kept = htl.distill_loss(x, w, items, logits)
        return (loss, lse, *htl.softmax_loss_backward(dloss, x, w, targets, lse), l2,
                *htl.distill_loss_backward(dloss, x, w, items, logits, kept))
    first = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        for a, b in zip((x, w, targets, dloss), _data(m, v, k, torch.bfloat16, seed)):
            a.copy_(b)
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
        if seed == 0:
            assert all(torch.equal(a, b) for a, b in zip(first, eager))


def test_two_streams_at_once(htl):
    """The same calls on two streams, which overlap: each has a workspace of its own."""
    data = [[a.cuda() for a in _data(500, 4000, 136, torch.bfloat16, s)] for s in range(2)]

    def step(x, w, targets, dloss):
        loss, lse = htl.softmax_loss(x, w, targets)
        return (loss, *htl.softmax_loss_backward(dloss, x, w, targets, lse))
    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = []
    for _ in range(4):
        got = []
        for s, d in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(step(*d))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("m", [5, 60, 300])
def test_vocabulary_past_4_gib(htl, m):
    """Matrices of more than 4 GiB: offsets past 32 bits, in each kind of tile; every thousandth item's gradient too."""
    v, k = 1_100_003, 2048
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, device="cuda", generator=gen).bfloat16()
    w = torch.empty(v, k, device="cuda", dtype=torch.bfloat16)
    for a in range(0, v, 100_000):
        w[a:a + 100_000] = (torch.randn(min(100_000, v - a), k, device="cuda", generator=gen) * 0.03).bfloat16()
    targets = torch.randint(0, v, (m,), device="cuda", generator=gen)
    targets[0] = v - 1
    dloss = torch.full((m,), 1.0 / m, device="cuda")
    loss, lse = htl.softmax_loss(x, w, targets)
    dx, dw = htl.softmax_loss_backward(dloss, x, w, targets, lse)
    x8 = x.double()
    s = torch.cat([torch.mm(x8, w[a:a + 50_000].double().t().contiguous()) for a in range(0, v, 50_000)], 1)
    want = torch.logsumexp(s, 1)
    # (terms and bounds as at the top: |x| |w| sums to less than 40 a score, scores are below 12)
    r = (k + 6) * U * 40 + (8 * 12 + v + 64 + 2 * 20) * U
    assert float((lse.double() - want).abs().max()) <= r
    assert float((loss.double() - (want - s.gather(1, targets[:, None])[:, 0])).abs().max()) <= 2 * r
    d = torch.exp(s - want[:, None])
    d[torch.arange(m, device="cuda"), targets] -= 1.0
    d /= m
    some = torch.cat([torch.arange(0, v, 1000, device="cuda"), targets])
    dw8 = torch.mm(d[:, some].t().contiguous(), x8)
    ed = d.abs() * (2 * r + 2.0 ** -8 * 1.1)
    tol = torch.mm(ed[:, some].t().contiguous(), x8.abs()) * 1.01 + 2.0 ** -8 * 1.01 * dw8.abs()
    assert bool(((dw[some].double() - dw8).abs() <= tol).all())
    # dx by norm: every term of it is off by its share of 2^-8, of either sign, and the result by a rounding
    dx8 = sum(torch.mm(d[:, a:a + 50_000].contiguous(), w[a:a + 50_000].double()) for a in range(0, v, 50_000))
    assert float((dx.double() - dx8).norm()) <= 2 * 2.0 ** -8 * float(dx8.norm())


@pytest.mark.parametrize("pad,first", [(9, 1), (8, 8), (8, 1)])
def test_wide_strides(htl, pad, first):
    """Rows of larger matrices, at any alignment, in the largest tiles."""
    m, v, k = 1100, 14500, 512
    x, w, targets, dloss = _data(m, v, k, torch.bfloat16)
    targets[targets >= v] = -1
    wide, wide_w = torch.full((m, k + pad + 1), float("nan")).bfloat16(), torch.full((v, k + pad), float("nan")).bfloat16()
    wide[:, first:k + first], wide_w[:, first % pad:k + first % pad] = x, w
    xs, ws = wide.cuda()[:, first:k + first], wide_w.cuda()[:, first % pad:k + first % pad]
    loss, lse = htl.softmax_loss(xs, ws, targets.cuda())
    dx, dw = htl.softmax_loss_backward(dloss.cuda(), xs, ws, targets.cuda(), lse)
    xc, wc = x.cuda(), w.cuda()
    want, want_lse = htl.softmax_loss(xc, wc, targets.cuda())
    assert torch.equal(loss, want) and torch.equal(lse, want_lse)
    for a, b in zip((dx, dw), htl.softmax_loss_backward(dloss.cuda(), xc, wc, targets.cuda(), lse)):
        assert torch.equal(a, b)
    rows = torch.randint(0, m, (40,), generator=torch.Generator().manual_seed(1))
    some = Want(x[rows], w, targets[rows][:, None], torch.zeros(40, 1).double(), 1.0, dloss[rows])
    _close(loss[rows], some.loss, some.tloss, "loss")
    _close(dx[rows], some.dx, some.tdx, "dx")


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heat", [1.0, 0.5])
def test_logits_of_the_lowest_value(htl, kind, heat):
    # Lists masked with their type's lowest value: all of it, equal shares; some of it, none for those.  A
    # logit's distance from the row's largest is below twice the ordinary logits' size wherever a share is not 0.
    m, v, k, t = 60, 700, 40, 6
    x, w, _, dloss = _data(m, v, k, torch.float32, seed=11)
    gen = torch.Generator().manual_seed(12)
    items = torch.stack([torch.randperm(v, generator=gen)[:t] for _ in range(m)])
    logits = (torch.randn(m, t, generator=gen) * 3.0).to(kind)
    size = 2.0 * float(logits.float().abs().max()) / heat
    low = torch.finfo(kind).min
    logits[:20] = low
    logits[20:40, ::2] = low
    items[5, 3:] = -1
    want = Want(x, w, items, _log_shares(items, logits, v, heat), heat, dloss, size)
    assert (want.loss[:20] != 0).all()
    xc, wc, ic, lc = x.cuda(), w.cuda(), items.cuda(), logits.cuda()
    loss, kept = htl.distill_loss(xc, wc, ic, lc, temperature=heat)
    _close(kept[0], want.lse, want.tlse, "lse")
    _close(loss, want.loss, want.tloss, "loss")
    dx, dw = htl.distill_loss_backward(dloss.cuda(), xc, wc, ic, lc, kept, temperature=heat)
    _close(dx, want.dx, want.tdx, "dx")
    _close(dw, want.dw, want.tdw, "dw")


@pytest.mark.parametrize("m,v,k", [(1024, 65_600, 32_768), (300, 33_000, 65_536)])
def test_rows_past_4_gib_a_piece(htl, m, v, k):
    """Rows so long that a piece of the vocabulary would span 4 GiB: cross entropy, and a teacher's lists with items of
    each piece.  Entries are -1, 0 and 1, and as many 128ths: scores are exact."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    f8 = dict(dtype=torch.float64, device="cuda")
    x = torch.randint(-1, 2, (m, k), device="cuda", generator=gen).bfloat16()
    w = torch.empty(v, k, device="cuda", dtype=torch.bfloat16)
    pieces = [slice(a, min(a + 8192, v)) for a in range(0, v, 8192)]
    for p in pieces:
        w[p] = (torch.randint(-1, 2, (p.stop - p.start, k), device="cuda", generator=gen) / 128.0).bfloat16()
    targets = torch.randint(0, v, (m,), device="cuda", generator=gen)
    targets[:3] = torch.tensor([v - 1, 0, -1], device="cuda")
    dloss = torch.rand(m, device="cuda", generator=gen) / m
    items = torch.stack([targets, (targets * 7 + 11) % v], 1)
    items[2] = -1
    x8 = x.double()
    s = torch.cat([torch.mm(x8, w[p].double().t().contiguous()) for p in pieces], 1)
    on = targets >= 0
    lse = torch.logsumexp(s, 1)
    r = (8 * s.abs().amax(1) + v + 64 + 2 * lse.abs()) * U          # (as at the top, of scores that are exact)
    at = targets.clamp(min=0)[:, None]
    for teach in (False, True):
        share = torch.zeros(m, v, **f8)
        if teach:
            loss, kept = htl.distill_loss(x, w, items, torch.zeros(m, 2, device="cuda"))
            share.scatter_add_(1, items.clamp(min=0), torch.full((m, 2), 0.5, **f8))
            want = lse - 0.5 * (s.gather(1, at)[:, 0] + s.gather(1, items[:, 1:].clamp(min=0))[:, 0]) - math.log(2.0)
            dx, dw = htl.distill_loss_backward(dloss, x, w, items, torch.zeros(m, 2, device="cuda"), kept)
        else:
            loss, kept = htl.softmax_loss(x, w, targets)
            share.scatter_(1, at, 1.0)
            want = lse - s.gather(1, at)[:, 0]
            dx, dw = htl.softmax_loss_backward(dloss, x, w, targets, kept)
        assert bool(((loss.double() - torch.where(on, want, 0.0)).abs() <= 2 * r + 64 * U).all())
        g = torch.where(on, dloss.double(), 0.0)[:, None]
        q = torch.exp(s - lse[:, None])
        d = (q - share) * g
        ed = g * (2 * r[:, None] * q + 16 * U * share) + 2 * U * d.abs()
        ed = ed + HALF[x.dtype] * (d.abs() + ed)
        dx8, tol = torch.zeros(m, k, **f8), torch.zeros(m, k, **f8)
        for p in pieces:
            wp = w[p].double()
            dx8 += torch.mm(d[:, p].contiguous(), wp)
            tol += torch.mm((ed[:, p] + (v + 2) * U * (d[:, p].abs() + ed[:, p])).contiguous(), wp.abs())
            dw8 = torch.mm(d[:, p].t().contiguous(), x8)
            t = torch.mm((ed[:, p] + (m + 2) * U * (d[:, p].abs() + ed[:, p])).t().contiguous(), x8.abs())
            assert bool(((dw[p].double() - dw8).abs() <= t + HALF[x.dtype] * (dw8.abs() + t)).all()), (teach, p)
        assert bool(((dx.double() - dx8).abs() <= tol + HALF[x.dtype] * (dx8.abs() + tol)).all()), teach


# Sizes of the tiles of 256 x 256 (tests/test_launches.py looks at the kernels that these calls take): scores in them
# too from rows of 384 elements on, and several pieces of the vocabulary.
WIDE = [(1100, 14500, 512, 9), (1100, 14500, 130, 65), (1100, 66000, 392, 9), (4500, 60000, 264, 12)]


def pieces(m, v, k):
    """Pieces of the vocabulary in a backward pass of bf16 rows below 1,024 elements: 512 MiB of gradients, 65,536 items."""
    each = min((512 << 20) // (2 * m) // 256 * 256, 65536)
    return -(-v // each)


@pytest.mark.parametrize("m,v,k,t", WIDE)
def test_wide_tiles(htl, m, v, k, t):
    """Both losses in the largest tiles: rows without entries, items listed twice, and items at the ends of pieces."""
    x, w, targets, dloss = _data(m, v, k, torch.bfloat16)
    gen = torch.Generator().manual_seed(t)
    items, logits = torch.randint(0, v, (m, t), generator=gen), torch.randn(m, t, generator=gen) * 3.0
    each = -(-v // pieces(m, v, k)) if pieces(m, v, k) == 1 else min((512 << 20) // (2 * m) // 256 * 256, 65536)
    ends = torch.tensor([0, min(each, v) - 1, min(each, v - 1), v - 1])
    items[:, 0] = ends[torch.arange(m) % 4]
    items[:, 1] = items[:, 0]
    items[torch.rand(m, t, generator=gen) < 0.1] = -1
    logits[torch.rand(m, t, generator=gen) < 0.05] = -math.inf
    items[::50] = -1                            # no entry
    logits[7::50] = -math.inf                   # entries of no share
    targets[:4] = ends
    xc, wc, dc = x.cuda(), w.cuda(), dloss.cuda()
    for heat, ic, lc in ((1.0, targets[:, None], torch.zeros(m, 1)), (2.0, items, logits)):
        size = float(lc[lc > -math.inf].abs().max()) / heat
        # (in 64 bits on the GPU: a reference of this size)
        want = Want(xc, wc, ic.cuda(), _log_shares(ic, lc, v, heat).cuda(), heat, dc, size)
        off = ~((ic >= 0) & (ic < v) & (lc > -math.inf)).any(1).cuda()
        xn, dn = xc.masked_fill(off[:, None], float("nan")), dc.masked_fill(off, float("inf"))
        if ic is items:
            loss, kept = htl.distill_loss(xn, wc, ic.cuda(), lc.cuda(), temperature=heat)
            lse = kept[0]
            dx, dw = htl.distill_loss_backward(dn, xn, wc, ic.cuda(), lc.cuda(), kept, temperature=heat)
        else:
            loss, lse = htl.softmax_loss(xn, wc, targets.cuda(), temperature=heat)
            dx, dw = htl.softmax_loss_backward(dn, xn, wc, targets.cuda(), lse, temperature=heat)
        for got, name in ((lse, "lse"), (loss, "loss"), (dx, "dx"), (dw, "dw")):
            _close(got, getattr(want, name).cpu(), getattr(want, "t" + name).cpu(), (heat, name))


EXACT = [(1, 40, 16), (20, 700, 32), (40, 500, 16), (300, 1500, 32), (1100, 14500, 512)]


def _whole(m, v, k, dtype):
    """Rows and items of whole numbers and 16ths, so few of them not zero that scores are exact in fp32 in any order."""
    gen = torch.Generator().manual_seed(m + v)
    x = torch.randint(-8, 9, (m, k), generator=gen).float()
    w = torch.randint(-8, 9, (v, k), generator=gen).float() / 16.0
    x[:, 16:], w[:, :2] = 0.0, 0.0
    return x.to(dtype), w.to(dtype), torch.randint(0, v, (m,), generator=gen), (torch.rand(m, generator=gen) - 0.3) / m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heat", [1.0, 0.3, 0.07])
@pytest.mark.parametrize("m,v,k", EXACT)
def test_an_item_far_above_the_rest(htl, m, v, k, heat, dtype):
    """Its share is 1 and the others' are 0, in fp32 and in 64 bits: the loss is 0, neither above nor below, and so are all
    gradients, whatever the score.  (The others' scores are below 64, this one's over 400 and not a whole number.)"""
    x, w, _, dloss = _whole(m, v, k, dtype)
    best = v // 3
    w[best] = 0.0
    w[best, :2] = 1.0
    x[:, 0] = 512.0 + 4.0 * (torch.arange(m) % 100)
    x[:, 1] = (torch.arange(m) % 200).float() / 128.0 + 0.0078125
    targets = torch.full((m,), best)
    xc, wc, tc = x.cuda(), w.cuda(), targets.cuda()
    loss, lse = htl.softmax_loss(xc, wc, tc, temperature=heat)
    assert not loss.any(), (float(loss.min()), float(loss.max()))
    for t in htl.softmax_loss_backward(dloss.cuda(), xc, wc, tc, lse, temperature=heat):
        assert not t.any(), float(t.abs().max())
    # a target that is another item: never below 0 either, but the distance
    loss, _ = htl.softmax_loss(xc, wc, (tc + 1) % v, temperature=heat)
    assert v == 1 or float(loss.min()) > 400.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heat", [1.0, 0.3, 0.01])
@pytest.mark.parametrize("m,v,k", EXACT)
def test_gradients_of_large_scores(htl, m, v, k, heat, dtype):
    """Scores up to some thousands, which are exact before they are divided by the temperature (e at the top is 0): losses
    and gradients of both kinds.  Shares and products below fp32's least normal number, 2^-126, may be taken as 0: at most
    14,500 terms, each of a |g| below 128 and an |x| or |w| of at most 8, are off by 2^-126 * 2^14 * 2^7 * 2^3 < 2^-100."""
    x, w, targets, dloss = _whole(m, v, k, dtype)
    items, logits = torch.stack([targets, (targets + 7) % v], 1), torch.zeros(m, 2)
    xc, wc, dc = x.cuda(), w.cuda(), dloss.cuda()
    x8, w8 = xc.double(), wc.double()
    s = torch.mm(x8, w8.t().contiguous()) / heat
    lse = torch.logsumexp(s, 1)
    r = (8 * s.abs().amax(1) + v + 64 + 2 * lse.abs()) * U
    q = torch.exp(s - lse[:, None])
    half, g = HALF[dtype], dc.double()[:, None] / heat
    for ic in (targets[:, None].cuda(), items.cuda()):
        t = ic.shape[1]
        share = torch.zeros_like(q).scatter_add_(1, ic, torch.full(ic.shape, 1.0 / t, dtype=torch.float64, device="cuda"))
        want = lse - s.gather(1, ic).mean(1) - math.log(t)
        if t == 1:
            loss, kept = htl.softmax_loss(xc, wc, ic[:, 0], temperature=heat)
            dx, dw = htl.softmax_loss_backward(dc, xc, wc, ic[:, 0], kept, temperature=heat)
            assert bool((loss >= 0.0).all())
        else:
            loss, kept = htl.distill_loss(xc, wc, ic, logits.cuda(), temperature=heat)
            dx, dw = htl.distill_loss_backward(dc, xc, wc, ic, logits.cuda(), kept, temperature=heat)
        assert bool(((loss.double() - want).abs() <= 3 * r + 64 * U).all()), t
        d = (q - share) * g
        ed = g.abs() * (2 * r[:, None] * q + 16 * U * share) + 2 * U * d.abs()
        ed = ed + half * (d.abs() + ed)
        e = torch.mm(ed + (v + 2) * U * (d.abs() + ed), w8.abs())
        want = torch.mm(d, w8)
        assert bool(((dx.double() - want).abs() <= e + half * (want.abs() + e) + 2.0 ** -100).all()), (t, "dx")
        e = torch.mm((ed + (m + 2) * U * (d.abs() + ed)).t().contiguous(), x8.abs())
        want = torch.mm(d.t().contiguous(), x8)
        assert bool(((dw.double() - want).abs() <= e + half * (want.abs() + e) + 2.0 ** -100).all()), (t, "dw")
