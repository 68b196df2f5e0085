"""Host-side checks of gated projections and of the losses over a vocabulary: what they refuse, before any device call."""
import ctypes

import pytest
import torch

INVALID = 1
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    import hash_table_lookup_amd as h
    return h.lib()


def _gated(L, m=4, n=8, k=8, ldx=8, g=1, order=None, offsets=None, dtype=1, yd=1, act=2, x=P, w=P, y=P, kept=None, ws=P,
           nb=None):
    nb = max(L.gated_mm_workspace_bytes(m, g, n, k, dtype), 256) if nb is None else nb
    return L.gated_mm(x, ldx, w, dtype, m, n, k, order, offsets, g, act, y, yd, kept, ws, nb, None)


def _gated_back(L, m=4, n=8, k=8, ld=8, g=1, order=None, offsets=None, dtype=1, xd=1, act=2, dy=P, x=P, w=P, kept=None,
                dx=P, dw=P, ws=P, nb=None):
    nb = L.gated_mm_backward_workspace_bytes(m, g, n, k, dtype) if nb is None else nb
    return L.gated_mm_backward(dy, ld, x, ld, w, dtype, kept, m, n, k, order, offsets, g, act, dx, xd, dw, ws, nb, None)


def _loss(L, m=4, v=8, k=8, ldx=8, ldw=8, dtype=1, bits=32, heat=1.0, x=P, w=P, t=P, loss=P, lse=P, ws=P, nb=None):
    nb = L.softmax_loss_workspace_bytes(m, v, k, dtype) if nb is None else nb
    return L.softmax_loss(x, ldx, w, ldw, dtype, m, v, k, t, bits, heat, loss, lse, ws, nb, None)


def _loss_back(L, m=4, v=8, k=8, ldx=8, ldw=8, dtype=1, bits=32, heat=1.0, x=P, w=P, t=P, dloss=P, lse=P, dx=P, xd=1,
               dw=P, ws=P, nb=None):
    nb = L.softmax_loss_backward_workspace_bytes(m, v, k, dtype) if nb is None else nb
    return L.softmax_loss_backward(dloss, x, ldx, w, ldw, dtype, m, v, k, t, bits, lse, heat, dx, xd, dw, ws, nb, None)


def _distill(L, m=4, v=8, k=8, ldx=8, ldw=8, dtype=1, bits=32, heat=1.0, top=3, ldl=3, ld=0, items=P, logits=P, loss=P,
             lse=P, scores=P, ws=P, nb=None):
    nb = L.softmax_loss_workspace_bytes(m, v, k, dtype) if nb is None else nb
    return L.distill_loss(P, ldx, P, ldw, dtype, m, v, k, items, bits, logits, ld, ldl, top, heat, loss, lse, scores, ws,
                          nb, None)


def _distill_back(L, m=4, v=8, k=8, top=3, ldl=3, ld=0, dloss=P, logits=P, lse=P, scores=P, dx=P, xd=1, dw=P, ws=P,
                  nb=None, heat=1.0):
    nb = L.distill_loss_backward_workspace_bytes(m, v, k, top, 1) if nb is None else nb
    return L.distill_loss_backward(dloss, P, k, P, k, 1, m, v, k, P, 32, logits, ld, ldl, top, lse, scores, heat, dx, xd,
                                   dw, ws, nb, None)


def test_gated_refuses(L):
    for kw in (dict(m=-1), dict(m=1 << 31), dict(n=0), dict(n=32769), dict(k=0, ldx=0), dict(k=65537, ldx=65537),
               dict(ldx=7), dict(g=0), dict(g=4096, offsets=P), dict(g=2), dict(order=P), dict(dtype=2), dict(yd=2),
               dict(act=3), dict(act=-1), dict(x=None), dict(w=None), dict(y=None), dict(x=ODD), dict(kept=ODD),
               dict(offsets=ODD, g=2), dict(ws=None), dict(ws=ODD), dict(nb=1)):
        assert _gated(L, **kw) == INVALID, kw
    assert b"gated_mm" in L.htl_last_error()
    for kw in (dict(m=-1), dict(n=32769), dict(ld=7), dict(g=2), dict(dtype=3), dict(xd=4), dict(act=9), dict(dy=None),
               dict(w=None), dict(x=None), dict(kept=ODD), dict(dw=ODD), dict(ws=None), dict(ws=ODD), dict(nb=1)):
        assert _gated_back(L, **kw) == INVALID, kw
    assert _gated(L, m=0, x=None, y=None) == 0
    assert _gated_back(L, dx=None, dw=None) == 0         # nothing wanted: nothing to do
    assert L.gated_mm_workspace_bytes(-1, 1, 8, 8, 1) == 0 and L.gated_mm_backward_workspace_bytes(4, 0, 8, 8, 1) == 0
    # copies of rows that 16-byte pieces do not make up take room; others none
    assert L.gated_mm_workspace_bytes(1000, 1, 64, 65, 1) > L.gated_mm_workspace_bytes(1000, 1, 64, 64, 1) == 256


@pytest.mark.parametrize("m,n,k", [(260_200, 4096, 2048), (261_000, 4096, 2048), (262_080, 4096, 2048), (520_000, 2048, 4096),
                                   (32_760, 32768, 256)])
def test_sums_of_operands_past_4_gib(L, m, n, k):
    """dz and du of so many rows, 64 elements more than 2 n apart, take over 4 GiB, which the sums of dw reach in no less
    than two chunks: room for both chunks' sums beside those rows and a copy of x (as far apart)."""
    assert 2 * n % 512 == 0 and m * (2 * n + 64) * 2 > 1 << 32
    ld_x = k + (0 if k % 512 else 64)
    assert L.gated_mm_backward_workspace_bytes(m, 1, n, k, 1) >= m * (2 * n + 64 + ld_x) * 2 + 2 * 2 * n * k * 4


def test_softmax_refuses(L):
    for kw in (dict(m=-1), dict(m=1 << 31), dict(v=0), dict(v=(1 << 30) + 1), dict(k=0, ldx=0), dict(k=65537, ldx=65537),
               dict(ldx=7), dict(ldw=7), dict(dtype=2), dict(bits=16), dict(heat=0.0), dict(heat=-1.0),
               dict(heat=float("nan")), dict(heat=float("inf")), dict(heat=1e-40), dict(x=None), dict(w=None), dict(t=None),
               dict(t=ODD), dict(x=ODD), dict(loss=None), dict(lse=ODD), dict(ws=None), dict(ws=ODD), dict(nb=1)):
        assert _loss(L, **kw) == INVALID, kw
    assert b"softmax_loss" in L.htl_last_error()
    for kw in (dict(m=-1), dict(v=0), dict(ldw=7), dict(dtype=2), dict(bits=8), dict(heat=0.0), dict(xd=2), dict(dloss=None),
               dict(lse=None), dict(dx=ODD), dict(dw=ODD), dict(ws=None), dict(nb=1)):
        assert _loss_back(L, **kw) == INVALID, kw
    assert _loss(L, m=0, x=None, t=None, loss=None, lse=None) == 0
    assert _loss_back(L, dx=None, dw=None) == 0
    assert L.softmax_loss_workspace_bytes(4, 0, 8, 1) == 0 and L.softmax_loss_backward_workspace_bytes(4, 8, 0, 1) == 0
    # the scores of 8,192 rows with 131,072 items, 4 GiB in fp32, are never held
    assert L.softmax_loss_workspace_bytes(8192, 131072, 2048, 1) < 1 << 28
    assert L.softmax_loss_backward_workspace_bytes(8192, 131072, 2048, 1) < 1 << 30


@pytest.mark.parametrize("k", [36_000, 40_960, 65_536])
def test_pieces_of_long_rows(L, k):
    """Backward passes hold a piece of the vocabulary, less than 4 GiB of its rows (and here less than 1 GiB beside them)."""
    for top in (0, 7):
        nb = (L.distill_loss_backward_workspace_bytes(256, 131_072, k, top, 1) if top else
              L.softmax_loss_backward_workspace_bytes(256, 131_072, k, 1))
        assert 1 << 31 < nb < (1 << 32) + (1 << 28)


def test_distill_refuses(L):
    for kw in (dict(m=-1), dict(v=0), dict(top=0), dict(top=1025, ldl=1025), dict(ldl=2), dict(ld=2), dict(bits=31),
               dict(heat=0.0), dict(items=None), dict(items=ODD), dict(logits=None), dict(logits=ODD), dict(loss=None),
               dict(lse=None), dict(scores=None), dict(scores=ODD), dict(ws=None), dict(nb=1)):
        assert _distill(L, **kw) == INVALID, kw
    assert b"distill_loss" in L.htl_last_error()
    for kw in (dict(m=-1), dict(top=0), dict(ldl=2), dict(dloss=None), dict(logits=None), dict(lse=None), dict(scores=None),
               dict(xd=7), dict(dx=ODD), dict(dw=ODD), dict(ws=ODD), dict(nb=1), dict(heat=1e31)):
        assert _distill_back(L, **kw) == INVALID, kw
    assert _distill(L, m=0, items=None, logits=None, loss=None, lse=None, scores=None) == 0
    assert L.distill_loss_backward_workspace_bytes(4, 8, 8, 0, 1) == 0


def test_binding_refuses():
    import hash_table_lookup_amd as htl
    x, w = torch.zeros(4, 8), torch.ones(16, 8)
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: htl.gated_mm(x, w), lambda: htl.gated_mm_backward(x, x, w),
                 lambda: htl.softmax_loss(x, w, t), lambda: htl.softmax_loss_backward(x[:, 0], x, w, t, x[:, 0]),
                 lambda: htl.distill_loss(x, w, t[:, None], x[:, :1]),
                 lambda: htl.distill_loss_backward(x[:, 0], x, w, t[:, None], x[:, :1], (x[:, 0], x[:, :1]))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="act"):
        htl.gated_mm(x, w, act="relu")
    for heat in (0.0, -1.0, float("nan"), float("inf"), 1e-31):
        with pytest.raises(ValueError, match="temperature"):
            htl.softmax_loss(x, w, t, temperature=heat)
