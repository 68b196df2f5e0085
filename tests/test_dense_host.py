"""Host-side checks of the dense operators: what they refuse, before any device call."""
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


def _norm(L, m=4, dim=8, ldx=8, g=1, ids=None, xd=0, yd=0, kind=0, eps=1e-6, x=P, y=P, w=P, codes=None, scales=None,
          fmt=0, x_scales=None, x_fmt=0):
    return L.norm_rows(x, xd, ldx, x_scales, x_fmt, m, dim, w, None, ids, g, kind, eps, y, yd, codes, scales, fmt, None)


def _norm_back(L, m=4, dim=8, ld=8, g=1, order=None, offsets=None, dy=P, dw=P, ws=P, nb=None, kind=0, xd=0):
    nb = L.norm_back_workspace_bytes(m, g, dim) if nb is None else nb
    return L.norm_rows_backward(dy, 0, ld, P, xd, ld, None, 0, None, 0, m, dim, P, order, offsets, g, kind, 1e-6, P,
                                dw, None, ws, nb, None)


def _gate(L, m=4, dim=8, ld=8, g=1, act=0, kind=0, zc=None, uc=None, ids=None, z=P):
    return L.norm_gate(P, 0, ld, z, ld, P, ld, 0, m, dim, P, None, ids, g, kind, 1e-6, act, 1.0, P, zc, zc, uc, uc, 0,
                       None)


def _gate_back(L, m=4, dim=8, ld=8, g=1, act=0, zs=None, us=None, offsets=None, ws=P, nb=None):
    nb = L.norm_back_workspace_bytes(m, g, dim) if nb is None else nb
    return L.norm_gate_backward(P, 0, ld, P, ld, zs, P, ld, us, 0, 0, m, dim, P, None, None, offsets, g, 0, 1e-6, act,
                                1.0, P, P, P, None, ws, nb, None)


def _mm(L, m=4, n=8, k=8, ldx=8, g=1, order=None, offsets=None, dtype=0, yd=0, x=P, w=P, y=P):
    return L.grouped_mm(x, ldx, w, dtype, m, n, k, order, offsets, g, y, yd, None)


def _mm_back(L, m=4, n=8, k=8, ld=8, g=1, order=None, offsets=None, dx=P, dw=P, ws=P, nb=None, dy=P, w=P):
    nb = L.grouped_mm_backward_workspace_bytes(m, g, n, k) if nb is None else nb
    return L.grouped_mm_backward(dy, ld, P, ld, w, 1, m, n, k, order, offsets, g, dx, 1, dw, ws, nb, None)


def test_row_groups_refuses(L):
    nb = L.row_groups_workspace_bytes(100, 4)
    assert nb > 0 and nb % 256 == 0
    assert L.row_groups_workspace_bytes(-1, 4) == 0 and L.row_groups_workspace_bytes(100, 0) == 0
    assert L.row_groups_workspace_bytes(100, 4096) == 0 and L.row_groups_workspace_bytes(1 << 31, 4) == 0
    for m, g, ids, order, off, ws, n in ((-1, 4, P, P, P, P, nb), (1 << 31, 4, P, P, P, P, nb), (100, 0, P, P, P, P, nb),
                                         (100, 4096, P, P, P, P, nb), (100, 4, None, P, P, P, nb),
                                         (100, 4, P, None, P, P, nb), (100, 4, P, P, None, P, nb),
                                         (100, 4, ODD, P, P, P, nb), (100, 4, P, P, P, ODD, nb),
                                         (100, 4, P, P, P, None, nb), (100, 4, P, P, P, P, nb - 1)):
        assert L.row_groups(ids, m, g, order, off, ws, n, None) == INVALID
    assert b"row_groups" in L.htl_last_error()


def test_rows8_refuses(L):
    for m, dim, ld, fmt, dt, x in ((-1, 8, 8, 0, 0, P), (4, 0, 8, 0, 0, P), (4, 65537, 65537, 0, 0, P),
                                   (4, 8, 7, 0, 0, P), (4, 8, 8, 2, 0, P), (4, 8, 8, 0, 2, P), (4, 8, 8, 0, 0, None),
                                   (4, 8, 8, 0, 0, ODD)):
        assert L.rows8_save(x, dt, ld, m, dim, fmt, P, P, None) == INVALID
    for m, dim, fmt, dt, y in ((-1, 8, 0, 0, P), (4, 0, 0, 0, P), (4, 8, -1, 0, P), (4, 8, 0, 7, P), (4, 8, 0, 0, None)):
        assert L.rows8_load(P, P, fmt, m, dim, y, dt, None) == INVALID
    assert L.rows8_save(None, 0, 8, 0, 8, 0, None, None, None) == 0      # no rows: nothing to do


def test_norms_refuse(L):
    for kw in (dict(m=-1), dict(m=1 << 31), dict(dim=0, ldx=0), dict(dim=16385, ldx=16385), dict(ldx=7), dict(g=0),
               dict(g=4096, ids=P), dict(g=2), dict(xd=2), dict(yd=5), dict(kind=2), dict(eps=-1.0), dict(x=None),
               dict(y=None), dict(w=None), dict(x=ODD), dict(codes=P), dict(scales=P), dict(fmt=3), dict(x_fmt=9),
               dict(codes=P, scales=P, x_scales=P), dict(eps=float("nan"))):
        assert _norm(L, **kw) == INVALID, kw
    assert b"norm_rows" in L.htl_last_error()
    for kw in (dict(m=-1), dict(dim=16385, ld=16385), dict(ld=7), dict(g=3), dict(order=P), dict(dy=None),
               dict(dw=None), dict(ws=None), dict(ws=ODD), dict(nb=16), dict(kind=-1), dict(xd=9), dict(dy=ODD)):
        assert _norm_back(L, **kw) == INVALID, kw
    for kw in (dict(m=-1), dict(dim=0, ld=0), dict(ld=7), dict(g=2), dict(act=3), dict(kind=5), dict(zc=P), dict(uc=P),
               dict(z=None), dict(z=ODD)):
        assert _gate(L, **kw) == INVALID, kw
    for kw in (dict(m=-1), dict(ld=7), dict(g=2), dict(act=-1), dict(zs=P), dict(us=P), dict(ws=None), dict(nb=0)):
        assert _gate_back(L, **kw) == INVALID, kw
    assert L.norm_back_workspace_bytes(4, 1, 0) == 0 and L.norm_back_workspace_bytes(4, 0, 8) == 0
    assert _norm(L, m=0, x=None, y=None) == 0


def test_products_refuse(L):
    for kw in (dict(m=-1), dict(m=1 << 31), dict(n=0), dict(k=0, ldx=0), dict(n=65537), dict(ldx=7), dict(g=0),
               dict(g=2), dict(order=P), dict(dtype=2), dict(yd=2), dict(x=None), dict(w=None), dict(y=None),
               dict(x=ODD), dict(offsets=ODD, g=2)):
        assert _mm(L, **kw) == INVALID, kw
    assert b"grouped_mm" in L.htl_last_error()
    for kw in (dict(m=-1), dict(n=65537), dict(ld=7), dict(g=2), dict(dy=None), dict(w=None), dict(ws=None),
               dict(ws=ODD), dict(nb=1)):
        assert _mm_back(L, **kw) == INVALID, kw
    assert L.grouped_mm_backward_workspace_bytes(-1, 1, 8, 8) == 0
    assert _mm(L, m=0, x=None, y=None) == 0


def test_binding_refuses():
    import hash_table_lookup_amd as htl
    x = torch.zeros(4, 8)
    w = torch.ones(1, 8)
    with pytest.raises(ValueError, match="GPU"):
        htl.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    for f in (lambda: htl.save_rows8(x, "i8"), lambda: htl.norm_rows(x, w), lambda: htl.norm_gate(x, x, x, w),
              lambda: htl.norm_rows_backward(x, x, w), lambda: htl.norm_gate_backward(x, x, x, w),
              lambda: htl.grouped_mm(x, w), lambda: htl.grouped_mm_backward(x, x, w)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(ValueError, match="kind"):
        htl.norm_rows(x, w, kind="batch")
    with pytest.raises(ValueError, match="act"):
        htl.norm_gate(x, x, x, w, act="tanh")
    r = htl.Rows8(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8), "int4", torch.float32)
    with pytest.raises(ValueError, match="format"):
        htl.load_rows8(r)
    with pytest.raises(ValueError, match="8 bits"):
        htl.norm_rows(r._replace(fmt="i8"), w, save="i8")
    with pytest.raises(ValueError, match="both"):
        htl.norm_gate_backward(x, r._replace(fmt="i8"), x, w)


class _OnGpu:
    """What the checks of a plan ask of a tensor."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, n, dtype=torch.int32):
        self.n, self.dtype = n, dtype

    def numel(self):
        return self.n

    def contiguous(self):
        return self


def test_plans_are_checked():
    """A plan's tensors are read by address: their type, size and place are checked before."""
    import hash_table_lookup_amd as htl
    from hash_table_lookup_amd import dense
    good = htl.RowGroups(_OnGpu(6), _OnGpu(6), _OnGpu(4), 3)
    assert dense._ids(good, 6) is good.ids and dense._plan(good, 6) == (good.order, good.offsets)
    assert dense._plan(good._replace(order=None), 6) == (None, good.offsets)
    assert dense._ids(None, 6) is None and dense._plan(None, 6) == (None, None)
    for bad in (_OnGpu(6, torch.int64), _OnGpu(5), _OnGpu(7), torch.zeros(6, dtype=torch.int32)):
        with pytest.raises(ValueError, match="groups.ids must be a GPU tensor of 6 int32"):
            dense._ids(good._replace(ids=bad), 6)
        with pytest.raises(ValueError, match="groups.order must be a GPU tensor of 6 int32"):
            dense._plan(good._replace(order=bad), 6)
    for bad in (_OnGpu(4, torch.int64), _OnGpu(3), _OnGpu(5), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="groups.offsets must be a GPU tensor of 4 int32"):
            dense._plan(good._replace(offsets=bad), 6)
    with pytest.raises(ValueError, match="offsets"):
        dense._plan(good._replace(n_groups=5), 6)


class _Shaped(_OnGpu):
    def __init__(self, shape, dtype):
        super().__init__(0, dtype)
        self.shape = shape

    def stride(self):
        return self.shape[-1], 1

    def dim(self):
        return len(self.shape)


def test_sizes_past_32_bits_are_refused():
    """Row lengths and group counts go to the library as int32: none may be cut to its low bits on the way."""
    import hash_table_lookup_amd as htl
    from hash_table_lookup_amd import dense
    big = 2**32 + 8
    with pytest.raises(ValueError, match="n_groups"):
        htl.group_rows(torch.zeros(4, dtype=torch.int32), big)
    assert dense._rows(_Shaped((2, 8), torch.float32), "x")[1] == 8
    with pytest.raises(ValueError, match="rows of at most"):
        dense._rows(_Shaped((2, big), torch.float32), "x")
    with pytest.raises(ValueError, match="at most .* outputs"):
        dense._weights(_Shaped((1, big, 1), torch.float32), None, torch.float32)
    kept = htl.Rows8(_Shaped((2, big), torch.uint8), _Shaped((2, (big + 31) // 32), torch.uint8), "i8", torch.float32)
    with pytest.raises(ValueError, match="rows of at most"):
        dense._check_rows8(kept, "kept")


def test_workspaces_of_sums_go_by_rows(L):
    """Partial sums take room for the chunks of groups that have several, not for every group."""
    mm, norm = L.grouped_mm_backward_workspace_bytes, L.norm_back_workspace_bytes
    # 16 experts, 2,048 -> 4,096: at most four chunks of split groups (a group's matrix is 33.6 MB)
    assert mm(16384, 16, 4096, 2048) <= 4 * 4096 * 2048 * 4 + 256
    assert mm(16384, 256, 1024, 1024) <= 256 * 1024 * 1024 * 4 // 4
    for m, n, k in ((16384, 1024, 1024), (100001, 513, 777), (1 << 20, 128, 256), (5000, 64, 64)):
        assert mm(m, 1, n, k) <= mm(m, 300, n, k) <= mm(m, 4095, n, k) <= 2 * mm(m, 1, n, k)
    for m, dim in ((8192, 16384), (1 << 20, 128), (100, 4096)):
        assert norm(m, 4095, dim) <= 2 * norm(m, 1, dim) and norm(m, 4095, dim) % 256 == 0
    assert mm(10, 4095, 512, 512) == norm(10, 4095, 128) == 256
