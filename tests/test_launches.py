"""What calls launch: a launch that fails is an error of its call, whichever of them it is, and the sizes at which GPU
tests compare a kernel reach that kernel.

Launches are stood in for by a small library of these tests' own, preloaded into a child process: one that is chosen
fails, the others do nothing, and their kernels' names are kept.  No GPU takes part, and no pointer is followed.
"""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

LAUNCHES = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stddef.h>
#include <string.h>
typedef struct { unsigned x, y, z; } D3;
static int at, chosen = -1, pending;
static struct { const void* f; const char* name; } known[1 << 14];
static int knows;
static char names[1 << 16];
void choose(int n) { at = 0; chosen = n; pending = 0; names[0] = 0; }
int launched(void) { return at; }
const char* launched_names(void) { return names; }
void __hipRegisterFunction(void** module, const void* f, char* device, const char* name, unsigned threads, void* tid,
                           void* bid, D3* block, D3* grid, int* warp) {
    static void (*next)(void**, const void*, char*, const char*, unsigned, void*, void*, D3*, D3*, int*);
    if (!next) *(void**)&next = dlsym(RTLD_NEXT, "__hipRegisterFunction");
    if (knows < 1 << 14 && strstr(name, "N3htl")) {
        known[knows].f = f;
        known[knows++].name = name;
    }
    if (next) next(module, f, device, name, threads, tid, bid, block, grid, warp);
}
int hipLaunchKernel(const void* f, D3 grid, D3 block, void** args, size_t lds, void* stream) {
    for (int i = 0; i < knows; ++i)
        if (known[i].f == f && strlen(names) + strlen(known[i].name) + 2 < sizeof names) strcat(strcat(names, known[i].name), " ");
    (void)grid, (void)block, (void)args, (void)lds, (void)stream;
    if (at++ == chosen) pending = 719;               /* hipErrorLaunchFailure */
    return pending;
}
int hipGetLastError(void) { int e = pending; pending = 0; return e; }
int __hipPushCallConfiguration(D3 grid, D3 block, size_t lds, void* stream) {
    (void)grid, (void)block, (void)lds, (void)stream;
    return 0;
}
int __hipPopCallConfiguration(D3* grid, D3* block, size_t* lds, void** stream) {
    D3 one = {1, 1, 1};
    *grid = one, *block = one, *lds = 0, *stream = 0;
    return 0;
}
"""

COMMON = r"""
import ctypes, sys
import hash_table_lookup_amd as h
L, S = h.lib(), ctypes.CDLL(sys.argv[1])
S.launched_names.restype = ctypes.c_char_p
P = ctypes.c_void_p(0x100000)

def gated(m, n, k, g, dtype, kept, offsets=True):
    o = P if offsets else None
    nb = L.gated_mm_workspace_bytes(m, g, n, k, dtype)
    yield "gated_mm", lambda: L.gated_mm(P, k, P, dtype, m, n, k, o, o, g, 2, P, dtype, kept, P, nb, None)
    bb = L.gated_mm_backward_workspace_bytes(m, g, n, k, dtype)
    yield "gated_mm_backward", lambda: L.gated_mm_backward(P, n, P, k, P, dtype, kept, m, n, k, o, o, g, 2, P, dtype, P, P, bb, None)

def losses(m, v, k, dtype):
    nb, bb = L.softmax_loss_workspace_bytes(m, v, k, dtype), L.softmax_loss_backward_workspace_bytes(m, v, k, dtype)
    db = L.distill_loss_backward_workspace_bytes(m, v, k, 5, dtype)
    yield "softmax_loss", lambda: L.softmax_loss(P, k, P, k, dtype, m, v, k, P, 32, 1.0, P, P, P, nb, None)
    yield "softmax_loss_backward", lambda: L.softmax_loss_backward(P, P, k, P, k, dtype, m, v, k, P, 32, P, 1.0, P, dtype, P, P, bb, None)
    yield "distill_loss", lambda: L.distill_loss(P, k, P, k, dtype, m, v, k, P, 32, P, 0, 5, 5, 1.0, P, P, P, P, nb, None)
    yield "distill_loss_backward", lambda: L.distill_loss_backward(P, P, k, P, k, dtype, m, v, k, P, 32, P, 0, 5, 5, P, P, 1.0, P, dtype, P, P, db, None)
"""

FAILING = COMMON + r"""
sets = []
for dtype in (0, 1):
    for m, n, k, g, offsets in ((1, 8, 16, 1, False), (300, 24, 40, 3, True), (300, 24, 41, 3, True), (8192, 2048, 512, 3, True),
                                (8192, 2048, 500, 1, False), (70000, 256, 128, 26, True), (70000, 40, 128, 1, False)):
        for kept in (None, P):
            sets.append(((m, n, k, g, dtype, bool(kept)), gated(m, n, k, g, dtype, kept, offsets)))
    for m, v, k in ((4, 900, 24), (40, 900, 24), (300, 2000, 41), (1100, 20000, 512), (1100, 70000, 130), (3000, 20000, 128)):
        sets.append(((m, v, k, dtype), losses(m, v, k, dtype)))
for sizes, calls in sets:
    for name, call in calls:
        S.choose(-1)
        assert call() == 0, (name, sizes, L.htl_last_error())
        count = S.launched()
        assert count > 0, (name, sizes)
        for i in range(count):
            S.choose(i)
            assert call() != 0, (name, sizes, "launch %d of %d failed, and the call did not" % (i, count))
print("every launch counts")
"""


CHOOSING = COMMON + r"""
sys.path.insert(0, "tests")
import test_gpu_gated as tg
import test_gpu_scores as ts

def names(call):
    S.choose(-1)
    assert call() == 0, L.htl_last_error()
    return S.launched_names().decode()

def has(what, got, *kernels):
    for k in kernels:
        assert k in got, (what, k, got)

for m, n, k, g in tg.WIDE:
    for kept in (None, P):
        calls = dict(gated(m, n, k, g, 1, kept, g > 1))
        has((m, n, k, g), names(calls["gated_mm"]), "k_gated_wide", *(["k_zero_rest"] if g > 1 else []))
        has((m, n, k, g), names(calls["gated_mm_backward"]), "k_gated_slopes" if kept else "k_gated_back_wide", "k_wide_dx", "k_wide_dw")
for m, v, k, t in ts.WIDE:
    calls = dict(losses(m, v, k, 1))
    tiles = "k_scores_wide" if k >= 384 else "k_scores"
    for name in calls:
        got = names(calls[name])
        has((m, v, k), got, *(["k_wide_dx", "k_wide_dw", tiles] if "backward" in name else [tiles]))
        if name == "distill_loss_backward":
            assert got.count("k_put_items") == ts.pieces(m, v, k), (m, v, k, got)
print("every size as it says")
"""


def _child(tmp_path, code):
    import torch
    if torch.cuda.is_available():
        pytest.skip("for hosts without a GPU")
    src, so = tmp_path / "launches.c", tmp_path / "launches.so"
    src.write_text(LAUNCHES)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(so), str(src), "-ldl"], check=True)
    env = dict(os.environ, LD_PRELOAD=" ".join(filter(None, [str(so), os.environ.get("LD_PRELOAD")])))
    r = subprocess.run([sys.executable, "-c", code, str(so)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return r.stdout


def test_no_launch_fails_unseen(tmp_path):
    assert "every launch counts" in _child(tmp_path, FAILING)


def test_wide_sizes_take_wide_tiles(tmp_path):
    assert "every size as it says" in _child(tmp_path, CHOOSING)
