// Products of few rows, where each matrix row is read once and there are not
// rows enough to share it: matrix rows go straight from global memory to the
// registers of the matrix instructions, many loads ahead, and nothing waits at a
// barrier until the end.
//
// A wave takes 32 matrix rows (16 of each projection where they are pairs) and
// 16 TR rows.  With KS waves for the same rows each has a KS-th of the
// reduction, and the first adds up: enough loads are then under way where the
// matrix has few rows.  The four lanes that share a matrix row read 128
// bytes of it in two loads each; the reduction's elements meet in another order
// than they lie in, the same for both operands.
#pragma once

#include "tile.h"

namespace htl {
namespace {

template <int TR_> struct Few {
    static constexpr int TR = TR_, TC = 2, BR = 16 * TR_;
};
constexpr int kFewThreads = 256;

template <int T, int KS, class C, class End>
__device__ __forceinline__ void few_tiles(const ProdArgs& p, const End& end) {
    constexpr bool kPairs = End::kPairs;
    constexpr int ES = T == kSrcF32 ? 4 : 2, VE = 16 / ES, kStep = 8 * VE, kBatch = 2;
    constexpr int kWaves = kFewThreads / 64, WC = kWaves / KS, kCols = kPairs ? 16 : 32;   // columns a wave
    __shared__ f32x4 s_part[KS > 1 ? KS - 1 : 1][WC][C::TC * C::TR][64];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const int wc = wv % WC, ks = wv / WC;
    const int col_tiles = (p.n + WC * kCols - 1) / (WC * kCols);
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        TileAt t;
        if (p.offsets) {
            const int found = find_tile(p.offsets, p.n_groups, p.m, C::BR, 0, false, col_tiles, b, t);
            if (found < 0) return;
            if (!found) continue;
        } else {                                         // one group: no search (it takes as long as a short reduction)
            const uint32_t chunk = (uint32_t)b / (uint32_t)col_tiles;
            t.g = 0;
            t.col = (int)((uint32_t)b - chunk * (uint32_t)col_tiles);
            t.beg = (int64_t)chunk * C::BR;
            t.end = t.beg + C::BR < p.m ? t.beg + C::BR : p.m;
            if (t.beg >= p.m) return;
        }
        const bool grouped = t.g < p.n_groups;
        const int c0 = (t.col * WC + wc) * kCols;
        int64_t row[C::TR];
        const char* x[C::TR];
#pragma unroll
        for (int j = 0; j < C::TR; ++j) {
            const int64_t pos = t.beg + j * 16 + (lane & 15);
            const int64_t r = pos < t.end ? (p.order ? (int64_t)p.order[pos] : pos) : -1;
            row[j] = r >= 0 && r < p.m ? r : -1;
            x[j] = (const char*)p.a + ((row[j] < 0 ? 0 : row[j]) * p.lda + q * 2 * VE) * ES;   // (products of no row are not stored)
        }
        const char* w[C::TC];
        const int64_t wg = grouped ? (int64_t)t.g * (kPairs ? 2 : 1) * p.n * p.ldw : 0;
#pragma unroll
        for (int i = 0; i < C::TC; ++i) {
            int c = c0 + (kPairs ? 0 : i * 16) + (lane & 15);
            c = c < p.n ? c : p.n - 1;
            w[i] = (const char*)p.b + (wg + ((kPairs && i ? p.n : 0) + (int64_t)c) * p.ldw + q * 2 * VE) * ES;
        }
        f32x4 acc[C::TC][C::TR];
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int j = 0; j < C::TR; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        struct Pieces { Frag<T> w[C::TC][2], x[C::TR][2]; };
        auto products = [&](const Pieces& f) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < kSteps<T>; ++e)
#pragma unroll
                    for (int j = 0; j < C::TR; ++j)
#pragma unroll
                        for (int i = 0; i < C::TC; ++i) multiply(f.w[i][h], f.x[j][h], e, acc[i][j]);
        };
        const int whole = p.k / kStep, mine = (whole + KS - 1) / KS;     // steps of 128 bytes
        int s = ks * mine, last = s + mine < whole ? s + mine : whole;
        if (grouped && c0 < p.n) {
            auto read = [&](int at, Pieces& f) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < C::TC; ++i) load_at<ES>(w[i] + (int64_t)at * 128 + h * 16, f.w[i][h].v);
#pragma unroll
                    for (int j = 0; j < C::TR; ++j) load_at<ES>(x[j] + (int64_t)at * 128 + h * 16, f.x[j][h].v);
                }
            };
            if (s + kBatch <= last) {                    // a batch of steps ahead
                Pieces now[kBatch], next[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) read(s + u, now[u]);
                for (; s + 2 * kBatch <= last; s += kBatch) {
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) read(s + kBatch + u, next[u]);
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) products(now[u]);
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) now[u] = next[u];
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) products(now[u]);
                s += kBatch;
            }
            for (; s < last; ++s) {
                Pieces f;
                read(s, f);
                products(f);
            }
            if (ks == KS - 1 && whole * kStep < p.k) {   // the rest of the rows
                Pieces f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t left = p.k - whole * kStep - (q * 2 + h) * VE;
#pragma unroll
                    for (int i = 0; i < C::TC; ++i) {
                        const u32x4 v = held_piece<ES>(w[i] + (int64_t)whole * 128 + h * 16, left);
                        __builtin_memcpy(&f.w[i][h].v, &v, 16);
                    }
#pragma unroll
                    for (int j = 0; j < C::TR; ++j) {
                        const u32x4 v = held_piece<ES>(x[j] + (int64_t)whole * 128 + h * 16, left);
                        __builtin_memcpy(&f.x[j][h].v, &v, 16);
                    }
                }
                products(f);
            }
        }
        if (KS > 1) {
            __syncthreads();                             // the sums of the tile before are read
            if (ks > 0) {
#pragma unroll
                for (int i = 0; i < C::TC; ++i)
#pragma unroll
                    for (int j = 0; j < C::TR; ++j) s_part[ks - 1][wc][i * C::TR + j][lane] = acc[i][j];
            }
            __syncthreads();
            if (ks > 0) continue;
#pragma unroll
            for (int i = 0; i < C::TC; ++i)
#pragma unroll
                for (int j = 0; j < C::TR; ++j)
#pragma unroll
                    for (int o = 0; o < KS - 1; ++o) acc[i][j] += s_part[o][wc][i * C::TR + j][lane];
        }
        if (c0 >= p.n) continue;
#pragma unroll
        for (int j = 0; j < C::TR; ++j) {
            f32x4 v[C::TC];
#pragma unroll
            for (int i = 0; i < C::TC; ++i) v[i] = acc[i][j];
            end(t, grouped, j * 16 + (lane & 15), row[j], c0, v);
        }
    }
}

// Waves that share a reduction, by the waves that there would be without and
// the length of a row (us, with 1, 2, 4: one row, 4,096 x 2 rows of 4 KiB 20.9,
// 13.4, 9.7; 64 rows in 16 groups of as many 81, 78, 83; 16 rows, 65,536 rows of
// 2 KiB 26, 27, 30; 8 rows, 65,536 of 256 bytes 6.1, 8.1, 12.1).  Two steps ahead
// are as good as four (9.7, 78, 28, 7.5): more waves fit.
inline int few_splits(int64_t waves, int64_t row_bytes) {
    if (row_bytes < 1024) return 1;
    return waves >= 1024 ? 2 : 4;
}
template <class F> void with_splits(int splits, F&& f) {
    if (splits == 4) f(std::integral_constant<int, 4>());
    else if (splits == 2) f(std::integral_constant<int, 2>());
    else f(std::integral_constant<int, 1>());
}
template <int KS> constexpr int few_waves = 4 / KS;   // of a workgroup beside each other

}  // namespace
}  // namespace htl
