// Gated projections by group: both projections of a feed-forward block, the
// activation and the product in one kernel, and the backward pass.
//
//   [z_i; u_i] = w_g x_i      (x [m][k], w [groups][2 n][k]: n rows of z's, n of u's)
//   y_i  = act(z_i) u_i
//   dz_i = dy_i u_i act'(z_i),  du_i = dy_i act(z_i)
//   dx_i = w_g^T [dz_i; du_i],  dw_g = sum over the group's rows of [dz_i; du_i] x_i^T
// Rows of no group: y = 0, dx = 0.  z and u are formed in fp32 and only what is
// kept of them, y, and dz and du (operands of the matrix instructions that
// follow) are rounded to the rows' type: bf16 costs each term half a step, 2^-8.
//
// Bound: products, and bytes where matrices are small or rows few.  Measured:
// 16,384 bf16 rows over 16 ragged groups, 2,048 -> 2 x 4,096: forward 598 us
// (577-654; 919 TFLOP/s), dz and du with z and u again 719 (695-803), dx 639, dw 683.
// 426,000 rows of 26 groups, 128 -> 2 x 256: forward with z and u kept 234 us (763 MB:
// 3.3 TB/s), dz, du and dx from them 294 (1.2 GB: 4.1 TB/s).  One row, 2,048 -> 2 x
// 4,096: 9.7 us (33.6 MB: 3.5 TB/s); 64 rows in 16 groups: 74 us (7.2 TB/s, in part
// from the last-level cache).  5,001 fp32 rows, 513 -> 2 x 777: 110 us (72 TFLOP/s).
#include "few.h"
#include "wide.h"

namespace htl {
namespace {

// The end of a tile of pairs: a wave's first TC / 2 results of a row are z and
// the others u of the same columns.
template <class C> struct GatedEnd {
    static constexpr bool kPairs = true;
    static constexpr int F = C::TC / 2;
    int n, act;
    void* y;                 // [m][n]
    bool y_f32, row_f32;
    void* kept;              // nullable: [m][2 n] of the rows' type
    __device__ __forceinline__ void operator()(const TileAt&, bool, int, int64_t row, int col, f32x4 (&v)[C::TC]) const {
        f32x4 out[F];
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float slope;
                out[i][e] = gate_act(v[i][e], act, slope) * v[F + i][e];
            }
        store_rows<F>(y, y_f32, row, n, col, n, out);
        if (kept) {
            store_rows<F>(kept, row_f32, row, 2 * (int64_t)n, col, n, v);
            store_rows<F>((char*)kept + n * (row_f32 ? 4ll : 2ll), row_f32, row, 2 * (int64_t)n, col, n, v + F);
        }
    }
};

// The same with dy: dz and du, rows of 2 n of the rows' type, `ld` apart, by
// row or (packed) by position in the plan.
template <class C, int T> struct GatedBackEnd {
    static constexpr bool kPairs = true;
    static constexpr int F = C::TC / 2;
    int n, act;
    RowsIn dy;
    void* d;
    int64_t ld;
    bool packed;
    __device__ __forceinline__ void operator()(const TileAt& t, bool grouped, int r, int64_t row, int col,
                                               f32x4 (&v)[C::TC]) const {
        if (!grouped) return;                // nothing reads their gradients
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int c = col + i * 16 + (__lane_id() >> 4) * 4;
            float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row >= 0) {
                const char* at = (const char*)dy.p + (row * dy.ld + c) * (T == kSrcF32 ? 4 : 2);
                if (c + 4 <= n) {
                    if (T == kSrcF32) {
                        load_at<4>(at, g);
                    } else {
                        u32x2 w;
                        load_at<2>(at, w);
                        g[0] = bf16_lo(w[0]), g[1] = bf16_hi(w[0]), g[2] = bf16_lo(w[1]), g[3] = bf16_hi(w[1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < n) g[e] = T == kSrcF32 ? ((const float*)at)[e] : bf16_lo(((const uint16_t*)at)[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float slope;
                const float a = gate_act(v[i][e], act, slope);
                v[i][e] = g[e] * v[F + i][e] * slope;
                v[F + i][e] = g[e] * a;
            }
        }
        // (a position that names no row has zeros: sums over positions read it)
        const int64_t to = !packed ? row : t.beg + r < t.end ? t.beg + r : -1;
        store_rows<F>(d, T == kSrcF32, to, ld, col, n, v);
        store_rows<F>((char*)d + n * (T == kSrcF32 ? 4ll : 2ll), T == kSrcF32, to, ld, col, n, v + F);
    }
};

template <int T, class C, bool ASYNC>
__global__ __launch_bounds__(C::kThreads, 2) void k_gated(ProdArgs p, GatedEnd<C> end) {
    product_tiles<T, kFwd, C, ASYNC>(p, end);
}
template <int T, class C, bool ASYNC>
__global__ __launch_bounds__(C::kThreads, 2) void k_gated_back(ProdArgs p, GatedBackEnd<C, T> end) {
    product_tiles<T, kFwd, C, ASYNC>(p, end);
}

__global__ __launch_bounds__(256, 1) void k_gated_wide(ProdArgs p, GatedEnd<Wide> end) { wide_tiles<kFwd>(p, end); }
__global__ __launch_bounds__(256, 1) void k_gated_back_wide(ProdArgs p, GatedBackEnd<Wide, kSrcBf16> end) {
    wide_tiles<kFwd>(p, end);
}

// dz and du from what was kept of z and u: eight columns a lane.  order
// (nullable): d's rows lie by position in it.
template <int T>
__global__ __launch_bounds__(256) void k_gated_slopes(RowsIn dy, RowsIn kept, RowsOut d, const int32_t* __restrict__ order,
                                                      int64_t m, int n, int act) {
    const int64_t each = (n + 7) / 8, all = m * each;
    const RowsIn up = {(const char*)kept.p + n * (T == kSrcF32 ? 4ll : 2ll), nullptr, kept.ld, 0};
    const RowsOut du = {(char*)d.p + n * (T == kSrcF32 ? 4ll : 2ll), d.ld};
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int64_t to = i / each, row = order ? (int64_t)order[to] : to;
        const int col = (int)(i - to * each) * 8;
        const bool in = row >= 0 && row < m;             // (a position that names no row: zeros)
        const int have = in ? n : 0;
        const int64_t from = in ? row : 0;
        Raw8<T> rg, rz, ru;
        load8(dy, from, col, have, rg);
        load8(kept, from, col, have, rz);
        load8(up, from, col, have, ru);
        float g[8], z[8], u[8];
        unpack8(dy, rg, g);
        unpack8(kept, rz, z);
        unpack8(up, ru, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float slope;
            const float a = gate_act(z[e], act, slope);
            z[e] = g[e] * u[e] * slope;
            u[e] = g[e] * a;
        }
        store8<T>(d, to, col, n, z);
        store8<T>(du, to, col, n, u);
    }
}

template <int T, int KS, class C, class End> __global__ __launch_bounds__(kFewThreads) void k_gated_few(ProdArgs p, End end) {
    few_tiles<T, KS, C>(p, end);
}

// Projections that fit in LDS (a feature table's block): a workgroup loads its
// group's once, and its waves walk the chunk's rows, 32 at a time and without
// waiting for each other, as product.hip's kernel for such matrices does.  LDS
// holds for every 64 outputs (whole lines of y) their rows of z's and then of u's,
// LP * 32 elements each, zeros beyond the matrix, 16 bytes apart so that 16 rows
// read together hit different banks.  Bound: bytes.
struct Resident {
    static constexpr int TC = 8;
};
template <int LP, int BYTES>
__global__ __launch_bounds__(512, 2) void k_gated_resident(ProdArgs p, GatedEnd<Resident> end) {
    constexpr int kLd = LP * 64 + 16;
    __shared__ __attribute__((aligned(16))) char lds[BYTES];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = (p.n + 63) / 64;
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        TileAt t;
        const int found = find_tile(p.offsets, p.n_groups, p.m, p.rows, 0, false, 1, b, t);
        if (found < 0) return;
        if (!found) continue;
        const bool grouped = t.g < p.n_groups;
        auto row_at = [&](int64_t pos) {
            const int32_t row = pos < t.end ? (p.order ? p.order[pos] : (int32_t)pos) : -1;
            return row >= 0 && row < p.m ? row : -1;
        };
        int64_t pos = t.beg + wv * 32;
        int32_t row[2] = {row_at(pos + (lane & 15)), row_at(pos + 16 + (lane & 15))};
        __syncthreads();                     // the matrix before is read
        if (grouped) {
            const char* w = (const char*)p.b + (int64_t)t.g * 2 * p.n * p.ldw * 2;
#pragma unroll 4
            for (int i = threadIdx.x; i < blocks * 128 * LP * 4; i += 512) {
                const int c = i / (LP * 4), e = i % (LP * 4) * 8, col = c / 128 * 64 + c % 64;
                const int64_t at = (int64_t)(c % 128 < 64 ? 0 : p.n) + col;
                *(u32x4*)(lds + c * kLd + e * 2) = held_piece<2>(w + (at * p.ldw + e) * 2, col < p.n ? p.k - e : 0);
            }
        }
        __syncthreads();
        for (; pos < t.end; pos += 256) {
            Frag<kSrcBf16> x[2][LP];
#pragma unroll
            for (int l = 0; l < LP; ++l)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int e = l * 32 + (lane >> 4) * 8;
                    const char* at = (const char*)p.a + ((row[j] < 0 ? 0 : row[j]) * p.lda + e) * 2;
                    if (p.k == LP * 32) {    // every piece whole; a row that is not there is read as the first
                        load_at<2>(at, x[j][l].v);
                    } else {
                        const u32x4 v = held_piece<2>(at, p.k - e);
                        __builtin_memcpy(&x[j][l].v, &v, 16);
                    }
                }
            const int32_t next[2] = {row_at(pos + 256 + (lane & 15)), row_at(pos + 272 + (lane & 15))};
            for (int nb = 0; nb < blocks; ++nb) {
                f32x4 acc[2][8];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[j][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (grouped) {
#pragma unroll
                    for (int l = 0; l < LP; ++l)
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            Frag<kSrcBf16> c;
                            c.v = *(const bf16x8*)(lds + (nb * 128 + q * 16 + (lane & 15)) * kLd + l * 64 + (lane >> 4) * 16);
                            multiply(c, x[0][l], 0, acc[0][q]);
                            multiply(c, x[1][l], 0, acc[1][q]);
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) end(t, grouped, j * 16 + (lane & 15), row[j], nb * 64, acc[j]);
            }
            row[0] = next[0];
            row[1] = next[1];
        }
    }
}
// Positions per chunk: so many that no more chunks than workgroups run at once load a matrix,
// each once.  (426,000 rows of 26 groups, 128 -> 2 x 256, one sweep: 234 us with 2,048, 246
// with 1,024, 271 with 512; the backward pass below 285, 313 and 341; its median elsewhere 294.)
uint32_t resident_rows(int64_t m, int n_groups, int at_once) {
    return (uint32_t)align_up((size_t)(n_groups <= at_once / 4 ? ceil_div(m, at_once - n_groups) : ceil_div(m, 1024)), 256);
}
template <int LP> void launch_resident(ProdArgs p, int64_t bytes, const GatedEnd<Resident>& end, hipStream_t s) {
    const int64_t chunks = p.m / p.rows + p.n_groups + 1;
    const dim3 grid(grid_for(align_up((size_t)chunks, kXcds), 1));
    if (bytes <= 81920) hipLaunchKernelGGL((k_gated_resident<LP, 81920>), grid, dim3(512), 0, s, p, end);
    else hipLaunchKernelGGL((k_gated_resident<LP, 163840>), grid, dim3(512), 0, s, p, end);
}

// Backward of such blocks from what was kept of z and u: a workgroup holds its
// group's matrix transposed, and its waves take 32 rows at a time from dy, z and u
// to dz and du in registers, out to d, and through the matrix to dx.  Loads and
// d are whole 128-byte lines, 64 outputs of eight rows a time, and lanes exchange dz and
// du to where the matrix instructions have them.  In LDS, for each of 128 columns, the
// z's rows and then the u's, NP * 32 elements each with zeros behind, 16 bytes apart
// as above.  Bound: bytes.  WHOLE: n is NP * 32.
template <int NP, bool WHOLE>
__global__ __launch_bounds__(512, 2) void k_gated_back_resident(ProdArgs p, RowsIn dy, RowsIn kept, RowsOut d, int act) {
    constexpr int kLd = NP * 128 + 16;
    __shared__ __attribute__((aligned(16))) char lds[128 * kLd];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int piece = (lane & 7) * 8, from_lane = ((lane & 7) * 8 + (lane >> 3 & 1) * 4 + (lane >> 4)) * 4;
    const RowsIn up = {(const char*)kept.p + p.n * 2ll, nullptr, kept.ld, 0};
    const RowsOut du = {(char*)d.p + p.n * 2ll, d.ld};
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        TileAt t;
        const int found = find_tile(p.offsets, p.n_groups, p.m, p.rows, 0, false, 1, b, t);
        if (found < 0) return;
        if (!found) continue;
        const bool grouped = t.g < p.n_groups;
        auto row_at = [&](int64_t pos) {
            const int32_t row = pos < t.end ? (p.order ? p.order[pos] : (int32_t)pos) : -1;
            return row >= 0 && row < p.m ? row : -1;
        };
        int64_t pos = t.beg + wv * 32;
        if (!grouped) {                      // no matrix, and nothing reads their d
            f32x4 zero[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) zero[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (; pos < t.end; pos += 256)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    for (int c = 0; c < p.k; c += 64)
                        store_rows<4>(p.out, p.out_f32, row_at(pos + j * 16 + (lane & 15)), p.k, c, p.k, zero);
            continue;
        }
        // eight rows and 64 columns of each: row lane / 8, piece lane % 8
        struct Raw { Raw8<kSrcBf16> g, z, u; } raw[4];
        int32_t row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = row_at(pos + i * 8 + (lane >> 3));
        // a row that is not there: as the first, or zeros
        auto fetch = [&](int l, int32_t from, Raw& o) __attribute__((always_inline)) {
            const int64_t r = from < 0 ? 0 : from;
            const int col = l * 64 + piece;
            if (WHOLE) {
                load_at<2>((const uint16_t*)dy.p + r * dy.ld + col, o.g.w);
                load_at<2>((const uint16_t*)kept.p + r * kept.ld + col, o.z.w);
                load_at<2>((const uint16_t*)up.p + r * up.ld + col, o.u.w);
            } else {
                const int have = from < 0 ? 0 : p.n;
                load8(dy, r, col, have, o.g);
                load8(kept, r, col, have, o.z);
                load8(up, r, col, have, o.u);
            }
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch(0, row[i], raw[i]);
        __syncthreads();                     // the matrix before is read
        const char* w = (const char*)p.b + (int64_t)t.g * 2 * p.n * p.ldw * 2;
        // two rows of w and eight columns: pairs of neighbours in eight rows of LDS.  A wave has 16 such pairs
        // of rows beside each other, so that it writes to all banks.
#pragma unroll 2
        for (int i = threadIdx.x; i < NP * 32 * 16; i += 512) {
            const int c = ((i >> 4) & 15) * 8, at_e = ((i >> 8) * 16 + (i & 15)) * 2;   // of both halves
            const bool half = at_e >= NP * 32;
            const int e = at_e - (half ? NP * 32 : 0);
            const char* at = w + (((int64_t)(half ? p.n : 0) + e) * p.ldw + c) * 2;
            const u32x4 lo = held_piece<2>(at, e < p.n ? p.k - c : 0);
            const u32x4 hi = held_piece<2>(at + p.ldw * 2, e + 1 < p.n ? p.k - c : 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t a = lo[j >> 1] >> (16 * (j & 1)) & 0xFFFFu, v = hi[j >> 1] >> (16 * (j & 1));
                *(uint32_t*)(lds + (c + j) * kLd + at_e * 2) = a | v << 16;
            }
        }
        __syncthreads();
        for (; pos < t.end; pos += 256) {
            int32_t next[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = row_at(pos + 256 + i * 8 + (lane >> 3));
            f32x4 acc[2][8];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[j][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int l = 0; l < NP / 2; ++l) {
                const bool more = l + 1 < NP / 2;
                u32x4 w8[2][4];              // dz and du of each eight rows
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float g[8], z[8], u[8];
                    unpack8(dy, raw[i].g, g);
                    unpack8(kept, raw[i].z, z);
                    unpack8(up, raw[i].u, u);
                    fetch(more ? l + 1 : 0, more ? row[i] : next[i], raw[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float slope;
                        const float a = gate_act(z[e], act, slope);
                        z[e] = g[e] * u[e] * slope;
                        u[e] = g[e] * a;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w8[0][i][e] = pack_bf16(z[2 * e], z[2 * e + 1]);
                        w8[1][i][e] = pack_bf16(u[2 * e], u[2 * e + 1]);
                    }
                    if (row[i] >= 0) {
                        const int col = l * 64 + piece;
                        if (WHOLE) {
                            store_at<2>((uint16_t*)d.p + row[i] * d.ld + col, w8[0][i]);
                            store_at<2>((uint16_t*)du.p + row[i] * du.ld + col, w8[1][i]);
                        } else {
                            store8<kSrcBf16>(d, row[i], col, p.n, z);
                            store8<kSrcBf16>(du, row[i], col, p.n, u);
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)  // 32 of the columns: pieces s * 4 .. + 4
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        Frag<kSrcBf16> x[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            u32x4 o;
                            // rows 8 .. 15 to the lanes whose pieces are not of this half, then all to row lane % 16,
                            // piece lane / 16
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int low = (int)w8[h][j * 2][e], high = (int)w8[h][j * 2 + 1][e];
                                const int v = s == 0 ? __builtin_amdgcn_update_dpp(low, high, 0x114, 0xF, 0xA, false)
                                                     : __builtin_amdgcn_update_dpp(high, low, 0x104, 0xF, 0x5, false);
                                o[e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from_lane, v);
                            }
                            __builtin_memcpy(&x[j].v, &o, 16);
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            Frag<kSrcBf16> c;
                            c.v = *(const bf16x8*)(lds + (q * 16 + (lane & 15)) * kLd + (h * NP + l * 2 + s) * 64 + (lane >> 4) * 16);
                            multiply(c, x[0], 0, acc[0][q]);
                            multiply(c, x[1], 0, acc[1][q]);
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                store_rows<8>(p.out, p.out_f32, row_at(pos + j * 16 + (lane & 15)), p.k, 0, p.k, acc[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) row[i] = next[i];
        }
    }
}
// Whether a backward pass from z and u goes that way: 426,000 rows of 26 groups, 128 ->
// 2 x 256: 294 us, where dz and du by themselves and then dx in tiles take 415.  (Lines
// read and written in two halves, 16 rows a time: 356.)
bool back_resident(int64_t m, int n_groups, int n, int k, htl_dtype dtype) {
    return dtype == HTL_BF16 && n <= 256 && k <= 128 && m / n_groups >= 512 && m >= 1 << 16;
}
htl_status launch_back_resident(ProdArgs p, const RowsIn& dy, const RowsIn& kept, const RowsOut& d, int act, hipStream_t s) {
    p.rows = resident_rows(p.m, p.n_groups, 256);
    const dim3 grid(grid_for(align_up((size_t)(p.m / p.rows + p.n_groups + 1), kXcds), 1));
    auto go = [&](auto steps) {
        constexpr int NP = decltype(steps)::value;
        if (p.n == NP * 32) hipLaunchKernelGGL((k_gated_back_resident<NP, true>), grid, dim3(512), 0, s, p, dy, kept, d, act);
        else hipLaunchKernelGGL((k_gated_back_resident<NP, false>), grid, dim3(512), 0, s, p, dy, kept, d, act);
    };
    if (p.n <= 64) go(std::integral_constant<int, 2>());
    else if (p.n <= 128) go(std::integral_constant<int, 4>());
    else go(std::integral_constant<int, 8>());
    return check_launch("gated_mm_backward");
}

template <int T, class C, bool ASYNC>
void launch_gated(const ProdArgs& p, int64_t chunks, const GatedEnd<C>* fwd, const GatedBackEnd<C, T>* back, hipStream_t s) {
    const dim3 grid(grid_for(align_up((size_t)(chunks * ceil_div(p.n, C::BC / 2)), kXcds), 1));
    if (fwd) hipLaunchKernelGGL((k_gated<T, C, ASYNC>), grid, dim3(C::kThreads), 0, s, p, *fwd);
    else hipLaunchKernelGGL((k_gated_back<T, C, ASYNC>), grid, dim3(C::kThreads), 0, s, p, *back);
}

struct GatedCall {
    int act;
    void* y;
    bool y_f32;
    void* kept;
    RowsIn dy;               // null: forward
    void* d;
    int64_t ld;
    bool packed;             // d by position
};

// Whether wide.h's tiles fill the device (`tiles` of them) with whole rows.
bool many(int64_t m, int n_groups, int64_t tiles) { return tiles >= 224 && m / n_groups >= 256; }

// Rows that few.h's kernel is for (all of them in one group, or few in each).
bool few(int64_t m, int n_groups) { return m <= 32 || m / n_groups <= 8; }
template <int T> void launch_few(const ProdArgs& p, const GatedCall& c, hipStream_t s) {
    auto go = [&](auto shape, auto splits) {
        using C = decltype(shape);
        constexpr int KS = decltype(splits)::value;
        const int64_t tiles = (p.m / C::BR + p.n_groups + 1) * ceil_div(p.n, 16 * few_waves<KS>);
        const dim3 grid(grid_for(align_up((size_t)tiles, kXcds), 1));
        if (c.dy.p) {
            const GatedBackEnd<C, T> end = {p.n, c.act, c.dy, c.d, c.ld, c.packed};
            hipLaunchKernelGGL((k_gated_few<T, KS, C, GatedBackEnd<C, T>>), grid, dim3(kFewThreads), 0, s, p, end);
        } else {
            const GatedEnd<C> end = {p.n, c.act, c.y, c.y_f32, T == kSrcF32, c.kept};
            hipLaunchKernelGGL((k_gated_few<T, KS, C, GatedEnd<C>>), grid, dim3(kFewThreads), 0, s, p, end);
        }
    };
    const int64_t groups = p.m < p.n_groups ? p.m : p.n_groups;
    const int splits = few_splits(groups * ceil_div(p.n, 16), (int64_t)p.k * (T == kSrcF32 ? 4 : 2));
    auto with = [&](auto shape) {
        with_splits(splits, [&](auto ks) { go(shape, ks); });
    };
    if (p.m <= 16 || p.m / p.n_groups <= 8) with(Few<1>());
    else with(Few<2>());
}

// The kernel by size, as the plain products' (product.hip) at twice the columns.
// Few fp32 rows a tile leave the device's last round almost empty: 5,001 rows,
// 513 -> 777 pairs, 137 us in tiles of 128 rows, 127 in tiles of 32.
htl_status launch_pairs(ProdArgs p, htl_dtype dtype, const GatedCall& c, hipStream_t s) {
    const int es = elem(dtype);
    const bool fast = p.lda * es % 16 == 0 && aligned(p.a, 16) && p.ldw * es % 16 == 0 && (int64_t)p.k * es % 16 == 0 &&
                      aligned(p.b, 16) && p.m * p.lda * es <= kBufferBytes && 2 * (int64_t)p.n * p.ldw * es <= kBufferBytes;
    const int64_t each = p.m / p.n_groups;
    const int lp = p.k <= 32 ? 1 : p.k <= 64 ? 2 : p.k <= 128 ? 4 : 8;
    const int64_t bytes = ceil_div(p.n, 64) * 128 * (lp * 64 + 16);
    if (!c.dy.p && dtype == HTL_BF16 && p.k <= 256 && bytes <= 163840 && each >= 512 && p.m >= 1 << 16) {
        p.rows = resident_rows(p.m, p.n_groups, bytes <= 81920 ? 512 : 256);
        const GatedEnd<Resident> end = {p.n, c.act, c.y, c.y_f32, false, c.kept};
        if (lp == 1) launch_resident<1>(p, bytes, end, s);
        else if (lp == 2) launch_resident<2>(p, bytes, end, s);
        else if (lp == 4) launch_resident<4>(p, bytes, end, s);
        else launch_resident<8>(p, bytes, end, s);
        return check_launch("gated projections");
    }
    if (p.packed || (p.k >= 256 && dtype == HTL_BF16 && fast && many(p.m, p.n_groups, ceil_div(p.m, 256) * ceil_div(p.n, 128)))) {
        p.rows = 256;
        p.no_rest = true;
        const dim3 grid(wide_grid((p.m / 256 + p.n_groups) * ceil_div(p.n, 128)));
        if (c.dy.p) {
            const GatedBackEnd<Wide, kSrcBf16> end = {p.n, c.act, c.dy, c.d, c.ld, c.packed};
            hipLaunchKernelGGL(k_gated_back_wide, grid, dim3(Wide::kThreads), 0, s, p, end);
        } else {
            const GatedEnd<Wide> end = {p.n, c.act, c.y, c.y_f32, false, c.kept};
            hipLaunchKernelGGL(k_gated_wide, grid, dim3(Wide::kThreads), 0, s, p, end);
        }
        htl_status st = check_launch("gated projections");
        if (c.dy.p || !p.offsets) return st;
        if (st == HTL_OK) st = zero_rest(c.y, (int64_t)p.n * (c.y_f32 ? 4 : 2), p.m, p.order, p.offsets + p.n_groups, s);
        if (st == HTL_OK && c.kept) st = zero_rest(c.kept, (int64_t)p.n * 4, p.m, p.order, p.offsets + p.n_groups, s);
        return st;
    }
    if (few(p.m, p.n_groups)) {
        if (dtype == HTL_F32) launch_few<kSrcF32>(p, c, s);
        else launch_few<kSrcBf16>(p, c, s);
        return check_launch("gated projections");
    }
    const int64_t small = (ceil_div(p.m, 32) + p.n_groups) * ceil_div(p.n, 64);
    const int tile = each <= 48 || small <= (dtype == HTL_F32 ? 4096 : 512) ? 32 : 128;
    p.rows = (uint32_t)tile;
    const int64_t chunks = p.m / tile + p.n_groups + 1;
    auto go = [&](auto t, auto shape, auto async) {
        constexpr int T = decltype(t)::value;
        using C = decltype(shape);
        const GatedEnd<C> fwd = {p.n, c.act, c.y, c.y_f32, T == kSrcF32, c.kept};
        const GatedBackEnd<C, T> back = {p.n, c.act, c.dy, c.d, c.ld, c.packed};
        launch_gated<T, C, decltype(async)::value>(p, chunks, c.dy.p ? nullptr : &fwd, c.dy.p ? &back : nullptr, s);
    };
    using F32 = std::integral_constant<int, kSrcF32>;
    using B16 = std::integral_constant<int, kSrcBf16>;
    using Yes = std::true_type;
    using No = std::false_type;
    if (dtype == HTL_BF16) {
        if (tile == 128 && fast) go(B16(), Mid(), Yes());
        else if (tile == 128) go(B16(), Mid(), No());
        else if (fast) go(B16(), Small(), Yes());
        else go(B16(), Small(), No());
    } else {
        if (tile == 128 && fast) go(F32(), Mid(), Yes());
        else if (tile == 128) go(F32(), Mid(), No());
        else if (fast) go(F32(), Small(), Yes());
        else go(F32(), Small(), No());
    }
    return check_launch("gated projections");
}

// Copies of x and w whose rows whole 16-byte pieces make up, for rows that they
// do not: tiles' loads then go straight to LDS.  With few rows a matrix is read
// once, and they cost more than they save.
bool copies(int64_t m, int n_groups, int k, htl_dtype dtype) {
    return k % (dtype == HTL_F32 ? 4 : 8) && m / n_groups >= 64;
}
size_t x_copy_bytes(int64_t m, int k, htl_dtype dtype) { return align_up((size_t)m * spread_ld(k) * elem(dtype), 256); }
size_t w_copy_bytes(int n_groups, int n, int k, htl_dtype dtype) {
    return align_up((size_t)n_groups * 2 * n * packed_ld(k) * elem(dtype), 256);
}

struct BackSpace {
    bool wide, copied;
    int64_t ld;              // of d
    int splits;
    char *d, *sums, *x, *w;
    float* parts;
    size_t bytes;
    // tiles: whether wide.h's may be used
    BackSpace(void* ws, int64_t m, int n_groups, int n, int k, htl_dtype dtype, bool tiles) {
        wide = tiles && dtype == HTL_BF16 && k >= 256 && n >= 128 && 4 * n * packed_ld(k) <= kBufferBytes &&
               many(m, n_groups, ceil_div(m, 256) * ceil_div(2 * n, 256));
        copied = copies(m, n_groups, k, dtype);
        ld = wide || copied ? spread_ld(2 * n) : 2 * (int64_t)n;
        splits = wide ? wide_dx_splits(m, 2 * n, k) : 1;
        size_t at = 0;
        auto take = [&](size_t b) {
            char* p = (char*)ws + at;
            at += align_up(b + 1, 256);
            return p;
        };
        d = take((size_t)m * ld * elem(dtype));
        sums = take(wide ? wide_dw_bytes(m, n_groups, 2 * n, k, ld, spread_ld(k)) : sums_dw_bytes(m, n_groups, 2 * n, k));
        x = take(wide || copied ? x_copy_bytes(m, k, dtype) : 0);
        w = take(copied ? w_copy_bytes(n_groups, n, k, dtype) : 0);
        parts = (float*)take(splits > 1 ? (size_t)splits * m * k * 4 : 0);
        bytes = at;
    }
};

}  // namespace
}  // namespace htl

using namespace htl;

#define GATED_CHECK(name)                                                                                        \
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, name ": row count out of range");                                       \
    HTL_REQUIRE(n >= 1 && n <= HTL_MAX_PRODUCT_DIM / 2 && k >= 1 && k <= HTL_MAX_PRODUCT_DIM, name ": n or k out of range"); \
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, name ": group count out of range");                     \
    HTL_REQUIRE(known(dtype), name ": dtype must be HTL_F32 or HTL_BF16");                                       \
    HTL_REQUIRE(act == HTL_ACT_NONE || act == HTL_ACT_SIGMOID || act == HTL_ACT_SILU, name ": unknown activation"); \
    HTL_REQUIRE(offsets || (n_groups == 1 && !order), name ": several groups need offsets");                     \
    HTL_REQUIRE(aligned(order, 4) && aligned(offsets, 4), name ": misaligned pointer")

extern "C" size_t gated_mm_workspace_bytes(int64_t m, int n_groups, int n, int k, htl_dtype dtype) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || n < 1 || n > HTL_MAX_PRODUCT_DIM / 2 || k < 1 ||
        k > HTL_MAX_PRODUCT_DIM || !known(dtype))
        return 0;
    return 256 + (copies(m, n_groups, k, dtype) ? x_copy_bytes(m, k, dtype) + w_copy_bytes(n_groups, n, k, dtype) : 0);
}

extern "C" htl_status gated_mm(const void* x, int64_t ldx, const void* w, htl_dtype dtype, int64_t m, int n, int k,
                               const int32_t* order, const int32_t* offsets, int n_groups, htl_act act, void* y,
                               htl_dtype y_dtype, void* kept, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    GATED_CHECK("gated_mm");
    HTL_REQUIRE(known(y_dtype), "gated_mm: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(ldx >= k, "gated_mm: row stride below k");
    if (m == 0) return HTL_OK;
    const int es = elem(dtype);
    HTL_REQUIRE(x && w && y, "gated_mm: null pointer");
    HTL_REQUIRE(aligned(x, es) && aligned(w, es) && aligned(y, elem(y_dtype)) && aligned(kept, es),
                "gated_mm: misaligned pointer");
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= gated_mm_workspace_bytes(m, n_groups, n, k, dtype),
                "gated_mm: workspace too small or misaligned");
    ProdArgs p = {x, w, nullptr, order, offsets, m, ldx, k, k, n, k, n_groups, 0, nullptr, 0, 0};
    if (copies(m, n_groups, k, dtype)) {
        char* const xc = (char*)ws;
        char* const wc = xc + x_copy_bytes(m, k, dtype);
        const int64_t rows = (int64_t)n_groups * 2 * n;
        htl_status st = pack_rows(x, ldx, dtype, nullptr, m, m, k, xc, spread_ld(k), stream);
        if (st == HTL_OK) st = pack_rows(w, k, dtype, nullptr, rows, rows, k, wc, packed_ld(k), stream);
        if (st != HTL_OK) return st;
        p = {xc, wc, nullptr, order, offsets, m, spread_ld(k), k, packed_ld(k), n, (int)packed_ld(k), n_groups, 0, nullptr, 0, 0};
    }
    return launch_pairs(p, dtype, {(int)act, y, y_dtype == HTL_F32, kept, {}, nullptr, 0, false}, stream);
}

extern "C" size_t gated_mm_backward_workspace_bytes(int64_t m, int n_groups, int n, int k, htl_dtype dtype) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || n < 1 || n > HTL_MAX_PRODUCT_DIM / 2 || k < 1 ||
        k > HTL_MAX_PRODUCT_DIM || !known(dtype))
        return 0;
    const size_t a = BackSpace(nullptr, m, n_groups, n, k, dtype, true).bytes;
    const size_t b = BackSpace(nullptr, m, n_groups, n, k, dtype, false).bytes;
    return a > b ? a : b;
}

extern "C" htl_status gated_mm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w,
                                        htl_dtype dtype, const void* kept, int64_t m, int n, int k, const int32_t* order,
                                        const int32_t* offsets, int n_groups, htl_act act, void* dx, htl_dtype dx_dtype,
                                        void* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    GATED_CHECK("gated_mm_backward");
    HTL_REQUIRE(known(dx_dtype), "gated_mm_backward: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(ld_dy >= n && ldx >= k, "gated_mm_backward: row stride below the row's length");
    if (!dx && !dw) return HTL_OK;
    const int es = elem(dtype);
    HTL_REQUIRE(m == 0 || (dy && w && x), "gated_mm_backward: null pointer");
    HTL_REQUIRE(aligned(dy, es) && aligned(x, es) && aligned(w, es) && aligned(kept, es) && aligned(dx, elem(dx_dtype)) &&
                    aligned(dw, es),
                "gated_mm_backward: misaligned pointer");
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= gated_mm_backward_workspace_bytes(m, n_groups, n, k, dtype),
                "gated_mm_backward: workspace too small or misaligned");
    const BackSpace s(ws, m, n_groups, n, k, dtype, k % 8 || aligned(w, 16));
    htl_status st = HTL_OK;
    const int64_t rows = (int64_t)n_groups * 2 * n;
    if (s.copied) st = pack_rows(w, k, dtype, nullptr, rows, rows, k, s.w, packed_ld(k), stream);
    // wide.h takes x by position in the plan, and sums over as many rows as lie in 4 GiB
    const bool as_is = s.wide ? !order && packed_as_is(x, ldx, k) && m * ldx * 2 <= kBufferBytes : !s.copied;
    if (st == HTL_OK && !as_is)
        st = pack_rows(x, ldx, dtype, s.wide ? order : nullptr, m, m, k, s.x, spread_ld(k), stream);
    if (st != HTL_OK) return st;
    const void* xs = as_is ? x : s.x;
    const void* wp = s.copied ? s.w : w;
    const int64_t ldxs = as_is ? ldx : spread_ld(k), ldw = s.copied ? packed_ld(k) : k;
    const bool fused = m > 0 && kept && dx && !s.wide && back_resident(m, n_groups, n, k, dtype);
    if (m > 0) {
        const RowsIn in = {dy, nullptr, ld_dy, 0};
        if (fused) {
            const ProdArgs p = {nullptr, wp, dx, order, offsets, m, 0, k, ldw, n, k, n_groups, 0, nullptr, dx_dtype == HTL_F32, 0};
            st = launch_back_resident(p, in, {kept, nullptr, 2 * (int64_t)n, 0}, {s.d, s.ld}, (int)act, stream);
        } else if (kept) {
            const RowsIn from = {kept, nullptr, 2 * (int64_t)n, 0};
            const RowsOut to = {s.d, s.ld};
            const int32_t* by = s.wide ? order : nullptr;
            const dim3 grid(grid_for(m * ceil_div(n, 8), 256));
            if (dtype == HTL_F32) hipLaunchKernelGGL(k_gated_slopes<kSrcF32>, grid, dim3(256), 0, stream, in, from, to, by, m, n, (int)act);
            else hipLaunchKernelGGL(k_gated_slopes<kSrcBf16>, grid, dim3(256), 0, stream, in, from, to, by, m, n, (int)act);
        } else {
            ProdArgs p = {xs, wp, nullptr, order, offsets, m, ldxs, k, ldw, n, s.copied ? (int)ldw : k, n_groups, 0, nullptr, 0, 0};
            p.packed = s.wide;
            st = launch_pairs(p, dtype, {(int)act, nullptr, false, nullptr, in, s.d, s.ld, s.wide}, stream);
        }
        if (st == HTL_OK) st = check_launch("gated_mm_backward");
        if (st == HTL_OK && s.ld > 2 * n) st = zero_behind(s.d, dtype, m, 2 * n, s.ld, stream);
        if (st != HTL_OK) return st;
    }
    if (dx && s.wide) {
        st = wide_dx(s.d, s.ld, wp, ldw, m, 2 * n, k, order, offsets, n_groups, dx, dx_dtype,
                     s.splits > 1 ? s.parts : nullptr, s.splits, false, stream);
        if (st == HTL_OK && s.splits > 1)
            st = sum_parts(s.parts, s.splits, false, m, k, order, offsets ? offsets + n_groups : nullptr, dx, dx_dtype, stream);
        else if (st == HTL_OK && offsets)
            st = zero_rest(dx, (int64_t)k * elem(dx_dtype), m, order, offsets + n_groups, stream);
    } else if (dx && !fused) {
        st = rows_dx(s.d, s.ld, wp, ldw, dtype, m, 2 * n, k, order, offsets, n_groups, dx, dx_dtype, s.copied, stream);
    }
    if (st != HTL_OK || !dw) return st;
    if (s.wide) return wide_dw(s.d, s.ld, xs, ldxs, m, 2 * n, k, offsets, n_groups, dw, dtype, s.sums, stream);
    return sums_dw(s.d, s.ld, xs, ldxs, dtype, m, 2 * n, k, order, offsets, n_groups, dw, dtype, s.sums, s.copied, stream);
}
