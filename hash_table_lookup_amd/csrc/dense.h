// Shared by the dense operators beside the lookup (rows8.hip, norm.hip,
// gate.hip, product.hip, gated.hip, scores.hip): rows read and written eight elements per lane, the
// 8-bit row format, and the map from workgroups to the rows of a group.
#pragma once

#include "htl_common.h"

namespace htl {

constexpr int kMaxGroups = HTL_MAX_GROUPS;
constexpr int kMaxNormDim = HTL_MAX_NORM_DIM;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 4096;   // row positions are int32

// Where a row's elements come from: fp32, bf16, or 8-bit codes with scales.
enum { kSrcF32 = 0, kSrcBf16 = 1, kSrcRows8 = 2 };

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Rows in device memory, at any alignment of the element: a lane moves eight
// elements at once wherever they start (the memory system takes a 16-byte
// access at any byte; rows of odd length ran 4 times slower element by
// element), and one at a time only past the last whole eight of a row.
struct RowsIn {
    const void* p;
    const uint8_t* scales;   // 8-bit rows only: [rows][ceil(dim / 32)]
    int64_t ld;              // elements from row to row
    int fmt;                 // 8-bit rows only: HTL_ROWS8_*
};
struct RowsOut {
    void* p;
    int64_t ld;
};

// Lanes exchanged without LDS, within 16: x of lane l ^ 1 or l ^ 2 (of a
// quad), or of the lane that mirrors l in its 8 or 16, which stands for l ^ 4
// and l ^ 8 where the lanes of a quad, or of 8, hold the same; rotated by 8 of
// 16, of lane l ^ 8.
enum { kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kRotate8 = 0x128 };
template <int HOW> __device__ __forceinline__ int move_lanes(int x) {
    return __builtin_amdgcn_update_dpp(0, x, HOW, 0xF, 0xF, true);
}
template <int HOW> __device__ __forceinline__ float add_moved(float x) {
    return x + __int_as_float(move_lanes<HOW>(__float_as_int(x)));
}

// A vector at any address that is a multiple of A.
template <int A, class V> __device__ __forceinline__ void load_at(const void* p, V& v) {
    __builtin_memcpy(&v, __builtin_assume_aligned(p, A), sizeof(V));
}
template <int A, class V> __device__ __forceinline__ void store_at(void* p, const V& v) {
    __builtin_memcpy(__builtin_assume_aligned(p, A), &v, sizeof(V));
}
// The same past the caches: rows of a result, of which nothing is read again here.
template <int A, class V> __device__ __forceinline__ void stream_at(void* p, const V& v) {
    typedef V Loose __attribute__((aligned(A)));
    __builtin_nontemporal_store(v, (Loose*)p);
}

template <int SRC> struct Raw8;
template <> struct Raw8<kSrcF32> { u32x4 lo, hi; };
template <> struct Raw8<kSrcBf16> { u32x4 w; };
template <> struct Raw8<kSrcRows8> { u32x2 c; uint32_t scale; };

__device__ __forceinline__ u32x4 zeros4() {
    u32x4 z = {0u, 0u, 0u, 0u};
    return z;
}

// Eight elements of a row from `col` on, as they lie in memory; zeros from
// dim on.  Loads only: nothing waits for them here.
__device__ __forceinline__ void load8(const RowsIn& r, int64_t row, int col, int dim, Raw8<kSrcF32>& o) {
    const float* p = (const float*)r.p + row * r.ld + col;
    o.lo = o.hi = zeros4();
    if (col + 8 <= dim) {
        load_at<4>(p, o.lo);
        load_at<4>(p + 4, o.hi);
    } else if (col < dim) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (col + j < dim) o.lo[j] = __float_as_uint(p[j]);
            if (col + 4 + j < dim) o.hi[j] = __float_as_uint(p[4 + j]);
        }
    }
}
__device__ __forceinline__ void load8(const RowsIn& r, int64_t row, int col, int dim, Raw8<kSrcBf16>& o) {
    const uint16_t* p = (const uint16_t*)r.p + row * r.ld + col;
    o.w = zeros4();
    if (col + 8 <= dim) {
        load_at<2>(p, o.w);
    } else if (col < dim) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < dim) o.w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    }
}
__device__ __forceinline__ void load8(const RowsIn& r, int64_t row, int col, int dim, Raw8<kSrcRows8>& o) {
    const uint8_t* p = (const uint8_t*)r.p + row * r.ld + col;
    o.c = {0u, 0u};
    o.scale = 0;
    if (col < dim) o.scale = r.scales[row * ((dim + 31) >> 5) + (col >> 5)];
    if (col + 8 <= dim) {
        load_at<1>(p, o.c);
    } else if (col < dim) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < dim) o.c[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
}

__device__ __forceinline__ void unpack8(const RowsIn&, const Raw8<kSrcF32>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = __uint_as_float(r.lo[j]);
        v[4 + j] = __uint_as_float(r.hi[j]);
    }
}
__device__ __forceinline__ void unpack8(const RowsIn&, const Raw8<kSrcBf16>& r, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(r.w[j]);
        v[2 * j + 1] = bf16_hi(r.w[j]);
    }
}

// The 8-bit row format.  A block of 32 elements of one row shares the scale
// 2^e, with e >= -126 the least that brings the block's largest magnitude to
// at most 127 (HTL_ROWS8_I8) or 448 (HTL_ROWS8_E4M3); an element x is kept as
// the nearest integer, or the nearest e4m3 number, to x / 2^e, ties to even,
// or as the nearest that stands for a finite value: with the largest scales
// 64 * 2^122 and 256 * 2^120 would be infinities, so 63 and 240 are the last.
// The scale byte is e + 127 (1..249), or 255 for a block that holds an
// infinity or a NaN, which reads back as NaN throughout.  A power of two
// costs up to one bit of the code's range against a free scale, and in
// return multiplying by it is exact: codes times scales have at most 8
// significant bits, so they are exact in bf16, and every reader sees the same
// values whatever type it reads them in.
__device__ __forceinline__ float rows8_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte << 23);
}
__device__ __forceinline__ void unpack8(const RowsIn& r, const Raw8<kSrcRows8>& q, float* v) {
    const float s = rows8_scale(q.scale);
    if (r.fmt == HTL_ROWS8_I8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)(q.c[j >> 2] >> (8 * (j & 3))) * s;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)q.c[h], 0) * s;
            v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)q.c[h], 1) * s;
            v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)q.c[h], 2) * s;
            v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)q.c[h], 3) * s;
        }
    }
}

// Rounded to nearest even by the one instruction that converts a pair (the
// bit arithmetic costs ten, and the norms are bound by instructions).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 f = {lo, hi};
    const bf16x2 b = __builtin_convertvector(f, bf16x2);
    uint32_t w;
    __builtin_memcpy(&w, &b, 4);
    return w;
}

template <int DST>
__device__ __forceinline__ void store8(const RowsOut& r, int64_t row, int col, int dim, const float* v) {
    if (DST == kSrcF32) {
        float* p = (float*)r.p + row * r.ld + col;
        if (col + 8 <= dim) {
            const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
            stream_at<4>(p, a);
            stream_at<4>(p + 4, b);
        } else if (col < dim) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < dim) p[j] = v[j];
        }
    } else {
        uint16_t* p = (uint16_t*)r.p + row * r.ld + col;
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
        if (col + 8 <= dim) {
            stream_at<2>(p, a);
        } else if (col < dim) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < dim) p[j] = (uint16_t)(a[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// 8-bit rows to be written beside another result (codes null: none).
struct Rows8Out {
    uint8_t* codes;
    uint8_t* scales;
    int fmt;
};
// Four neighbouring lanes (col = 8 * lane) hold a block of 32 and call this
// together; columns from dim on hold zeros.
__device__ __forceinline__ void save8(const Rows8Out& r, int64_t row, int col, int dim, const float* v) {
    uint32_t top = 0;                    // magnitudes compare as their bits; a NaN is above all
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        top = a > top ? a : top;
    }
    uint32_t o = (uint32_t)move_lanes<kXor1>((int)top);
    top = o > top ? o : top;
    o = (uint32_t)move_lanes<kXor2>((int)top);
    top = o > top ? o : top;
    const bool i8 = r.fmt == HTL_ROWS8_I8;
    // top = f * 2^k with f in [1, 2): e = k - 6 while f <= 127/64 (0x7E0000
    // is 127/64's fraction), or k - 8 while f <= 448/256 (0x600000), else one
    // more.  A subnormal top has e = -126.
    int e = (int)(top >> 23) - 127 - (i8 ? 6 : 8) + ((top & 0x7FFFFFu) > (i8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
    e = e < -126 ? -126 : e;
    const bool finite = top < 0x7F800000u;
    const float inv = finite ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.0f;
    u32x2 c = {0u, 0u};
    if (finite) {
        if (i8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // 1.5 * 2^23 + q: the sum is rounded to a whole q, to even, and its low byte is q's
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(__builtin_fmaf(v[4 * h + j], inv, 12582912.0f));
                c[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0C0C0400u),
                                             __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u), 0x05040100u);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
                w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
                c[h] = (uint32_t)w;
            }
        }
        if (e > (i8 ? 121 : 119)) {      // +-64 (0x40, 0xC0) to +-63, or +-256 (0x78, 0xF8) to +-240
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w = c[h], ones = 0x01010101u;
                if (i8) c[h] = w - (w >> 6 & ~(w >> 7) & ones) + (w >> 7 & ~((w & 63u * ones) + 63u * ones >> 6) & ones);
                else c[h] = w - (w >> 6 & w >> 5 & w >> 4 & w >> 3 & ones);
            }
        }
    }
    if (col < dim) {
        if ((col & 31) == 0)
            r.scales[row * ((dim + 31) >> 5) + (col >> 5)] = finite ? (uint8_t)(e + 127) : (uint8_t)255;
        uint8_t* p = r.codes + row * (int64_t)dim + col;
        if (col + 8 <= dim) {
            stream_at<1>(p, c);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < dim) p[j] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// Eight floats of a parameter row (fp32 [groups][dim]), zeros from dim on.
__device__ __forceinline__ void load_param(const float* p, int g, int col, int dim, float* v) {
    const RowsIn r = {p, nullptr, dim, 0};
    Raw8<kSrcF32> raw;
    load8(r, g, col, dim, raw);
    unpack8(r, raw, v);
}

// -------------------------------------------------------------- gates ----
// exp(-x) for x >= 0, within two last places, 0 below 2^-126: 2^h with h the
// product x log2(e) rounded, times 1 + l ln 2 with l what the rounding left.
__device__ __forceinline__ float exp_down(float x) {
    const float y = x > 128.0f ? 128.0f : x;                       // (an infinity less an infinity)
    const float kLog2e = 1.44269502f, kRest = 1.92596299e-8f;      // log2(e) in two parts
    const float h = -y * kLog2e, l = __builtin_fmaf(-y, kRest, __builtin_fmaf(-y, kLog2e, -h));
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, l * 0.693147182f, e);
}

// act(u) and its slope.  The sigmoid s and t = 1 - s come from exp(-|u|), which
// does not overflow, and neither is a difference: 1 - s would have no digits
// left of the slope s t of an open gate (none at all from u = 17 on).  The
// reciprocal is refined by one step to fp32's last place or so; a division
// costs ten instructions.
__device__ __forceinline__ float gate_act(float u, int act, float& slope) {
    if (act == HTL_ACT_NONE) {
        slope = 1.0f;
        return u;
    }
    const float e = exp_down(fabsf(u)), d = 1.0f + e, q0 = __builtin_amdgcn_rcpf(d);
    const float q = __builtin_fmaf(q0, __builtin_fmaf(-d, q0, 1.0f), q0), eq = e * q;
    const float s = u < 0.0f ? eq : q, t = u < 0.0f ? q : eq;
    if (act == HTL_ACT_SIGMOID) {
        slope = s * t;
        return s;
    }
    slope = s * (1.0f + u * t);
    return u * s;
}

// ---------------------------------------------------- teams of lanes ----
// Sums over a team of L lanes (L <= 64: aligned lanes of one wave; larger: the
// whole workgroup of L threads, through LDS), the same in every lane.  Two
// places in LDS take turns, so that one barrier a sum is enough: whoever
// writes a place again has passed the barrier of the sum between, and with it
// every wave's reading.
constexpr int kSumWords = 2 * 2 * 16;
struct Sums {
    float* lds;              // kSumWords
    int turn;
};
template <int L, int N> __device__ __forceinline__ void team_sums(float (&v)[N], Sums& s) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = add_moved<kXor2>(add_moved<kXor1>(v[n]));
        if (L >= 8) v[n] = add_moved<kMirror8>(v[n]);
        if (L >= 16) v[n] = add_moved<kMirror16>(v[n]);
        if (L >= 32) v[n] += __shfl_xor(v[n], 16);
        if (L >= 64) v[n] += __shfl_xor(v[n], 32);
    }
    if (L > 64) {
        float* at = s.lds + s.turn * 32;
        s.turn ^= 1;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) at[n * 16 + (threadIdx.x >> 6)] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.0f;
#pragma unroll
            for (int w = 0; w < L / 64; ++w) v[n] += at[n * 16 + w];
        }
    }
}
template <int L> __device__ __forceinline__ float team_sum(float v, Sums& s) {
    float a[1] = {v};
    team_sums<L>(a, s);
    return a[0];
}

// How a row is held: L lanes with I groups of eight elements each, so a row of
// up to 8 * L * I elements stays in registers between the statistics and the
// result, and is read once.  Up to 64 lanes a workgroup holds several rows.
template <int L_, int I_> struct Hold {
    static constexpr int L = L_, I = I_;
    static constexpr int kThreads = L_ > 64 ? L_ : 256;
    static constexpr int kTeams = kThreads / L_;
    // A workgroup that is one team waits at barriers, and few such fit: the
    // next row's loads run ahead.  Waves that hold rows of their own hide one
    // another's waiting better than they could with the registers for that
    // (norm_rows_backward of 1.7M rows of 128, when it took 441 us without: 517).
    static constexpr bool kAhead = L_ > 64;
    static constexpr int kGrid = kAhead ? 524288 / kThreads : 1 << 20;   // workgroups of a launch at most
    static constexpr int kChunks = kAhead ? 262144 / kThreads : 2048;    // chunks of rows, about
};
// Calls f with the smallest Hold for a row of dim elements (<= kMaxNormDim).
template <class F> void with_hold(int dim, F&& f) {
    if (dim <= 32) f(Hold<4, 1>());
    else if (dim <= 64) f(Hold<8, 1>());
    else if (dim <= 128) f(Hold<16, 1>());
    else if (dim <= 256) f(Hold<32, 1>());
    else if (dim <= 512) f(Hold<64, 1>());
    else if (dim <= 1024) f(Hold<64, 2>());
    else if (dim <= 2048) f(Hold<256, 1>());
    else if (dim <= 4096) f(Hold<512, 1>());
    else if (dim <= 8192) f(Hold<1024, 1>());
    else f(Hold<1024, 2>());
}

// 1 / deviation and, in v, the centred and scaled row: v <- (v - [mean]) * r.
// The mean is taken out before the squares are summed, so a row far from zero
// keeps its deviation.  The mean itself is off by the rounding of its sum,
// which is in units of the row's distance from zero: at 10,000 it would be
// 1e-3, beside deviations as small as that.  So what is left of it after the
// first subtraction is summed with the squares and taken out too:
//   c = x - mean,  v = c - mean(c),  var = mean(c^2) - mean(c)^2.
template <class H>
__device__ __forceinline__ float normalize(float v[][8], bool center, int tl, int dim, float eps, Sums& sums) {
    float var, rest = 0.0f;
    if (center) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < H::I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        const float mean = team_sum<H::L>(s, sums) / (float)dim;   // divided: exact for a constant row of few bits
        float cq[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = (i * H::L + tl) * 8;
            const float mid = col < dim ? mean : 0.0f;             // columns past the row stay zeros
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] -= mid;
            if (dim % 8 != 0 && col + 8 > dim) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j >= dim) v[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cq[0] += v[i][j];
                cq[1] += v[i][j] * v[i][j];
            }
        }
        team_sums<H::L>(cq, sums);
        const float inv_dim = 1.0f / (float)dim;                   // (the same for every row)
        rest = cq[0] * inv_dim;
        var = __builtin_fmaf(-rest, rest, cq[1] * inv_dim);        // (an infinite sum of squares stays one)
        var = var < 0.0f ? 0.0f : var;
    } else {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < H::I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) q += v[i][j] * v[i][j];
        var = team_sum<H::L>(q, sums) / (float)dim;
    }
    const float r = 1.0f / sqrtf(var + eps), shift = rest != 0.0f ? -rest * r : -0.0f;   // (r may be infinite)
#pragma unroll
    for (int i = 0; i < H::I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j], r, shift);
    return r;
}

// Column sums of a workgroup's teams, written to dst[dim] (the partial row of
// a chunk, or the group's result): lanes of a wave that hold the same columns
// first, then the waves through s_col (kThreads / 64 rows of 8 * L * I
// floats; none needed when one team fills the workgroup).
template <class H>
__device__ __forceinline__ void write_columns(float acc[][8], int tl, int dim, float* s_col, float* dst) {
    constexpr int kWaves = H::kThreads / 64;
    if (H::L <= 64) {
#pragma unroll
        for (int i = 0; i < H::I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int off = H::L; off < 64; off <<= 1) acc[i][j] += __shfl_xor(acc[i][j], off);
        const int w = threadIdx.x >> 6;
        __syncthreads();                 // s_col may still be read from the call before
        if ((threadIdx.x & 63) < H::L)
#pragma unroll
            for (int i = 0; i < H::I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s_col[(w * H::I * H::L + i * H::L + tl) * 8 + j] = acc[i][j];
        __syncthreads();
        for (int d = threadIdx.x; d < dim; d += H::kThreads) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) s += s_col[q * H::I * H::L * 8 + d];
            dst[d] = s;
        }
    } else {
        const RowsOut o = {dst, 0};
#pragma unroll
        for (int i = 0; i < H::I; ++i) store8<kSrcF32>(o, 0, (i * H::L + tl) * 8, dim, acc[i]);
    }
}

// ------------------------------------------------- rows of a group ----
// Position range [beg, end) of group g: offsets clamped into [0, m] and to a
// non-negative length, so offsets that break the CSR rules read no row
// outside the m given.
__device__ __forceinline__ void group_range(const int32_t* offsets, int n_groups, int64_t m, int g, int64_t& beg,
                                            int64_t& end) {
    if (!offsets) {
        beg = 0;
        end = m;
        return;
    }
    const int64_t a = offsets[g], b = g < n_groups ? (int64_t)offsets[g + 1] : m;
    beg = a < 0 ? 0 : (a > m ? m : a);
    end = b < beg ? beg : (b > m ? m : b);
}

// Work item `item` of the chunks of at most R positions that the groups are
// cut into, group by group, each group with at least min_chunks (0 or 1);
// the rows of no group follow as group n_groups.  count: chunks of the group.
// All lanes of a wave call it together with the same arguments.  Returns
// false past the last chunk.
//
// A group of one chunk writes its sums itself; the chunks of the others leave
// partial sums, and slots number those chunks alone (split_chunks bounds
// them), so that partial sums take room by the rows, however many groups
// there are.
struct Chunk {
    int g;
    int64_t beg, end;
    int index, count;       // which of the group's chunks
    int64_t slot;           // of its partial sums, where count > 1
};
// Chunks of groups that have several, at most: such a group has more than R
// rows, so there are at most m / R of them, each with one chunk that is not full.
inline int64_t split_chunks(int64_t m, int n_groups, int64_t R) {
    const int64_t full = m / R;
    return full + (n_groups < full ? n_groups : full);
}
__device__ __forceinline__ bool find_chunk(const int32_t* offsets, int n_groups, int64_t m, uint32_t R, int min_chunks,
                                           int64_t item, Chunk& c) {
    const int lane = __lane_id();
    int64_t run = 0, alone = 0;          // chunks before, and those that are their group's only one
    for (int g0 = 0; g0 <= n_groups; g0 += 64) {
        const int g = g0 + lane;
        int64_t beg = 0, end = 0;
        int cnt = 0;
        if (g < n_groups || (g == n_groups && offsets)) {
            group_range(offsets, n_groups, m, g, beg, end);
            cnt = (int)(((uint32_t)(end - beg) + R - 1u) / R);
            if (g < n_groups && cnt < min_chunks) cnt = min_chunks;
        }
        int incl = cnt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int y = __shfl_up(incl, off);
            if (lane >= off) incl += y;
        }
        const uint64_t past = __ballot(run + incl > item), one = __ballot(cnt == 1);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            c.slot = item - alone - __popcll(one & ((1ull << l) - 1));
            c.g = g0 + l;
            c.count = __shfl(cnt, l);
            c.index = (int)(item - run) - (__shfl(incl, l) - c.count);
            const int64_t b = (int64_t)__shfl((int)beg, l), e = (int64_t)__shfl((int)end, l);
            c.beg = b + (int64_t)c.index * R;
            c.end = c.beg + R < e ? c.beg + R : e;
            return true;
        }
        run += __shfl(incl, 63);
        alone += __popcll(one);
    }
    return false;
}

// The slot of group g's first chunk and how many it has, as find_chunk numbers them.
__device__ __forceinline__ void chunks_of_group(const int32_t* offsets, int n_groups, int64_t m, uint32_t R,
                                                int min_chunks, int g, int64_t& first, int& count) {
    const int lane = __lane_id();
    int64_t sum = 0;
    for (int q = lane; q < g; q += 64) {
        int64_t beg, end;
        group_range(offsets, n_groups, m, q, beg, end);
        const int c = (int)(((uint32_t)(end - beg) + R - 1u) / R);
        sum += c > 1 ? c : 0;
    }
    int s = (int)sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off);
    first = s;
    int64_t beg, end;
    group_range(offsets, n_groups, m, g, beg, end);
    count = (int)(((uint32_t)(end - beg) + R - 1u) / R);
    if (count < min_chunks) count = min_chunks;
}

// Sums of a group's partial rows: out[g][d] = sum over its chunks of
// partial[slot][d], for the groups with more than one chunk (a lone chunk
// writes its sums itself).  Chunks are added in order, so the result does
// not depend on which workgroup ended first.  limit: rows that partial holds;
// a second set of sums (out2, nullable) has its partial rows after those.
// out is fp32, or with bf16 (and no second set) rounded.
htl_status sum_chunks(const float* partial, int64_t limit, void* out, float* out2, const int32_t* offsets,
                      int n_groups, int64_t m, uint32_t R, int64_t width, hipStream_t stream, bool bf16 = false);

}  // namespace htl
