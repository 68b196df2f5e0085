// Losses of a softmax over a whole vocabulary, which never hold the scores of
// a row with all of it, and their gradients.
//
//   s_iv = x_i w_v / T                  (x [m][k], w [vocab][k], T the temperature)
//   lse_i = log sum_v exp(s_iv)
//   loss_i = lse_i - s_i,target         (softmax_loss)
//   p_i = softmax over a teacher's listed items of its logits / T
//   loss_i = lse_i + sum_j p_ij (log p_ij - s_i,item j)       (distill_loss)
//   d_iv = (exp(s_iv - lse_i) - p_iv) dloss_i / T             (p 1 at the target)
//   dx_i = sum_v d_iv w_v,   dw_v = sum_i d_iv x_i
//
// Forward: tiles of the product x w^T whose end leaves, for each row and each
// of its waves' columns, the largest score and the sum of exponentials below
// it; a second kernel joins these.  Backward: pieces of the vocabulary, each
// three products: the scores again, their end writing d in the rows' type (an
// operand of the matrix instructions that follow: bf16 costs each term half a
// step, 2^-8), then dx += d w and dw = d^T x.
//
// Bound: products.  Measured: 8,192 bf16 rows of 2,048 (one in twenty without a
// target) against 131,072 items: forward 3.60 ms (1,180 TFLOP/s with its end, where the
// library's product of such sizes alone reaches 1,198), a piece of 16,384 items 541
// us for d, 426 for dx and 409 for dw (1,251 and 1,278 TFLOP/s).  16,384 fp32 rows of 128
// against 65,536: forward 2.60 ms (106 TFLOP/s of 154), a piece of 8,192 items 376, 294
// and 287 us.  16 rows of 1,024 against 65,536: 26 us (134 MB: 5.1 TB/s).
#include "few.h"
#include "wide.h"

namespace htl {
namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// Indices of items, int32 or int64; -1 for one outside the vocabulary.
struct Items {
    const void* p;
    bool wide;
    int vocab;
    __device__ __forceinline__ int at(int64_t i) const {
        const int64_t v = wide ? ((const int64_t*)p)[i] : (int64_t)((const int32_t*)p)[i];
        return v >= 0 && v < vocab ? (int)v : -1;
    }
};

// Of some products x w: the largest, and the sum of 2^((product - largest) unit), unit = log2(e) / T.  The
// largest is taken off before anything is multiplied: an item far above the rest has a sum of exactly 1, and its
// score rounds once on its way to lse, as the target's does, so that no loss is below 0.
struct Best {
    float top, sum;
};
__device__ __forceinline__ Best join(const Best& a, const Best& b, float unit) {
    const float top = fmaxf(a.top, b.top), at = top == -INFINITY ? 0.0f : top;
    return {top, a.sum * __builtin_amdgcn_exp2f((a.top - at) * unit) + b.sum * __builtin_amdgcn_exp2f((b.top - at) * unit)};
}
// log2 of a score's share, s - lse with s rounded as lse has it (kept in one rounding, an item far above the
// rest would be off its share of 1 by the rounding of its score).
__device__ __forceinline__ float log2_share(float product, float scale, float lse) {
#pragma clang fp contract(off)
    return (product * scale - lse) * kLog2e;
}

// Forward end: partial[block][row] of each wave's columns, and the target's score.
template <class C> struct ScoreEnd {
    static constexpr bool kPairs = false;
    int64_t m;
    int cols, v0, block0;    // columns of this piece, its first item and its first block
    float scale;             // 1 / T
    Best* partial;           // [blocks][m]
    Items targets;           // p null: none
    float* target_score;     // [m]
    __device__ __forceinline__ void operator()(const TileAt&, bool grouped, int, int64_t row, int col, f32x4 (&v)[C::TC]) const {
        if (!grouped) return;
        constexpr int W = C::TC * 16;
        const int q = __lane_id() >> 4;
        const float unit = scale * kLog2e;
        if (col + W > cols) {
#pragma unroll
            for (int i = 0; i < C::TC; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + i * 16 + q * 4 + e >= cols) v[i][e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, v[i][e]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float at = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f((v[i][e] - at) * unit);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (row < 0) return;
        if (q == 0) partial[(int64_t)(block0 + col / W) * m + row] = {top, sum};
        if (targets.p) {
            const int t = targets.at(row) - v0 - col;
            if ((uint32_t)t < (uint32_t)W) {
#pragma unroll
                for (int i = 0; i < C::TC; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i * 16 + q * 4 + e == t) target_score[row] = v[i][e] * scale;
            }
        }
    }
};

// Backward end: d of a piece's columns, rows of the rows' type `ld` apart, by
// row or (packed) by position in the plan.
template <class C> struct SlopeEnd {
    static constexpr bool kPairs = false;
    int cols, v0;
    int64_t ld;
    float scale;
    const float* lse;
    const float* dloss;
    Items targets;           // p null: none (a teacher's items are put in afterwards)
    void* d;
    bool f32, packed;
    __device__ __forceinline__ void operator()(const TileAt& t, bool grouped, int r, int64_t row, int col,
                                               f32x4 (&v)[C::TC]) const {
        if (!grouped) return;
        constexpr int W = C::TC * 16;
        const int q = __lane_id() >> 4;
        const float l = row < 0 ? 0.0f : lse[row], g = row < 0 ? 0.0f : dloss[row] * scale;
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = __builtin_amdgcn_exp2f(log2_share(v[i][e], scale, l));
        if (targets.p && row >= 0) {
            const int at_target = targets.at(row) - v0 - col;
            if ((uint32_t)at_target < (uint32_t)W) {
#pragma unroll
                for (int i = 0; i < C::TC; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i * 16 + q * 4 + e == at_target) v[i][e] -= 1.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < C::TC; ++i) v[i] *= g;
        store_rows<C::TC>(d, f32, !packed ? row : t.beg + r < t.end ? t.beg + r : -1, ld, col, cols, v);
    }
};

template <int T, class C, bool ASYNC, class End>
__global__ __launch_bounds__(C::kThreads, 2) void k_scores(ProdArgs p, End end) {
    product_tiles<T, kFwd, C, ASYNC>(p, end);
}

template <int T, int KS, class C, class End> __global__ __launch_bounds__(kFewThreads) void k_scores_few(ProdArgs p, End end) {
    few_tiles<T, KS, C>(p, end);
}
template <class End>
__global__ __launch_bounds__(256, 1) void k_scores_wide(ProdArgs p, End end) {
    wide_tiles<kFwd>(p, end);
}

// A row's partial sums joined by the workgroup, the same in every thread.
__device__ __forceinline__ Best row_best(const Best* partial, int blocks, int64_t m, int64_t row, float unit, Best* s) {
    Best b = {-INFINITY, 0.0f};
#pragma unroll 4
    for (int i = threadIdx.x; i < blocks; i += 256) b = join(b, partial[(int64_t)i * m + row], unit);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) b = join(b, {__shfl_xor(b.top, off), __shfl_xor(b.sum, off)}, unit);
    __syncthreads();                                     // (the row before is read)
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = b;
    __syncthreads();
    return join(join(s[0], s[1], unit), join(s[2], s[3], unit), unit);
}
__device__ __forceinline__ float lse_of(const Best& b, float scale) {
    return __builtin_fmaf(b.top, scale, __builtin_amdgcn_logf(b.sum) * kLn2);
}

// lse of rows from their partial sums, and the losses: a row a workgroup, or
// (many rows: whole lines of partial sums are read) 16.
__global__ __launch_bounds__(256) void k_softmax_finish(const Best* __restrict__ partial, int blocks, int64_t m,
                                                        float scale, Items targets,
                                                        const float* __restrict__ target_score,
                                                        float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ Best s[4];
    const int64_t row = blockIdx.x;
    const bool on = targets.at(row) >= 0;                // (the same for the workgroup)
    const float l = on ? lse_of(row_best(partial, blocks, m, row, scale * kLog2e, s), scale) : 0.0f;
    if (threadIdx.x) return;
    lse[row] = l;
    loss[row] = on ? l - target_score[row] : 0.0f;
}
__global__ __launch_bounds__(256) void k_softmax_finish16(const Best* __restrict__ partial, int blocks, int64_t m,
                                                          float scale, Items targets,
                                                          const float* __restrict__ target_score,
                                                          float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ Best s[16][16];
    const int r = threadIdx.x & 15, part = threadIdx.x >> 4;
    for (int64_t row0 = blockIdx.x * 16ll; row0 < m; row0 += gridDim.x * 16ll) {
        const int64_t row = row0 + r;
        const bool on = row < m && targets.at(row) >= 0;
        Best b = {-INFINITY, 0.0f};
        if (on) {
#pragma unroll 4
            for (int i = part; i < blocks; i += 16) b = join(b, partial[(int64_t)i * m + row], scale * kLog2e);
        }
        __syncthreads();                                 // the rows before are read
        s[part][r] = b;
        __syncthreads();
        if (part || row >= m) continue;
        for (int i = 1; i < 16; ++i) b = join(b, s[i][r], scale * kLog2e);
        const float l = on ? lse_of(b, scale) : 0.0f;
        lse[row] = l;
        loss[row] = on ? l - target_score[row] : 0.0f;
    }
}

// A wave's dot products of row i with two rows, the same in every lane.
template <int T>
__device__ __forceinline__ void row_dots(const RowsIn& a, int64_t i, const RowsIn& b, const int64_t (&j)[2], int k, float (&s)[2]) {
    s[0] = s[1] = 0.0f;
    for (int c = __lane_id() * 8; c < k; c += 512) {
        Raw8<T> ra, rb[2];
        float va[8], vb[8];
        load8(a, i, c, k, ra);
        load8(b, j[0], c, k, rb[0]);
        load8(b, j[1], c, k, rb[1]);
        unpack8(a, ra, va);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unpack8(b, rb[h], vb);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[h] = __builtin_fmaf(va[e], vb[e], s[h]);
        }
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        s[0] += __shfl_xor(s[0], off);
        s[1] += __shfl_xor(s[1], off);
    }
}

struct Teacher {
    Items items;
    const void* logits;
    int64_t ld;              // of logits' rows
    bool f32;
    int top;
    float scale;             // 1 / T
    // -inf for an entry that is not there
    __device__ __forceinline__ float logit(int64_t row, int j) const {
        if (items.at(row * top + j) < 0) return -INFINITY;
        return f32 ? ((const float*)logits)[row * ld + j] : bf16_lo(((const uint16_t*)logits)[row * ld + j]);
    }
};
// A row's shares: log2 of an entry's is (logit - top) unit - log.  (The largest logit is taken off before
// anything is multiplied: lists of the type's lowest value keep their equal shares.)
struct Shares {
    float top, unit, log;
    __device__ __forceinline__ float log2_of(float logit) const { return __builtin_fmaf(logit - top, unit, -log); }
};
// Found by one wave; false where no entry is there.
__device__ __forceinline__ bool teacher_sum(const Teacher& t, int64_t row, Shares& all) {
    float top = -INFINITY;
    for (int j = __lane_id(); j < t.top; j += 64) {
        const float v = t.logit(row, j);
        top = v != v ? INFINITY : fmaxf(top, v);             // (a NaN makes the sum one)
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (top == -INFINITY) return false;
    const float unit = t.scale * kLog2e;
    float s = 0.0f;
    for (int j = __lane_id(); j < t.top; j += 64) s += __builtin_amdgcn_exp2f((t.logit(row, j) - top) * unit);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off);
    all = {top, unit, __builtin_amdgcn_logf(s)};
    return true;
}

// The scores of a teacher's items, lse and the loss: a row a workgroup.
template <int T>
__global__ __launch_bounds__(256) void k_distill_finish(RowsIn x, RowsIn w, int k, const Best* __restrict__ partial,
                                                        int blocks, int64_t m, Teacher t, float* __restrict__ scores,
                                                        float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ Best s[4];
    __shared__ float s_score[HTL_MAX_TOP];
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        Shares all;
        const bool on = teacher_sum(t, row, all);        // (every wave finds the same)
        __syncthreads();                                 // the scores before are read
        for (int j = (threadIdx.x >> 6) * 2; j < t.top; j += 8) {
            const int v[2] = {t.items.at(row * t.top + j), j + 1 < t.top ? t.items.at(row * t.top + j + 1) : -1};
            float d[2] = {0.0f, 0.0f};
            if (on && (v[0] >= 0 || v[1] >= 0)) {
                const int64_t at[2] = {v[0] < 0 ? v[1] : v[0], v[1] < 0 ? v[0] : v[1]};
                row_dots<T>(x, row, w, at, k, d);
            }
            if (__lane_id() < 2 && j + __lane_id() < t.top) {
                const float dot = __lane_id() ? d[1] : d[0];
                const float score = (__lane_id() ? v[1] : v[0]) < 0 ? 0.0f : dot * t.scale;
                scores[row * t.top + j + __lane_id()] = score;
                s_score[j + __lane_id()] = score;
            }
        }
        if (!on) {
            if (threadIdx.x == 0) loss[row] = lse[row] = 0.0f;
            continue;
        }
        const float l = lse_of(row_best(partial, blocks, m, row, t.scale * kLog2e, s), t.scale);
        if (threadIdx.x >= 64) continue;
        float sum = 0.0f;
        for (int j = threadIdx.x; j < t.top; j += 64) {
            const float logp = all.log2_of(t.logit(row, j));
            if (logp > -INFINITY || logp != logp)        // an entry of share 0 adds nothing
                sum += __builtin_amdgcn_exp2f(logp) * (logp * kLn2 + (l - s_score[j]));
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
        if (threadIdx.x) continue;
        loss[row] = sum;
        lse[row] = l;
    }
}

// Which rows take part (0, or -1: none), and, of a teacher's entries, d: an
// item listed twice has the shares of both in each.  A wave a row, which compares all
// pairs of its list: little for lists of 64, not for long ones (4,096 bf16 rows of 512
// against 65,536 items, step: 1.55 ms with 64 or 128 entries, 1.76, 2.29 and 4.01 with
// 256, 512 and 1,024, whose scores are part of that too).
__global__ __launch_bounds__(256) void k_active(int64_t m, Items targets, int32_t* __restrict__ ids) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m; i += gridDim.x * 256ll) ids[i] = targets.at(i) >= 0 ? 0 : -1;
}
__global__ __launch_bounds__(256) void k_teach(int64_t m, Teacher t, const float* __restrict__ scores,
                                               const float* __restrict__ lse, const float* __restrict__ dloss,
                                               int32_t* __restrict__ ids, float* __restrict__ d) {
    for (int64_t row = blockIdx.x * 4ll + (threadIdx.x >> 6); row < m; row += gridDim.x * 4ll) {
        Shares all;
        const bool on = teacher_sum(t, row, all);
        if (__lane_id() == 0) ids[row] = on ? 0 : -1;
        if (!on) continue;
        const float g = dloss[row] * t.scale, l = lse[row];
        for (int j0 = 0; j0 < t.top; j0 += 64) {
            const int j = j0 + __lane_id();
            const int item = j < t.top ? t.items.at(row * t.top + j) : -1;
            float share = 0.0f;
            for (int i0 = 0; i0 < t.top; i0 += 64) {
                const int i = i0 + __lane_id();
                const int other = i < t.top ? t.items.at(row * t.top + i) : -1;
                const float p = other >= 0 ? __builtin_amdgcn_exp2f(all.log2_of(t.logit(row, i))) : 0.0f;
                const int count = t.top - i0 < 64 ? t.top - i0 : 64;
                for (int n = 0; n < count; ++n) {
                    const int it = __shfl(other, n);
                    const float pn = __shfl(p, n);
                    if (it == item) share += pn;
                }
            }
            if (item >= 0)
                d[row * t.top + j] = (__builtin_amdgcn_exp2f((scores[row * t.top + j] - l) * kLog2e) - share) * g;
        }
    }
}
// Which rows a teacher has entries for.
__global__ __launch_bounds__(256) void k_taught(int64_t m, Teacher t, int32_t* __restrict__ ids) {
    for (int64_t row = blockIdx.x * 4ll + (threadIdx.x >> 6); row < m; row += gridDim.x * 4ll) {
        bool on = false;
        for (int j = __lane_id(); j < t.top; j += 64) on |= t.logit(row, j) != -INFINITY;
        const bool any = __ballot(on) != 0;
        if (__lane_id() == 0) ids[row] = any ? 0 : -1;
    }
}
// Puts the teacher's entries of a piece of the vocabulary into d, of which rows
// lie by row or (packed) by position.
template <int T>
__global__ __launch_bounds__(256) void k_put_items(int64_t m, Items items, int top, const int32_t* __restrict__ order,
                                                   const int32_t* __restrict__ offsets, bool packed,
                                                   const float* __restrict__ entries, int v0, int cols, int64_t ld,
                                                   void* __restrict__ d) {
    const int64_t all = (int64_t)offsets[1] * top;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int64_t pos = i / top, row = order[pos], at = row * top + (i - pos * top), to = packed ? pos : row;
        const int item = items.at(at), c = item - v0;
        if (item < 0 || (uint32_t)c >= (uint32_t)cols) continue;
        if (T == kSrcF32) ((float*)d)[to * ld + c] = entries[at];
        else ((uint16_t*)d)[to * ld + c] = (uint16_t)f32_to_bf16_bits(entries[at]);
    }
}

// ------------------------------------------------------------ launches ----
struct Rows2 {               // x and w as the calls have them
    const void* x;
    const void* w;
    int64_t ldx, ldw, m;
    int vocab, k;
    htl_dtype dtype;
};

// The product x w^T of `cols` items (r.w: the first one's row), with an end made
// by `make` for the tile's shape.  Tiles by size, as the plain products' (product.hip).
constexpr int64_t kFewRows = 48;
// Tiles of 32 rows rather than 128: for few rows, and where those of 128 would
// leave units idle (2,838 fp32 rows of 1,115 against 893: 161 of them).
bool narrow_of(int64_t m, int vocab, htl_dtype dtype) {
    return m <= kFewRows || ceil_div(m, 32) * ceil_div(vocab, 128) <= (dtype == HTL_F32 ? 1024 : 512);
}
int tile_of(const Rows2& r, int64_t cols, bool& fast) {
    const int es = elem(r.dtype);
    fast = r.ldx * es % 16 == 0 && r.ldw * es % 16 == 0 && (int64_t)r.k * es % 16 == 0 && aligned(r.x, 16) &&
           aligned(r.w, 16) && r.m * r.ldx * es <= kBufferBytes && cols * r.ldw * es <= kBufferBytes;
    return narrow_of(r.m, r.vocab, r.dtype) ? 32 : 128;
}
// Scores of rows shorter than this run as well or better in tiles of 128, of which
// two fill a unit and one's end passes under the other's products (4,096 rows
// against 65,536, step: 801 and 830 us of 128 elements, 953 and 967 of 256, but 1,639
// and 1,448 of 504).
constexpr int kWideK = 384;
// Whether wide.h's tiles fill the device.
bool wide_of(int64_t m, int vocab, htl_dtype dtype) {
    return dtype == HTL_BF16 && m >= 256 && ceil_div(m, 256) * ceil_div(vocab, 256) >= 224;
}
// A wave's columns: those of a block of partial sums.
int wave_cols(int64_t m, int vocab, htl_dtype dtype, bool wide) {
    return wide ? Wide::TC * 16 : narrow_of(m, vocab, dtype) ? Small::TC * 16 : Mid::TC * 16;
}

template <class Make>
void launch_scores(const Rows2& r, int tile, bool fast, int cols, const int32_t* order, const int32_t* offsets, Make make,
                   hipStream_t s, bool packed = false) {
    ProdArgs p = {r.x, r.w, nullptr, order, offsets, r.m, r.ldx, r.ldw, r.ldw, cols, r.k, 1, (uint32_t)tile, nullptr, 0, 0};
    p.packed = packed;
    p.no_rest = offsets != nullptr;
    auto few = [&](auto t, auto shape) {                 // (tile: rows)
        constexpr int T = decltype(t)::value;
        using C = decltype(shape);
        const auto end = make(shape);
        with_splits(few_splits(ceil_div(cols, 32), (int64_t)r.k * (T == kSrcF32 ? 4 : 2)), [&](auto splits) {
            constexpr int KS = decltype(splits)::value;
            const dim3 grid(grid_for(align_up((size_t)((r.m / C::BR + 2) * ceil_div(cols, 32 * few_waves<KS>)), kXcds), 1));
            hipLaunchKernelGGL((k_scores_few<T, KS, C, decltype(end)>), grid, dim3(kFewThreads), 0, s, p, end);
        });
    };
    auto go = [&](auto t, auto shape, auto async) {
        using C = decltype(shape);
        const auto end = make(shape);
        const dim3 grid(grid_for(align_up((size_t)((r.m / tile + 2) * ceil_div(cols, C::BC)), kXcds), 1));
        hipLaunchKernelGGL((k_scores<decltype(t)::value, C, decltype(async)::value, decltype(end)>), grid,
                           dim3(C::kThreads), 0, s, p, end);
    };
    using F32 = std::integral_constant<int, kSrcF32>;
    using B16 = std::integral_constant<int, kSrcBf16>;
    using Yes = std::true_type;
    using No = std::false_type;
    if (r.m <= 32) {
        if (r.dtype == HTL_BF16) r.m <= 16 ? few(B16(), Few<1>()) : few(B16(), Few<2>());
        else r.m <= 16 ? few(F32(), Few<1>()) : few(F32(), Few<2>());
        return;
    }
    if (r.dtype == HTL_BF16) {
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
}

// Items whose matrix rows span less than 4 GiB (buffer offsets have 32 bits).
int most_cols(const Rows2& r) {
    const int64_t c = (kBufferBytes / (r.ldw * elem(r.dtype))) & ~255ll;
    return (int)(c < 256 ? 256 : c > (1 << 30) ? 1 << 30 : c);
}

struct Carve {               // a workspace cut into 256-byte aligned parts
    char* p;
    size_t at;
    template <class V> V* take(int64_t count) {
        V* v = (V*)(p + at);
        at += align_up((size_t)count * sizeof(V) + 1, 256);
        return p ? v : nullptr;
    }
};

// Whether tiles take copies of x and w, whose rows whole 16-byte pieces make up,
// where theirs do not: loads then go straight to LDS.
bool copied_of(int64_t m, int k, htl_dtype dtype) { return m > kFewRows && k % (dtype == HTL_F32 ? 4 : 8); }

// Items whose copied matrix rows are held at a time (128 MiB), and of a piece at most.
constexpr int kMostCols = 65536;
int pack_cols(int vocab, int k, htl_dtype dtype) {
    int64_t c = (128ll << 20) / (packed_ld(k) * elem(dtype)) / 256 * 256;
    c = c < 256 ? 256 : c > kMostCols ? kMostCols : c;
    return (int)(c < vocab ? c : vocab);
}

struct ForwardSpace {
    bool wide, copied;
    Best* partial;
    float* target_score;
    int32_t *ids, *order, *offsets;
    void* groups;
    size_t group_bytes;
    char *x, *w;
    size_t bytes;
    ForwardSpace(void* ws, int64_t m, int vocab, int k, htl_dtype dtype) {
        wide = wide_of(m, vocab, dtype) && k >= kWideK;
        Carve c = {(char*)ws, 0};
        partial = c.take<Best>(m * ceil_div(vocab, wave_cols(m, vocab, dtype, wide)));
        target_score = c.take<float>(m);
        ids = c.take<int32_t>(wide ? m : 0);
        order = c.take<int32_t>(wide ? m : 0);
        offsets = c.take<int32_t>(2);
        group_bytes = wide ? row_groups_workspace_bytes(m, 1) : 0;
        groups = c.take<char>(group_bytes);
        copied = copied_of(m, k, dtype);
        x = c.take<char>(wide || copied ? m * spread_ld(k) * elem(dtype) : 0);
        w = c.take<char>(wide || copied ? pack_cols(vocab, k, dtype) * packed_ld(k) * elem(dtype) : 0);
        bytes = c.at;
    }
};

// Gradients of scores held at a time: columns of a piece of the vocabulary.  Short
// rows make little work of a piece, and longer pieces leave fewer partial sums:
// 16,384 fp32 rows of 128 against 65,536, step: 12.4, 10.9, 10.3 and 10.0 ms with
// 128, 256, 512 and 1,024 MiB; 4,096 rows of 2,048 against 131,072, step: 7.4, 7.5,
// 7.9 and 7.8 ms.  The matrix rows of a piece span less than 4 GiB (offsets have 32 bits).
int piece_cols(int64_t m, int vocab, int k, htl_dtype dtype) {
    int64_t c = ((k < 1024 ? 512ll : 256ll) << 20) / (elem(dtype) * (m < 1 ? 1 : m)) / 256 * 256;
    const int64_t most = kBufferBytes / (packed_ld(k) * elem(dtype)) / 256 * 256;
    if (c < 256) c = 256;
    if (c > kMostCols) c = kMostCols;
    if (c > most) c = most;
    return (int)(c < vocab ? c : vocab);
}

struct BackwardSpace {
    bool wide, copied;
    int step, splits;        // columns of a piece, parts of dx's sums
    int32_t *ids, *order, *offsets;
    void* groups;
    size_t group_bytes;
    float *entries, *parts;
    char *d, *sums, *x, *w;
    size_t bytes;
    BackwardSpace(void* ws, int64_t m, int vocab, int k, int top, htl_dtype dtype) {
        wide = wide_of(m, vocab, dtype);
        step = piece_cols(m, vocab, k, dtype);
        splits = wide ? wide_dx_splits(m, step, k) : rows_dx_splits(m, step, k);
        Carve c = {(char*)ws, 0};
        ids = c.take<int32_t>(m);
        order = c.take<int32_t>(m);
        offsets = c.take<int32_t>(2);
        group_bytes = row_groups_workspace_bytes(m, 1);
        groups = c.take<char>(group_bytes);
        entries = c.take<float>(m * top);
        parts = c.take<float>(step < vocab || splits > 1 ? splits * m * k : 0);
        d = c.take<char>(m * spread_ld(step) * elem(dtype));
        const int last = vocab % step ? vocab % step : step;
        auto sums_of = [&](int cols) {
            return wide ? wide_dw_bytes(m, 1, cols, k, spread_ld(step), spread_ld(k)) : sums_dw_bytes(m, 1, cols, k);
        };
        const size_t a = sums_of(step), b = sums_of(last);
        sums = c.take<char>(a > b ? a : b);
        copied = copied_of(m, k, dtype);
        x = c.take<char>(wide || copied ? m * spread_ld(k) * elem(dtype) : 0);
        w = c.take<char>(wide || copied ? step * packed_ld(k) * elem(dtype) : 0);
        bytes = c.at;
    }
};

bool sizes_ok(int64_t m, int vocab, int k) {
    return m >= 0 && m <= kMaxRows && vocab >= 1 && vocab <= HTL_MAX_VOCAB && k >= 1 && k <= HTL_MAX_PRODUCT_DIM;
}

// The same in wide.h's tiles; w: the piece's rows.
template <class End>
void launch_wide(const void* x, int64_t ldx, bool packed, const void* w, int64_t ldw, int64_t m, int cols, int k,
                 const int32_t* order, const int32_t* offsets, const End& end, hipStream_t s) {
    const ProdArgs p = {x, w, nullptr, order, offsets, m, ldx, 0, ldw, cols, k, 1, 256, nullptr, 0, 0, packed, true};
    const dim3 grid(wide_grid((m / 256 + 1) * ceil_div(cols, 256)));
    hipLaunchKernelGGL(k_scores_wide<End>, grid, dim3(Wide::kThreads), 0, s, p, end);
}

// A piece of w as an operand of tiles: as it lies, or copied to `room`.
htl_status piece_of(const Rows2& r, int v0, int cols, char* room, const void*& w, int64_t& ldw, hipStream_t stream) {
    w = (const char*)r.w + (int64_t)v0 * r.ldw * elem(r.dtype);
    ldw = r.ldw;
    if (packed_as_is(r.w, r.ldw, r.k, r.dtype) && cols * r.ldw * elem(r.dtype) <= kBufferBytes) return HTL_OK;
    const htl_status st = pack_rows(w, r.ldw, r.dtype, nullptr, cols, cols, r.k, room, packed_ld(r.k), stream);
    w = room;
    ldw = packed_ld(r.k);
    return st;
}

// Partial sums of all scores' exponentials; ids (wide tiles only): which rows take part.
htl_status forward_scores(const Rows2& r, float scale, const ForwardSpace& s, const Items& targets, int& blocks,
                          hipStream_t stream) {
    const int W = wave_cols(r.m, r.vocab, r.dtype, s.wide);
    blocks = (int)ceil_div(r.vocab, W);
    if (s.wide) {
        htl_status st = row_groups(s.ids, r.m, 1, s.order, s.offsets, s.groups, s.group_bytes, stream);
        if (st != HTL_OK) return st;
        const bool as_is = packed_as_is(r.x, r.ldx, r.k) && r.m * r.ldx * 2 <= kBufferBytes;
        if (!as_is) st = pack_rows(r.x, r.ldx, r.dtype, s.order, r.m, r.m, r.k, s.x, spread_ld(r.k), stream);
        const int most = packed_as_is(r.w, r.ldw, r.k) && 256 * r.ldw * 2 <= kBufferBytes ? most_cols(r) : pack_cols(r.vocab, r.k, r.dtype);
        for (int v0 = 0; v0 < r.vocab && st == HTL_OK;) {
            const int cols = r.vocab - v0 < most ? r.vocab - v0 : most;
            const void* w;
            int64_t ldw;
            st = piece_of(r, v0, cols, s.w, w, ldw, stream);
            if (st != HTL_OK) return st;
            const ScoreEnd<Wide> end = {r.m, cols, v0, v0 / W, scale, s.partial, targets, s.target_score};
            launch_wide(as_is ? r.x : s.x, as_is ? r.ldx : spread_ld(r.k), !as_is, w, ldw, r.m, cols, r.k, s.order, s.offsets,
                        end, stream);
            st = check_launch("scores");
            v0 += cols;
        }
        return st;
    }
    Rows2 t = r;                             // operands as the tiles take them
    htl_status st = HTL_OK;
    if (s.copied) {
        st = pack_rows(r.x, r.ldx, r.dtype, nullptr, r.m, r.m, r.k, s.x, spread_ld(r.k), stream);
        t.x = s.x;
        t.ldx = spread_ld(r.k);
        t.k = (int)packed_ld(r.k);
    }
    const int step = s.copied ? pack_cols(r.vocab, r.k, r.dtype) : most_cols(r);
    for (int v0 = 0; v0 < r.vocab && st == HTL_OK;) {
        const int cols = r.vocab - v0 < step ? r.vocab - v0 : step;
        if (s.copied) st = piece_of(r, v0, cols, s.w, t.w, t.ldw, stream);
        else t.w = (const char*)r.w + (int64_t)v0 * r.ldw * elem(r.dtype);
        if (st != HTL_OK) return st;
        bool fast;
        const int tile = tile_of(t, cols, fast);
        launch_scores(t, tile, fast, cols, nullptr, nullptr, [&](auto shape) {
            return ScoreEnd<decltype(shape)>{r.m, cols, v0, v0 / W, scale, s.partial, targets, s.target_score};
        }, stream);
        st = check_launch("scores");
        v0 += cols;
    }
    return st;
}

// All of a backward pass once ids and the teacher's entries stand.
htl_status backward_pieces(const Rows2& r, float scale, const BackwardSpace& s, const Items& targets, const Items& items,
                           int top, const float* lse, const float* dloss, void* dx, htl_dtype dx_dtype, void* dw,
                           hipStream_t stream) {
    const int64_t m = r.m, ld = spread_ld(s.step);
    const int es = elem(r.dtype);
    htl_status st = row_groups(s.ids, m, 1, s.order, s.offsets, s.groups, s.group_bytes, stream);
    if (st == HTL_OK && (s.wide || s.copied)) st = pack_rows(r.x, r.ldx, r.dtype, s.wide ? s.order : nullptr, m, m, r.k, s.x, spread_ld(r.k), stream);
    if (st != HTL_OK) return st;
    Rows2 t = r;                             // operands as the tiles take them
    if (s.wide || s.copied) {
        t.x = s.x;
        t.ldx = spread_ld(r.k);
        t.k = (int)packed_ld(r.k);
    }
    // dx in parts (wide tiles: by position) or whole
    float* parts = s.step < r.vocab || s.splits > 1 ? s.parts : nullptr;
    for (int v0 = 0; v0 < r.vocab;) {
        const int cols = r.vocab - v0 < s.step ? r.vocab - v0 : s.step;
        const void* w = (const char*)r.w + (int64_t)v0 * r.ldw * es;
        int64_t ldw = r.ldw;
        if (s.wide || s.copied) st = piece_of(r, v0, cols, s.w, w, ldw, stream);
        if (st != HTL_OK) return st;
        if (s.wide && r.k >= kWideK) {
            const SlopeEnd<Wide> end = {cols, v0, ld, scale, lse, dloss, targets, s.d, false, true};
            launch_wide(s.x, spread_ld(r.k), true, w, ldw, m, cols, r.k, s.order, s.offsets, end, stream);
        } else {
            t.w = w;
            t.ldw = ldw;
            bool fast;
            const int tile = tile_of(t, cols, fast);
            launch_scores(t, tile, fast, cols, s.order, s.offsets, [&](auto shape) {
                return SlopeEnd<decltype(shape)>{cols, v0, ld, scale, lse, dloss, targets, s.d, r.dtype == HTL_F32, s.wide};
            }, stream, s.wide);
        }
        if (top) {
            const dim3 grid(grid_for(m * top, 256));
            if (r.dtype == HTL_F32)
                hipLaunchKernelGGL(k_put_items<kSrcF32>, grid, dim3(256), 0, stream, m, items, top, s.order, s.offsets, s.wide,
                                   s.entries, v0, cols, ld, s.d);
            else
                hipLaunchKernelGGL(k_put_items<kSrcBf16>, grid, dim3(256), 0, stream, m, items, top, s.order, s.offsets, s.wide,
                                   s.entries, v0, cols, ld, s.d);
        }
        st = check_launch("slopes");
        if (st == HTL_OK) st = zero_behind(s.d, r.dtype, m, cols, ld, stream);
        // rows of d have zeros behind them; those of x and w are copies, or whole pieces
        const bool whole = s.copied || (packed_as_is(r.x, r.ldx, r.k, r.dtype) && packed_as_is(r.w, r.ldw, r.k, r.dtype));
        if (st == HTL_OK && dx) {
            if (s.wide)
                st = wide_dx(s.d, ld, w, ldw, m, cols, r.k, s.order, s.offsets, 1, dx, dx_dtype, parts, s.splits, v0 > 0, stream);
            else
                st = parts ? rows_dx_parts(s.d, ld, w, ldw, r.dtype, m, cols, r.k, s.order, s.offsets, 1, parts, s.splits, v0 > 0, whole, stream)
                           : rows_dx(s.d, ld, w, ldw, r.dtype, m, cols, r.k, s.order, s.offsets, 1, dx, dx_dtype, whole, stream);
        }
        if (st == HTL_OK && dw) {
            char* to = (char*)dw + (int64_t)v0 * r.k * es;
            if (s.wide)
                st = wide_dw(s.d, ld, s.x, spread_ld(r.k), m, cols, r.k, s.offsets, 1, to, r.dtype, s.sums, stream);
            else
                st = sums_dw(s.d, ld, t.x, t.ldx, r.dtype, m, cols, r.k, s.order, s.offsets, 1, to, r.dtype, s.sums, whole, stream);
        }
        if (st != HTL_OK) return st;
        v0 += cols;
    }
    if (!dx) return HTL_OK;
    if (parts) return sum_parts(parts, s.splits, !s.wide, m, r.k, s.order, s.offsets + 1, dx, dx_dtype, stream);
    return s.wide ? zero_rest(dx, (int64_t)r.k * elem(dx_dtype), m, s.order, s.offsets + 1, stream) : HTL_OK;
}

}  // namespace
}  // namespace htl

using namespace htl;

#define SCORE_CHECK(name)                                                                                    \
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, name ": row count out of range");                                   \
    HTL_REQUIRE(vocab >= 1 && vocab <= HTL_MAX_VOCAB, name ": vocabulary size out of range");                \
    HTL_REQUIRE(k >= 1 && k <= HTL_MAX_PRODUCT_DIM, name ": k out of range");                                \
    HTL_REQUIRE(known(dtype), name ": dtype must be HTL_F32 or HTL_BF16");                                   \
    HTL_REQUIRE(ldx >= k && ldw >= k, name ": row stride below k");                                          \
    HTL_REQUIRE(temperature >= 1.0e-30f && temperature <= 1.0e30f, name ": temperature out of range");       \
    HTL_REQUIRE(index_bits == 32 || index_bits == 64, name ": indices have 32 or 64 bits")
#define SCORE_POINTERS(name, index)                                                                          \
    HTL_REQUIRE(w && (m == 0 || (x && index)), name ": null pointer");                                       \
    HTL_REQUIRE(aligned(x, elem(dtype)) && aligned(w, elem(dtype)) && aligned(index, index_bits / 8), name ": misaligned pointer")
#define SCORE_SPACE(name, bytes) \
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= (bytes), name ": workspace too small or misaligned")

extern "C" size_t softmax_loss_workspace_bytes(int64_t m, int vocab, int k, htl_dtype dtype) {
    return sizes_ok(m, vocab, k) && known(dtype) ? ForwardSpace(nullptr, m, vocab, k, dtype).bytes : 0;
}

extern "C" htl_status softmax_loss(const void* x, int64_t ldx, const void* w, int64_t ldw, htl_dtype dtype, int64_t m,
                                   int vocab, int k, const void* targets, int index_bits, float temperature, float* loss,
                                   float* lse, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    SCORE_CHECK("softmax_loss");
    SCORE_POINTERS("softmax_loss", targets);
    HTL_REQUIRE(m == 0 || (loss && lse), "softmax_loss: null pointer");
    HTL_REQUIRE(aligned(loss, 4) && aligned(lse, 4), "softmax_loss: misaligned pointer");
    SCORE_SPACE("softmax_loss", softmax_loss_workspace_bytes(m, vocab, k, dtype));
    if (m == 0) return HTL_OK;
    const Rows2 r = {x, w, ldx, ldw, m, vocab, k, dtype};
    const float scale = 1.0f / temperature;
    const Items t = {targets, index_bits == 64, vocab};
    const ForwardSpace s(ws, m, vocab, k, dtype);
    int blocks;
    if (s.wide) hipLaunchKernelGGL(k_active, dim3(grid_for(m, 256, 1 << 12)), dim3(256), 0, stream, m, t, s.ids);
    const htl_status st = forward_scores(r, scale, s, t, blocks, stream);
    if (st != HTL_OK) return st;
    // 8 rows of 2,048 blocks: 34 us at 16 rows a workgroup
    if (m < 2048)
        hipLaunchKernelGGL(k_softmax_finish, dim3((unsigned)m), dim3(256), 0, stream, s.partial, blocks, m, scale, t, s.target_score,
                           loss, lse);
    else
        hipLaunchKernelGGL(k_softmax_finish16, dim3(grid_for(m, 16)), dim3(256), 0, stream, s.partial, blocks, m, scale, t,
                           s.target_score, loss, lse);
    return check_launch("softmax_loss");
}

extern "C" size_t softmax_loss_backward_workspace_bytes(int64_t m, int vocab, int k, htl_dtype dtype) {
    return sizes_ok(m, vocab, k) && known(dtype) ? BackwardSpace(nullptr, m, vocab, k, 0, dtype).bytes : 0;
}

extern "C" htl_status softmax_loss_backward(const float* dloss, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                            htl_dtype dtype, int64_t m, int vocab, int k, const void* targets,
                                            int index_bits, const float* lse, float temperature, void* dx,
                                            htl_dtype dx_dtype, void* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    SCORE_CHECK("softmax_loss_backward");
    SCORE_POINTERS("softmax_loss_backward", targets);
    HTL_REQUIRE(m == 0 || (dloss && lse), "softmax_loss_backward: null pointer");
    HTL_REQUIRE(known(dx_dtype), "softmax_loss_backward: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(aligned(dloss, 4) && aligned(lse, 4) && aligned(dx, elem(dx_dtype)) && aligned(dw, elem(dtype)),
                "softmax_loss_backward: misaligned pointer");
    SCORE_SPACE("softmax_loss_backward", softmax_loss_backward_workspace_bytes(m, vocab, k, dtype));
    if (!dx && !dw) return HTL_OK;
    const Rows2 r = {x, w, ldx, ldw, m, vocab, k, dtype};
    const Items t = {targets, index_bits == 64, vocab};
    const BackwardSpace s(ws, m, vocab, k, 0, dtype);
    if (m > 0) hipLaunchKernelGGL(k_active, dim3(grid_for(m, 256, 1 << 12)), dim3(256), 0, stream, m, t, s.ids);
    return backward_pieces(r, 1.0f / temperature, s, t, t, 0, lse, dloss, dx, dx_dtype, dw, stream);
}

#define DISTILL_CHECK(name)                                                                                  \
    SCORE_CHECK(name);                                                                                       \
    HTL_REQUIRE(top >= 1 && top <= HTL_MAX_TOP, name ": list length out of range");                          \
    HTL_REQUIRE(ld_logits >= top, name ": row stride below the list's length");                              \
    HTL_REQUIRE(known(logits_dtype), name ": dtype must be HTL_F32 or HTL_BF16");                            \
    SCORE_POINTERS(name, items);                                                                             \
    HTL_REQUIRE(m == 0 || (logits && scores && lse), name ": null pointer");                                 \
    HTL_REQUIRE(aligned(logits, elem(logits_dtype)) && aligned(scores, 4) && aligned(lse, 4), name ": misaligned pointer")

extern "C" htl_status distill_loss(const void* x, int64_t ldx, const void* w, int64_t ldw, htl_dtype dtype, int64_t m,
                                   int vocab, int k, const void* items, int index_bits, const void* logits,
                                   htl_dtype logits_dtype, int64_t ld_logits, int top, float temperature, float* loss,
                                   float* lse, float* scores, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    DISTILL_CHECK("distill_loss");
    HTL_REQUIRE(m == 0 || loss, "distill_loss: null pointer");
    HTL_REQUIRE(aligned(loss, 4), "distill_loss: misaligned pointer");
    SCORE_SPACE("distill_loss", softmax_loss_workspace_bytes(m, vocab, k, dtype));
    if (m == 0) return HTL_OK;
    const Rows2 r = {x, w, ldx, ldw, m, vocab, k, dtype};
    const float scale = 1.0f / temperature;
    const Teacher t = {{items, index_bits == 64, vocab}, logits, ld_logits, logits_dtype == HTL_F32, top, scale};
    const ForwardSpace s(ws, m, vocab, k, dtype);
    int blocks;
    if (s.wide) hipLaunchKernelGGL(k_taught, dim3(grid_for(m, 4)), dim3(256), 0, stream, m, t, s.ids);
    const htl_status st = forward_scores(r, scale, s, Items{nullptr, false, vocab}, blocks, stream);
    if (st != HTL_OK) return st;
    const RowsIn xr = {x, nullptr, ldx, 0}, wr = {w, nullptr, ldw, 0};
    const dim3 grid(grid_for(m, 1));
    if (dtype == HTL_F32)
        hipLaunchKernelGGL(k_distill_finish<kSrcF32>, grid, dim3(256), 0, stream, xr, wr, k, s.partial, blocks, m, t, scores, loss, lse);
    else
        hipLaunchKernelGGL(k_distill_finish<kSrcBf16>, grid, dim3(256), 0, stream, xr, wr, k, s.partial, blocks, m, t, scores, loss, lse);
    return check_launch("distill_loss");
}

extern "C" size_t distill_loss_backward_workspace_bytes(int64_t m, int vocab, int k, int top, htl_dtype dtype) {
    return sizes_ok(m, vocab, k) && known(dtype) && top >= 1 && top <= HTL_MAX_TOP
               ? BackwardSpace(nullptr, m, vocab, k, top, dtype).bytes : 0;
}

extern "C" htl_status distill_loss_backward(const float* dloss, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                            htl_dtype dtype, int64_t m, int vocab, int k, const void* items, int index_bits,
                                            const void* logits, htl_dtype logits_dtype, int64_t ld_logits, int top,
                                            const float* lse, const float* scores, float temperature, void* dx,
                                            htl_dtype dx_dtype, void* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    DISTILL_CHECK("distill_loss_backward");
    HTL_REQUIRE(m == 0 || dloss, "distill_loss_backward: null pointer");
    HTL_REQUIRE(known(dx_dtype), "distill_loss_backward: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(aligned(dloss, 4) && aligned(dx, elem(dx_dtype)) && aligned(dw, elem(dtype)),
                "distill_loss_backward: misaligned pointer");
    SCORE_SPACE("distill_loss_backward", distill_loss_backward_workspace_bytes(m, vocab, k, top, dtype));
    if (!dx && !dw) return HTL_OK;
    const Rows2 r = {x, w, ldx, ldw, m, vocab, k, dtype};
    const float scale = 1.0f / temperature;
    const Teacher t = {{items, index_bits == 64, vocab}, logits, ld_logits, logits_dtype == HTL_F32, top, scale};
    const BackwardSpace s(ws, m, vocab, k, top, dtype);
    if (m > 0)
        hipLaunchKernelGGL(k_teach, dim3(grid_for(m, 4)), dim3(256), 0, stream, m, t, scores, lse, dloss, s.ids, s.entries);
    return backward_pieces(r, scale, s, Items{nullptr, false, vocab}, t.items, top, lse, dloss, dx, dx_dtype, dw, stream);
}
