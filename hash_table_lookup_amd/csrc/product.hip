// Matrix products grouped by row: every row times its group's matrix (the
// projection of its feature table, or its expert), and the gradients.
//
//   y_i  = w_g x_i            (x [m][k], w [groups][n][k], g the row's group)
//   dx_i = w_g^T dy_i
//   dw_g = sum over the group's rows of dy_i x_i^T   (fp32)
// Rows of no group: y = 0, dx = 0.  Rows are read and written in place
// through the plan's order, so nothing is sorted or copied around the product.
//
// Measured: 16,384 bf16 rows in 16 ragged groups, 2,048 -> 4,096: forward
// 321 us (316-330; 860 TFLOP/s), dx 349 (348-354), dw 388 (385-392, with 537 MB of
// fp32 results); one group, 32,768 rows, 2,048 -> 2,048: 260, 270 and 292 us
// (940-1,060 TFLOP/s, where the library's product of such sizes reaches
// 1,340-1,600).  Without its loads the forward kernel runs at 1,450-1,550: it
// is bound by how soon operands arrive in LDS (a request takes 577 cycles
// against 282 in the library's kernel of the same tile, at equal hits in L2).
// Counted from the code, a step of a 256 x 256 tile moves 96 KiB out of LDS and
// 32 KiB into it, 1,024 cycles at 128 bytes each, and its matrix instructions
// take as many: loads find LDS busy.
// 1.7M rows in 26 groups, 128 -> 256: 312, 303 and 353 us, bound by bytes
// (1,308 MB each: 3.7-4.3 TB/s; the results alone are 2.9 TB/s of scattered rows);
// 66 of the last are the sums of its partial sums.
// fp32: 20,000 rows, 1,024 x 1,024: 328, 348 and 370 us (113-128 TFLOP/s of 157).
#include "tile.h"

namespace htl {
namespace {

template <int T, int MODE, class C, bool ASYNC, bool BF16 = false>
__global__ __launch_bounds__(C::kThreads, 2) void k_product(ProdArgs p) {
    product_tiles<T, MODE, C, ASYNC>(p, StoreRows<MODE, C, BF16>{p});
}
template <int T, class C, bool ASYNC, bool ADD> __global__ __launch_bounds__(C::kThreads, 2) void k_dx_parts(ProdArgs p) {
    product_tiles<T, kDx, C, ASYNC, true>(p, StoreParts<C, ADD>{p});
}

// Products whose matrix fits in LDS (the projections of a feature table's
// rows): a workgroup loads its group's matrix once and its waves then walk
// the chunk's rows, 32 at a time and without waiting for each other, from
// global memory to registers, through the matrix, and out.
//
// LDS holds one row of LP * 32 elements per output, zeros beyond the matrix,
// 16 bytes apart so that 16 rows read together hit different banks.
template <int LP, int BYTES, int MODE>
__global__ __launch_bounds__(512, BYTES <= 81920 && LP <= 4 ? 4 : 2) void k_resident(ProdArgs p) {
    constexpr int kLd = LP * 64 + 16;
    __shared__ __attribute__((aligned(16))) char lds[BYTES];
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = MODE == kFwd ? p.n : p.k, len = MODE == kFwd ? p.k : p.n;
    const int blocks = (cols + 63) / 64;
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
            const char* w = (const char*)p.b + (int64_t)t.g * p.n * p.k * 2;
            if (MODE == kFwd) {
#pragma unroll 4
                for (int i = threadIdx.x; i < blocks * 64 * LP * 4; i += 512) {
                    const int c = i / (LP * 4), e = i % (LP * 4) * 8;
                    *(u32x4*)(lds + c * kLd + e * 2) =
                        held_piece<2>(w + ((int64_t)c * p.k + e) * 2, c < p.n ? p.k - e : 0);
                }
            } else {
                // two rows of w and eight columns: pairs of neighbours in eight rows of LDS
#pragma unroll 2
                for (int i = threadIdx.x; i < LP * 16 * blocks * 8; i += 512) {
                    const int e = i / (blocks * 8) * 2, c = i % (blocks * 8) * 8;
                    const char* at = w + ((int64_t)e * p.k + c) * 2;
                    const u32x4 lo = held_piece<2>(at, e < p.n ? p.k - c : 0);
                    const u32x4 hi = held_piece<2>(at + p.k * 2, e + 1 < p.n ? p.k - c : 0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t a = lo[j >> 1] >> (16 * (j & 1)) & 0xFFFFu, d = hi[j >> 1] >> (16 * (j & 1));
                        *(uint32_t*)(lds + (c + j) * kLd + e * 2) = a | d << 16;
                    }
                }
            }
        }
        __syncthreads();
        for (; pos < t.end; pos += 256) {
            Frag<kSrcBf16> x[2][LP];
            if (len == LP * 32) {            // every piece whole; a row that is not there is read as the first
#pragma unroll
                for (int l = 0; l < LP; ++l)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        load_at<2>((const char*)p.a + ((row[j] < 0 ? 0 : row[j]) * p.lda + l * 32 + (lane >> 4) * 8) * 2,
                                   x[j][l].v);
            } else {
#pragma unroll
                for (int l = 0; l < LP; ++l)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int e = l * 32 + (lane >> 4) * 8;
                        const char* at = (const char*)p.a + (row[j] * p.lda + e) * 2;
                        const u32x4 v = held_piece<2>(at, row[j] >= 0 ? len - e : 0);
                        __builtin_memcpy(&x[j][l].v, &v, 16);
                    }
            }
            const int32_t next[2] = {row_at(pos + 256 + (lane & 15)), row_at(pos + 272 + (lane & 15))};
            for (int nb = 0; nb < blocks; ++nb) {
                f32x4 acc[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[j][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (grouped) {
#pragma unroll
                    for (int l = 0; l < LP; ++l)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            Frag<kSrcBf16> c;
                            c.v = *(const bf16x8*)(lds + (nb * 64 + q * 16 + (lane & 15)) * kLd + l * 64 + (lane >> 4) * 16);
                            multiply(c, x[0][l], 0, acc[0][q]);
                            multiply(c, x[1][l], 0, acc[1][q]);
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    store_rows<4>(p.out, p.out_f32, row[j], cols, nb * 64, cols, acc[j]);
                }
            }
            row[0] = next[0];
            row[1] = next[1];
        }
    }
}

// chunks: at most this many in all
template <int T, int MODE, class C, bool ASYNC, bool BF16 = false>
void launch(const ProdArgs& p, int64_t chunks, hipStream_t s) {
    const int64_t cols = ceil_div(MODE == kFwd ? p.n : p.k, C::BC) * (MODE == kDw ? ceil_div(p.n, C::BR) : 1);
    const dim3 grid(grid_for(align_up((size_t)(chunks * cols), kXcds), 1));
    hipLaunchKernelGGL((k_product<T, MODE, C, ASYNC, BF16>), grid, dim3(C::kThreads), 0, s, p);
}

template <int MODE, int LP> void launch_resident(const ProdArgs& p, int64_t chunks, int64_t bytes, hipStream_t s) {
    const dim3 grid(grid_for(align_up((size_t)chunks, kXcds), 1));
    if (bytes <= 81920) hipLaunchKernelGGL((k_resident<LP, 81920, MODE>), grid, dim3(512), 0, s, p);
    else hipLaunchKernelGGL((k_resident<LP, 163840, MODE>), grid, dim3(512), 0, s, p);
}

// Forward product or dx: `cols` outputs a row, reduced over `len`.  The kernel
// goes by size (us, forward / dx, bf16, groups x rows, k -> n):
// - a matrix kept in LDS pays its loading back over many rows: 26 x 65,536,
//   128 -> 256: 315 / 302 against 512 / 361 in tiles; 26 x 4,096: 26 / 36
//   against 32 / 27; 26 x 1,024: 16 / 17 against 11 / 11.  (The transposed
//   matrix of 256 reduced elements takes longest to load: from 2^20 rows on.)
// - tiles of 32 rows where groups have few rows, or the output few tiles:
//   8 x 128, 1,024 -> 1,024: 11 / 15 against 15 / 20 with 128; 8 x 512: 28 / 30
//   against 18 / 22.
// - tiles of 256 x 256 once they fill the device: 8 x 2,048, 1,024 -> 1,024:
//   43 / 47 against 51 / 53 with 128; 8 x 1,024: 37 / 38 against 28 / 28.
template <int MODE> void launch_rows(ProdArgs p, htl_dtype dtype, hipStream_t s, bool padded = false) {
    const int cols = MODE == kFwd ? p.n : p.k, es = elem(dtype);
    const bool fast = p.lda * es % 16 == 0 && aligned(p.a, 16) && p.ldw * es % 16 == 0 && aligned(p.b, 16) &&
                      (padded || ((int64_t)p.k * es % 16 == 0 && (MODE == kFwd || (int64_t)p.n * es % 16 == 0))) &&
                      p.m * p.lda * es <= kBufferBytes && (int64_t)p.n * p.ldw * es <= kBufferBytes;
    const int64_t each = p.m / p.n_groups;
    const int len = MODE == kFwd ? p.k : p.n, lp = len <= 32 ? 1 : len <= 64 ? 2 : len <= 128 ? 4 : 8;
    const int64_t bytes = ceil_div(cols, 64) * 64 * (lp * 64 + 16);
    if (dtype == HTL_BF16 && p.ldw == p.k && len <= 256 && bytes <= 163840 && each >= 512 && p.m >= (lp == 8 ? 1 << 20 : 1 << 16)) {
        p.rows = (uint32_t)align_up((size_t)ceil_div(p.m, 1024), 256);
        const int64_t chunks = p.m / p.rows + p.n_groups + 1;
        if (lp == 1) launch_resident<MODE, 1>(p, chunks, bytes, s);
        else if (lp == 2) launch_resident<MODE, 2>(p, chunks, bytes, s);
        else if (lp == 4) launch_resident<MODE, 4>(p, chunks, bytes, s);
        else launch_resident<MODE, 8>(p, chunks, bytes, s);
        return;
    }
    int tile = each <= 48 || (ceil_div(p.m, 32) + p.n_groups) * ceil_div(cols, 128) <= 512 ? 32 : 128;
    if (dtype == HTL_BF16 && fast && ceil_div(p.m, 256) * ceil_div(cols, 256) >= 224 && each >= 256) tile = 256;
    p.rows = (uint32_t)tile;
    const int64_t chunks = p.m / tile + p.n_groups + 1;
    if (dtype == HTL_BF16) {
        if (tile == 256) launch<kSrcBf16, MODE, Big, true>(p, chunks, s);
        else if (tile == 128 && fast) launch<kSrcBf16, MODE, Mid, true>(p, chunks, s);
        else if (tile == 128) launch<kSrcBf16, MODE, Mid, false>(p, chunks, s);
        else if (fast) launch<kSrcBf16, MODE, Small, true>(p, chunks, s);
        else launch<kSrcBf16, MODE, Small, false>(p, chunks, s);
    } else {
        if (tile == 128 && fast) launch<kSrcF32, MODE, Mid, true>(p, chunks, s);
        else if (tile == 128) launch<kSrcF32, MODE, Mid, false>(p, chunks, s);
        else if (fast) launch<kSrcF32, MODE, Small, true>(p, chunks, s);
        else launch<kSrcF32, MODE, Small, false>(p, chunks, s);
    }
}

// Rows per chunk of dw's sums.  A tile of a chunk leaves a partial sum to be
// written and read again, so chunks are as long as fills the device once with
// tiles of 256 x 256 (16 ragged experts, 2,048 x 4,096: 391 us, with twice as
// many 469; 8 x 1,024 rows, 1,024 x 1,024: 67 against 94), and twice with those
// that move by way of registers (100,001 rows, 513 x 777: 495 us, once 560) or
// a few times over with small matrices, whose partial sums are small.
uint32_t dw_chunk_rows(int64_t m, int n, int k) {
    const int side = n >= 256 && k >= 256 ? 256 : 128;
    const int64_t tiles = ceil_div(n, side) * ceil_div(k, side);
    int64_t r = ceil_div(m * tiles, side == 128 ? 1024 : (n % 8 == 0 && k % 8 == 0 ? 256 : 512));
    if (r < 256) r = 256;
    if (r > m) r = m < 1 ? 1 : m;
    return (uint32_t)r;
}
int64_t dw_chunks(int64_t m, int n_groups, int n, int k) { return m / dw_chunk_rows(m, n, k) + n_groups + 1; }
int64_t dw_slots(int64_t m, int n_groups, int n, int k) { return split_chunks(m, n_groups, dw_chunk_rows(m, n, k)); }

}  // namespace

htl_status rows_dx(const void* dy, int64_t ld_dy, const void* w, int64_t ldw, htl_dtype dtype, int64_t m, int n, int k,
                   const int32_t* order, const int32_t* offsets, int n_groups, void* dx, htl_dtype dx_dtype, bool padded,
                   hipStream_t stream) {
    if (m == 0) return HTL_OK;
    const ProdArgs p = {dy, w, dx, order, offsets, m, ld_dy, k, ldw, n, k, n_groups, 0, nullptr, dx_dtype == HTL_F32, 0};
    launch_rows<kDx>(p, dtype, stream, padded);
    return check_launch("input gradients");
}

// Parts of at least 256 elements that fill the device with tiles three times
// over, and sums of at most 256 MiB.
int rows_dx_splits(int64_t m, int n, int k) {
    const int64_t tiles = ceil_div(m, m <= 32 ? 32 : 128) * ceil_div(k, 128);
    int64_t s = 768 / (tiles < 1 ? 1 : tiles);
    if (s > n / 256) s = n / 256;
    if (m > 0 && s > (64 << 20) / (m * k)) s = (64 << 20) / (m * k);
    return s < 1 ? 1 : (int)s;
}

htl_status rows_dx_parts(const void* dy, int64_t ld_dy, const void* w, int64_t ldw, htl_dtype dtype, int64_t m, int n, int k,
                         const int32_t* order, const int32_t* offsets, int n_groups, float* parts, int splits, bool add,
                         bool padded, hipStream_t stream) {
    if (m == 0) return HTL_OK;
    const int es = elem(dtype);
    const bool fast = ld_dy * es % 16 == 0 && aligned(dy, 16) &&
                      (padded || ((int64_t)n * es % 16 == 0 && (int64_t)k * es % 16 == 0)) && ldw * es % 16 == 0 && aligned(w, 16) && m * ld_dy * es <= kBufferBytes && n * ldw * es <= kBufferBytes;
    // (one fp32 row of 1,096 against 193,959 items, in tiles of 128 rows: 590 us, bound by products of rows that are not there)
    const int rows = m <= 32 ? 32 : 128;
    ProdArgs p = {dy, w, nullptr, order, offsets, m, ld_dy, k, ldw, n, k, n_groups, (uint32_t)rows, parts, 1, 0};
    p.splits = splits;
    const int64_t tiles = (m / rows + n_groups + 1) * ceil_div(k, 128) * splits;
    const dim3 grid(grid_for(align_up((size_t)tiles, kXcds), 1));
    auto go = [&](auto t, auto shape, auto async, auto adds) {
        using C = decltype(shape);
        hipLaunchKernelGGL((k_dx_parts<decltype(t)::value, C, decltype(async)::value, decltype(adds)::value>), grid,
                           dim3(C::kThreads), 0, stream, p);
    };
    auto of = [&](auto t, auto shape) {
        using Yes = std::true_type;
        using No = std::false_type;
        if (fast && add) go(t, shape, Yes(), Yes());
        else if (fast) go(t, shape, Yes(), No());
        else if (add) go(t, shape, No(), Yes());
        else go(t, shape, No(), No());
    };
    auto with = [&](auto t) {
        if (rows == 32) of(t, Small());
        else of(t, Mid());
    };
    if (dtype == HTL_F32) with(std::integral_constant<int, kSrcF32>());
    else with(std::integral_constant<int, kSrcBf16>());
    return check_launch("input gradients");
}

size_t sums_dw_bytes(int64_t m, int n_groups, int n, int k) {
    if (m <= (int64_t)dw_chunk_rows(m, n, k)) return 256;
    return align_up((size_t)dw_slots(m, n_groups, n, k) * n * k * 4, 256);
}

htl_status sums_dw(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, htl_dtype dtype, int64_t m, int n, int k,
                   const int32_t* order, const int32_t* offsets, int n_groups, void* dw, htl_dtype dw_dtype, void* ws,
                   bool padded, hipStream_t stream) {
    const int es = elem(dtype);
    const ProdArgs p = {dy, x, dw, order, offsets, m, ld_dy, ldx, k, n, k, n_groups, dw_chunk_rows(m, n, k),
                        (float*)ws, dw_dtype == HTL_F32, dw_slots(m, n_groups, n, k)};
    const int64_t chunks = dw_chunks(m, n_groups, n, k);
    const bool fast = ld_dy * es % 16 == 0 && ldx * es % 16 == 0 && aligned(dy, 16) && aligned(x, 16) &&
                      (padded || ((int64_t)n * es % 16 == 0 && (int64_t)k * es % 16 == 0)) && m * ld_dy * es <= kBufferBytes &&
                      m * ldx * es <= kBufferBytes;
    if (dw_dtype == HTL_BF16) {              // of bf16 operands
        if (fast && n >= 256 && k >= 256) launch<kSrcBf16, kDw, Big, true, true>(p, chunks, stream);
        else if (fast) launch<kSrcBf16, kDw, Mid, true, true>(p, chunks, stream);
        else launch<kSrcBf16, kDw, Mid, false, true>(p, chunks, stream);
    } else if (dtype == HTL_BF16) {
        if (fast && n >= 256 && k >= 256) launch<kSrcBf16, kDw, Big, true>(p, chunks, stream);
        else if (fast) launch<kSrcBf16, kDw, Mid, true>(p, chunks, stream);
        else launch<kSrcBf16, kDw, Mid, false>(p, chunks, stream);
    } else {
        if (fast) launch<kSrcF32, kDw, Mid, true>(p, chunks, stream);
        else launch<kSrcF32, kDw, Mid, false>(p, chunks, stream);
    }
    const htl_status st = check_launch("weight gradients");
    if (st != HTL_OK) return st;
    return sum_chunks(p.partial, p.limit, dw, nullptr, offsets, n_groups, m, p.rows, (int64_t)n * k, stream,
                      dw_dtype == HTL_BF16);
}

}  // namespace htl

using namespace htl;

#define PROD_CHECK(name)                                                                                         \
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, name ": row count out of range");                                       \
    HTL_REQUIRE(n >= 1 && n <= HTL_MAX_PRODUCT_DIM && k >= 1 && k <= HTL_MAX_PRODUCT_DIM, name ": n or k out of range"); \
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, name ": group count out of range");                     \
    HTL_REQUIRE(known(dtype), name ": dtype must be HTL_F32 or HTL_BF16");                                       \
    HTL_REQUIRE(offsets || (n_groups == 1 && !order), name ": several groups need offsets");                     \
    HTL_REQUIRE(aligned(order, 4) && aligned(offsets, 4), name ": misaligned pointer")

extern "C" htl_status grouped_mm(const void* x, int64_t ldx, const void* w, htl_dtype dtype, int64_t m, int n, int k,
                                 const int32_t* order, const int32_t* offsets, int n_groups, void* y,
                                 htl_dtype y_dtype, hipStream_t stream) {
    clear_error();
    PROD_CHECK("grouped_mm");
    HTL_REQUIRE(known(y_dtype), "grouped_mm: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(ldx >= k, "grouped_mm: row stride below k");
    if (m == 0) return HTL_OK;
    const int es = elem(dtype);
    HTL_REQUIRE(x && w && y, "grouped_mm: null pointer");
    HTL_REQUIRE(aligned(x, es) && aligned(w, es) && aligned(y, elem(y_dtype)), "grouped_mm: misaligned pointer");
    ProdArgs p = {x, w, y, order, offsets, m, ldx, k, k, n, k, n_groups, 0, nullptr, y_dtype == HTL_F32, 0};
    launch_rows<kFwd>(p, dtype, stream);
    return check_launch("grouped_mm");
}

extern "C" size_t grouped_mm_backward_workspace_bytes(int64_t m, int n_groups, int n, int k) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || n < 1 || n > HTL_MAX_PRODUCT_DIM || k < 1 ||
        k > HTL_MAX_PRODUCT_DIM)
        return 0;
    return sums_dw_bytes(m, n_groups, n, k);
}

extern "C" htl_status grouped_mm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ldx, const void* w,
                                          htl_dtype dtype, int64_t m, int n, int k, const int32_t* order,
                                          const int32_t* offsets, int n_groups, void* dx, htl_dtype dx_dtype,
                                          float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    PROD_CHECK("grouped_mm_backward");
    HTL_REQUIRE(known(dx_dtype), "grouped_mm_backward: dtype must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(ld_dy >= n && (!dw || ldx >= k), "grouped_mm_backward: row stride below the row's length");
    const int es = elem(dtype);
    HTL_REQUIRE((m == 0 || dy) && (!dx || w) && (!dw || x || m == 0), "grouped_mm_backward: null pointer");
    HTL_REQUIRE(aligned(dy, es) && aligned(x, es) && aligned(w, es) && aligned(dx, elem(dx_dtype)) && aligned(dw, 4),
                "grouped_mm_backward: misaligned pointer");
    HTL_REQUIRE(!dw || (ws && aligned(ws, 256) && ws_bytes >= grouped_mm_backward_workspace_bytes(m, n_groups, n, k)),
                "grouped_mm_backward: workspace too small or misaligned");
    if (dx && m > 0) {
        const htl_status st = rows_dx(dy, ld_dy, w, k, dtype, m, n, k, order, offsets, n_groups, dx, dx_dtype, false, stream);
        if (st != HTL_OK) return st;
    }
    if (!dw) return HTL_OK;
    return sums_dw(dy, ld_dy, x, ldx, dtype, m, n, k, order, offsets, n_groups, dw, HTL_F32, ws, false, stream);
}
