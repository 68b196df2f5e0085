// Matrix products grouped by row: every row times its group's matrix (the
// projection of its feature table, or its expert), and the gradients.
//
//   y_i  = w_g x_i            (x [m][k], w [groups][n][k], g the row's group)
//   dx_i = w_g^T dy_i
//   dw_g = sum over the group's rows of dy_i x_i^T   (fp32)
// Rows of no group: y = 0, dx = 0.  Rows are read and written in place
// through the plan's order, so nothing is sorted or copied around the product.
#include "dense.h"

namespace htl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct ProdArgs {
    const void* a;           // x (forward), dy (dx and dw)
    const void* b;           // w, or x (dw)
    void* out;
    const int32_t* order;    // nullable: rows lie in group order
    const int32_t* offsets;  // nullable: one group
    int64_t m, lda, ldb;     // ldb: row stride of x in dw
    int n, k, n_groups;
    uint32_t rows;           // dw: rows per chunk
    int64_t chunks;          // of rows, over all groups (an upper bound)
    float* partial;          // dw: [chunks][n][k]
    int out_f32;
};

enum { kFwd = 0, kDx = 1, kDw = 2 };

template <int T> __device__ __forceinline__ float elem_at(const void* p, int64_t i) {
    return T == kSrcF32 ? ((const float*)p)[i] : __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

// Any widths, strides and types: 64 x 64 tiles of the output, operands
// widened to fp32 in LDS element by element, 16x16x4 fp32 matrix
// instructions.  out[r][c] = sum over e of A(r, e) B(c, e).
constexpr int kT = 64, kE = 32;

template <int T, int MODE>
__global__ __launch_bounds__(256) void k_product_any(ProdArgs p) {
    __shared__ float sa[kT][kE + 1], sb[kT][kE + 1];
    __shared__ int32_t s_row[kT];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int cols = MODE == kFwd ? p.n : p.k;
    const int col_tiles = (cols + kT - 1) / kT;
    const int64_t tiles = MODE == kDw ? (int64_t)col_tiles * ((p.n + kT - 1) / kT) : col_tiles;
    for (int64_t item = blockIdx.x; item < p.chunks * tiles; item += gridDim.x) {
        const int64_t chunk = item / tiles;
        const int tile = (int)(item - chunk * tiles);
        Chunk c;
        if (!find_chunk(p.offsets, p.n_groups, p.m, p.rows, MODE == kDw ? 1 : 0, chunk, c))
            return;
        const bool grouped = c.g < p.n_groups;
        const int r0 = MODE == kDw ? tile / col_tiles * kT : 0;
        const int c0 = tile % col_tiles * kT;
        __syncthreads();                     // the tile before is written
        if (MODE == kDw) {
            if (!grouped) return;
        } else {
            if (threadIdx.x < kT) {
                const int64_t pos = c.beg + threadIdx.x;
                const int32_t row = pos < c.end ? (p.order ? p.order[pos] : (int32_t)pos) : -1;
                s_row[threadIdx.x] = row >= 0 && row < p.m ? row : -1;
            }
        }
        const int64_t len = MODE == kFwd ? p.k : (MODE == kDx ? p.n : c.end - c.beg);
        f32x4 acc[4];
    #pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t wg = grouped ? (int64_t)c.g * p.n * p.k : 0;
        for (int64_t e0 = 0; grouped && e0 < len; e0 += kE) {
            __syncthreads();
            if (MODE == kDw) {
                for (int i = threadIdx.x; i < kT * kE; i += 256) {
                    const int e = i / kT, q = i % kT;
                    const int64_t pos = c.beg + e0 + e;
                    const int64_t row = pos < c.end ? (p.order ? p.order[pos] : pos) : -1;
                    const bool in = row >= 0 && row < p.m;
                    sa[q][e] = in && r0 + q < p.n ? elem_at<T>(p.a, row * p.lda + r0 + q) : 0.0f;
                    sb[q][e] = in && c0 + q < p.k ? elem_at<T>(p.b, row * p.ldb + c0 + q) : 0.0f;
                }
            } else {
                for (int i = threadIdx.x; i < kT * kE; i += 256) {
                    const int q = i / kE, e = i % kE;
                    const int32_t row = s_row[q];
                    sa[q][e] = row >= 0 && e0 + e < len ? elem_at<T>(p.a, row * p.lda + e0 + e) : 0.0f;
                }
                for (int i = threadIdx.x; i < kT * kE; i += 256) {
                    // along the weight's rows in both cases
                    const int q = MODE == kFwd ? i / kE : i % kT, e = MODE == kFwd ? i % kE : i / kT;
                    const bool in = c0 + q < cols && e0 + e < len;
                    const int64_t at = MODE == kFwd ? wg + (int64_t)(c0 + q) * p.k + e0 + e
                                                    : wg + (e0 + e) * p.k + c0 + q;
                    sb[q][e] = in ? elem_at<T>(p.b, at) : 0.0f;
                }
            }
            __syncthreads();
            // wave wv: rows 16 wv .. + 16; lane l: element l / 16 of four
    #pragma unroll
            for (int e = 0; e < kE; e += 4) {
                const float va = sa[wv * 16 + (lane & 15)][e + (lane >> 4)];
    #pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(va, sb[t * 16 + (lane & 15)][e + (lane >> 4)], acc[t], 0,
                                                                  0, 0);
            }
        }
        __syncthreads();
    #pragma unroll
        for (int t = 0; t < 4; ++t)
    #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = wv * 16 + (lane >> 4) * 4 + j, col = c0 + t * 16 + (lane & 15);
                if (col >= cols) continue;
                if (MODE == kDw) {
                    if (r0 + q >= p.n) continue;
                    float* dst = c.count == 1 ? (float*)p.out + wg : p.partial + chunk * p.n * p.k;
                    dst[(int64_t)(r0 + q) * p.k + col] = acc[t][j];
                } else if (s_row[q] >= 0) {
                    const int64_t at = (int64_t)s_row[q] * cols + col;
                    if (p.out_f32) ((float*)p.out)[at] = acc[t][j];
                    else ((uint16_t*)p.out)[at] = (uint16_t)f32_to_bf16_bits(acc[t][j]);
                }
            }
    }
}

// Rows per chunk of dw's sums: chunks times tiles fill the device a few
// times over, and a chunk is long against the partial sums it leaves.
uint32_t dw_chunk_rows(int64_t m, int n_groups, int n, int k) {
    const int64_t tiles = ceil_div(n, kT) * ceil_div(k, kT);
    int64_t r = ceil_div(m * tiles, 2048);
    if (r < 256) r = 256;
    if (r > m) r = m < 1 ? 1 : m;
    return (uint32_t)r;
}
int64_t dw_chunks(int64_t m, int n_groups, int n, int k) { return m / dw_chunk_rows(m, n_groups, n, k) + n_groups + 1; }

int elem(htl_dtype t) { return t == HTL_F32 ? 4 : 2; }
bool known(htl_dtype t) { return t == HTL_F32 || t == HTL_BF16; }

}  // namespace
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
    ProdArgs p = {x, w, y, order, offsets, m, ldx, k, n, k, n_groups, (uint32_t)kT,
                  m / kT + n_groups + 1, nullptr, y_dtype == HTL_F32};
    const dim3 grid(grid_for(p.chunks * ceil_div(n, kT), 1));
    if (dtype == HTL_F32) hipLaunchKernelGGL((k_product_any<kSrcF32, kFwd>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((k_product_any<kSrcBf16, kFwd>), grid, dim3(256), 0, stream, p);
    return check_launch("grouped_mm");
}

extern "C" size_t grouped_mm_backward_workspace_bytes(int64_t m, int n_groups, int n, int k) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || n < 1 || n > HTL_MAX_PRODUCT_DIM || k < 1 ||
        k > HTL_MAX_PRODUCT_DIM)
        return 0;
    if (m <= (int64_t)dw_chunk_rows(m, n_groups, n, k)) return 256;
    return align_up((size_t)dw_chunks(m, n_groups, n, k) * n * k * 4, 256);
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
        ProdArgs p = {dy, w, dx, order, offsets, m, ld_dy, k, n, k, n_groups, (uint32_t)kT,
                      m / kT + n_groups + 1, nullptr, dx_dtype == HTL_F32};
        const dim3 grid(grid_for(p.chunks * ceil_div(k, kT), 1));
        if (dtype == HTL_F32) hipLaunchKernelGGL((k_product_any<kSrcF32, kDx>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((k_product_any<kSrcBf16, kDx>), grid, dim3(256), 0, stream, p);
        const htl_status st = check_launch("grouped_mm_backward");
        if (st != HTL_OK) return st;
    }
    if (!dw) return HTL_OK;
    ProdArgs p = {dy, x, dw, order, offsets, m, ld_dy, ldx, n, k, n_groups, dw_chunk_rows(m, n_groups, n, k),
                  dw_chunks(m, n_groups, n, k), (float*)ws, 1};
    const dim3 grid(grid_for(p.chunks * ceil_div(n, kT) * ceil_div(k, kT), 1));
    if (dtype == HTL_F32) hipLaunchKernelGGL((k_product_any<kSrcF32, kDw>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((k_product_any<kSrcBf16, kDw>), grid, dim3(256), 0, stream, p);
    const htl_status st = check_launch("grouped_mm_backward");
    if (st != HTL_OK) return st;
    return sum_chunks(p.partial, dw, offsets, n_groups, m, p.rows, (int64_t)n * k, stream);
}
