// The gradients' products of operators with much to multiply, in wide.h's tiles,
// and the copies that lay their operands out.  Measured (bf16, 7,782 of 8,192 rows, 2,048
// columns, 16,384 elements of the reduction or as many sums): dx 417 us (1,277
// TFLOP/s), dw 399 us (1,309).
#include "wide.h"

namespace htl {
namespace {

// Parts of input gradients: rows of p.out by the plan, or by position in a part's sums.
struct DxEnd {
    static constexpr bool kPairs = false;
    void* dx;
    bool f32;
    float* parts;            // nullable
    bool add;
    int64_t m;
    int k;
    __device__ __forceinline__ void operator()(const TileAt& t, bool, int r, int64_t row, int col, f32x4 (&v)[8]) const {
        if (!parts) {
            store_rows<8>(dx, f32, row, k, col, k, v);
            return;
        }
        float* part = parts + t.slot * m * k;
        const int64_t pos = row < 0 ? -1 : t.beg + r;
        if (add) add_rows<8>(part, pos, k, col, k, v);
        else store_rows<8>(part, true, pos, k, col, k, v);
    }
};

struct DwEnd {
    static constexpr bool kPairs = false;
    void* dw;
    bool f32;
    float* partial;
    int n, k;
    __device__ __forceinline__ void operator()(const TileAt& t, bool, int, int64_t row, int col, f32x4 (&v)[8]) const {
        const bool whole = t.count == 1, out32 = f32 || !whole;
        const int64_t each = (int64_t)n * k;
        void* to = whole ? (char*)dw + t.g * each * (f32 ? 4 : 2) : (char*)(partial + t.slot * each);
        store_rows<8>(to, out32, row, k, col, k, v);
    }
};

__global__ __launch_bounds__(256, 1) void k_wide_dx(ProdArgs p, DxEnd end) { wide_tiles<kDx>(p, end); }
__global__ __launch_bounds__(256, 1) void k_wide_dw(ProdArgs p, DwEnd end) { wide_tiles<kDw>(p, end); }

// 16 bytes a thread.
template <int ES>
__global__ __launch_bounds__(256) void k_pack_rows(const char* __restrict__ x, int64_t ldx, const int32_t* __restrict__ order,
                                                   int64_t m, int64_t src_rows, int k, char* __restrict__ out, int64_t ld) {
    constexpr int VE = 16 / ES;
    const int64_t each = ld / VE, all = m * each;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int64_t pos = i / each, row = order ? (int64_t)order[pos] : pos;
        const int col = (int)(i - pos * each) * VE;
        const int64_t left = row >= 0 && row < src_rows ? k - col : 0;
        *(u32x4*)(out + (pos * ld + col) * ES) = held_piece<ES>(x + (row * ldx + col) * ES, left);
    }
}

template <class E>
__global__ __launch_bounds__(256) void k_zero_behind(E* __restrict__ d, int64_t m, int cols, int64_t ld) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m; i += gridDim.x * 256ll)
        for (int64_t c = cols; c < packed_ld(cols); ++c) d[i * ld + c] = 0;
}

// Four columns a thread.
template <bool BF16>
__global__ __launch_bounds__(256) void k_sum_parts(const float* __restrict__ parts, int splits, bool by_row,
                                                   int64_t m, int k, const int32_t* __restrict__ order, const int32_t* __restrict__ count,
                                                   void* __restrict__ dx) {
    const int64_t each = (k + 3) / 4, all = m * each, on = count ? (int64_t)*count : m;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int64_t pos = i / each, row = order ? (int64_t)order[pos] : pos;
        const int col = (int)(i - pos * each) * 4;
        if (row < 0 || row >= m) continue;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        const int have = k - col < 4 ? k - col : 4;
        if (pos < on) {
            const float* at = parts + (by_row ? row : pos) * k + col;
            if (have == 4) {
#pragma unroll 8
                for (int s = 0; s < splits; ++s) {
                    f32x4 a;
                    load_at<4>(at + (int64_t)s * m * k, a);
                    v += a;
                }
            } else {
                for (int s = 0; s < splits; ++s)
                    for (int e = 0; e < have; ++e) v[e] += at[(int64_t)s * m * k + e];
            }
        }
        if (BF16) {
            uint16_t* o = (uint16_t*)dx + row * k + col;
            const u32x2 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            if (have == 4) store_at<2>(o, w);
            else
                for (int e = 0; e < have; ++e) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        } else {
            float* o = (float*)dx + row * k + col;
            if (have == 4) store_at<4>(o, v);
            else
                for (int e = 0; e < have; ++e) o[e] = v[e];
        }
    }
}

// 16 bytes a thread, or two.
__global__ __launch_bounds__(256) void k_zero_rest(char* __restrict__ out, int64_t bytes, int64_t m,
                                                   const int32_t* __restrict__ order, const int32_t* __restrict__ count) {
    const int64_t from = *count < 0 ? 0 : *count, unit = bytes % 16 || !((uintptr_t)out % 16 == 0) ? 2 : 16, each = bytes / unit;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < (m - from) * each; i += gridDim.x * 256ll) {
        const int64_t pos = from + i / each, row = order ? (int64_t)order[pos] : pos;
        if (row < 0 || row >= m) continue;
        char* o = out + row * bytes + i % each * unit;
        if (unit == 16) *(u32x4*)o = zeros4();
        else *(uint16_t*)o = 0;
    }
}

// Positions per chunk of dw's sums: as long as fills the device once with
// tiles, and less than 4 GiB of an operand that is longer in all (offsets have 32
// bits; groups round a chunk up to 64 positions).
uint32_t wide_dw_rows(int64_t m, int n, int k, int64_t ldd, int64_t ldx) {
    int64_t r = ceil_div(m * ceil_div(n, 256) * ceil_div(k, 256), 256);
    if (r < 512) r = 512;
    for (const int64_t ld : {ldd, ldx}) {
        const int64_t most = kBufferBytes / 2 / ld / 64 * 64;
        if (m * ld * 2 > kBufferBytes && r > most) r = most;
    }
    if (r > m) r = m < 1 ? 1 : m;
    return (uint32_t)r;
}

}  // namespace

htl_status pack_rows(const void* x, int64_t ldx, htl_dtype dtype, const int32_t* order, int64_t m, int64_t src_rows, int k,
                     void* out, int64_t ld, hipStream_t stream) {
    if (m == 0) return HTL_OK;
    const dim3 grid(grid_for(m * (ld / 4), 256, 1 << 16));
    if (dtype == HTL_F32)
        hipLaunchKernelGGL(k_pack_rows<4>, grid, dim3(256), 0, stream, (const char*)x, ldx, order, m, src_rows, k, (char*)out, ld);
    else
        hipLaunchKernelGGL(k_pack_rows<2>, grid, dim3(256), 0, stream, (const char*)x, ldx, order, m, src_rows, k, (char*)out, ld);
    return check_launch("pack rows");
}

htl_status zero_behind(void* d, htl_dtype dtype, int64_t m, int cols, int64_t ld, hipStream_t stream) {
    if (cols % 8 == 0 || m == 0) return HTL_OK;
    const dim3 grid(grid_for(m, 256, 1 << 14));
    if (dtype == HTL_F32) hipLaunchKernelGGL(k_zero_behind<uint32_t>, grid, dim3(256), 0, stream, (uint32_t*)d, m, cols, ld);
    else hipLaunchKernelGGL(k_zero_behind<uint16_t>, grid, dim3(256), 0, stream, (uint16_t*)d, m, cols, ld);
    return check_launch("zeros behind rows");
}

// Tiles enough for the device once, of at least 1,024 elements of the reduction
// each, and parts of at most 256 MiB.
int wide_dx_splits(int64_t m, int n, int k) {
    const int64_t tiles = ceil_div(m, 256) * ceil_div(k, 256);
    int64_t s = 256 / (tiles < 1 ? 1 : tiles);
    if (s > n / 1024) s = n / 1024;
    if (m > 0 && s > (64 << 20) / (m * k)) s = (64 << 20) / (m * k);
    return s < 1 ? 1 : (int)s;
}

htl_status wide_dx(const void* d, int64_t ldd, const void* w, int64_t ldw, int64_t m, int n, int k, const int32_t* order,
                   const int32_t* offsets, int n_groups, void* dx, htl_dtype dx_dtype, float* parts, int splits, bool add,
                   hipStream_t stream) {
    if (m == 0) return HTL_OK;
    const ProdArgs p = {d, w, nullptr, order, offsets, m, ldd, 0, ldw, n, k, n_groups, 256, nullptr, 0, 0, true, true, splits};
    const DxEnd end = {dx, dx_dtype == HTL_F32, parts, add, m, k};
    const dim3 grid(wide_grid((m / 256 + n_groups) * ceil_div(k, 256) * splits));
    hipLaunchKernelGGL(k_wide_dx, grid, dim3(Wide::kThreads), 0, stream, p, end);
    return check_launch("input gradients");
}

htl_status sum_parts(const float* parts, int splits, bool by_row, int64_t m, int k, const int32_t* order,
                     const int32_t* count, void* dx, htl_dtype dx_dtype, hipStream_t stream) {
    if (m == 0) return HTL_OK;
    const dim3 grid(grid_for(m * ceil_div(k, 4), 256, 1 << 16));
    if (dx_dtype == HTL_F32) hipLaunchKernelGGL(k_sum_parts<false>, grid, dim3(256), 0, stream, parts, splits, by_row, m, k, order, count, dx);
    else hipLaunchKernelGGL(k_sum_parts<true>, grid, dim3(256), 0, stream, parts, splits, by_row, m, k, order, count, dx);
    return check_launch("input gradients");
}

htl_status zero_rest(void* out, int64_t bytes, int64_t m, const int32_t* order, const int32_t* count, hipStream_t stream) {
    if (m == 0) return HTL_OK;
    hipLaunchKernelGGL(k_zero_rest, dim3(grid_for(m * ceil_div(bytes, 16), 4096, 1 << 12)), dim3(256), 0, stream, (char*)out,
                       bytes, m, order, count);
    return check_launch("rows of no group");
}

size_t wide_dw_bytes(int64_t m, int n_groups, int n, int k, int64_t ldd, int64_t ldx) {
    const uint32_t r = wide_dw_rows(m, n, k, ldd, ldx);
    if (m <= (int64_t)r) return 256;
    return align_up((size_t)split_chunks(m, n_groups, r) * n * k * 4, 256);
}

htl_status wide_dw(const void* d, int64_t ldd, const void* x, int64_t ldx, int64_t m, int n, int k, const int32_t* offsets,
                   int n_groups, void* dw, htl_dtype dw_dtype, void* ws, hipStream_t stream) {
    const uint32_t r = wide_dw_rows(m, n, k, ldd, ldx);
    const ProdArgs p = {d, x, nullptr, nullptr, offsets, m, ldd, ldx, 0, n, k, n_groups, r, nullptr, 0, split_chunks(m, n_groups, r), true};
    const DwEnd end = {dw, dw_dtype == HTL_F32, (float*)ws, n, k};
    const int64_t tiles = (m / r + n_groups + 1) * ceil_div(n, 256) * ceil_div(k, 256);
    // (groups differ in length: their tiles are dealt out as units come free)
    const unsigned grid = n_groups == 1 ? wide_grid(tiles) : grid_for(align_up((size_t)tiles, kXcds), 1);
    hipLaunchKernelGGL(k_wide_dw, dim3(grid), dim3(Wide::kThreads), 0, stream, p, end);
    const htl_status st = check_launch("weight gradients");
    if (st != HTL_OK) return st;
    return sum_chunks((const float*)ws, p.limit, dw, nullptr, offsets, n_groups, m, r, (int64_t)n * k, stream, dw_dtype == HTL_BF16);
}

}  // namespace htl
