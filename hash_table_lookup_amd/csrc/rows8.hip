// Rows kept in 8 bits (activations held for a backward pass at half of bf16's
// bytes) and read back: the format is at dense.h's unpack8 / save8.
//
// Bound: bytes.  1.7M bf16 rows of 128: 131 us to write (661 MB: 5.0 TB/s), 245
// to write and read back (5.4 TB/s).  A lane moves eight elements (16 or 32
// bytes in, 8 codes out); four lanes share a block's scale.
#include "dense.h"

namespace htl {
namespace {

constexpr int kThreads = 256;

// Row and first column of this thread's eight elements, the workgroup's first
// being number i0: one 64-bit division for the workgroup, a 32-bit one per lane.
__device__ __forceinline__ void place(int64_t i0, int lanes, int64_t& row, int& col) {
    const int64_t row0 = i0 / lanes;
    const uint32_t in = (uint32_t)(i0 - row0 * lanes) + threadIdx.x, q = in / (uint32_t)lanes;
    row = row0 + q;
    col = (int)(in - q * lanes) * 8;
}

// One lane per eight elements, a row padded to whole blocks of 32 (so that
// the lanes of a block are always neighbours).
template <int TX>
__global__ __launch_bounds__(kThreads) void k_rows8_save(RowsIn x, int64_t m, int dim, int lanes, Rows8Out out) {
    const int64_t n = m * lanes, stride = (int64_t)gridDim.x * kThreads;
    // whole waves loop together: the shuffles of a block need its four lanes
    for (int64_t i0 = blockIdx.x * (int64_t)kThreads; i0 < n; i0 += stride) {
        int64_t row;
        int col;
        place(i0, lanes, row, col);
        if (i0 + threadIdx.x >= n) {     // past the end: nothing to read or write
            row = 0;
            col = dim;
        }
        Raw8<TX> raw;
        load8(x, row, col, dim, raw);
        float v[8];
        unpack8(x, raw, v);
        save8(out, row, col, dim, v);
    }
}

template <int TY>
__global__ __launch_bounds__(kThreads) void k_rows8_load(RowsIn q, int64_t m, int dim, int lanes, RowsOut y) {
    const int64_t n = m * lanes, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i0 = blockIdx.x * (int64_t)kThreads; i0 < n; i0 += stride) {
        if (i0 + threadIdx.x >= n) continue;
        int64_t row;
        int col;
        place(i0, lanes, row, col);
        Raw8<kSrcRows8> raw;
        load8(q, row, col, dim, raw);
        float v[8];
        unpack8(q, raw, v);
        store8<TY>(y, row, col, dim, v);
    }
}

}  // namespace
}  // namespace htl

using namespace htl;

#define ROWS8_CHECK(name)                                                                                            \
    HTL_REQUIRE(m >= 0 && m <= kMaxRows && dim >= 1 && dim <= 65536, name ": rows or dim out of range");             \
    HTL_REQUIRE(fmt == HTL_ROWS8_I8 || fmt == HTL_ROWS8_E4M3, name ": unknown 8-bit format");                        \
    HTL_REQUIRE(dtype == HTL_F32 || dtype == HTL_BF16, name ": dtype must be HTL_F32 or HTL_BF16")

extern "C" htl_status rows8_save(const void* x, htl_dtype dtype, int64_t ldx, int64_t m, int dim, htl_rows8_fmt fmt,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    clear_error();
    ROWS8_CHECK("rows8_save");
    if (m == 0) return HTL_OK;
    const int es = dtype == HTL_F32 ? 4 : 2;
    HTL_REQUIRE(ldx >= dim, "rows8_save: row stride below dim");
    HTL_REQUIRE(x && codes && scales && aligned(x, es), "rows8_save: null or misaligned pointer");
    const RowsIn in = {x, nullptr, ldx, 0};
    const Rows8Out out = {codes, scales, (int)fmt};
    const int lanes = (dim + 31) / 32 * 4;
    const dim3 grid(grid_for(m * lanes, kThreads, 1 << 22));
    if (dtype == HTL_F32)
        hipLaunchKernelGGL((k_rows8_save<kSrcF32>), grid, dim3(kThreads), 0, stream, in, m, dim, lanes, out);
    else
        hipLaunchKernelGGL((k_rows8_save<kSrcBf16>), grid, dim3(kThreads), 0, stream, in, m, dim, lanes, out);
    return check_launch("rows8_save");
}

extern "C" htl_status rows8_load(const uint8_t* codes, const uint8_t* scales, htl_rows8_fmt fmt, int64_t m, int dim,
                                 void* y, htl_dtype dtype, hipStream_t stream) {
    clear_error();
    ROWS8_CHECK("rows8_load");
    if (m == 0) return HTL_OK;
    const int es = dtype == HTL_F32 ? 4 : 2;
    HTL_REQUIRE(y && codes && scales && aligned(y, es), "rows8_load: null or misaligned pointer");
    const RowsIn in = {codes, scales, dim, (int)fmt};
    const RowsOut out = {y, dim};
    const int lanes = (dim + 7) / 8;
    const dim3 grid(grid_for(m * lanes, kThreads, 1 << 22));
    if (dtype == HTL_F32)
        hipLaunchKernelGGL((k_rows8_load<kSrcF32>), grid, dim3(kThreads), 0, stream, in, m, dim, lanes, out);
    else
        hipLaunchKernelGGL((k_rows8_load<kSrcBf16>), grid, dim3(kThreads), 0, stream, in, m, dim, lanes, out);
    return check_launch("rows8_load");
}
