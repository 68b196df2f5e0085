// Rows by group: a stable counting sort of row ids (which feature table a row
// comes from, or the expert a router chose), the plan that the grouped
// products and per-group norms read.
//
// order lists the rows of group 0, then of group 1, ..., rows in their own
// order within a group, and last the rows of no group (id outside
// [0, n_groups)); offsets[g] is where group g starts.  Both are functions of
// the ids alone: ranks come from ballots and prefix sums, never from the
// order in which atomics land.
//
// Bound: latency (8 bytes a row are little): of launches on few rows, of the
// placement on many, which for every 64 ids of a wave is a chain of ballots and
// an LDS update, then 4-byte stores into the groups' runs.  Up to
// kOneBlockRows rows one workgroup does all in one launch.  Beyond, a count
// per (group, block) and the placement, whose blocks each add up the counts of
// those before them; where that would be too many counts to read in every
// block, a prefix sum over them in between.  1,000 rows: 4 us on the device;
// 16,384 in 16 groups: 13 us the call (one workgroup alone: 18 on the device);
// 1.7M in 26: 4 + 13.6 on the device (with a prefix sum between 5 more, and its
// launch).
#include "dense.h"
#include "scan.h"

namespace htl {
namespace {

constexpr int64_t kOneBlockRows = 4096;
constexpr int64_t kBlockRows = 1024;
constexpr int kMaxBlocks = 512, kSumBlocks = 256;
constexpr int64_t kSumCounts = 16384;      // counts that every block may read
constexpr int64_t kScanOneBlock = 4095;    // entries the prefix sum handles in one launch

__device__ __forceinline__ int bin_of(int32_t id, int n_groups) {
    return (uint32_t)id < (uint32_t)n_groups ? id : n_groups;
}

// counts[bin * nblocks + block] of each block's rows.
__global__ __launch_bounds__(1024) void k_group_count(const int32_t* __restrict__ ids, int64_t m, int64_t per_block,
                                                     int n_groups, int32_t* __restrict__ counts) {
    extern __shared__ int32_t s_cnt[];
    for (int b = threadIdx.x; b <= n_groups; b += blockDim.x) s_cnt[b] = 0;
    __syncthreads();
    const int64_t beg = blockIdx.x * per_block, end = beg + per_block < m ? beg + per_block : m;
    for (int64_t i = beg + threadIdx.x; i < end; i += blockDim.x) atomicAdd(&s_cnt[bin_of(ids[i], n_groups)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= n_groups; b += blockDim.x)
        counts[(int64_t)b * gridDim.x + blockIdx.x] = s_cnt[b];
}

// Each wave takes a contiguous run of the block's rows, so ranks within a
// wave, then waves in order, then blocks in order give the stable place.
// s_pos[wave][bin]: first the wave's counts, then the next place of the bin.
// base: the scanned counts.  Without them the block adds up counts (null when
// one block holds every row) and scans its bins itself (n_groups < 1024 then,
// and 1,024 threads).
__global__ __launch_bounds__(1024) void k_group_place(const int32_t* __restrict__ ids, int64_t m, int64_t per_block,
                                                     int n_groups, int id_bits, const int32_t* __restrict__ base,
                                                     const int32_t* __restrict__ counts,
                                                     int32_t* __restrict__ order, int32_t* __restrict__ offsets) {
    extern __shared__ int32_t s_pos[];
    __shared__ int32_t s_wave[16], s_before[1024], s_total[1024];
    const int nw = blockDim.x >> 6, w = threadIdx.x >> 6, lane = __lane_id();
    const int nb = n_groups + 1;
    for (int b = threadIdx.x; b < nw * nb; b += blockDim.x) s_pos[b] = 0;
    __syncthreads();
    const int64_t beg = blockIdx.x * per_block, end = beg + per_block < m ? beg + per_block : m;
    const int64_t run = ((uint32_t)(end - beg) / nw / 64 + 1) * 64;
    const int64_t wbeg = beg + w * run < end ? beg + w * run : end;
    const int64_t wend = wbeg + run < end ? wbeg + run : end;
    // eight loads at a time: one after the other, they were most of the time
    int bin[8];
    auto read = [&](int64_t i0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t i = i0 + q * 64 + lane;
            bin[q] = i < wend ? ids[i] : 0;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) bin[q] = bin_of(bin[q], n_groups);
    };
    for (int64_t i0 = wbeg; i0 < wend; i0 += 512) {
        read(i0);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (i0 + q * 64 + lane < wend) atomicAdd(&s_pos[w * nb + bin[q]], 1);
    }
    __syncthreads();
    if (base) {
        for (int b = threadIdx.x; b < nb; b += blockDim.x) {
            int32_t at = base[(int64_t)b * gridDim.x + blockIdx.x];
            if (blockIdx.x == 0) offsets[b] = at;
            for (int q = 0; q < nw; ++q) {
                const int32_t c = s_pos[q * nb + b];
                s_pos[q * nb + b] = at;
                at += c;
            }
        }
    } else {
        if (counts) {                       // a wave per bin
            for (int b = w; b < nb; b += nw) {
                int32_t before = 0, total = 0;
                for (int q = lane; q < (int)gridDim.x; q += 64) {
                    const int32_t c = counts[(int64_t)b * gridDim.x + q];
                    total += c;
                    if (q < (int)blockIdx.x) before += c;
                }
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    total += __shfl_xor(total, off);
                    before += __shfl_xor(before, off);
                }
                if (lane == 0) {
                    s_total[b] = total;
                    s_before[b] = before;
                }
            }
            __syncthreads();
        }
        const int b = threadIdx.x;
        int32_t total = 0;
        if (b < nb) {
            if (counts) total = s_total[b];
            else
                for (int q = 0; q < nw; ++q) total += s_pos[q * nb + b];
        }
        int32_t incl = total;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int32_t y = __shfl_up(incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 63) s_wave[w] = incl;
        __syncthreads();
        int32_t at = incl - total;
        for (int q = 0; q < w; ++q) at += s_wave[q];
        if (b < nb) {
            if (blockIdx.x == 0) offsets[b] = at;
            if (counts) at += s_before[b];
            for (int q = 0; q < nw; ++q) {
                const int32_t c = s_pos[q * nb + b];
                s_pos[q * nb + b] = at;
                at += c;
            }
        }
    }
    __syncthreads();
    for (int64_t i0 = wbeg; i0 < wend; i0 += 512) {
        if (run > 512) read(i0);            // else they are there from the count
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t i = i0 + q * 64 + lane;
            if (i - lane >= wend) break;
            const bool in = i < wend;
            const int b = bin[q];
            uint64_t same = __ballot(in);       // lanes of the same bin
            for (int k = 0; k < id_bits; ++k) {
                const bool bit = (b >> k) & 1;
                const uint64_t v = __ballot(bit);
                same &= bit ? v : ~v;
            }
            const int first = __ffsll((unsigned long long)same) - 1;
            int32_t at = 0;
            if (in && lane == first) at = atomicAdd(&s_pos[w * nb + b], __popcll(same));
            at = __shfl(at, in ? first : lane);
            if (in) order[at + __popcll(same & lanemask_lt())] = (int32_t)i;
        }
    }
}

// Blocks of rows, and whether the placement adds up their counts itself.
int64_t group_blocks(int64_t m, int n_groups, bool& summed) {
    int64_t nb = m / kBlockRows;
    nb = nb < 1 ? 1 : (nb > kMaxBlocks ? kMaxBlocks : nb);
    int64_t most = kSumCounts / (n_groups + 1);
    if (most > kSumBlocks) most = kSumBlocks;
    summed = n_groups < 1024 && (most >= nb || most >= 128);
    if (summed) return nb < most ? nb : most;
    nb = nb < m / 4096 ? nb : (m / 4096 < 1 ? 1 : m / 4096);
    // a prefix sum of one launch, where that leaves blocks enough to fill the device
    const int64_t one = kScanOneBlock / (n_groups + 1);
    return nb > one && one >= 128 ? one : nb;
}

}  // namespace
}  // namespace htl

using namespace htl;

extern "C" size_t row_groups_workspace_bytes(int64_t m, int n_groups) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups) return 0;
    bool summed;
    const int64_t entries = (int64_t)(n_groups + 1) * group_blocks(m, n_groups, summed);
    return align_up((size_t)entries * 4, 256) + align_up((size_t)(entries + 1) * 4, 256) +
           align_up(scan_temp_bytes(entries), 256);
}

extern "C" htl_status row_groups(const int32_t* ids, int64_t m, int n_groups, int32_t* order, int32_t* offsets,
                                 void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, "row_groups: row count out of range");
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, "row_groups: group count out of range");
    HTL_REQUIRE(offsets && (m == 0 || (ids && order)), "row_groups: null pointer");
    HTL_REQUIRE(aligned(ids, 4) && aligned(order, 4) && aligned(offsets, 4), "row_groups: misaligned pointer");
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= row_groups_workspace_bytes(m, n_groups),
                "row_groups: workspace too small or misaligned");
    int bits = 0;
    while (n_groups >> bits) ++bits;
    // the places of 16 waves fit in 64 KiB up to 1,023 groups, of 4 waves up to 4,095
    const int threads = n_groups < 1024 ? 1024 : 256;
    const size_t lds = (size_t)(threads / 64) * (n_groups + 1) * 4;
    if (m <= kOneBlockRows && n_groups < 1024) {
        hipLaunchKernelGGL(k_group_place, dim3(1), dim3(threads), lds, stream, ids, m, m, n_groups, bits,
                           (const int32_t*)nullptr, (const int32_t*)nullptr, order, offsets);
        return check_launch("row_groups");
    }
    bool summed;
    const int64_t nb = group_blocks(m, n_groups, summed), per = ceil_div(m, nb);
    const int64_t entries = (int64_t)(n_groups + 1) * nb;
    int32_t* counts = (int32_t*)ws;
    int32_t* base = (int32_t*)((char*)ws + align_up((size_t)entries * 4, 256));
    void* tmp = (char*)base + align_up((size_t)(entries + 1) * 4, 256);
    hipLaunchKernelGGL(k_group_count, dim3((unsigned)nb), dim3(1024), (size_t)(n_groups + 1) * 4, stream, ids, m, per,
                       n_groups, counts);
    if (summed) {
        hipLaunchKernelGGL(k_group_place, dim3((unsigned)nb), dim3(threads), lds, stream, ids, m, per, n_groups, bits,
                           (const int32_t*)nullptr, (const int32_t*)counts, order, offsets);
        return check_launch("row_groups");
    }
    const htl_status st = scan_exclusive_i32(counts, base, entries, nullptr, kScanIdentity, 0, tmp, stream);
    if (st != HTL_OK) return st;
    hipLaunchKernelGGL(k_group_place, dim3((unsigned)nb), dim3(threads), lds, stream, ids, m, per, n_groups, bits,
                       (const int32_t*)base, (const int32_t*)nullptr, order, offsets);
    return check_launch("row_groups");
}
