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
#include "dense.h"

#include <type_traits>

namespace htl {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct ProdArgs {
    const void* a;           // x (forward), dy (dx and dw)
    const void* b;           // w, or x (dw)
    void* out;
    const int32_t* order;    // nullable: rows lie in group order
    const int32_t* offsets;  // nullable: one group
    int64_t m, lda, ldb;     // ldb: row stride of x in dw
    int n, k, n_groups;
    uint32_t rows;           // positions per chunk
    float* partial;          // dw: [limit][n][k]
    int out_f32;
    int64_t limit;           // dw: chunks of split groups that `partial` has room for
};

enum { kFwd = 0, kDx = 1, kDw = 2 };

// The output is cut into tiles of BR x BC: rows are x's (dy's) rows of one
// group and columns n (k), or n and k for dw.  A tile is reduced 64 bytes of
// each operand row at a time (a step: 32 bf16 elements or 16 fp32), through a
// ring of four steps in LDS: two steps' loads are under way while a third
// lies ready and the fourth is multiplied, with one barrier a step.
//
// An operand whose reduction runs along its rows in memory ("along") is kept
// as [tile row][64 bytes]; one whose reduction runs across them ("across": w
// in dx, both operands in dw) as [step's elements][tile row], and is
// transposed on the way to the registers.  In both, 16-byte pieces of a row
// are permuted by an exclusive or with row bits, so that the lanes that a
// read serves together hit different banks (no conflict is left by count).
constexpr int kStepBytes = 64, kRing = 4;
template <int BR_, int BC_, int WR_, int WC_> struct Tile {
    static constexpr int BR = BR_, BC = BC_, WR = WR_, WC = WC_;
    static constexpr int kThreads = 64 * WR_ * WC_;
    static constexpr int TR = BR_ / WR_ / 16, TC = BC_ / WC_ / 16;   // 16 x 16 outputs per wave
};

// An operand in global memory, below 4 GiB: pieces come by 32-bit offset (a
// lane's and the wave's; the wave's stays within the operand), and one at
// kOutside (beyond `bytes`) is zeros.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kOutside = 0xFFFFFFF0u;
constexpr int64_t kBufferBytes = 0xFFFF0000ll;
__device__ __forceinline__ Buffer buffer_of(const void* p, int64_t bytes) {
    // raw 32-bit data, no stride: offsets are in bytes and checked against `bytes`
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)(uint32_t)bytes, 0x00020000);
}
// A 16-byte piece from global memory straight into LDS: lane l of the wave
// writes lds + 16 l.
__device__ __forceinline__ void load_piece(Buffer b, uint32_t at, uint32_t add, char* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)lds, 16, (int)at, (int)add, 0, 0);
}
// `left` elements of a piece at any alignment of the element, zeros beyond.
template <int ES> __device__ __forceinline__ u32x4 held_piece(const char* src, int64_t left) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (left >= 16 / ES) {
        __builtin_memcpy(&v, __builtin_assume_aligned(src, ES), 16);
    } else if (ES == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) v[j] = ((const uint32_t*)src)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) v[j >> 1] |= (uint32_t)((const uint16_t*)src)[j] << (16 * (j & 1));
    }
    return v;
}

// Piece number of pass i of a tile of N pieces; with fewer pieces than
// threads some are loaded twice over, so that every wave has the same number
// of loads under way.
template <int NT, int N> __device__ __forceinline__ int piece_at(int i, int t) { return N < NT ? t % N : i * NT + t; }
template <int NT, int N, bool ASYNC> __device__ __forceinline__ void store_pieces(const u32x4* held, char* lds) {
    if (ASYNC) return;
#pragma unroll
    for (int i = 0; i < (N + NT - 1) / NT; ++i) *(u32x4*)(lds + piece_at<NT, N>(i, threadIdx.x) * 16) = held[i];
}
// The wave's first piece of pass i, in bytes.
template <int NT, int N> __device__ __forceinline__ int wave_bytes(int i) {
    return __builtin_amdgcn_readfirstlane(piece_at<NT, N>(i, threadIdx.x & ~63)) * 16;
}

__device__ __forceinline__ int swap_along(int r) { return (r >> 2) & 3; }
// Rows of at least 16 pieces.  bf16: 32 lanes read 32 bytes of rows 0..3 and
// 8..11 (and the next 32 of rows 16 on); fp32: 64 lanes read 64 bytes of each
// of four rows 4 apart.
template <int ES> __device__ __forceinline__ int swap_across(int e) {
    return ES == 4 ? ((e >> 2) & 3) << 2 : ((e & 3) | ((e >> 3) & 1) << 2) << 1;
}

// Keeps the compiler from holding every address that follows from v in a
// register of its own across the loop.
template <class V> __device__ __forceinline__ V recompute(V v) {
    asm volatile("" : "+v"(v));
    return v;
}

// One operand's share of a step, kN pieces per thread, from rows (of x or dy)
// that `row_at` names.  ASYNC: whole pieces, 16-byte aligned, straight into
// LDS; otherwise by way of registers.
template <int ES, int B, int NT, bool ASYNC> struct Along {
    static constexpr int N = B * 4, kN = (N + NT - 1) / NT, VE = 16 / ES;
    static_assert(N % NT == 0 || NT % N == 0, "whole passes");
    Buffer buf;
    uint32_t at[ASYNC ? kN : 1];
    const char* src[ASYNC ? 1 : kN];
    int slot;
    u32x4 held[ASYNC ? 1 : kN];
    template <class F> __device__ __forceinline__ void begin(const void* p, int64_t ld_bytes, int64_t rows, F row_at) {
        // passes are a multiple of 16 rows apart: one permutation for all
        slot = (threadIdx.x & 3) ^ swap_along(threadIdx.x >> 2);
        if (ASYNC) buf = buffer_of(p, rows * ld_bytes);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t row = row_at(piece_at<NT, N>(i, threadIdx.x) >> 2);
            if (ASYNC) at[i] = (uint32_t)row * (uint32_t)ld_bytes + slot * 16;
            else src[i] = (const char*)p + row * ld_bytes + slot * 16;
        }
    }
    __device__ __forceinline__ void load(char* lds, int64_t e0, int64_t len) {
        const int64_t left = len - e0 - slot * VE;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if (ASYNC) load_piece(buf, left > 0 ? at[i] : kOutside, e0 < len ? (uint32_t)e0 * ES : 0, lds + wave_bytes<NT, N>(i));
            else held[i] = held_piece<ES>(src[i] + e0 * ES, left);
        }
    }
    __device__ __forceinline__ void store(char* lds) { store_pieces<NT, N, ASYNC>(held, lds); }
};

// The same from consecutive rows (of w), zeros from row `rows` on.
template <int ES, int B, int NT, bool ASYNC> struct AlongRows {
    static constexpr int N = B * 4, kN = (N + NT - 1) / NT, VE = 16 / ES;
    static_assert(N % NT == 0, "whole passes");
    Buffer buf;
    uint32_t at;
    const char* src;
    int64_t ld;              // bytes
    int slot, rows, all;     // rows: from this lane's first on; all: from the tile's
    u32x4 held[ASYNC ? 1 : kN];
    __device__ __forceinline__ void begin(const char* p, int64_t ld_bytes, int rows_left) {
        slot = (threadIdx.x & 3) ^ swap_along(threadIdx.x >> 2);
        ld = ld_bytes;
        all = rows_left;
        rows = rows_left - (int)(threadIdx.x >> 2);
        if (ASYNC) {
            buf = buffer_of(p, rows_left * ld);
            at = (threadIdx.x >> 2) * (uint32_t)ld + slot * 16;
        } else {
            src = p + (threadIdx.x >> 2) * ld + slot * 16;
        }
    }
    __device__ __forceinline__ void load(char* lds, int64_t e0, int64_t len) {
        const int64_t left = len - e0 - slot * VE;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int64_t have = i * (NT / 4) < rows ? left : 0;
            if (ASYNC)
                load_piece(buf, have > 0 ? at : kOutside,
                           e0 < len && i * (NT / 4) < all ? (uint32_t)e0 * ES + i * (NT / 4) * (uint32_t)ld : 0,
                           lds + wave_bytes<NT, N>(i));
            else
                held[i] = held_piece<ES>(src + e0 * ES + i * (NT / 4) * ld, have);
        }
    }
    __device__ __forceinline__ void store(char* lds) { store_pieces<NT, N, ASYNC>(held, lds); }
};

// Rows of consecutive positions of a chunk, kIds at a time in LDS: a block is
// on its way in registers while the one before is used.
constexpr int kIds = 1024;
template <int NT> struct Rows {
    static constexpr int kN = kIds / NT;
    const int32_t* order;
    int64_t pos, m;
    int32_t raw[kN];
    __device__ __forceinline__ void begin(const int32_t* ord, int64_t beg, int64_t rows) {
        order = ord;
        pos = beg;
        m = rows;
    }
    __device__ __forceinline__ void read(int64_t e0, int64_t len) {
        const int64_t e = e0 + threadIdx.x;
        if (order) {
            const int32_t* at = order + pos;
#pragma unroll
            for (int i = 0; i < kN; ++i) raw[i] = at[e + i * NT < len ? e + i * NT : 0];
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) raw[i] = (int32_t)(pos + e) + i * NT;
        }
    }
    // -1: no row
    __device__ __forceinline__ void store(int32_t* ids, int64_t e0, int64_t len) const {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            ids[threadIdx.x + i * NT] = e0 + threadIdx.x + i * NT < len && raw[i] < m ? raw[i] : -1;
    }
};

// One operand's share of a step whose reduction runs across the rows of a
// matrix: those that ids names (GATHER), or row e0 + e from `base` on.
template <int ES, int B, int NT, bool ASYNC, bool GATHER> struct Across {
    static constexpr int N = B * 4, kN = N / NT, VE = 16 / ES, S = B * ES / 16, kRows = NT / S;
    static_assert(kN * NT == N && S >= 16, "whole passes");
    Buffer buf;
    const char* base;
    int64_t ld;              // bytes
    int cols;                // elements of a row from this tile's first on
    u32x4 held[ASYNC ? 1 : kN];
    // p: the matrix of `rows` rows, c0: the tile's first column
    __device__ __forceinline__ void begin(const void* p, int64_t ld_bytes, int64_t rows, int c0, int cols_in_all) {
        if (ASYNC) buf = buffer_of(p, rows * ld_bytes);
        base = (const char*)p + (int64_t)c0 * ES;
        first = c0 * ES;
        ld = ld_bytes;
        cols = cols_in_all - c0;
    }
    // ids: of the step's elements
    __device__ __forceinline__ void load(char* lds, int64_t e0, int64_t len, const int32_t* ids) {
        const int t = recompute((int)threadIdx.x);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = t / S + i * kRows, col = ((t % S) ^ swap_across<ES>(e)) * VE;
            const int32_t row = GATHER ? ids[e] : 0;
            const int64_t left = (!GATHER || row >= 0) && e0 + e < len ? cols - col : 0;
            if (ASYNC) {
                const uint32_t at = (GATHER ? (uint32_t)row : (uint32_t)(t / S)) * (uint32_t)ld + (uint32_t)first + col * ES;
                load_piece(buf, left > 0 ? at : kOutside,
                           GATHER || e0 + i * kRows >= len ? 0 : (uint32_t)(e0 + i * kRows) * (uint32_t)ld,
                           lds + wave_bytes<NT, N>(i));
            } else {
                held[i] = held_piece<ES>(base + (GATHER ? (int64_t)row : e0 + e) * ld + col * ES, left);
            }
        }
    }
    __device__ __forceinline__ void store(char* lds) { store_pieces<NT, N, ASYNC>(held, lds); }
    int first;
};

template <int T> struct Frag;
template <> struct Frag<kSrcBf16> { bf16x8 v; };
template <> struct Frag<kSrcF32> { f32x4 v; };

// What a lane gives a matrix instruction of 16 tile rows: row l % 16, elements
// (l / 16) * 8 .. + 8 of the step in bf16, (l / 16) * 4 .. + 4 in fp32.
// at: lane_along / lane_across of the lane, once for a tile; i: which 16 rows.
__device__ __forceinline__ int lane_along(int r0) {
    const int lane = __lane_id();
    return (r0 + (lane & 15)) * 64 + ((lane >> 4) ^ swap_along(lane & 15)) * 16;
}
template <int T> __device__ __forceinline__ void frag_along(const char* lds, int at, int i, Frag<T>& f) {
    f.v = *(const decltype(f.v)*)(lds + at + i * 1024);
}
// bf16: 16 lanes read four rows of 16 elements, and each gets one column.
template <int T, int B> __device__ __forceinline__ int lane_across(int r0) {
    const int lane = __lane_id(), q = lane >> 4;
    if (T == kSrcBf16) {
        const int e = q * 8 + ((lane & 15) >> 2);
        return e * B * 2 + (((r0 >> 3) + ((lane & 3) >> 1)) ^ swap_across<2>(e)) * 16 + (lane & 1) * 8;
    }
    return q * 4 * B * 4 + (((r0 >> 2) + ((lane & 15) >> 2)) ^ swap_across<4>(q * 4)) * 16 + (lane & 3) * 4;
}
template <int B> __device__ __forceinline__ void frag_across(const char* lds, int at, int i, Frag<kSrcBf16>& f) {
    const char* p = lds + (at ^ i * 32);
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    union { i16x4 h[2]; bf16x8 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * B * 2));
    f.v = u.v;
}
template <int B> __device__ __forceinline__ void frag_across(const char* lds, int at, int i, Frag<kSrcF32>& f) {
    const char* p = lds + (at ^ i * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = *(const float*)(p + j * B * 4);
}

// Step e of kSteps<T>: one matrix instruction.
template <int T> constexpr int kSteps = T == kSrcF32 ? 4 : 1;
__device__ __forceinline__ void multiply(const Frag<kSrcBf16>& c, const Frag<kSrcBf16>& r, int, f32x4& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c.v, r.v, acc, 0, 0, 0);
}
// fp32 sums are one chain over the reduction.  Their error is 9.6 u of the
// results at 1,024 elements and 19 u at 4,096 (u = 2^-24, root mean squares),
// as the library's fp32 products' is where they do not split the reduction
// (4.9 and 9.6 u where they do).  Sums put aside every 256 elements leave 4.9 u
// at any length, but registers do not hold a second set of them: 20,000 rows,
// 1,024 x 1,024, 331 -> 465 us.
__device__ __forceinline__ void multiply(const Frag<kSrcF32>& c, const Frag<kSrcF32>& r, int e, f32x4& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(c.v[e], r.v[e], acc, 0, 0, 0);
}

// The tile that workgroup number b of the launch takes: consecutive tiles go
// to one XCD (workgroups go round the eight of them), so that its L2 serves
// what neighbours share.  Tiles run group by group, within a group over blocks
// of kBlock chunks, in a block column by column: what is at work at one time
// shares a few chunks' rows and a few columns of the group's matrix.  Sums
// over rows (min_chunks 1) take time by their chunk's length, which differs
// from group to group, so their tiles are dealt out in smaller lots.
struct TileAt {
    int g;
    int64_t beg, end;       // positions
    int64_t slot;           // of its partial sums, where count > 1 (sums over rows)
    int count;              // chunks of the group
    int col;                // which of the `cols` tiles beside each other
};
constexpr int kBlock = 8, kXcds = 8;
// 1: found; 0: nothing at this b; -1: nothing at this or any later b.
__device__ __forceinline__ int search_tile(const int32_t* offsets, int n_groups, int64_t m, uint32_t R, int min_chunks,
                                         int64_t cols, int64_t b, TileAt& t) {
    const int lane = __lane_id();
    auto chunks_at = [&](int g, int64_t& beg, int64_t& end) {
        beg = end = 0;
        int cnt = 0;
        if (g < n_groups || (g == n_groups && offsets)) {
            group_range(offsets, n_groups, m, g, beg, end);
            cnt = (int)(((uint32_t)(end - beg) + R - 1u) / R);
            if (g < n_groups && cnt < min_chunks) cnt = min_chunks;
            if (g == n_groups && min_chunks) cnt = 0;        // sums leave out the rows of no group
        }
        return cnt;
    };
    int64_t total = 0, beg, end;
    for (int g0 = 0; g0 <= n_groups; g0 += 64) {
        int s = chunks_at(g0 + lane, beg, end);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off);
        total += s;
    }
    total *= cols;
    const int64_t x = b % kXcds, i = b / kXcds;
    int64_t item;
    if (min_chunks) {
        const int64_t deal = cols < 2 * kXcds ? 1 : (cols < 16 * kXcds ? cols / kXcds : 16);
        item = (i / deal * kXcds + x) * deal + i % deal;
        if (item >= total) return i / deal * kXcds * deal >= total ? -1 : 0;
    } else {
        const int64_t each = total / kXcds, extra = total % kXcds;
        if (i >= each + (x < extra)) return i > each ? -1 : 0;
        item = x * each + (x < extra ? x : extra) + i;
    }
    int64_t run = 0, alone = 0;
    for (int g0 = 0; g0 <= n_groups; g0 += 64) {
        const int cnt = chunks_at(g0 + lane, beg, end);
        int incl = cnt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int y = __shfl_up(incl, off);
            if (lane >= off) incl += y;
        }
        const uint64_t past = __ballot((run + incl) * cols > item), one = __ballot(cnt == 1);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            t.g = g0 + l;
            t.count = __shfl(cnt, l);
            const int64_t before = run + __shfl(incl, l) - t.count;
            const int64_t local = item - before * cols;
            const int64_t block = local / (cols * kBlock), in = local - block * cols * kBlock;
            const int64_t left = t.count - block * kBlock, width = left < kBlock ? left : kBlock;
            const int col = (int)(in / width);
            const int64_t index = block * kBlock + (in - col * width);
            const int64_t gb = (int64_t)__shfl((int)beg, l), ge = (int64_t)__shfl((int)end, l);
            // sums over rows: chunks of about the same length
            const int64_t len = min_chunks ? ((uint32_t)((ge - gb + t.count - 1) / t.count) + 63u) / 64 * 64 : R;
            const int64_t b0 = gb + index * len < ge ? gb + index * len : ge;
            t.col = col;
            t.slot = before + index - alone - __popcll(one & ((1ull << l) - 1));
            t.beg = b0;
            t.end = b0 + len < ge ? b0 + len : ge;
            return 1;
        }
        run += __shfl(incl, 63);
        alone += __popcll(one);
    }
    return -1;
}

// The same, said to be the same in every lane: what follows from it stays in
// scalar registers.
__device__ __forceinline__ int find_tile(const int32_t* offsets, int n_groups, int64_t m, uint32_t R, int min_chunks,
                                         int64_t cols, int64_t b, TileAt& t) {
    TileAt v = {};
    const int found = search_tile(offsets, n_groups, m, R, min_chunks, cols, b, v);
    t.g = __builtin_amdgcn_readfirstlane(v.g);
    t.beg = __builtin_amdgcn_readfirstlane((int)v.beg);
    t.end = __builtin_amdgcn_readfirstlane((int)v.end);
    t.slot = __builtin_amdgcn_readfirstlane((int)v.slot);
    t.count = __builtin_amdgcn_readfirstlane(v.count);
    t.col = __builtin_amdgcn_readfirstlane(v.col);
    return __builtin_amdgcn_readfirstlane(found);
}

// Writes 16 rows of F * 16 outputs that begin at column `col` of rows of `cols`:
// lane l holds four neighbours of row l % 16 in each of F matrix results, `row`
// being where that row goes (-1: nowhere).  In bf16 four neighbours are 8
// bytes, and a row's 32 bytes of one result would be a store of their own.
// Lanes first exchange, without LDS: in bf16 between 16s of lanes two results
// for eight neighbours of one, then between row r's lane and row r + 8's, so
// that one store fills whole 128-byte lines of eight rows.  (Half lines cost the
// 1.7M x 256 outputs of 26 feature tables 300 us by themselves.)
template <int F>
__device__ __forceinline__ void store_rows(void* out, bool f32, int64_t row, int col, int cols, const f32x4* v) {
    const int lane = __lane_id(), q = lane >> 4;
    const bool high = lane & 8;
    const int64_t other = move_lanes<kRotate8>((int)row);
    const int64_t low_row = high ? other : row, high_row = high ? row : other;
    // a and b of row r's lane (low) and of row r + 8's (high): after it both lanes hold parts of row r in a,
    // the low lane its a and the high lane the low one's b, and parts of row r + 8 in b
    auto exchange = [&](u32x4& a, u32x4& b) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t got = (uint32_t)move_lanes<kRotate8>((int)(high ? a[e] : b[e]));
            a[e] = high ? got : a[e];
            b[e] = high ? b[e] : got;
        }
    };
    if (f32) {
        auto put = [&](int64_t r, int c, const u32x4& w) __attribute__((always_inline)) {
            if (r < 0 || c >= cols) return;
            uint32_t* o = (uint32_t*)out + r * cols + c;
            if (c + 4 <= cols) {
                store_at<4>(o, w);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) o[e] = w[e];
            }
        };
#pragma unroll
        for (int t = 0; t < F; t += 2) {
            u32x4 a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = __float_as_uint(v[t][e]);
                b[e] = __float_as_uint(v[t + 1][e]);
            }
            exchange(a, b);
            const int c = col + t * 16 + (high ? 16 : 0) + q * 4;
            put(low_row, c, a);
            put(high_row, c, b);
        }
        return;
    }
    auto put = [&](int64_t r, int c, const u32x4& w) __attribute__((always_inline)) {
        if (r < 0 || c >= cols) return;
        uint16_t* o = (uint16_t*)out + r * cols + c;
        if (c + 8 <= cols) {
            store_at<2>(o, w);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    };
    u32x4 eight[F / 2];      // result 2 h + q % 2, neighbours q / 2 * 8 on
#pragma unroll
    for (int h = 0; h < F / 2; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16(v[2 * h][2 * e], v[2 * h][2 * e + 1]),
                                                            pack_bf16(v[2 * h + 1][2 * e], v[2 * h + 1][2 * e + 1]), false, false);
            eight[h][e] = x[0];
            eight[h][2 + e] = x[1];
        }
    }
    const int c = col + (q & 1) * 16 + (q >> 1) * 8;
    if constexpr (F == 2) {
        put(row, c, eight[0]);
    } else {
        exchange(eight[0], eight[1]);
        put(low_row, c + (high ? 32 : 0), eight[0]);
        put(high_row, c + (high ? 32 : 0), eight[1]);
    }
}

template <int T, int MODE, class C, bool ASYNC>
__global__ __launch_bounds__(C::kThreads, 2) void k_product(ProdArgs p) {
    // Slots of the ring as variables of their own: the compiler then makes a
    // read of one wait for that slot's loads alone, not for every load into
    // LDS under way.
    constexpr int kSlot = (C::BR + C::BC) * kStepBytes;
    __shared__ int32_t s_ids[MODE == kDw ? 2 * kIds : 1];
    __shared__ int32_t s_row[MODE == kDw ? 1 : C::BR];
    __shared__ __attribute__((aligned(128))) char ring0[kSlot];
    __shared__ __attribute__((aligned(128))) char ring1[kSlot];
    __shared__ __attribute__((aligned(128))) char ring2[kSlot];
    __shared__ __attribute__((aligned(128))) char ring3[kSlot];
    constexpr int ES = T == kSrcF32 ? 4 : 2, NT = C::kThreads, kStep = kStepBytes / ES;
    constexpr int kCols = C::BR * kStepBytes;
    const int lane = __lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wv / C::WC * (C::TR * 16), wc = wv % C::WC * (C::TC * 16);
    const int cols = MODE == kFwd ? p.n : p.k;
    const int col_tiles = (cols + C::BC - 1) / C::BC;
    const int row_tiles = MODE == kDw ? (p.n + C::BR - 1) / C::BR : 1;
    for (int64_t b = blockIdx.x;; b += gridDim.x) {
        TileAt t;
        const int found = find_tile(p.offsets, p.n_groups, p.m, p.rows, MODE == kDw ? 1 : 0,
                                    (int64_t)col_tiles * row_tiles, b, t);
        if (found < 0) return;
        if (!found) continue;
        if (MODE == kDw && t.count > 1 && t.slot >= p.limit) continue;   // offsets that overlap
        const bool grouped = t.g < p.n_groups;
        const int r0 = MODE == kDw ? t.col % row_tiles * C::BR : 0;
        const int c0 = (MODE == kDw ? t.col / row_tiles : t.col) * C::BC;
        __syncthreads();                     // the tile before is read and stored
        if (MODE != kDw) {
            for (int i = threadIdx.x; i < C::BR; i += NT) {
                const int64_t pos = t.beg + i;
                const int32_t row = pos < t.end ? (p.order ? p.order[pos] : (int32_t)pos) : -1;
                s_row[i] = row >= 0 && row < p.m ? row : -1;
            }
            __syncthreads();
        }
        f32x4 acc[C::TC][C::TR];
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int j = 0; j < C::TR; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t len = !grouped ? 0 : (MODE == kFwd ? p.k : (MODE == kDx ? p.n : t.end - t.beg));
        const int64_t wg = grouped ? (int64_t)t.g * p.n * p.k : 0;
        // rows of this wave that exist
        const bool busy = (MODE == kDw ? r0 + wr < p.n : t.beg + wr < t.end) && c0 + wc < cols;
        if (len > 0) {
            using RowOp = typename std::conditional<MODE == kDw, Across<ES, C::BR, NT, ASYNC, true>,
                                                    Along<ES, C::BR, NT, ASYNC>>::type;
            using ColOp = typename std::conditional<MODE == kFwd, AlongRows<ES, C::BC, NT, ASYNC>,
                                                    Across<ES, C::BC, NT, ASYNC, MODE == kDw>>::type;
            RowOp ro;
            ColOp co;
            Rows<NT> rows;
            int ro_at, co_at;
            if constexpr (MODE == kDw) {
                rows.begin(p.order, t.beg, p.m);
                rows.read(0, len);
                ro.begin(p.a, p.lda * ES, p.m, r0, p.n);
                co.begin(p.b, p.ldb * ES, p.m, c0, p.k);
                ro_at = lane_across<T, C::BR>(wr);
                rows.store(s_ids, 0, len);
                rows.read(kIds, len);
                __syncthreads();
            } else {
                // a row that is not there is read as the first that may be: its products are not stored
                ro.begin(p.a, p.lda * ES, p.m, [&](int r) { return s_row[r] < 0 ? 0 : s_row[r]; });
                ro_at = lane_along(wr);
                if constexpr (MODE == kFwd)
                    co.begin((const char*)p.b + (wg + (int64_t)c0 * p.k) * ES, (int64_t)p.k * ES, p.n - c0);
                else
                    co.begin((const char*)p.b + wg * ES, (int64_t)p.k * ES, p.n, c0, p.k);
            }
            if constexpr (MODE == kFwd) co_at = lane_along(C::BR + wc);
            else co_at = kCols + lane_across<T, C::BC>(wc);
            const int steps = (int)((len + kStep - 1) / kStep);
            auto load = [&](char* to, const int32_t* ids, int s) __attribute__((always_inline)) {
                const int64_t e0 = (int64_t)s * kStep;
                if constexpr (MODE == kDw) {
                    ids += (int)(e0 % (2 * kIds));
                    ro.load(to, e0, len, ids);
                    co.load(to + kCols, e0, len, ids);
                } else {
                    ro.load(to, e0, len);
                    if constexpr (MODE == kFwd) co.load(to + kCols, e0, len);
                    else co.load(to + kCols, e0, len, ids);
                }
            };
            auto store = [&](char* to) __attribute__((always_inline)) {
                ro.store(to);
                co.store(to + kCols);
            };
            // Held from step to step: the next one's first pieces.
            constexpr int kHeld = C::TR > 4 ? 3 : 2;
            struct First { Frag<T> c[C::TC], r[kHeld]; } even, odd;
            auto row_frag = [&](const char* at, int j, Frag<T>& f) __attribute__((always_inline)) {
                const int ra = recompute(ro_at);
                if constexpr (MODE == kDw) frag_across<C::BR>(at, ra, j, f);
                else frag_along<T>(at, ra, j, f);
            };
            auto first_frags = [&](const char* at, First& f) __attribute__((always_inline)) {
                const int ca = recompute(co_at);
#pragma unroll
                for (int i = 0; i < C::TC; ++i) {
                    if constexpr (MODE == kFwd) frag_along<T>(at, ca, i, f.c[i]);
                    else frag_across<C::BC>(at, ca, i, f.c[i]);
                }
#pragma unroll
                for (int j = 0; j < kHeld; ++j) row_frag(at, j, f.r[j]);
            };
            constexpr int kAhead = ASYNC ? kRing - 1 : 2, kLoads = RowOp::kN + ColOp::kN;
            // Step s, which lies in `cur`: its products, the next one's first pieces
            // from `next`, and the loads of a later one under way into `to`.
            auto step = [&](const char* cur, const char* next, char* to, int s, First& now, First& then)
                __attribute__((always_inline)) {
                if (s >= -1) {
                    // this wave's loads of step s + 1 are in, and then the other waves' are
                    // (products before this point have what they read from the slot before)
                    __builtin_amdgcn_sched_barrier(0);
                    if (ASYNC) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
                    else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
                if constexpr (MODE == kDw) {
                    // the block of ids after the one that the loads now leave
                    constexpr int kEvery = kIds / kStep;
                    if (s >= 0 && s % kEvery == 0 && (int64_t)(s / kEvery + 1) * kIds < len) {
                        const int64_t e0 = (int64_t)(s / kEvery + 1) * kIds;
                        rows.store(s_ids + (s / kEvery + 1) % 2 * kIds, e0, len);
                        rows.read(e0 + kIds, len);
                    }
                }
                // past the last step pieces of zeros: every step has the same loads under way
                if (ASYNC || s + kAhead < steps) load(to, s_ids, s + kAhead);
                if (busy && s == -1) {
                    first_frags(next, then);
                } else if (busy && s >= 0) {
                    Frag<T> r[C::TR];
#pragma unroll
                    for (int j = kHeld; j < C::TR; ++j) row_frag(cur, j, r[j]);
                    first_frags(next, then);
#pragma unroll
                    for (int e = 0; e < kSteps<T>; ++e)
#pragma unroll
                        for (int j = 0; j < C::TR; ++j)
#pragma unroll
                            for (int i = 0; i < C::TC; ++i) multiply(now.c[i], j < kHeld ? now.r[j < kHeld ? j : 0] : r[j], e, acc[i][j]);
                    if constexpr (T == kSrcBf16 && C::TR >= 4) {
                        // a row piece is read kHeld rows of products ahead; then the next step's first
                        constexpr int RC = MODE == kFwd ? 1 : 2, RR = MODE == kDw ? 2 : 1;   // reads per piece
#pragma unroll
                        for (int j = 0; j < C::TR - kHeld; ++j) {
                            __builtin_amdgcn_sched_group_barrier(0x100, RR, 0);
                            __builtin_amdgcn_sched_group_barrier(0x008, C::TC, 0);
                        }
#pragma unroll
                        for (int j = 0; j < kHeld; ++j) {
                            __builtin_amdgcn_sched_group_barrier(0x100, (C::TC * RC + kHeld * RR + kHeld - 1) / kHeld, 0);
                            __builtin_amdgcn_sched_group_barrier(0x008, C::TC, 0);
                        }
                    }
                }
                if (!ASYNC && s + kAhead < steps) store(to);
            };
            static_assert(kRing == 4, "step s lies in slot s % 4");
            if (ASYNC) step(ring1, ring2, ring0, -3, odd, even);
            step(ring2, ring3, ASYNC ? ring1 : ring0, -2, even, odd);
            step(ring3, ring0, ASYNC ? ring2 : ring1, -1, odd, even);
            for (int s = 0;; s += 4) {
                step(ring0, ring1, ASYNC ? ring3 : ring2, s, even, odd);
                if (s + 1 >= steps) break;
                step(ring1, ring2, ASYNC ? ring0 : ring3, s + 1, odd, even);
                if (s + 2 >= steps) break;
                step(ring2, ring3, ASYNC ? ring1 : ring0, s + 2, even, odd);
                if (s + 3 >= steps) break;
                step(ring3, ring0, ASYNC ? ring2 : ring1, s + 3, odd, even);
                if (s + 4 >= steps) break;
            }
            __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0): nothing comes into LDS any more
        }
        if (!busy) continue;
        void* to = MODE != kDw ? p.out : (t.count == 1 ? (float*)p.out + wg : p.partial + t.slot * p.n * p.k);
#pragma unroll
        for (int j = 0; j < C::TR; ++j) {
            const int r = wr + j * 16 + (lane & 15);
            const int row = MODE != kDw ? s_row[r] : (r0 + r < p.n ? r0 + r : -1);
            f32x4 v[C::TC];
#pragma unroll
            for (int i = 0; i < C::TC; ++i) v[i] = acc[i][j];
            store_rows<C::TC>(to, MODE == kDw || p.out_f32, row, c0 + wc, cols, v);
        }
    }
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
        const int found = find_tile(p.offsets, p.n_groups, p.m, p.rows, 0, 1, b, t);
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
                    store_rows<4>(p.out, p.out_f32, row[j], nb * 64, cols, acc[j]);
                }
            }
            row[0] = next[0];
            row[1] = next[1];
        }
    }
}

typedef Tile<256, 256, 2, 4> Big;
typedef Tile<128, 128, 2, 2> Mid;
typedef Tile<32, 128, 1, 4> Small;

int elem(htl_dtype t) { return t == HTL_F32 ? 4 : 2; }
bool known(htl_dtype t) { return t == HTL_F32 || t == HTL_BF16; }

// chunks: at most this many in all
template <int T, int MODE, class C, bool ASYNC>
void launch(const ProdArgs& p, int64_t chunks, hipStream_t s) {
    const int64_t cols = ceil_div(MODE == kFwd ? p.n : p.k, C::BC) * (MODE == kDw ? ceil_div(p.n, C::BR) : 1);
    const dim3 grid(grid_for(align_up((size_t)(chunks * cols), kXcds), 1));
    hipLaunchKernelGGL((k_product<T, MODE, C, ASYNC>), grid, dim3(C::kThreads), 0, s, p);
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
template <int MODE> void launch_rows(ProdArgs p, htl_dtype dtype, hipStream_t s) {
    const int cols = MODE == kFwd ? p.n : p.k, es = elem(dtype);
    const bool fast = p.lda * es % 16 == 0 && aligned(p.a, 16) && (int64_t)p.k * es % 16 == 0 &&
                      (MODE == kFwd || (int64_t)p.n * es % 16 == 0) && aligned(p.b, 16) &&
                      p.m * p.lda * es <= kBufferBytes && (int64_t)p.n * p.k * es <= kBufferBytes;
    const int64_t each = p.m / p.n_groups;
    const int len = MODE == kFwd ? p.k : p.n, lp = len <= 32 ? 1 : len <= 64 ? 2 : len <= 128 ? 4 : 8;
    const int64_t bytes = ceil_div(cols, 64) * 64 * (lp * 64 + 16);
    if (dtype == HTL_BF16 && len <= 256 && bytes <= 163840 && each >= 512 && p.m >= (lp == 8 ? 1 << 20 : 1 << 16)) {
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
    ProdArgs p = {x, w, y, order, offsets, m, ldx, k, n, k, n_groups, 0, nullptr, y_dtype == HTL_F32, 0};
    launch_rows<kFwd>(p, dtype, stream);
    return check_launch("grouped_mm");
}

extern "C" size_t grouped_mm_backward_workspace_bytes(int64_t m, int n_groups, int n, int k) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || n < 1 || n > HTL_MAX_PRODUCT_DIM || k < 1 ||
        k > HTL_MAX_PRODUCT_DIM)
        return 0;
    if (m <= (int64_t)dw_chunk_rows(m, n, k)) return 256;
    return align_up((size_t)dw_slots(m, n_groups, n, k) * n * k * 4, 256);
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
        const ProdArgs p = {dy, w, dx, order, offsets, m, ld_dy, k, n, k, n_groups, 0, nullptr, dx_dtype == HTL_F32, 0};
        launch_rows<kDx>(p, dtype, stream);
        const htl_status st = check_launch("grouped_mm_backward");
        if (st != HTL_OK) return st;
    }
    if (!dw) return HTL_OK;
    const ProdArgs p = {dy, x, dw, order, offsets, m, ld_dy, ldx, n, k, n_groups, dw_chunk_rows(m, n, k),
                        (float*)ws, 1, dw_slots(m, n_groups, n, k)};
    const int64_t chunks = dw_chunks(m, n_groups, n, k);
    const bool fast = ld_dy * es % 16 == 0 && ldx * es % 16 == 0 && aligned(dy, 16) && aligned(x, 16) &&
                      (int64_t)n * es % 16 == 0 && (int64_t)k * es % 16 == 0 && m * ld_dy * es <= kBufferBytes &&
                      m * ldx * es <= kBufferBytes;
    if (dtype == HTL_BF16) {
        if (fast && n >= 256 && k >= 256) launch<kSrcBf16, kDw, Big, true>(p, chunks, stream);
        else if (fast) launch<kSrcBf16, kDw, Mid, true>(p, chunks, stream);
        else launch<kSrcBf16, kDw, Mid, false>(p, chunks, stream);
    } else {
        if (fast) launch<kSrcF32, kDw, Mid, true>(p, chunks, stream);
        else launch<kSrcF32, kDw, Mid, false>(p, chunks, stream);
    }
    const htl_status st = check_launch("grouped_mm_backward");
    if (st != HTL_OK) return st;
    return sum_chunks(p.partial, p.limit, dw, nullptr, offsets, n_groups, m, p.rows, (int64_t)n * k, stream);
}
