// bf16 products in tiles of 256 x 256, for operators with much to multiply:
// four waves, each 128 x 128 of the tile's outputs, so that a step's operands
// leave LDS twice (tile.h's eight waves: three times).
//
//   kFwd  out[row] = w_g x[row]       x's rows by the plan's order, or packed by position
//   kDx   out[row] = w_g^T d[pos]     d's rows by position in the plan
//   kDw   out_g = sum_pos d[pos] x[pos]^T     both by position
//
// A stage is 64 elements of the reduction, 32 KiB of each operand, in one of two
// slots.  Halves of a stage alternate: while one half's pieces are multiplied
// from registers the next one's are read, and a slot's loads are issued once all
// waves have read it, two for every sixteen products a wave: a burst of them
// holds up the wave that issues it (8,192-cubed, all at once 958 us, four
// 938, two 897, one and one 876).  A ring of four slots of half a stage, whose
// loads have three times as long, runs no faster (896): it is not their latency
// that bounds it.  Without loads it takes 679 us, without reads from LDS 865,
// with products alone 641: the clock is 1.8 GHz of 2.4 under this load, and at
// that clock the matrix units are busy for 64% of it.
#pragma once

#include "tile.h"

namespace htl {
namespace {

struct Wide {
    static constexpr int BR = 256, BC = 256, WR = 2, WC = 2, kThreads = 256, TR = 8, TC = 8;
};
constexpr int kStage = 64;                               // elements
constexpr int kStageBytes = 256 * kStage * 2;            // of one operand

// f(0), ..., f(N - 1) with numbers the compiler knows: a loop that it leaves as
// one would keep the products' registers in memory.
template <int N, class F, int I = 0> __device__ __forceinline__ void for_each(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        for_each<N, F, I + 1>(static_cast<F&&>(f));
    }
}

// What all loads of a wave write to: its sixteenth of every 4 KiB.
__device__ __forceinline__ char* wide_lds(char* lds, int i) {
    return lds + i * 4096 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
}

// Rows along the reduction, [256 rows][128 bytes]: 16-byte pieces of a row are
// permuted by row bits, so that 16 rows read together hit different banks.
struct WideAlong {
    Buffer buf;
    uint32_t at[8];
    int slot;
    // row_at: of the operand at p, below `rows`; -1: zeros
    template <class F> __device__ __forceinline__ void begin(const void* p, int64_t ld_bytes, int64_t rows, F row_at) {
        slot = (threadIdx.x & 7) ^ ((threadIdx.x >> 4) & 7);
        buf = buffer_of(p, rows * ld_bytes);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = row_at(i * 32 + (int)(threadIdx.x >> 3));
            at[i] = row < 0 ? kOutside : (uint32_t)row * (uint32_t)ld_bytes + slot * 16;
        }
    }
    __device__ __forceinline__ void load(int i, char* lds, int e0, int len) const {
        load_piece(buf, e0 + slot * 8 < len ? at[i] : kOutside, e0 < len ? (uint32_t)e0 * 2 : 0, wide_lds(lds, i));
    }
    // half: of the stage; at: of lane_wide
    static __device__ __forceinline__ int lane(int r0) {
        const int l = __lane_id(), r = l & 15;
        return (r0 + r) * 128 + ((l >> 4) ^ ((r >> 1) & 7)) * 16;
    }
    static __device__ __forceinline__ void read(const char* lds, int at, int i, int half, Frag<kSrcBf16>& f) {
        f.v = *(const bf16x8*)(lds + (at ^ half * 64) + i * 2048);
    }
};

// Consecutive rows across the reduction, [64 rows][256 elements].
struct WideAcross {
    Buffer buf;
    uint32_t ld, at[2];                                  // of even and odd groups of eight rows
    __device__ __forceinline__ void begin(const void* p, int64_t ld_bytes, int64_t rows, int c0, int cols) {
        buf = buffer_of(p, rows * ld_bytes);             // a row past the last lies past the buffer: zeros
        ld = (uint32_t)ld_bytes;
        const int e = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int col = c0 + (int)((threadIdx.x & 31) ^ swap_across<2>(i * 8 + e)) * 8;
            at[i] = col < cols ? e * ld + (uint32_t)col * 2 : kOutside;
        }
    }
    __device__ __forceinline__ void load(int i, char* lds, int e0, int len) const {
        const int e = e0 + i * 8;
        load_piece(buf, e < len ? at[i & 1] : kOutside, e < len ? (uint32_t)e * ld : 0, wide_lds(lds, i));
    }
    static __device__ __forceinline__ int lane(int r0) { return lane_across<kSrcBf16, 256>(r0); }
    static __device__ __forceinline__ void read(const char* lds, int at, int i, int half, Frag<kSrcBf16>& f) {
        frag_across<256>(lds + half * 16384, at, i, f);
    }
};

// A tile and its operands' places.
template <int MODE, bool PAIRS> struct WideTile {
    using RowOp = typename std::conditional<MODE == kDw, WideAcross, WideAlong>::type;
    using ColOp = typename std::conditional<MODE == kFwd, WideAlong, WideAcross>::type;
    static constexpr int BC = PAIRS ? Wide::BC / 2 : Wide::BC;
    TileAt t;
    bool grouped;
    int r0, c0, len;
    RowOp ro;
    ColOp co;

    // The first tile from workgroup number b on, which it leaves at that tile's; false past the last.
    __device__ __forceinline__ bool find(const ProdArgs& p, int64_t& b) {
        const int cols = MODE == kFwd ? p.n : p.k, col_tiles = (cols + BC - 1) / BC;
        const int row_tiles = MODE == kDw ? (p.n + Wide::BR - 1) / Wide::BR : MODE == kDx ? p.splits : 1;
        for (;; b += gridDim.x) {
            const int found = find_tile(p.offsets, p.n_groups, p.m, p.rows, MODE == kDw ? 1 : 0, p.no_rest,
                                        (int64_t)col_tiles * row_tiles, b, t);
            if (found < 0) return false;
            if (!found) continue;
            if (MODE == kDw && t.count > 1 && t.slot >= p.limit) continue;   // offsets that overlap
            break;
        }
        grouped = t.g < p.n_groups;
        r0 = MODE == kDw ? t.col % row_tiles * Wide::BR : 0;
        c0 = (MODE == kDw ? t.col / row_tiles : t.col % col_tiles) * BC;
        if (MODE == kDx) t.slot = t.col / col_tiles;     // a part's tiles lie together
        return true;
    }
    // Its operands, and where its rows go.
    __device__ __forceinline__ void begin(const ProdArgs& p, int32_t* s_row) {
        auto row_at = [&](int r) {
            const int64_t pos = t.beg + r;
            const int32_t row = pos < t.end ? (p.order ? p.order[pos] : (int32_t)pos) : -1;
            return row >= 0 && row < p.m ? row : -1;
        };
        if (MODE != kDw) s_row[threadIdx.x] = row_at(threadIdx.x);
        const int64_t wg = grouped ? (int64_t)t.g * (PAIRS ? 2 : 1) * p.n * p.ldw : 0;
        int first = 0;
        len = !grouped ? 0 : (MODE == kFwd ? p.k : (MODE == kDx ? p.n : (int)(t.end - t.beg)));
        if (MODE == kDx) part_of((int)t.slot, p.splits, kStage, first, len);
        if (len <= 0) return;
        const char* a = (const char*)p.a;
        const char* w = (const char*)p.b;
        if constexpr (MODE == kFwd) {
            if (p.packed) {
                const int rows = (int)(t.end - t.beg);
                ro.begin(a + t.beg * p.lda * 2, p.lda * 2, rows, [&](int r) { return r < rows ? (int64_t)r : -1; });
            } else {
                ro.begin(a, p.lda * 2, p.m, [&](int r) { return (int64_t)row_at(r); });
            }
        } else if constexpr (MODE == kDx) {
            const int rows = (int)(t.end - t.beg);
            ro.begin(a + (t.beg * p.lda + first) * 2, p.lda * 2, rows, [&](int r) { return r < rows ? (int64_t)r : -1; });
        } else {
            ro.begin(a + t.beg * p.lda * 2, p.lda * 2, len, r0, p.n);
        }
        if constexpr (PAIRS) {
            const int n = p.n;                           // of every 128 rows 64 of each half
            co.begin(w + wg * 2, p.ldw * 2, 2 * (int64_t)n, [&](int r) {
                const int col = c0 + r / 128 * 64 + r % 64;
                return col < n ? (int64_t)(r % 128 < 64 ? 0 : n) + col : -1;
            });
        } else if constexpr (MODE == kFwd) {
            const int rows = p.n - c0 < Wide::BC ? p.n - c0 : Wide::BC;
            co.begin(w + (wg + (int64_t)c0 * p.ldw) * 2, p.ldw * 2, rows, [&](int r) { return r < rows ? (int64_t)r : -1; });
        } else if constexpr (MODE == kDx) {
            co.begin(w + (wg + first * p.ldw) * 2, p.ldw * 2, len, c0, p.k);
        } else {
            co.begin(w + t.beg * p.ldb * 2, p.ldb * 2, len, c0, p.k);
        }
    }
    __device__ __forceinline__ void load(int i, char* rows, char* cls, int stage) const {
        ro.load(i, rows, stage * kStage, len);
        co.load(i, cls, stage * kStage, len);
    }
};

// kDx: the reduction is cut into p.splits parts, a tile each, whose number is
// t.slot.
//
// A workgroup takes one tile after another, and the next one's first two stages
// are under way while a tile's end runs (a tile of 2,048 elements took 66 us
// beside 55 of products where it began with the search and those loads).
template <int MODE, class End> __device__ __forceinline__ void wide_tiles(const ProdArgs& p, const End& end) {
    using C = Wide;
    constexpr bool kPairs = End::kPairs;
    __shared__ __attribute__((aligned(128))) char row0[kStageBytes];
    __shared__ __attribute__((aligned(128))) char col0[kStageBytes];
    __shared__ __attribute__((aligned(128))) char row1[kStageBytes];
    __shared__ __attribute__((aligned(128))) char col1[kStageBytes];
    __shared__ int32_t s_rows[2][MODE == kDw ? 1 : C::BR];
    using Tile_ = WideTile<MODE, kPairs>;
    using RowOp = typename Tile_::RowOp;
    using ColOp = typename Tile_::ColOp;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wv / C::WC * 128, wc = wv % C::WC * 128;
    const int cols = MODE == kFwd ? p.n : p.k;
    const int ro_at = RowOp::lane(wr), co_at = ColOp::lane(wc);
    Tile_ cur;
    int64_t b = blockIdx.x;
    if (!cur.find(p, b)) return;
    auto first_loads = [&](const Tile_& o) __attribute__((always_inline)) {
        if (o.len <= 0) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.load(i, row0, col0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) o.load(i, row1, col1, 1);
    };
    cur.begin(p, s_rows[0]);
    first_loads(cur);
    for (int turn = 0;; turn ^= 1) {
        f32x4 acc[C::TC][C::TR];
#pragma unroll
        for (int i = 0; i < C::TC; ++i)
#pragma unroll
            for (int j = 0; j < C::TR; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (cur.len > 0) {
            const int stages = (cur.len + kStage - 1) / kStage;
            struct Pieces { Frag<kSrcBf16> r[8], c[8]; } f0, f1;
            // Read q of a half's 16: the columns' pieces, all of which each row's products need, come first.
            auto read = [&](const char* rows, const char* cls, int q, int half, Pieces& f) __attribute__((always_inline)) {
                if (q < 8) ColOp::read(cls, co_at, q, half, f.c[q]);
                else if (q < 16) RowOp::read(rows, ro_at, q - 8, half, f.r[q - 8]);
            };
            // Eight products.  Their sums are named as both source and result: left to itself the compiler moves
            // them between registers, of which they take half.
            auto products = [&](const Pieces& f, int j) __attribute__((always_inline)) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(f.c[i].v), "v"(f.r[j].v));
                __builtin_amdgcn_sched_barrier(0);
            };
            auto stage = [&](char* rows, char* cls, const char* next_rows, const char* next_cls, int s) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int q = 0; q < 3; ++q) read(rows, cls, j * 3 + q, 1, f1);
                    products(f0, j);
                }
                // all waves have read this stage, and their loads of the next are in
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    cur.load(j, rows, cls, s + 2);       // (past the last stage: zeros)
#pragma unroll
                    for (int q = 0; q < 3; ++q) read(next_rows, next_cls, j * 3 + q, 0, f0);
                    products(f1, j);
                }
            };
            // the first two stages are in, and what the tile before left to be stored is on its way
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int q = 0; q < 16; ++q) read(row0, col0, q, 0, f0);
            // (a product's source stands two instructions after a vector instruction has written it: the zeros above)
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_nop 3");
            for (int s = 0; s < stages; s += 2) {        // an odd number is filled up with zeros
                stage(row0, col0, row1, col1, s);
                stage(row1, col1, row0, col0, s + 1);
            }
            // nothing comes into LDS any more, and the last products' results stand before anything reads them
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
        }
        __syncthreads();                                 // all waves have read the last stage
        Tile_ next;
        b += gridDim.x;
        const bool more = next.find(p, b);
        if (more) {
            next.begin(p, s_rows[turn ^ 1]);
            first_loads(next);
        }
        const bool busy = (MODE == kDw ? cur.r0 + wr < p.n : cur.t.beg + wr < cur.t.end) &&
                          cur.c0 + (kPairs ? wc / 2 : wc) < cols;
        if (busy) {
            for_each<8>([&](auto which) __attribute__((always_inline)) {
                constexpr int j = decltype(which)::value;
                // one row's results leave the products' registers at a time
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("" : "+a"(acc[0][j]), "+a"(acc[1][j]), "+a"(acc[2][j]), "+a"(acc[3][j]), "+a"(acc[4][j]),
                                  "+a"(acc[5][j]), "+a"(acc[6][j]), "+a"(acc[7][j]));
                const int r = wr + j * 16 + (__lane_id() & 15);
                f32x4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = acc[i][j];
                end(cur.t, cur.grouped, cur.r0 + r,
                    MODE != kDw ? (int64_t)s_rows[turn][MODE == kDw ? 0 : r] : (int64_t)(cur.r0 + r < p.n ? cur.r0 + r : -1),
                    cur.c0 + (kPairs ? wc / 2 : wc), v);
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        if (!more) return;
        cur = next;
    }
}

// Workgroups for `tiles` of about the same length: one a unit, which takes them in turn.
inline unsigned wide_grid(int64_t tiles) { return grid_for(align_up((size_t)(tiles < 256 ? tiles : 256), kXcds), 1); }

}  // namespace

// The products of wide.hip.  Rows lie by position in the plan (order nullable:
// rows lie group by group), row strides are multiples of 8 elements, pointers
// 16-byte aligned, and what lies between a row's length and the next multiple
// of 8 is zero in d and finite elsewhere.

// Rows (order nullable: by position in it), `ld` >= k apart (a multiple of 8), with zeros behind their k elements.
htl_status pack_rows(const void* x, int64_t ldx, htl_dtype dtype, const int32_t* order, int64_t m, int64_t src_rows, int k,
                     void* out, int64_t ld, hipStream_t stream);
inline __host__ __device__ int64_t packed_ld(int64_t k) { return (k + 7) / 8 * 8; }
// The same for rows laid out here: rows whole KiB apart share L2 channels (d of 32,768
// columns, dx's product: 874 us, with 64 elements more 808).
inline int64_t spread_ld(int64_t k) { return packed_ld(k) + (packed_ld(k) % 512 ? 0 : 64); }
// Zeros between the `cols` elements of each row and the next multiple of 8.
htl_status zero_behind(void* d, htl_dtype dtype, int64_t m, int cols, int64_t ld, hipStream_t stream);
// Whether rows can be an operand as they lie.
inline bool packed_as_is(const void* p, int64_t ld, int k, htl_dtype dtype = HTL_BF16) {
    const int piece = dtype == HTL_F32 ? 4 : 8;
    return ld % piece == 0 && k % piece == 0 && aligned(p, 16);
}

// dx[row] = w_g^T d[pos] in `splits` parts of the reduction.  With parts
// (float[splits][m][k], by position) they are put there (add: added to what is
// there) for sum_parts to join; without (splits 1) rows of a group are written.
int wide_dx_splits(int64_t m, int n, int k);
htl_status wide_dx(const void* d, int64_t ldd, const void* w, int64_t ldw, int64_t m, int n, int k, const int32_t* order,
                   const int32_t* offsets, int n_groups, void* dx, htl_dtype dx_dtype, float* parts, int splits, bool add,
                   hipStream_t stream);
// dx[order[pos]] = the sum of the parts' rows pos or (by_row) order[pos]; zeros from position *count on (null: m).
htl_status sum_parts(const float* parts, int splits, bool by_row, int64_t m, int k, const int32_t* order,
                     const int32_t* count, void* dx, htl_dtype dx_dtype, hipStream_t stream);
// Zeros for rows order[pos] of `bytes` each, from position *count on.
htl_status zero_rest(void* out, int64_t bytes, int64_t m, const int32_t* order, const int32_t* count, hipStream_t stream);

// dw_g = sum of d[pos] x[pos]^T over the group's positions.  The workspace goes by the row strides; x's
// may be larger in the call where all of x is less than 4 GiB.
size_t wide_dw_bytes(int64_t m, int n_groups, int n, int k, int64_t ldd, int64_t ldx);
htl_status wide_dw(const void* d, int64_t ldd, const void* x, int64_t ldx, int64_t m, int n, int k, const int32_t* offsets,
                   int n_groups, void* dw, htl_dtype dw_dtype, void* ws, hipStream_t stream);

}  // namespace htl
