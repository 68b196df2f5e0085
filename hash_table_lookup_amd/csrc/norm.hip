// A norm per row with its group's parameters, before a block ([MTGR] section
// 4 describes a layer norm per token group; RMS is the other kind), and its
// backward pass, from the input or from its 8-bit copy.
//
//   n = (x - [mean x]) * r,  r = 1 / sqrt(mean (x - [mean x])^2 + eps)
//   y = n w_g + b_g;                        rows of no group: y = 0
//   d = dy w_g;  dx = dres + r (d - [mean d] - n mean(d n))
//   dw_g = sum dy n,  db_g = sum dy;        rows of no group: dx = dres
//
// Bound: bytes and instructions alike.  On 1.7M bf16 rows of 128 in 26 groups
// the forward pass with its 8-bit copy takes 242 us (238-267; 1,097 MB: 4.5
// TB/s), from that copy 158 (668 MB: 4.2 TB/s), the backward pass from that
// copy with a residual gradient 332 (1,533 MB: 4.6 TB/s; 530 with bit
// arithmetic for bf16, LDS shuffles and selects in every element, which the
// lanes do without now).  On long rows bytes decide.  A row is read once into registers (see Hold in dense.h) and
// its statistics are recomputed in the backward pass rather than kept.
#include "dense.h"

namespace htl {
namespace {

struct NormArgs {
    RowsIn x;
    RowsOut y;
    Rows8Out save;
    const float* weight;
    const float* bias;       // nullable
    const int32_t* ids;      // nullable: one group
    int64_t m;
    int dim, n_groups;
    float eps;
    bool center;
};

// A team per row.
template <class H, int TX, int TY>
__global__ __launch_bounds__(H::kThreads) void k_norm(NormArgs a) {
    __shared__ float s_sum[kSumWords];
    Sums sums = {s_sum, 0};
    const int tl = threadIdx.x % H::L;
    const int64_t teams = (int64_t)gridDim.x * H::kTeams;
    int64_t row0 = (int64_t)blockIdx.x * H::kTeams;
    if (row0 >= a.m) return;
    Raw8<TX> raw[H::I];
    int g;
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        const int64_t r = row < a.m ? row : a.m - 1;    // lanes of a wave stay together for the sums
        g = a.ids ? a.ids[r] : 0;
#pragma unroll
        for (int i = 0; i < H::I; ++i) load8(a.x, r, (i * H::L + tl) * 8, a.dim, raw[i]);
    };
    if (H::kAhead) fetch(row0 + threadIdx.x / H::L);
    for (; row0 < a.m; row0 += teams) {
        const int64_t row = row0 + threadIdx.x / H::L;
        const bool in = row < a.m;
        if (!H::kAhead) fetch(row);
        const bool grouped = (uint32_t)g < (uint32_t)a.n_groups;
        float v[H::I][8], w[H::I][8], b[H::I][8];
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = (i * H::L + tl) * 8;
            load_param(a.weight, grouped ? g : 0, col, a.dim, w[i]);
            if (a.bias) load_param(a.bias, grouped ? g : 0, col, a.dim, b[i]);
        }
#pragma unroll
        for (int i = 0; i < H::I; ++i) unpack8(a.x, raw[i], v[i]);
        if (H::kAhead && row0 + teams < a.m) fetch(row + teams);
        if (a.save.codes) {
#pragma unroll
            for (int i = 0; i < H::I; ++i)
                save8(a.save, in ? row : 0, in ? (i * H::L + tl) * 8 : a.dim, a.dim, v[i]);
        }
        normalize<H>(v, a.center, tl, a.dim, a.eps, sums);
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = v[i][j] * w[i][j];
                if (a.bias) y += b[i][j];
                v[i][j] = grouped ? y : 0.0f;
            }
            if (in) store8<TY>(a.y, row, (i * H::L + tl) * 8, a.dim, v[i]);
        }
    }
}

struct NormBackArgs {
    RowsIn dy, x, dres;      // dres.p nullable
    RowsOut dx;
    const float* weight;
    const int32_t* order;    // nullable: rows lie in group order
    const int32_t* offsets;  // nullable: one group
    float* dweight;          // [n_groups][dim]
    float* dbias;            // nullable
    float* partial;          // [limit][dim], dbias's after dweight's
    int64_t chunks, limit;
    int64_t m;
    int dim, n_groups;
    uint32_t rows;           // positions per chunk
    float eps;
    bool center;
};

// One workgroup per chunk of a group's rows, so the group's weights and the
// column sums stay in registers over the chunk.  A row's place in order is
// read a row ahead.
template <class H, int TD, int TX, int TR>
__global__ __launch_bounds__(H::kThreads) void k_norm_back(NormBackArgs a) {
    __shared__ float s_sum[kSumWords];
    __shared__ float s_col[H::L <= 64 ? (H::kThreads / 64) * H::I * H::L * 8 : 1];
    Sums sums = {s_sum, 0};
    const int tl = threadIdx.x % H::L;
    const float inv_dim = 1.0f / (float)a.dim;
    Chunk c;
    if (!find_chunk(a.offsets, a.n_groups, a.m, a.rows, 1, blockIdx.x, c)) return;
    const bool grouped = c.g < a.n_groups;
    float w[H::I][8], sw[H::I][8], sb[H::I][8];
    int64_t row = -1, next = -1;
    Raw8<TX> rx[H::I];
    Raw8<TD> rd[H::I];
    Raw8<TR> rr[H::I];
    auto place = [&](int64_t p) {
        const int64_t r = p < c.end ? (a.order ? a.order[p] : p) : -1;
        return r < a.m ? r : -1;
    };
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = r >= 0 ? (i * H::L + tl) * 8 : a.dim;
            load8(a.x, r < 0 ? 0 : r, col, a.dim, rx[i]);
            load8(a.dy, r < 0 ? 0 : r, col, a.dim, rd[i]);
            if (a.dres.p) load8(a.dres, r < 0 ? 0 : r, col, a.dim, rr[i]);
        }
    };
    const int64_t first_p = c.beg + threadIdx.x / H::L;
    row = place(first_p);
    next = place(first_p + H::kTeams);
    if (H::kAhead) fetch(row);
#pragma unroll
    for (int i = 0; i < H::I; ++i) {
        load_param(a.weight, grouped ? c.g : 0, (i * H::L + tl) * 8, a.dim, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[i][j] = sb[i][j] = 0.0f;
    }
    for (int64_t p0 = c.beg; p0 < c.end; p0 += H::kTeams) {
        const bool in = row >= 0;
        const int64_t at = row;
        if (!H::kAhead) fetch(row);
        float v[H::I][8], d[H::I][8];
        Raw8<TR> res[H::I];
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            unpack8(a.x, rx[i], v[i]);
            unpack8(a.dy, rd[i], d[i]);
            res[i] = rr[i];
        }
        row = next;
        if (p0 + H::kTeams < c.end) {
            if (H::kAhead) fetch(row);
            next = place(p0 + 2 * H::kTeams + threadIdx.x / H::L);
        }
        const float r = normalize<H>(v, a.center, tl, a.dim, a.eps, sums);
        float c12[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < H::I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (in) {                // a row left out must not bring a NaN
                    sw[i][j] += d[i][j] * v[i][j];
                    sb[i][j] += d[i][j];
                }
                d[i][j] *= w[i][j];
                c12[0] += d[i][j];
                c12[1] += d[i][j] * v[i][j];
            }
        team_sums<H::L>(c12, sums);
        const float c1 = a.center ? c12[0] * inv_dim : 0.0f, c2 = c12[1] * inv_dim;
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            float add[8];
            if (a.dres.p) {
                unpack8(a.dres, res[i], add);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) add[j] = 0.0f;
            }
            if (grouped) {                   // (the same for the whole chunk)
#pragma unroll
                for (int j = 0; j < 8; ++j) add[j] += r * (d[i][j] - c1 - v[i][j] * c2);
            }
            if (in) store8<TR>(a.dx, at, (i * H::L + tl) * 8, a.dim, add);
        }
    }
    if (!grouped) return;
    const bool alone = c.count == 1;
    if (!alone && c.slot >= a.limit) return;                 // offsets that overlap
    const int64_t first = c.slot * a.dim, whole = (int64_t)c.g * a.dim;
    write_columns<H>(sw, tl, a.dim, s_col, alone ? a.dweight + whole : a.partial + first);
    if (a.dbias)
        write_columns<H>(sb, tl, a.dim, s_col, alone ? a.dbias + whole : a.partial + a.limit * a.dim + first);
}

// 64 columns per workgroup; its 16 waves take every 16th chunk of the group.
__global__ __launch_bounds__(1024) void k_sum_chunks(const float* __restrict__ partial, int64_t limit,
                                                    float* __restrict__ out, float* __restrict__ out2,
                                                    const int32_t* __restrict__ offsets, int n_groups, int64_t m,
                                                    uint32_t R, int64_t width) {
    __shared__ float s[16][64];
    if (blockIdx.z) {                        // the second set of sums
        partial += limit * width;
        out = out2;
    }
    const int g = blockIdx.y, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int64_t first;
    int count;
    chunks_of_group(offsets, n_groups, m, R, 1, g, first, count);
    if (count == 1) return;
    if (first + count > limit) count = first < limit ? (int)(limit - first) : 0;   // offsets that overlap
    for (int64_t d0 = blockIdx.x * 64ll; d0 < width; d0 += gridDim.x * 64ll) {
        const int64_t d = d0 + lane;
        float v = 0.0f;
        if (d < width) {
#pragma unroll 8
            for (int c = w; c < count; c += 16) v += partial[(first + c) * width + d];
        }
        s[w][lane] = v;
        __syncthreads();
        if (w == 0 && d < width) {
            for (int q = 1; q < 16; ++q) v += s[q][lane];
            out[g * width + d] = v;
        }
        __syncthreads();
    }
}

// Wide rows (a matrix each): four columns per thread, in fp32 or rounded to bf16.
template <bool BF16>
__global__ __launch_bounds__(256) void k_sum_wide(const float* __restrict__ partial, int64_t limit,
                                                  void* __restrict__ out, const int32_t* __restrict__ offsets,
                                                  int n_groups, int64_t m, uint32_t R, int64_t width) {
    const int g = blockIdx.y;
    int64_t first;
    int count;
    chunks_of_group(offsets, n_groups, m, R, 1, g, first, count);
    if (count == 1) return;
    if (first + count > limit) count = first < limit ? (int)(limit - first) : 0;   // offsets that overlap
    for (int64_t d = (blockIdx.x * 256ll + threadIdx.x) * 4; d < width; d += gridDim.x * 1024ll) {
        const float* p = partial + first * width + d;
        const int64_t at = g * width + d;
        if (width % 4 == 0) {
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int c = 0; c < count; ++c) v += *(const f32x4*)(p + c * width);
            if (BF16) {
                const u32x2 b = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                store_at<2>((uint16_t*)out + at, b);
            } else {
                store_at<4>((float*)out + at, v);
            }
        } else {
            for (int j = 0; j < 4 && d + j < width; ++j) {
                float v = 0.0f;
#pragma unroll 8
                for (int c = 0; c < count; ++c) v += p[c * width + j];
                if (BF16) ((uint16_t*)out)[at + j] = (uint16_t)f32_to_bf16_bits(v);
                else ((float*)out)[at + j] = v;
            }
        }
    }
}

// Positions per chunk: about H::kChunks chunks, at least four rows for each team.
uint32_t norm_chunk_rows(int64_t m, int dim) {
    int64_t r = 0;
    with_hold(dim, [&](auto h) {
        using H = decltype(h);
        r = ceil_div(m, H::kChunks);
        if (r < H::kTeams * 4) r = H::kTeams * 4;
    });
    return (uint32_t)r;
}

}  // namespace

int64_t norm_chunks(int64_t m, int n_groups, int dim) { return m / norm_chunk_rows(m, dim) + n_groups + 1; }
int64_t norm_slots(int64_t m, int n_groups, int dim) { return split_chunks(m, n_groups, norm_chunk_rows(m, dim)); }
uint32_t norm_rows_per_chunk(int64_t m, int dim) { return norm_chunk_rows(m, dim); }

htl_status sum_chunks(const float* partial, int64_t limit, void* out, float* out2, const int32_t* offsets, int n_groups,
                      int64_t m, uint32_t R, int64_t width, hipStream_t stream, bool bf16) {
    if (m <= (int64_t)R) return HTL_OK;      // every group is one chunk
    if (bf16 || (width >= 65536 && !out2)) {
        const int64_t blocks = ceil_div(width, 1024), most = ceil_div(4096, n_groups);
        const dim3 grid((unsigned)(blocks < most ? blocks : most), (unsigned)n_groups);
        if (bf16) hipLaunchKernelGGL(k_sum_wide<true>, grid, dim3(256), 0, stream, partial, limit, out, offsets, n_groups, m, R, width);
        else hipLaunchKernelGGL(k_sum_wide<false>, grid, dim3(256), 0, stream, partial, limit, out, offsets, n_groups, m, R, width);
        return check_launch("partial sums");
    }
    const int64_t cols = ceil_div(width, 64);
    hipLaunchKernelGGL(k_sum_chunks, dim3((unsigned)(cols < 4096 ? cols : 4096), (unsigned)n_groups, out2 ? 2 : 1),
                       dim3(1024), 0, stream, partial, limit, (float*)out, out2, offsets, n_groups, m, R, width);
    return check_launch("partial sums");
}

}  // namespace htl

using namespace htl;

namespace {

int elem(htl_dtype t) { return t == HTL_F32 ? 4 : 2; }
bool known(htl_dtype t) { return t == HTL_F32 || t == HTL_BF16; }

template <class H> void launch_norm(const NormArgs& a, int tx, int ty, hipStream_t s) {
    const dim3 grid(grid_for(a.m, H::kTeams, H::kGrid)), block(H::kThreads);
#define NORM_CASE(TX, TY) hipLaunchKernelGGL((k_norm<H, TX, TY>), grid, block, 0, s, a)
    if (tx == kSrcF32 && ty == kSrcF32) NORM_CASE(kSrcF32, kSrcF32);
    else if (tx == kSrcF32) NORM_CASE(kSrcF32, kSrcBf16);
    else if (tx == kSrcBf16 && ty == kSrcF32) NORM_CASE(kSrcBf16, kSrcF32);
    else if (tx == kSrcBf16) NORM_CASE(kSrcBf16, kSrcBf16);
    else if (ty == kSrcF32) NORM_CASE(kSrcRows8, kSrcF32);
    else NORM_CASE(kSrcRows8, kSrcBf16);
#undef NORM_CASE
}

template <class H, int TD, int TX, int TR>
void launch_norm_back(const NormBackArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.chunks), block(H::kThreads);
    hipLaunchKernelGGL((k_norm_back<H, TD, TX, TR>), grid, block, 0, s, a);
}

}  // namespace

extern "C" htl_status norm_rows(const void* x, htl_dtype x_dtype, int64_t ldx, const uint8_t* x_scales,
                                htl_rows8_fmt x_fmt, int64_t m, int dim, const float* weight, const float* bias,
                                const int32_t* ids, int n_groups, htl_norm_kind kind, float eps, void* y,
                                htl_dtype y_dtype, uint8_t* codes, uint8_t* scales, htl_rows8_fmt fmt,
                                hipStream_t stream) {
    clear_error();
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, "norm_rows: row count out of range");
    HTL_REQUIRE(dim >= 1 && dim <= kMaxNormDim, "norm_rows: dim out of range");
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, "norm_rows: group count out of range");
    HTL_REQUIRE(kind == HTL_NORM_RMS || kind == HTL_NORM_LAYER, "norm_rows: unknown kind");
    HTL_REQUIRE(known(x_dtype) && known(y_dtype), "norm_rows: dtypes must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(eps >= 0.0f, "norm_rows: eps must not be negative");
    HTL_REQUIRE(ids || n_groups == 1, "norm_rows: several groups need ids");
    HTL_REQUIRE(!codes == !scales, "norm_rows: codes and scales come together");
    HTL_REQUIRE((fmt == HTL_ROWS8_I8 || fmt == HTL_ROWS8_E4M3) && (x_fmt == HTL_ROWS8_I8 || x_fmt == HTL_ROWS8_E4M3),
                "norm_rows: unknown 8-bit format");
    HTL_REQUIRE(!(codes && x_scales), "norm_rows: x is in 8 bits already");
    HTL_REQUIRE(ldx >= dim, "norm_rows: row stride below dim");
    if (m == 0) return HTL_OK;
    const int xe = x_scales ? 1 : elem(x_dtype), ye = elem(y_dtype);
    HTL_REQUIRE(x && weight && y, "norm_rows: null pointer");
    HTL_REQUIRE(aligned(x, xe) && aligned(y, ye) && aligned(weight, 4) && aligned(bias, 4) && aligned(ids, 4),
                "norm_rows: misaligned pointer");
    NormArgs a;
    a.x = {x, x_scales, ldx, (int)x_fmt};
    a.y = {y, dim};
    a.save = {codes, scales, (int)fmt};
    a.weight = weight;
    a.bias = bias;
    a.ids = ids;
    a.m = m;
    a.dim = dim;
    a.n_groups = n_groups;
    a.eps = eps;
    a.center = kind == HTL_NORM_LAYER;
    const int tx = x_scales ? kSrcRows8 : (int)x_dtype;
    with_hold(dim, [&](auto h) { launch_norm<decltype(h)>(a, tx, (int)y_dtype, stream); });
    return check_launch("norm_rows");
}

extern "C" size_t norm_back_workspace_bytes(int64_t m, int n_groups, int dim) {
    if (m < 0 || m > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || dim < 1 || dim > kMaxNormDim) return 0;
    // partial sums of the weight's and the bias's gradients, a row per chunk of a split group each
    return align_up((size_t)(2 * norm_slots(m, n_groups, dim) * dim) * 4 + 1, 256);
}

extern "C" htl_status norm_rows_backward(const void* dy, htl_dtype dy_dtype, int64_t ld_dy, const void* x,
                                         htl_dtype x_dtype, int64_t ldx, const uint8_t* x_scales, htl_rows8_fmt x_fmt,
                                         const void* dres, int64_t ld_dres, int64_t m, int dim, const float* weight,
                                         const int32_t* order, const int32_t* offsets, int n_groups,
                                         htl_norm_kind kind, float eps, void* dx, float* dweight, float* dbias,
                                         void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, "norm_rows_backward: row count out of range");
    HTL_REQUIRE(dim >= 1 && dim <= kMaxNormDim, "norm_rows_backward: dim out of range");
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, "norm_rows_backward: group count out of range");
    HTL_REQUIRE(kind == HTL_NORM_RMS || kind == HTL_NORM_LAYER, "norm_rows_backward: unknown kind");
    HTL_REQUIRE(known(x_dtype) && known(dy_dtype), "norm_rows_backward: dtypes must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(x_fmt == HTL_ROWS8_I8 || x_fmt == HTL_ROWS8_E4M3, "norm_rows_backward: unknown 8-bit format");
    HTL_REQUIRE(eps >= 0.0f, "norm_rows_backward: eps must not be negative");
    HTL_REQUIRE(offsets || (n_groups == 1 && !order), "norm_rows_backward: several groups need offsets");
    HTL_REQUIRE(ldx >= dim && ld_dy >= dim && (!dres || ld_dres >= dim), "norm_rows_backward: row stride below dim");
    const int xe = x_scales ? 1 : elem(x_dtype), de = elem(dy_dtype), re = elem(x_dtype);
    HTL_REQUIRE(weight && dweight && (m == 0 || (dy && x && dx)), "norm_rows_backward: null pointer");
    HTL_REQUIRE(aligned(x, xe) && aligned(dy, de) && aligned(dres, re) && aligned(dx, re) && aligned(weight, 4) &&
                    aligned(dweight, 4) && aligned(dbias, 4) && aligned(order, 4) && aligned(offsets, 4),
                "norm_rows_backward: misaligned pointer");
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= norm_back_workspace_bytes(m, n_groups, dim),
                "norm_rows_backward: workspace too small or misaligned");
    NormBackArgs a;
    a.dy = {dy, nullptr, ld_dy, 0};
    a.x = {x, x_scales, ldx, (int)x_fmt};
    a.dres = {dres, nullptr, ld_dres, 0};
    a.dx = {dx, dim};
    a.weight = weight;
    a.order = order;
    a.offsets = offsets;
    a.dweight = dweight;
    a.dbias = dbias;
    a.partial = (float*)ws;
    a.rows = norm_rows_per_chunk(m, dim);
    a.chunks = norm_chunks(m, n_groups, dim);
    a.limit = norm_slots(m, n_groups, dim);
    a.m = m;
    a.dim = dim;
    a.n_groups = n_groups;
    a.eps = eps;
    a.center = kind == HTL_NORM_LAYER;
    const bool d32 = dy_dtype == HTL_F32, x32 = x_dtype == HTL_F32;
    with_hold(dim, [&](auto h) {
        using H = decltype(h);
        if (x_scales) {
            if (d32 && x32) launch_norm_back<H, kSrcF32, kSrcRows8, kSrcF32>(a, stream);
            else if (d32) launch_norm_back<H, kSrcF32, kSrcRows8, kSrcBf16>(a, stream);
            else if (x32) launch_norm_back<H, kSrcBf16, kSrcRows8, kSrcF32>(a, stream);
            else launch_norm_back<H, kSrcBf16, kSrcRows8, kSrcBf16>(a, stream);
        } else {
            if (d32 && x32) launch_norm_back<H, kSrcF32, kSrcF32, kSrcF32>(a, stream);
            else if (d32) launch_norm_back<H, kSrcF32, kSrcBf16, kSrcBf16>(a, stream);
            else if (x32) launch_norm_back<H, kSrcBf16, kSrcF32, kSrcF32>(a, stream);
            else launch_norm_back<H, kSrcBf16, kSrcBf16, kSrcBf16>(a, stream);
        }
    });
    const htl_status st = check_launch("norm_rows_backward");
    if (st != HTL_OK) return st;
    return sum_chunks(a.partial, a.limit, dweight, dbias, offsets, n_groups, m, a.rows, dim, stream);
}
