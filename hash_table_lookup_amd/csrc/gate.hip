// The norm after a block, its gate and the residual sum in one pass, and the
// backward pass, from the block's outputs or from their 8-bit copies.
//
//   n = norm(z) (as norm.hip's),  v = n w_g + b_g
//   out = x + scale * act(u) * v;           rows of no group: out = x
//   D = scale * dout
//   du = D act'(u) v
//   d = D act(u) w_g;  dz = r (d - [mean d] - n mean(d n))
//   dw_g = sum D act(u) n,  db_g = sum D act(u);  rows of no group: dz = du = 0
// (the gradient of x is dout itself).  act: u, 1 / (1 + exp(-u)), or
// u / (1 + exp(-u)), as the gates of [MTGR] section 4's encoder (silu) are.
//
// Bound: bytes, and in the backward pass instructions, as norm.hip.  16,384
// bf16 rows of 4,096: forward 110 us (107-126; 537 MB: 4.9 TB/s), backward 153
// (151-157; 671 MB: 4.4 TB/s); 426,000 rows of 128 in 26 groups, fp32 residual,
// e4m3 copies: 147 us (766 MB: 5.2 TB/s) and 144 (548 MB: 3.8 TB/s).
#include "dense.h"

namespace htl {

int64_t norm_chunks(int64_t m, int n_groups, int dim);
int64_t norm_slots(int64_t m, int n_groups, int dim);
uint32_t norm_rows_per_chunk(int64_t m, int dim);

namespace {

struct GateArgs {
    RowsIn x, z, u;
    RowsOut out;
    Rows8Out save_z, save_u;
    const float* weight;
    const float* bias;       // nullable
    const int32_t* ids;      // nullable: one group
    int64_t m;
    int dim, n_groups, act;
    float eps, scale;
    bool center;
};

template <class H, int TX, int TZ>
__global__ __launch_bounds__(H::kThreads) void k_gate(GateArgs a) {
    __shared__ float s_sum[kSumWords];
    Sums sums = {s_sum, 0};
    const int tl = threadIdx.x % H::L;
    const int64_t teams = (int64_t)gridDim.x * H::kTeams;
    int64_t row0 = (int64_t)blockIdx.x * H::kTeams;
    if (row0 >= a.m) return;
    Raw8<TZ> rz[H::I], ru[H::I];
    Raw8<TX> rx[H::I];
    int g;
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        const int64_t r = row < a.m ? row : a.m - 1;
        g = a.ids ? a.ids[r] : 0;
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = (i * H::L + tl) * 8;
            load8(a.z, r, col, a.dim, rz[i]);
            load8(a.u, r, col, a.dim, ru[i]);
            load8(a.x, r, col, a.dim, rx[i]);
        }
    };
    if (H::kAhead) fetch(row0 + threadIdx.x / H::L);
    for (; row0 < a.m; row0 += teams) {
        const int64_t row = row0 + threadIdx.x / H::L;
        const bool in = row < a.m;
        if (!H::kAhead) fetch(row);
        const bool grouped = (uint32_t)g < (uint32_t)a.n_groups;
        float v[H::I][8], w[H::I][8], b[H::I][8], u[H::I][8];
        Raw8<TX> xs[H::I];
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = (i * H::L + tl) * 8;
            load_param(a.weight, grouped ? g : 0, col, a.dim, w[i]);
            if (a.bias) load_param(a.bias, grouped ? g : 0, col, a.dim, b[i]);
        }
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            unpack8(a.z, rz[i], v[i]);
            unpack8(a.u, ru[i], u[i]);
            xs[i] = rx[i];
        }
        if (H::kAhead && row0 + teams < a.m) fetch(row + teams);
        if (a.save_z.codes) {
#pragma unroll
            for (int i = 0; i < H::I; ++i) {
                const int col = in ? (i * H::L + tl) * 8 : a.dim;
                save8(a.save_z, in ? row : 0, col, a.dim, v[i]);
                save8(a.save_u, in ? row : 0, col, a.dim, u[i]);
            }
        }
        normalize<H>(v, a.center, tl, a.dim, a.eps, sums);
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            float x[8];
            unpack8(a.x, xs[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = v[i][j] * w[i][j], slope;
                if (a.bias) y += b[i][j];
                y = a.scale * gate_act(u[i][j], a.act, slope) * y;
                v[i][j] = grouped ? x[j] + y : x[j];
            }
            if (in) store8<TX>(a.out, row, (i * H::L + tl) * 8, a.dim, v[i]);
        }
    }
}

struct GateBackArgs {
    RowsIn dout, z, u;
    RowsOut dz, du;
    const float* weight;
    const float* bias;       // nullable
    const int32_t* order;    // nullable: rows lie in group order
    const int32_t* offsets;  // nullable: one group
    float* dweight;          // [n_groups][dim]
    float* dbias;            // nullable
    float* partial;          // [limit][dim], dbias's after dweight's
    int64_t chunks, limit;
    int64_t m;
    int dim, n_groups, act;
    uint32_t rows;           // positions per chunk
    float eps, scale;
    bool center;
};

template <class H, int TD, int TZ, int TG>
__global__ __launch_bounds__(H::kThreads) void k_gate_back(GateBackArgs a) {
    __shared__ float s_sum[kSumWords];
    __shared__ float s_col[H::L <= 64 ? (H::kThreads / 64) * H::I * H::L * 8 : 1];
    Sums sums = {s_sum, 0};
    const int tl = threadIdx.x % H::L;
    const float inv_dim = 1.0f / (float)a.dim;
    Chunk c;
    if (!find_chunk(a.offsets, a.n_groups, a.m, a.rows, 1, blockIdx.x, c)) return;
    const bool grouped = c.g < a.n_groups;
    float w[H::I][8], b[H::I][8], sw[H::I][8], sb[H::I][8];
    int64_t row = -1, next = -1;
    Raw8<TZ> rz[H::I], ru[H::I];
    Raw8<TD> rd[H::I];
    auto place = [&](int64_t p) {
        const int64_t r = p < c.end ? (a.order ? a.order[p] : p) : -1;
        return r < a.m ? r : -1;
    };
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            const int col = r >= 0 ? (i * H::L + tl) * 8 : a.dim;
            load8(a.z, r < 0 ? 0 : r, col, a.dim, rz[i]);
            load8(a.u, r < 0 ? 0 : r, col, a.dim, ru[i]);
            load8(a.dout, r < 0 ? 0 : r, col, a.dim, rd[i]);
        }
    };
    const int64_t first_p = c.beg + threadIdx.x / H::L;
    row = place(first_p);
    next = place(first_p + H::kTeams);
    if (H::kAhead) fetch(row);
#pragma unroll
    for (int i = 0; i < H::I; ++i) {
        const int col = (i * H::L + tl) * 8;
        load_param(a.weight, grouped ? c.g : 0, col, a.dim, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[i][j] = sb[i][j] = b[i][j] = 0.0f;
        if (a.bias) load_param(a.bias, grouped ? c.g : 0, col, a.dim, b[i]);
    }
    for (int64_t p0 = c.beg; p0 < c.end; p0 += H::kTeams) {
        const bool in = row >= 0;
        const int64_t at = row;
        if (!H::kAhead) fetch(row);
        float v[H::I][8], d[H::I][8], u[H::I][8];
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
            unpack8(a.z, rz[i], v[i]);
            unpack8(a.u, ru[i], u[i]);
            unpack8(a.dout, rd[i], d[i]);
        }
        row = next;
        if (p0 + H::kTeams < c.end) {
            if (H::kAhead) fetch(row);
            next = place(p0 + 2 * H::kTeams + threadIdx.x / H::L);
        }
        const float r = normalize<H>(v, a.center, tl, a.dim, a.eps, sums);
        float c12[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float slope;
                const float D = a.scale * d[i][j], act = gate_act(u[i][j], a.act, slope), e = D * act;
                u[i][j] = D * slope * (v[i][j] * w[i][j] + b[i][j]);
                if (in) {                // a row left out must not bring a NaN
                    sw[i][j] += e * v[i][j];
                    sb[i][j] += e;
                }
                d[i][j] = e * w[i][j];
                c12[0] += d[i][j];
                c12[1] += d[i][j] * v[i][j];
            }
            if (!grouped) {                  // (the same for the whole chunk)
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] = 0.0f;
            }
            if (in) store8<TG>(a.du, at, (i * H::L + tl) * 8, a.dim, u[i]);
        }
        team_sums<H::L>(c12, sums);
        const float c1 = a.center ? c12[0] * inv_dim : 0.0f, c2 = c12[1] * inv_dim;
#pragma unroll
        for (int i = 0; i < H::I; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = r * (d[i][j] - c1 - v[i][j] * c2);
            if (!grouped) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = 0.0f;
            }
            if (in) store8<TG>(a.dz, at, (i * H::L + tl) * 8, a.dim, d[i]);
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

int elem(htl_dtype t) { return t == HTL_F32 ? 4 : 2; }
bool known(htl_dtype t) { return t == HTL_F32 || t == HTL_BF16; }

template <class H, int TX, int TZ> void launch_gate(const GateArgs& a, hipStream_t s) {
    const dim3 grid(grid_for(a.m, H::kTeams, H::kGrid)), block(H::kThreads);
    hipLaunchKernelGGL((k_gate<H, TX, TZ>), grid, block, 0, s, a);
}

template <class H, int TD, int TZ, int TG> void launch_gate_back(const GateBackArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.chunks), block(H::kThreads);
    hipLaunchKernelGGL((k_gate_back<H, TD, TZ, TG>), grid, block, 0, s, a);
}

}  // namespace
}  // namespace htl

using namespace htl;

extern "C" htl_status norm_gate(const void* x, htl_dtype x_dtype, int64_t ldx, const void* z, int64_t ldz,
                                const void* u, int64_t ldu, htl_dtype z_dtype, int64_t m, int dim,
                                const float* weight, const float* bias, const int32_t* ids, int n_groups,
                                htl_norm_kind kind, float eps, htl_act act, float scale, void* out, uint8_t* z_codes,
                                uint8_t* z_scales, uint8_t* u_codes, uint8_t* u_scales, htl_rows8_fmt fmt,
                                hipStream_t stream) {
    clear_error();
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, "norm_gate: row count out of range");
    HTL_REQUIRE(dim >= 1 && dim <= kMaxNormDim, "norm_gate: dim out of range");
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, "norm_gate: group count out of range");
    HTL_REQUIRE(kind == HTL_NORM_RMS || kind == HTL_NORM_LAYER, "norm_gate: unknown kind");
    HTL_REQUIRE(act == HTL_ACT_NONE || act == HTL_ACT_SIGMOID || act == HTL_ACT_SILU, "norm_gate: unknown activation");
    HTL_REQUIRE(known(x_dtype) && known(z_dtype), "norm_gate: dtypes must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(fmt == HTL_ROWS8_I8 || fmt == HTL_ROWS8_E4M3, "norm_gate: unknown 8-bit format");
    HTL_REQUIRE(eps >= 0.0f, "norm_gate: eps must not be negative");
    HTL_REQUIRE(ids || n_groups == 1, "norm_gate: several groups need ids");
    HTL_REQUIRE(!z_codes == !z_scales && !z_codes == !u_codes && !z_codes == !u_scales,
                "norm_gate: the codes and scales of z and u come together");
    HTL_REQUIRE(ldx >= dim && ldz >= dim && ldu >= dim, "norm_gate: row stride below dim");
    if (m == 0) return HTL_OK;
    const int xe = elem(x_dtype), ze = elem(z_dtype);
    HTL_REQUIRE(x && z && u && weight && out, "norm_gate: null pointer");
    HTL_REQUIRE(aligned(x, xe) && aligned(out, xe) && aligned(z, ze) && aligned(u, ze) && aligned(weight, 4) &&
                    aligned(bias, 4) && aligned(ids, 4),
                "norm_gate: misaligned pointer");
    GateArgs a;
    a.x = {x, nullptr, ldx, 0};
    a.z = {z, nullptr, ldz, 0};
    a.u = {u, nullptr, ldu, 0};
    a.out = {out, dim};
    a.save_z = {z_codes, z_scales, (int)fmt};
    a.save_u = {u_codes, u_scales, (int)fmt};
    a.weight = weight;
    a.bias = bias;
    a.ids = ids;
    a.m = m;
    a.dim = dim;
    a.n_groups = n_groups;
    a.act = (int)act;
    a.eps = eps;
    a.center = kind == HTL_NORM_LAYER;
    a.scale = scale;
    const bool x32 = x_dtype == HTL_F32, z32 = z_dtype == HTL_F32;
    with_hold(dim, [&](auto h) {
        using H = decltype(h);
        if (x32 && z32) launch_gate<H, kSrcF32, kSrcF32>(a, stream);
        else if (x32) launch_gate<H, kSrcF32, kSrcBf16>(a, stream);
        else if (z32) launch_gate<H, kSrcBf16, kSrcF32>(a, stream);
        else launch_gate<H, kSrcBf16, kSrcBf16>(a, stream);
    });
    return check_launch("norm_gate");
}

extern "C" htl_status norm_gate_backward(const void* dout, htl_dtype dout_dtype, int64_t ld_dout, const void* z,
                                         int64_t ldz, const uint8_t* z_scales, const void* u, int64_t ldu,
                                         const uint8_t* u_scales, htl_dtype z_dtype, htl_rows8_fmt fmt, int64_t m,
                                         int dim, const float* weight, const float* bias, const int32_t* order,
                                         const int32_t* offsets, int n_groups, htl_norm_kind kind, float eps,
                                         htl_act act, float scale, void* dz, void* du, float* dweight, float* dbias,
                                         void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    HTL_REQUIRE(m >= 0 && m <= kMaxRows, "norm_gate_backward: row count out of range");
    HTL_REQUIRE(dim >= 1 && dim <= kMaxNormDim, "norm_gate_backward: dim out of range");
    HTL_REQUIRE(n_groups >= 1 && n_groups <= kMaxGroups, "norm_gate_backward: group count out of range");
    HTL_REQUIRE(kind == HTL_NORM_RMS || kind == HTL_NORM_LAYER, "norm_gate_backward: unknown kind");
    HTL_REQUIRE(act == HTL_ACT_NONE || act == HTL_ACT_SIGMOID || act == HTL_ACT_SILU,
                "norm_gate_backward: unknown activation");
    HTL_REQUIRE(known(dout_dtype) && known(z_dtype), "norm_gate_backward: dtypes must be HTL_F32 or HTL_BF16");
    HTL_REQUIRE(fmt == HTL_ROWS8_I8 || fmt == HTL_ROWS8_E4M3, "norm_gate_backward: unknown 8-bit format");
    HTL_REQUIRE(eps >= 0.0f, "norm_gate_backward: eps must not be negative");
    HTL_REQUIRE(offsets || (n_groups == 1 && !order), "norm_gate_backward: several groups need offsets");
    HTL_REQUIRE(!z_scales == !u_scales, "norm_gate_backward: z and u are both in 8 bits or neither");
    HTL_REQUIRE(ld_dout >= dim && ldz >= dim && ldu >= dim, "norm_gate_backward: row stride below dim");
    const bool q = z_scales != nullptr;
    const int de = elem(dout_dtype), ge = elem(z_dtype), ze = q ? 1 : ge;
    HTL_REQUIRE(weight && dweight && (m == 0 || (dout && z && u && dz && du)), "norm_gate_backward: null pointer");
    HTL_REQUIRE(aligned(dout, de) && aligned(z, ze) && aligned(u, ze) && aligned(dz, ge) && aligned(du, ge) &&
                    aligned(weight, 4) && aligned(bias, 4) && aligned(dweight, 4) && aligned(dbias, 4) &&
                    aligned(order, 4) && aligned(offsets, 4),
                "norm_gate_backward: misaligned pointer");
    HTL_REQUIRE(ws && aligned(ws, 256) && ws_bytes >= norm_back_workspace_bytes(m, n_groups, dim),
                "norm_gate_backward: workspace too small or misaligned");
    GateBackArgs a;
    a.dout = {dout, nullptr, ld_dout, 0};
    a.z = {z, z_scales, ldz, (int)fmt};
    a.u = {u, u_scales, ldu, (int)fmt};
    a.dz = {dz, dim};
    a.du = {du, dim};
    a.weight = weight;
    a.bias = bias;
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
    a.act = (int)act;
    a.eps = eps;
    a.center = kind == HTL_NORM_LAYER;
    a.scale = scale;
    const bool d32 = dout_dtype == HTL_F32, g32 = z_dtype == HTL_F32;
    with_hold(dim, [&](auto h) {
        using H = decltype(h);
        if (q) {
            if (d32 && g32) launch_gate_back<H, kSrcF32, kSrcRows8, kSrcF32>(a, stream);
            else if (d32) launch_gate_back<H, kSrcF32, kSrcRows8, kSrcBf16>(a, stream);
            else if (g32) launch_gate_back<H, kSrcBf16, kSrcRows8, kSrcF32>(a, stream);
            else launch_gate_back<H, kSrcBf16, kSrcRows8, kSrcBf16>(a, stream);
        } else {
            if (d32 && g32) launch_gate_back<H, kSrcF32, kSrcF32, kSrcF32>(a, stream);
            else if (d32) launch_gate_back<H, kSrcF32, kSrcBf16, kSrcBf16>(a, stream);
            else if (g32) launch_gate_back<H, kSrcBf16, kSrcF32, kSrcF32>(a, stream);
            else launch_gate_back<H, kSrcBf16, kSrcBf16, kSrcBf16>(a, stream);
        }
    });
    const htl_status st = check_launch("norm_gate_backward");
    if (st != HTL_OK) return st;
    return sum_chunks(a.partial, a.limit, dweight, dbias, offsets, n_groups, m, a.rows, dim, stream);
}
