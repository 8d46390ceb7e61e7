// dr_seqops_abi.hip -- host side of the RMS norm, the short causal convolution and
// the gated linear recurrence: argument validation, workspace sizes, how the work
// is split, dispatch.  Nothing here allocates device memory.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "deltarule.h"
#include "dr_host.h"
#include "dr_internal.h"
#include "dr_rows.h"
#include "dr_seqops.h"

using dr::align256;
using dr::check_aligned;
using dr::check_disjoint;
using dr::check_elements;
using dr::check_rows_apart;
using dr::check_strides;
using dr::check_workspace;
using dr::elem_size;
using dr::fail;
using dr::hip_status;
using dr::Rows;
using dr::rows_span;
using dr::Span;
using dr::valid_dtype;

namespace {

// A tensor starts at any of its elements.
struct Start {
    const void* p;
    size_t elem;
    const char* name;
};
dr_status check_starts(std::initializer_list<Start> t) {
    dr_status s;
    for (const Start& x : t)
        if (x.p && (s = check_elements(x.p, x.elem, x.name)) != DR_OK) return s;
    return DR_OK;
}

dr_status check_rows(std::initializer_list<const Rows*> in, std::initializer_list<const Rows*> out) {
    dr_status s;
    for (const Rows* r : in)
        if ((s = check_strides(*r, false)) != DR_OK) return s;
    for (const Rows* r : out)
        if ((s = check_strides(*r, false)) != DR_OK || (s = check_rows_apart(*r)) != DR_OK) return s;
    return DR_OK;
}

}  // namespace

// ------------------------------------------------------------ RMS norm
namespace {

constexpr int kRnMaxD = 16384;

dr_status check_rn_desc(const dr_rmsnorm_desc* d, bool e4m3) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    if (d->B < 0 || d->H < 0 || d->L < 0)
        return fail(DR_ERR_SHAPE, "negative dimension (B=%d H=%d L=%d)", d->B, d->H, d->L);
    if (d->D < 1 || d->D > kRnMaxD)
        return fail(DR_ERR_UNSUPPORTED, "D=%d: rows of 1 to %d values are supported", d->D, kRnMaxD);
    if (!valid_dtype(d->x_dtype) || !valid_dtype(d->res_dtype) || !valid_dtype(d->y_dtype) || !valid_dtype(d->dy_dtype))
        return fail(DR_ERR_UNSUPPORTED, "unknown dtype (x %d, residual %d, y %d, dy %d)", d->x_dtype, d->res_dtype,
                    d->y_dtype, d->dy_dtype);
    if (d->per_head != 0 && d->per_head != 1) return fail(DR_ERR_UNSUPPORTED, "per_head=%d: 0 or 1", d->per_head);
    if (!(d->eps >= 0.f) || std::isinf(d->eps)) return fail(DR_ERR_UNSUPPORTED, "eps must be finite and not negative");
    if (e4m3 && d->block != 0 && d->block != 128)
        return fail(DR_ERR_UNSUPPORTED, "block=%d: scales for 128 columns or (0) for a row are supported", d->block);
    if ((double)d->B * d->H * d->L > 2147483647.0 || d->H > (1 << 20))
        return fail(DR_ERR_UNSUPPORTED, "B*H*L=%.0f: at most 2^31 - 1 rows (and 2^20 heads) are supported",
                    (double)d->B * d->H * d->L);
    return DR_OK;
}

// Groups of rows with one weight, and the workgroups of each: no more than stay on
// the chip, so that all walk their rows with the next ones in flight.  Forward: four per
// compute unit, two for rows of more than 1024 (of 8191 x 2048 bf16 with a residual 4:
// 26.2 us, 2: 25.5, 1: 26.5).  Backward, which leaves a row of sums for each: two, or
// one where a lane holds four octets and more (of 16384 x 1024 2: 27.1, 4: 30.4, 1: 27.8;
// of 8191 x 2048 1: 29.4, 2: 35.0, 4: 46.7).
void rn_groups(const dr_rmsnorm_desc& d, dr::RnArgs& a, bool bwd) {
    a.groups = d.per_head ? d.H : 1;
    a.rows = d.per_head ? (unsigned)d.B * d.L : (unsigned)d.B * d.H * d.L;
    const unsigned pass = (unsigned)dr::rn_pass_rows(d.D, (size_t)a.groups * a.rows);
    const unsigned passes = (a.rows + pass - 1) / pass;
    const unsigned most = bwd ? (dr::rn_shape(d.D, (size_t)a.groups * a.rows).vecs >= 4 ? 256 : 512)
                              : d.D <= 1024 ? 1024 : 512;
    const unsigned want = std::max(1u, (most + a.groups - 1) / a.groups);
    a.blocks = std::max(1u, std::min(want, passes));
}

dr::LnRows rn_strides(const dr_rmsnorm_desc& d, const dr_strides& s) {
    return {d.B > 1 ? s.b : 0, d.H > 1 ? s.h : 0, d.L > 1 ? s.t : 0};
}

size_t rn_part_bytes(const dr_rmsnorm_desc& d) {
    dr::RnArgs a{};
    rn_groups(d, a, true);
    return (size_t)a.groups * a.blocks * d.D * sizeof(float);
}

Rows rn_tensor(const dr_rmsnorm_desc& d, const char* name, const void* p, const dr_strides& s, int dtype) {
    return {name, p, s, {d.B, d.H, d.L}, d.D, dtype};
}

dr_status rn_forward(const dr_rmsnorm_desc* d, const void* x, const void* residual, const float* weight, void* y,
                     float* scale, void* total, float* rstd, bool e4m3, void* stream) {
    dr_status s = check_rn_desc(d, e4m3);
    if (s != DR_OK) return s;
    const size_t nrow = (size_t)d->B * d->H * d->L;
    if (nrow == 0) return DR_OK;
    if (!x || !y || (e4m3 && !scale)) return fail(DR_ERR_NULL, "x, y%s are required", e4m3 ? " and scale" : "");
    if ((residual == nullptr) != (total == nullptr))
        return fail(DR_ERR_NULL, "total must be given exactly when the residual is");
    if (residual && d->res_dtype != d->x_dtype && d->res_dtype != DR_F32)
        return fail(DR_ERR_UNSUPPORTED, "the residual must have x's type or fp32");
    const Rows rx = rn_tensor(*d, "x", x, d->x, d->x_dtype), rr = rn_tensor(*d, "residual", residual, d->res, d->res_dtype),
               ry = rn_tensor(*d, "y", y, d->y, e4m3 ? DR_BF16 : d->y_dtype),
               rt = rn_tensor(*d, "total", total, d->total, d->res_dtype);
    if ((s = check_rows({&rx}, {&ry})) != DR_OK || (residual && (s = check_rows({&rr}, {&rt})) != DR_OK)) return s;
    const size_t wb = (size_t)(d->per_head ? d->H : 1) * d->D * 4;
    const size_t nscale = e4m3 ? nrow * (d->block ? (d->D + 127) / 128 : 1) : 0;
    Span sy = rows_span(ry);
    if (e4m3) sy.bytes /= 2;   // counted as 16-bit values
    const Span ins[] = {rows_span(rx), rows_span(rr), {weight, wb, "weight"}};
    const Span outs[] = {sy, rows_span(rt), {scale, nscale * 4, "scale"}, {rstd, nrow * 4, "rstd"}};
    if ((s = check_starts({{x, elem_size(d->x_dtype), "x"}, {residual, elem_size(d->res_dtype), "residual"},
                           {weight, 4, "weight"}, {y, e4m3 ? 1 : elem_size(d->y_dtype), "y"},
                           {total, elem_size(d->res_dtype), "total"}, {scale, 4, "scale"}, {rstd, 4, "rstd"}})) != DR_OK)
        return s;
    // the sum may take the residual's place, row by row
    auto same = [](int n, long long p, long long q) { return n <= 1 || p == q; };
    const bool in_place = same(d->B, d->res.b, d->total.b) && same(d->H, d->res.h, d->total.h) &&
                          same(d->L, d->res.t, d->total.t);
    if ((s = check_disjoint(outs, 4, ins, 3, in_place ? total : nullptr, in_place ? residual : nullptr)) != DR_OK) return s;
    dr::RnArgs a{};
    a.x = x;
    a.r = residual;
    a.w = weight;
    a.y = y;
    a.total = total;
    a.scale = scale;
    a.rstd_out = rstd;
    a.sx = rn_strides(*d, d->x);
    a.sr = rn_strides(*d, d->res);
    a.sy = rn_strides(*d, d->y);
    a.st = rn_strides(*d, d->total);
    a.B = d->B;
    a.H = d->H;
    a.L = d->L;
    a.D = d->D;
    a.per_head = d->per_head;
    a.eps = d->eps;
    a.block = d->block;
    a.x_f32 = d->x_dtype == DR_F32;
    a.r_f32 = d->res_dtype == DR_F32;
    a.y_f32 = d->y_dtype == DR_F32;
    rn_groups(*d, a, false);
    return hip_status(dr::launch_rn_fwd(a, dr::kProfRnFwd, (hipStream_t)stream), "RMS norm launch");
}

}  // namespace

extern "C" {

dr_status dr_rmsnorm_fwd(const dr_rmsnorm_desc* d, const void* x, const void* residual, const float* weight, void* y,
                         void* total, float* rstd, void* stream) {
    return rn_forward(d, x, residual, weight, y, nullptr, total, rstd, false, stream);
}

dr_status dr_rmsnorm_fwd_e4m3(const dr_rmsnorm_desc* d, const void* x, const void* residual, const float* weight,
                              void* y, float* scale, void* total, float* rstd, void* stream) {
    return rn_forward(d, x, residual, weight, y, scale, total, rstd, true, stream);
}

size_t dr_rmsnorm_bwd_workspace_bytes(const dr_rmsnorm_desc* d) {
    if (check_rn_desc(d, false) != DR_OK || (size_t)d->B * d->H * d->L == 0) return 0;
    return rn_part_bytes(*d);
}

dr_status dr_rmsnorm_bwd(const dr_rmsnorm_desc* d, const void* x, const float* weight, const float* rstd,
                         const void* dy, const void* ds, void* dx, float* dweight, void* workspace,
                         size_t workspace_bytes, void* stream) {
    dr_status s = check_rn_desc(d, false);
    if (s != DR_OK) return s;
    const size_t nrow = (size_t)d->B * d->H * d->L, wn = (size_t)(d->per_head ? d->H : 1) * d->D;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfRnBwd;
    if (nrow && (!x || !rstd || !dy || !dx)) return fail(DR_ERR_NULL, "x, rstd, dy and dx are required");
    const Rows rx = rn_tensor(*d, "x", x, d->x, d->x_dtype), rdy = rn_tensor(*d, "dy", dy, d->dy, d->dy_dtype),
               rds = rn_tensor(*d, "ds", ds, d->res, d->res_dtype), rdx = rn_tensor(*d, "dx", dx, d->y, d->y_dtype);
    if ((s = check_rows({&rx, &rdy}, {&rdx})) != DR_OK || (ds && (s = check_rows({&rds}, {})) != DR_OK)) return s;
    const size_t need = nrow && dweight ? rn_part_bytes(*d) : 0;
    const Span ins[] = {rows_span(rx), {weight, wn * 4, "weight"}, {rstd, nrow * 4, "rstd"}, rows_span(rdy),
                        rows_span(rds)};
    const Span outs[] = {rows_span(rdx), {dweight, wn * 4, "dweight"}, {workspace, need, "workspace"}};
    if ((s = check_starts({{x, elem_size(d->x_dtype), "x"}, {weight, 4, "weight"}, {rstd, 4, "rstd"},
                           {dy, elem_size(d->dy_dtype), "dy"}, {ds, elem_size(d->res_dtype), "ds"},
                           {dx, elem_size(d->y_dtype), "dx"}, {dweight, 4, "dweight"}})) != DR_OK ||
        (s = check_aligned(outs + 2, 1)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 3, ins, 5)) != DR_OK) return s;
    if ((s = check_workspace(need, workspace, workspace_bytes)) != DR_OK) return s;
    if (nrow == 0) {
        // no rows: the sums are zero
        if (!dweight || !wn) return DR_OK;
        return hip_status(dr::launch_seq_copy(dweight, nullptr, wn * 4, slot, st), "RMS norm backward launch");
    }
    dr::RnArgs a{};
    a.x = x;
    a.r = ds;
    a.w = weight;
    a.rstd = rstd;
    a.dy = dy;
    a.y = dx;
    a.part = dweight ? (float*)workspace : nullptr;
    a.dw = dweight;
    a.sx = rn_strides(*d, d->x);
    a.sr = rn_strides(*d, d->res);
    a.sdy = rn_strides(*d, d->dy);
    a.sy = rn_strides(*d, d->y);
    a.B = d->B;
    a.H = d->H;
    a.L = d->L;
    a.D = d->D;
    a.per_head = d->per_head;
    a.x_f32 = d->x_dtype == DR_F32;
    a.r_f32 = d->res_dtype == DR_F32;
    a.y_f32 = d->y_dtype == DR_F32;
    a.dy_f32 = d->dy_dtype == DR_F32;
    rn_groups(*d, a, true);
    return hip_status(dr::launch_rn_bwd(a, slot, st), "RMS norm backward launch");
}

}  // extern "C"

// ------------------------------------------------------------ rows [B][L][C]
namespace {

constexpr int64_t kMaxSeqRows = 2147483647;   // B * ceil(C / 128), and tiles along a sequence

Rows seq_tensor(const char* name, const void* p, int B, int L, int C, const dr_strides& s, int dtype) {
    return {name, p, {s.b, 0, s.t}, {B, 1, L}, C, dtype};
}

dr::SeqRows seq_strides(int B, int L, const dr_strides& s) { return {B > 1 ? s.b : 0, L > 1 ? s.t : 0}; }

int64_t channel_tiles(int C) { return ((int64_t)C + 127) / 128; }

dr_status check_seq_dims(int B, int L, int C) {
    if (B < 0 || L < 0) return fail(DR_ERR_SHAPE, "negative dimension (B=%d L=%d)", B, L);
    if (C < 1) return fail(DR_ERR_SHAPE, "C=%d: at least one channel is needed", C);
    if (C > (1 << 23)) return fail(DR_ERR_UNSUPPORTED, "C=%d: at most 2^23 channels are supported", C);
    if (L > 2147483647 - 4096) return fail(DR_ERR_UNSUPPORTED, "L=%d too large", L);
    if ((int64_t)B * 2 * channel_tiles(C) > kMaxSeqRows)
        return fail(DR_ERR_UNSUPPORTED, "B*C=%.0f too large", (double)B * C);
    return DR_OK;
}

}  // namespace

// ------------------------------------------------------------ short convolution
namespace {

dr_status check_sc_desc(const dr_short_conv_desc* d) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    dr_status s = check_seq_dims(d->B, d->L, d->C);
    if (s != DR_OK) return s;
    if (d->W < 2 || d->W > 8) return fail(DR_ERR_UNSUPPORTED, "W=%d: 2 to 8 taps are supported", d->W);
    if (!valid_dtype(d->x_dtype) || !valid_dtype(d->y_dtype) || !valid_dtype(d->dy_dtype))
        return fail(DR_ERR_UNSUPPORTED, "unknown dtype (x %d, y %d, dy %d)", d->x_dtype, d->y_dtype, d->dy_dtype);
    if (d->act != DR_ACT_NONE && d->act != DR_ACT_SILU) return fail(DR_ERR_UNSUPPORTED, "unknown activation %d", d->act);
    return DR_OK;
}

// Tokens of a thread: as many (up to 16 times the kernel's step; a run reads W - 1 rows
// of the one before) as leave the chip about four workgroups per compute unit.
void sc_split(const dr_short_conv_desc& d, dr::ScArgs& a) {
    const int64_t nct = channel_tiles(d.C);
    const int step = dr::sc_run(d.W);
    a.run = 16 * step;
    auto tiles = [&] { return (d.B * (((int64_t)d.L + a.run - 1) / a.run) + 15) / 16; };
    while (a.run > step && tiles() * nct < 1024) a.run /= 2;
    a.tiles = (unsigned)std::min<int64_t>(tiles(), kMaxSeqRows);
    a.blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>(a.tiles, (1024 + nct - 1) / nct));
}

dr_status check_sc_tiles(const dr_short_conv_desc& d) {
    // runs are counted in 32 bits
    if ((double)d.B * (((double)d.L + 63) / 64) > (double)kMaxSeqRows)
        return fail(DR_ERR_UNSUPPORTED, "B*L=%.0f too large", (double)d.B * d.L);
    return DR_OK;
}

size_t sc_part_bytes(const dr_short_conv_desc& d) {
    dr::ScArgs a{};
    sc_split(d, a);
    return (size_t)a.blocks * d.C * (d.W + 1) * sizeof(float);
}

void sc_args(const dr_short_conv_desc& d, const void* x, const float* weight, const float* bias, const void* state,
             dr::ScArgs& a) {
    a.x = x;
    a.w = weight;
    a.bias = bias;
    a.state = state;
    a.sx = seq_strides(d.B, d.L, d.x);
    a.sy = seq_strides(d.B, d.L, d.y);
    a.sdy = seq_strides(d.B, d.L, d.dy);
    a.B = d.B;
    a.L = d.L;
    a.C = d.C;
    a.W = d.W;
    a.silu = d.act == DR_ACT_SILU;
    a.x_f32 = d.x_dtype == DR_F32;
    a.y_f32 = d.y_dtype == DR_F32;
    a.dy_f32 = d.dy_dtype == DR_F32;
}

}  // namespace

extern "C" {

dr_status dr_short_conv_fwd(const dr_short_conv_desc* d, const void* x, const float* weight, const float* bias,
                            const void* state, void* y, void* state_out, void* stream) {
    dr_status s = check_sc_desc(d);
    if (s != DR_OK || (s = check_sc_tiles(*d)) != DR_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfScFwd;
    if (d->B == 0) return DR_OK;
    if (d->L && (!x || !weight || !y)) return fail(DR_ERR_NULL, "x, weight and y are required");
    const size_t xb = elem_size(d->x_dtype), sb = (size_t)d->B * (d->W - 1) * d->C * xb;
    const Rows rx = seq_tensor("x", x, d->B, d->L, d->C, d->x, d->x_dtype),
               ry = seq_tensor("y", y, d->B, d->L, d->C, d->y, d->y_dtype);
    if ((s = check_rows({&rx}, {&ry})) != DR_OK) return s;
    const Span ins[] = {rows_span(rx), {weight, (size_t)d->C * d->W * 4, "weight"}, {bias, (size_t)d->C * 4, "bias"},
                        {state, sb, "state"}};
    const Span outs[] = {rows_span(ry), {state_out, sb, "state_out"}};
    if ((s = check_starts({{x, xb, "x"}, {weight, 4, "weight"}, {bias, 4, "bias"}, {state, xb, "state"},
                           {y, elem_size(d->y_dtype), "y"}, {state_out, xb, "state_out"}})) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 2, ins, 4, state_out, state)) != DR_OK) return s;
    if (d->L == 0) {
        // no tokens: the final state is the initial state
        if (!state_out || state_out == state) return DR_OK;
        return hip_status(dr::launch_seq_copy(state_out, state, sb, slot, st), "state copy launch");
    }
    dr::ScArgs a{};
    sc_args(*d, x, weight, bias, state, a);
    a.y = y;
    a.state_out = state_out;
    sc_split(*d, a);
    return hip_status(dr::launch_sc_fwd(a, slot, st), "short convolution launch");
}

size_t dr_short_conv_bwd_workspace_bytes(const dr_short_conv_desc* d) {
    if (check_sc_desc(d) != DR_OK || check_sc_tiles(*d) != DR_OK || d->B == 0 || d->L == 0) return 0;
    return sc_part_bytes(*d);
}

dr_status dr_short_conv_bwd(const dr_short_conv_desc* d, const void* x, const float* weight, const float* bias,
                            const void* state, const void* dy, const float* dstate_out, void* dx, float* dweight,
                            float* dbias, float* dstate, void* workspace, size_t workspace_bytes, void* stream) {
    dr_status s = check_sc_desc(d);
    if (s != DR_OK || (s = check_sc_tiles(*d)) != DR_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfScBwd;
    const bool tokens = d->B && d->L, sums = dweight || dbias;
    if (tokens && (!x || !weight || !dy || !dx)) return fail(DR_ERR_NULL, "x, weight, dy and dx are required");
    const size_t xb = elem_size(d->x_dtype), rows = (size_t)d->B * (d->W - 1) * d->C;
    const size_t wb = (size_t)d->C * d->W * 4, bb = (size_t)d->C * 4;
    const Rows rx = seq_tensor("x", x, d->B, d->L, d->C, d->x, d->x_dtype),
               rdy = seq_tensor("dy", dy, d->B, d->L, d->C, d->dy, d->dy_dtype),
               rdx = seq_tensor("dx", dx, d->B, d->L, d->C, d->y, d->y_dtype);
    if ((s = check_rows({&rx, &rdy}, {&rdx})) != DR_OK) return s;
    const size_t need = tokens && sums ? sc_part_bytes(*d) : 0;
    const Span ins[] = {rows_span(rx), {weight, wb, "weight"}, {bias, bb, "bias"}, {state, rows * xb, "state"},
                        rows_span(rdy), {dstate_out, rows * 4, "dstate_out"}};
    const Span outs[] = {rows_span(rdx), {dweight, wb, "dweight"}, {dbias, bb, "dbias"}, {dstate, rows * 4, "dstate"},
                         {workspace, need, "workspace"}};
    if ((s = check_starts({{x, xb, "x"}, {weight, 4, "weight"}, {bias, 4, "bias"}, {state, xb, "state"},
                           {dy, elem_size(d->dy_dtype), "dy"}, {dstate_out, 4, "dstate_out"},
                           {dx, elem_size(d->y_dtype), "dx"}, {dweight, 4, "dweight"}, {dbias, 4, "dbias"},
                           {dstate, 4, "dstate"}})) != DR_OK ||
        (s = check_aligned(outs + 4, 1)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 5, ins, 6)) != DR_OK) return s;
    if ((s = check_workspace(need, workspace, workspace_bytes)) != DR_OK) return s;
    if (!tokens) {
        // no tokens: the state's gradient goes through, and the sums are zero
        if (dstate && rows && (s = hip_status(dr::launch_seq_copy(dstate, dstate_out, rows * 4, slot, st), "launch")) != DR_OK)
            return s;
        if (dweight && (s = hip_status(dr::launch_seq_copy(dweight, nullptr, wb, slot, st), "launch")) != DR_OK) return s;
        return dbias ? hip_status(dr::launch_seq_copy(dbias, nullptr, bb, slot, st), "launch") : DR_OK;
    }
    dr::ScArgs a{};
    sc_args(*d, x, weight, bias, state, a);
    a.dy = dy;
    a.dstate_in = dstate_out;
    a.y = dx;
    a.dw = dweight;
    a.db = dbias;
    a.dstate = dstate;
    a.part = sums ? (float*)workspace : nullptr;
    sc_split(*d, a);
    return hip_status(dr::launch_sc_bwd(a, slot, st), "short convolution backward launch");
}

dr_status dr_short_conv_step(const dr_short_conv_desc* d, const void* x, const float* weight, const float* bias,
                             void* state, void* y, void* stream) {
    dr_status s = check_sc_desc(d);
    if (s != DR_OK) return s;
    if (d->B == 0) return DR_OK;
    if (!x || !weight || !state || !y) return fail(DR_ERR_NULL, "x, weight, state and y are required");
    const size_t xb = elem_size(d->x_dtype), n = (size_t)d->B * d->C;
    const Span ins[] = {{x, n * xb, "x"}, {weight, (size_t)d->C * d->W * 4, "weight"}, {bias, (size_t)d->C * 4, "bias"}};
    const Span outs[] = {{y, n * elem_size(d->y_dtype), "y"}, {state, n * (d->W - 1) * xb, "state"}};
    if ((s = check_starts({{x, xb, "x"}, {weight, 4, "weight"}, {bias, 4, "bias"}, {state, xb, "state"},
                           {y, elem_size(d->y_dtype), "y"}})) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 2, ins, 3)) != DR_OK) return s;
    dr::ScArgs a{};
    sc_args(*d, x, weight, bias, nullptr, a);
    a.y = y;
    a.state_out = state;
    return hip_status(dr::launch_sc_step(a, dr::kProfScStep, (hipStream_t)stream), "short convolution step launch");
}

}  // extern "C"

// ------------------------------------------------------------ gated linear recurrence
namespace {

dr_status check_gs_desc(const dr_gated_scan_desc* d) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    dr_status s = check_seq_dims(d->B, d->L, d->C);
    if (s != DR_OK) return s;
    if (!valid_dtype(d->x_dtype) || !valid_dtype(d->gate_dtype) || !valid_dtype(d->h_dtype) ||
        !valid_dtype(d->dh_dtype) || !valid_dtype(d->grad_dtype))
        return fail(DR_ERR_UNSUPPORTED, "unknown dtype (x %d, gate %d, h %d, dh %d, gradients %d)", d->x_dtype,
                    d->gate_dtype, d->h_dtype, d->dh_dtype, d->grad_dtype);
    if (d->gate_dtype != d->x_dtype && d->gate_dtype != DR_F32)
        return fail(DR_ERR_UNSUPPORTED, "the gate must have x's type or fp32");
    if (d->decay != DR_SCAN_LOG && d->decay != DR_SCAN_LOGIT) return fail(DR_ERR_UNSUPPORTED, "unknown decay %d", d->decay);
    if (d->inputs != DR_INPUT_PLAIN && d->inputs != DR_INPUT_BLEND && d->inputs != DR_INPUT_UNIT)
        return fail(DR_ERR_UNSUPPORTED, "unknown inputs %d", d->inputs);
    return DR_OK;
}

// The kernels reach the rows of a tile by 32-bit offsets.
dr_status check_gs_rows(std::initializer_list<const Rows*> in, std::initializer_list<const Rows*> out) {
    for (auto list : {in, out})
        for (const Rows* r : list)
            if (r->n[2] > 1 && r->s.t > ((int64_t)1 << 23))
                return fail(DR_ERR_UNSUPPORTED, "%s: tokens %lld elements apart, at most 2^23 are supported", r->name,
                            (long long)r->s.t);
    return check_rows(in, out);
}

int64_t gs_tiles(int C) { return ((int64_t)C + dr::kGsTile - 1) / dr::kGsTile; }

// Runs side by side in a workgroup: 8 (a wave), 16 or 32, the least that cover the
// tokens.  Sequences of several such tiles whose columns (64 channels of one) are too
// few to fill the chip have a workgroup for each tile; else a workgroup walks a column.
// Both, forward and backward in us, bf16, sigmoid gates, unit inputs:
//              256 tokens                 1024 tokens                4096 tokens
//   columns    walked        by tile      walked        by tile      walked        by tile
//     256      14,  21       17,  22       37,  60       31,  52     150, 245       94, 182
//     768      22,  43       26,  40       74, 158       69, 133     287, 612      270, 486
//    1024      27,  51       29,  49      100, 202       94, 179     394, 810      354, 646
//    2048      47, 107       51,  94      186, 388      171, 336
//    4096      88, 198       90, 175      360, 751      354, 673
// So walking gains a few percent forward at two tiles, and costs the backward up to a
// fifth; the border was set before the walked form was timed.
constexpr int64_t kGsColumns = 1024;

struct GsLayout {
    int groups, nseg;
    size_t maps, total;   // bytes; the counters stand first
};

GsLayout gs_layout(const dr_gated_scan_desc& d) {
    GsLayout w{};
    constexpr int run = dr::kGsRun;
    w.groups = 8;
    while (w.groups < 32 && (int64_t)w.groups * run < d.L) w.groups *= 2;
    const int64_t columns = d.B * gs_tiles(d.C), span = (int64_t)w.groups * run, tiles = (d.L + span - 1) / span;
    w.nseg = (int)tiles;
    if (tiles > 1 && columns < kGsColumns) {
        w.maps = (size_t)columns * dr::kGsCounter * 4;
        w.total = w.maps + (size_t)columns * w.nseg * 2 * dr::kGsTile * 8;
    }
    return w;
}

dr_status check_gs_tiles(const dr_gated_scan_desc& d, const GsLayout& w) {
    // a launch holds fewer than 2^32 threads
    if (w.total && ((double)d.B * gs_tiles(d.C) + 7) * w.nseg * 256 > 4294967295.0)
        return fail(DR_ERR_UNSUPPORTED, "B*C*L=%.0f too large", (double)d.B * d.C * d.L);
    return DR_OK;
}

void gs_split(const dr_gated_scan_desc& d, const GsLayout& w, void* workspace, dr::GsArgs& a) {
    a.groups = w.groups;
    a.nseg = w.nseg;
    a.tiles = (unsigned)gs_tiles(d.C);
    a.columns = d.B * a.tiles;
    // a multiple of eight, but for few columns, of which no die may stay without
    a.padded = a.columns < 64 ? a.columns : (a.columns + 7) / 8 * 8;
    a.by_columns = dr::gs_divider(a.padded);
    a.by_tiles = dr::gs_divider(a.tiles);
    char* ws = (char*)workspace;
    if (w.total) {
        a.counters = (unsigned*)ws;
        a.maps = (uint64_t*)(ws + w.maps);
        a.words = w.total / 8;
    }
}

void gs_args(const dr_gated_scan_desc& d, const void* x, const void* gate, const float* h0, dr::GsArgs& a) {
    a.x = x;
    a.g = gate;
    a.h0 = h0;
    a.sx = seq_strides(d.B, d.L, d.x);
    a.sg = seq_strides(d.B, d.L, d.gate);
    a.B = d.B;
    a.L = d.L;
    a.C = d.C;
    a.x_f32 = d.x_dtype == DR_F32;
    a.g_f32 = d.gate_dtype == DR_F32;
    a.h_f32 = d.h_dtype == DR_F32;
    a.dh_f32 = d.dh_dtype == DR_F32;
    a.logit = d.decay == DR_SCAN_LOGIT;
    a.inputs = d.inputs;
}

}  // namespace

extern "C" {

size_t dr_gated_scan_fwd_workspace_bytes(const dr_gated_scan_desc* d) {
    if (check_gs_desc(d) != DR_OK || d->B == 0 || d->L == 0) return 0;
    const GsLayout w = gs_layout(*d);
    return check_gs_tiles(*d, w) == DR_OK ? w.total : 0;
}

size_t dr_gated_scan_bwd_workspace_bytes(const dr_gated_scan_desc* d) {
    if (check_gs_desc(d) != DR_OK || d->B == 0 || d->L == 0) return 0;
    const GsLayout w = gs_layout(*d);
    return check_gs_tiles(*d, w) == DR_OK ? w.total : 0;
}

dr_status dr_gated_scan_fwd(const dr_gated_scan_desc* d, const void* x, const void* gate, const float* h0, void* h,
                            float* h_final, void* workspace, size_t workspace_bytes, void* stream) {
    dr_status s = check_gs_desc(d);
    if (s != DR_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfGsFwd;
    if (d->B == 0) return DR_OK;
    if (d->L && (!x || !gate || !h)) return fail(DR_ERR_NULL, "x, gate and h are required");
    const size_t state = (size_t)d->B * d->C * 4;
    const Rows rx = seq_tensor("x", x, d->B, d->L, d->C, d->x, d->x_dtype),
               rg = seq_tensor("gate", gate, d->B, d->L, d->C, d->gate, d->gate_dtype),
               rh = seq_tensor("h", h, d->B, d->L, d->C, d->h, d->h_dtype);
    if ((s = check_gs_rows({&rx, &rg}, {&rh})) != DR_OK) return s;
    const GsLayout w = d->L ? gs_layout(*d) : GsLayout{};
    if ((s = check_gs_tiles(*d, w)) != DR_OK) return s;
    const size_t need = w.total;
    const Span ins[] = {rows_span(rx), rows_span(rg), {h0, state, "h0"}};
    const Span outs[] = {rows_span(rh), {h_final, state, "h_final"}, {workspace, need, "workspace"}};
    if ((s = check_starts({{x, elem_size(d->x_dtype), "x"}, {gate, elem_size(d->gate_dtype), "gate"}, {h0, 4, "h0"},
                           {h, elem_size(d->h_dtype), "h"}, {h_final, 4, "h_final"}})) != DR_OK ||
        (s = check_aligned(outs + 2, 1)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 3, ins, 3, h_final, h0)) != DR_OK) return s;
    if ((s = check_workspace(need, workspace, workspace_bytes)) != DR_OK) return s;
    if (d->L == 0) {
        // no tokens: the final state is the initial state
        if (!h_final || h_final == h0) return DR_OK;
        return hip_status(dr::launch_seq_copy(h_final, h0, state, slot, st), "state copy launch");
    }
    dr::GsArgs a{};
    gs_args(*d, x, gate, h0, a);
    gs_split(*d, w, workspace, a);
    a.out = h;
    a.so = seq_strides(d->B, d->L, d->h);
    a.out_f32 = d->h_dtype == DR_F32;
    a.last = h_final;
    return hip_status(dr::launch_gs_fwd(a, slot, st), "gated recurrence launch");
}

dr_status dr_gated_scan_bwd(const dr_gated_scan_desc* d, const void* x, const void* gate, const float* h0,
                            const void* h, const void* dh, const float* dh_final, void* dx, void* dgate, float* dh0,
                            void* workspace, size_t workspace_bytes, void* stream) {
    dr_status s = check_gs_desc(d);
    if (s != DR_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfGsBwd;
    if (d->B == 0) return DR_OK;
    if (d->L && (!x || !gate || !h || !dh || !dx || !dgate))
        return fail(DR_ERR_NULL, "x, gate, h, dh, dx and dgate are required");
    const size_t state = (size_t)d->B * d->C * 4;
    const Rows rx = seq_tensor("x", x, d->B, d->L, d->C, d->x, d->x_dtype),
               rg = seq_tensor("gate", gate, d->B, d->L, d->C, d->gate, d->gate_dtype),
               rh = seq_tensor("h", h, d->B, d->L, d->C, d->h, d->h_dtype),
               rdh = seq_tensor("dh", dh, d->B, d->L, d->C, d->dh, d->dh_dtype),
               rdx = seq_tensor("dx", dx, d->B, d->L, d->C, d->dx, d->grad_dtype),
               rdg = seq_tensor("dgate", dgate, d->B, d->L, d->C, d->dgate, d->grad_dtype);
    if ((s = check_gs_rows({&rx, &rg, &rh, &rdh}, {&rdx, &rdg})) != DR_OK) return s;
    const GsLayout w = d->L ? gs_layout(*d) : GsLayout{};
    if ((s = check_gs_tiles(*d, w)) != DR_OK) return s;
    const size_t need = w.total;
    const Span ins[] = {rows_span(rx), rows_span(rg), {h0, state, "h0"}, rows_span(rh), rows_span(rdh),
                        {dh_final, state, "dh_final"}};
    const Span outs[] = {rows_span(rdx), rows_span(rdg), {dh0, state, "dh0"}, {workspace, need, "workspace"}};
    if ((s = check_starts({{x, elem_size(d->x_dtype), "x"}, {gate, elem_size(d->gate_dtype), "gate"}, {h0, 4, "h0"},
                           {h, elem_size(d->h_dtype), "h"}, {dh, elem_size(d->dh_dtype), "dh"},
                           {dh_final, 4, "dh_final"}, {dx, elem_size(d->grad_dtype), "dx"},
                           {dgate, elem_size(d->grad_dtype), "dgate"}, {dh0, 4, "dh0"}})) != DR_OK ||
        (s = check_aligned(outs + 3, 1)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 4, ins, 6)) != DR_OK) return s;
    if ((s = check_workspace(need, workspace, workspace_bytes)) != DR_OK) return s;
    if (d->L == 0) {
        // no tokens: the state's gradient goes through
        return dh0 ? hip_status(dr::launch_seq_copy(dh0, dh_final, state, slot, st), "state copy launch") : DR_OK;
    }
    dr::GsArgs a{};
    gs_args(*d, x, gate, h0, a);
    gs_split(*d, w, workspace, a);
    a.h = h;
    a.dh = dh;
    a.dlast = dh_final;
    a.out = dx;
    a.dg = dgate;
    a.last = dh0;
    a.sh = seq_strides(d->B, d->L, d->h);
    a.sdh = seq_strides(d->B, d->L, d->dh);
    a.so = seq_strides(d->B, d->L, d->dx);
    a.sdg = seq_strides(d->B, d->L, d->dgate);
    a.out_f32 = d->grad_dtype == DR_F32;
    return hip_status(dr::launch_gs_bwd(a, slot, st), "gated recurrence backward launch");
}

dr_status dr_gated_scan_step(const dr_gated_scan_desc* d, const void* x, const void* gate, float* state, void* h,
                             void* stream) {
    dr_status s = check_gs_desc(d);
    if (s != DR_OK) return s;
    if (d->B == 0) return DR_OK;
    if (!x || !gate || !state || !h) return fail(DR_ERR_NULL, "x, gate, state and h are required");
    const size_t n = (size_t)d->B * d->C;
    const Span ins[] = {{x, n * elem_size(d->x_dtype), "x"}, {gate, n * elem_size(d->gate_dtype), "gate"}};
    const Span outs[] = {{h, n * elem_size(d->h_dtype), "h"}, {state, n * 4, "state"}};
    if ((s = check_starts({{x, elem_size(d->x_dtype), "x"}, {gate, elem_size(d->gate_dtype), "gate"},
                           {state, 4, "state"}, {h, elem_size(d->h_dtype), "h"}})) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 2, ins, 2)) != DR_OK) return s;
    dr::GsArgs a{};
    gs_args(*d, x, gate, nullptr, a);
    a.out = h;
    a.last = state;
    a.out_f32 = d->h_dtype == DR_F32;
    return hip_status(dr::launch_gs_step(a, dr::kProfGsStep, (hipStream_t)stream), "gated recurrence step launch");
}

}  // extern "C"
