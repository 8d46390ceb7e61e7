// dr_linattn_abi.hip -- host side of linear attention with a decay per head
// and of the layer norm: argument validation, workspace layout, the split into
// segments, dispatch.  Nothing here allocates device memory.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "deltarule.h"
#include "dr_host.h"
#include "dr_internal.h"
#include "dr_layernorm.h"
#include "dr_linattn.h"

using dr::align256;
using dr::aligned16;
using dr::check_disjoint;
using dr::fail;
using dr::Span;
using dr::valid_dtype;

namespace {

constexpr size_t kMaxGrid = (size_t)std::numeric_limits<int>::max() - 8;

size_t elem_size(int dtype) { return dtype == DR_F32 ? 4 : 2; }

// A strided argument of n[0] x n[1] x n[2] rows of `d` channels.
struct Rows {
    const char* name;
    const void* p;
    dr_strides s;
    int64_t n[3];
    int64_t d;
    int dtype;
};

bool rows_empty(const Rows& r) { return r.n[0] == 0 || r.n[1] == 0 || r.n[2] == 0 || r.d == 0; }

// Strides: not negative, and (vec) whole 16-byte pieces.  A dimension of one
// has no stride.
dr_status check_strides(const Rows& r, bool vec) {
    const int64_t s[3] = {r.s.b, r.s.h, r.s.t};
    const int64_t unit = 16 / (int64_t)elem_size(r.dtype);
    for (int i = 0; i < 3; ++i) {
        if (r.n[i] <= 1) continue;
        if (s[i] < 0) return fail(DR_ERR_SHAPE, "%s has a negative stride (%lld)", r.name, (long long)s[i]);
        if (vec && s[i] % unit)
            return fail(DR_ERR_ALIGN, "%s: stride %lld is not a multiple of 16 bytes", r.name, (long long)s[i]);
        if (vec && i == 2 && s[i] > ((int64_t)1 << 23))
            return fail(DR_ERR_UNSUPPORTED, "%s: tokens %lld elements apart, at most 2^23 are supported", r.name,
                        (long long)s[i]);
        if (s[i] > ((int64_t)1 << 48) / (r.n[i] - 1))
            return fail(DR_ERR_SHAPE, "%s: stride %lld too large", r.name, (long long)s[i]);
    }
    return DR_OK;
}

// An output's rows must not share memory: taken by size, every stride reaches
// behind what the smaller ones cover.
dr_status check_rows_apart(const Rows& r) {
    if (rows_empty(r)) return DR_OK;
    int64_t s[3] = {r.s.b, r.s.h, r.s.t}, n[3] = {r.n[0], r.n[1], r.n[2]};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(n[i], n[j]);
            }
    int64_t extent = r.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < extent) return fail(DR_ERR_UNSUPPORTED, "%s: its strides make rows overlap", r.name);
        extent += (n[i] - 1) * s[i];
    }
    return DR_OK;
}

Span rows_span(const Rows& r) {
    if (!r.p || rows_empty(r)) return {nullptr, 0, r.name};
    int64_t last = r.d;
    const int64_t s[3] = {r.s.b, r.s.h, r.s.t};
    for (int i = 0; i < 3; ++i)
        if (r.n[i] > 1) last += (r.n[i] - 1) * s[i];
    return {r.p, (size_t)last * elem_size(r.dtype), r.name};
}

// A single token's row is as far from the next as it is wide: the kernels tell
// the rows of a chunk apart by their addresses.
dr::LaTensor tensor(const Rows& r, int group) {
    return {r.p, r.n[0] > 1 ? r.s.b : 0, r.n[1] > 1 ? r.s.h : 0, r.n[2] > 1 ? r.s.t : r.d, group};
}

// ------------------------------------------------------------ linear attention
bool valid_decay(int x) { return x == DR_DECAY_NONE || x == DR_DECAY_HEAD || x == DR_DECAY_TOKEN; }

dr_status check_heads(int H, int Hk, int Dk, int Dv, int in_dtype, int out_dtype, int decay) {
    if (H > 0 && Hk <= 0) return fail(DR_ERR_SHAPE, "Hk=%d: at least one q and k head is needed", Hk);
    if (H > 0 && H % Hk)
        return fail(DR_ERR_UNSUPPORTED, "H=%d state heads do not divide among Hk=%d q and k heads", H, Hk);
    if (Dk < 8 || Dk > 128 || Dk % 8 || Dv < 8 || Dv > 128 || Dv % 8)
        return fail(DR_ERR_UNSUPPORTED, "Dk=%d, Dv=%d: multiples of 8 in [8, 128] are supported", Dk, Dv);
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return fail(DR_ERR_UNSUPPORTED, "unknown dtype (in %d, out %d)", in_dtype, out_dtype);
    if (!valid_decay(decay)) return fail(DR_ERR_UNSUPPORTED, "unknown decay mode %d", decay);
    return DR_OK;
}

// How the work is split: workgroups of two to eight waves (16 columns each) that
// hold all columns of a state, and segments of whole chunks.
struct Split {
    int nseg, cps;
};

int waves_of(int D) { return D <= 32 ? 2 : D <= 64 ? 4 : 8; }

// Segments: as many as make two workgroups for each of 256 compute units, of
// four chunks at least; or, where that leaves compute units without work, one
// workgroup for each, of two chunks at least.  A segment costs its state (64 KB
// at 128 x 128) written, joined and read; a chunk takes a workgroup about 4 us
// where it has a compute unit to itself (3.1 at 64 x 64).
// bf16, 128 x 128, 16 heads: 512 tokens 36.6 us in two segments, 27.1 in four;
// 1024 tokens 39.3 in four, 31.5 in eight; 4096 tokens 47.6 in 16, 55.8 in 32;
// 256 tokens 21.6 in one, 24.9 in two (the two more launches).
// The rule does not count rounds: with two workgroups of 128 x 128 to a compute
// unit, 576 sequences of 2048 tokens are one round and a ninth, 363 us against 289
// for 512.
constexpr int64_t kUnits = 256;

Split la_split_of(int L, int64_t nseq) {
    const int NC = (int)(((int64_t)L + 63) / 64);
    auto segments = [&](int64_t workgroups, int chunks) {
        return std::min<int64_t>((workgroups + nseq - 1) / std::max<int64_t>(nseq, 1), NC / chunks);
    };
    int64_t want = segments(2 * kUnits, 4);
    if (NC >= 8) want = std::max(want, segments(kUnits, 2));
    want = std::max<int64_t>(want, 1);
    const int cps = (int)((NC + want - 1) / want);
    return {(NC + cps - 1) / cps, cps};
}

struct LaLayout {
    size_t seg[2], dec[2], S_end, dots[2], dqk[2], part, total;
    Split split;
};

int64_t seqs(const dr_linattn_desc& d) { return (int64_t)d.B * d.H; }

LaLayout la_layout(const dr_linattn_desc& d, bool bwd) {
    LaLayout w{};
    const size_t nseq = (size_t)seqs(d), elems = (size_t)d.Dk * d.Dv;
    w.split = la_split_of(d.L, (int64_t)nseq);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    if (w.split.nseg > 1)
        for (int i = 0; i < (bwd ? 2 : 1); ++i) {
            w.seg[i] = take(nseq * w.split.nseg * elems * sizeof(float));
            w.dec[i] = take(nseq * w.split.nseg * sizeof(float));
        }
    if (bwd && d.decay != DR_DECAY_NONE) {
        w.S_end = take(nseq * elems * sizeof(float));
        for (int i = 0; i < 2; ++i) w.dots[i] = take(nseq * d.L * sizeof(float));
        if (d.decay == DR_DECAY_HEAD) w.part = take(nseq * w.split.nseg * sizeof(double));
    }
    if (bwd && d.H > d.Hk)
        for (int i = 0; i < 2; ++i) w.dqk[i] = take(nseq * d.L * d.Dk * sizeof(float));
    w.total = off;
    return w;
}

dr_status check_la_desc(const dr_linattn_desc* d, bool bwd) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    if (d->B < 0 || d->H < 0 || d->L < 0)
        return fail(DR_ERR_SHAPE, "negative dimension (B=%d H=%d L=%d)", d->B, d->H, d->L);
    dr_status s = check_heads(d->H, d->Hk, d->Dk, d->Dv, d->in_dtype, d->out_dtype, d->decay);
    if (s != DR_OK) return s;
    if (d->L > std::numeric_limits<int>::max() - 128) return fail(DR_ERR_UNSUPPORTED, "L=%d too large", d->L);
    if (d->B == 0 || d->H == 0 || d->L == 0) return DR_OK;
    const LaLayout w = la_layout(*d, bwd);
    if ((size_t)seqs(*d) * w.split.nseg * 8 > kMaxGrid || (size_t)seqs(*d) > kMaxGrid / 64 / 16)
        return fail(DR_ERR_UNSUPPORTED, "B*H=%lld too large", (long long)seqs(*d));
    return DR_OK;
}

dr_status check_workspace(size_t need, const void* ws, size_t bytes) {
    if (!need) return DR_OK;
    if (!ws) return fail(DR_ERR_WORKSPACE, "workspace is NULL, %zu bytes needed", need);
    if (bytes < need) return fail(DR_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
    return DR_OK;
}

dr_status check_aligned(const Span* t, int n) {
    for (int i = 0; i < n; ++i)
        if (t[i].p && !aligned16(t[i].p)) return fail(DR_ERR_ALIGN, "%s is not 16-byte aligned", t[i].name);
    return DR_OK;
}

// Read and written one element at a time.
dr_status check_elements(const void* p, size_t elem, const char* name) {
    if ((uintptr_t)p % elem) return fail(DR_ERR_ALIGN, "%s is not %zu-byte aligned", name, elem);
    return DR_OK;
}

// log alpha, and its gradient, are taken one value at a time: a table's row of one
// value per head, or the sequences of a batch that are no multiples of 16 bytes,
// start at any of them.
dr_status check_decay_aligned(int decay, int64_t row, const float* p, const char* name) {
    if (decay == DR_DECAY_HEAD || row % 4) return check_elements(p, 4, name);
    const Span t{p, 4, name};
    return check_aligned(&t, 1);
}

dr_status hip_status(hipError_t e, const char* what) {
    return e == hipSuccess ? DR_OK : fail(DR_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// One launch of passes that run in the same kernel on the same tiling.
hipError_t run_passes(dr::LaArgs a, const dr::LaPass* p, int n, bool f32in, int terms, bool state_only, int slot,
                      hipStream_t st) {
    const int dx = p[0].Dx <= 64 ? 64 : 128, waves = waves_of(p[0].Dz);
    a.npass = n;
    for (int i = 0; i < n; ++i) a.pass[i] = p[i];
    a.total = (int)((int64_t)n * a.B * a.H * a.nseg);
    return f32in ? dr::launch_la32(a, dx, waves, state_only, slot, st)
                 : dr::launch_la16(a, dx, waves, terms, state_only, slot, st);
}

dr::LaArgs la_args(const dr_linattn_desc& d, const float* log_alpha, const Split& sp) {
    dr::LaArgs a{};
    a.la = log_alpha;
    a.la_head = d.decay == DR_DECAY_HEAD;
    a.B = d.B;
    a.H = d.H;
    a.L = d.L;
    a.NC = (int)(((int64_t)d.L + 63) / 64);
    a.nseg = sp.nseg;
    a.cps = sp.cps;
    return a;
}

size_t la_elems(const dr_linattn_desc& d) {
    return d.decay == DR_DECAY_NONE ? 0 : d.decay == DR_DECAY_HEAD ? (size_t)d.H : (size_t)seqs(d) * d.L;
}

dr_status check_decay_arg(int decay, const float* log_alpha) {
    if ((decay == DR_DECAY_NONE) != (log_alpha == nullptr))
        return fail(DR_ERR_NULL, "log_alpha must be NULL exactly when decay is DR_DECAY_NONE");
    return DR_OK;
}

}  // namespace

extern "C" {

size_t dr_linear_attn_fwd_workspace_bytes(const dr_linattn_desc* d) {
    if (check_la_desc(d, false) != DR_OK || seqs(*d) == 0 || d->L == 0) return 0;
    return la_layout(*d, false).total;
}

size_t dr_linear_attn_bwd_workspace_bytes(const dr_linattn_desc* d) {
    if (check_la_desc(d, true) != DR_OK || seqs(*d) == 0 || d->L == 0) return 0;
    return la_layout(*d, true).total;
}

dr_status dr_linear_attn_fwd(const dr_linattn_desc* d, const void* q, const void* k, const void* v,
                             const float* log_alpha, const float* S0, void* o, float* S_final, void* workspace,
                             size_t workspace_bytes, void* stream) {
    dr_status s = check_la_desc(d, false);
    if (s != DR_OK) return s;
    const size_t nseq = (size_t)seqs(*d), state = nseq * d->Dk * d->Dv;
    const hipStream_t st = (hipStream_t)stream;
    const bool tokens = nseq > 0 && d->L > 0;
    if (tokens) {
        if (!q || !k || !v || !o) return fail(DR_ERR_NULL, "q, k, v and o are required");
        if ((s = check_decay_arg(d->decay, log_alpha)) != DR_OK) return s;
    }
    const Rows rq{"q", q, d->q, {d->B, d->Hk, d->L}, d->Dk, d->in_dtype};
    const Rows rk{"k", k, d->k, {d->B, d->Hk, d->L}, d->Dk, d->in_dtype};
    const Rows rv{"v", v, d->v, {d->B, d->H, d->L}, d->Dv, d->in_dtype};
    const Rows ro{"o", o, d->o, {d->B, d->H, d->L}, d->Dv, d->out_dtype};
    const Rows* rows[] = {&rq, &rk, &rv, &ro};
    for (const Rows* r : rows)
        if ((s = check_strides(*r, true)) != DR_OK) return s;
    if ((s = check_rows_apart(ro)) != DR_OK) return s;
    const LaLayout w = tokens ? la_layout(*d, false) : LaLayout{};
    const Span ins[] = {rows_span(rq), rows_span(rk), rows_span(rv), {S0, state * 4, "S0"},
                        {log_alpha, la_elems(*d) * 4, "log_alpha"}};
    // what is written, the workspace too
    const Span outs[] = {rows_span(ro), {S_final, state * 4, "S_final"}, {workspace, w.total, "workspace"}};
    if ((s = check_aligned(ins, 4)) != DR_OK || (s = check_aligned(outs, 3)) != DR_OK ||
        (s = check_decay_aligned(d->decay, d->L, log_alpha, "log_alpha")) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 3, ins, 5, S_final, S0)) != DR_OK) return s;
    if ((s = check_workspace(w.total, workspace, workspace_bytes)) != DR_OK) return s;
    if (nseq == 0) return DR_OK;
    if (d->L == 0) {
        // no tokens: the final state is the initial state
        if (!S_final || S_final == S0) return DR_OK;
        return hip_status(dr::launch_la_copy(S_final, S0, state, dr::kProfLaFwd, st), "state copy launch");
    }
    const bool f32in = d->in_dtype == DR_F32;
    char* ws = (char*)workspace;
    const dr::LaArgs a = la_args(*d, log_alpha, w.split);
    dr::LaPass p{};
    const int group = d->H / d->Hk;
    p.x = tensor(rq, group);
    p.y = tensor(rk, group);
    p.z = tensor(rv, 1);
    p.w = {nullptr, 0, 0, 0, 1};
    p.out = o;
    const dr::LaTensor to = tensor(ro, 1);
    p.ob = to.b;
    p.oh = to.h;
    p.ot = to.t;
    p.out_bf16 = d->out_dtype == DR_BF16;
    p.Dx = d->Dk;
    p.Dz = d->Dv;
    p.start = S0;
    p.end = S_final;
    if (a.nseg > 1) {
        p.seg = (float*)(ws + w.seg[0]);
        p.segdec = (float*)(ws + w.dec[0]);
        s = hip_status(run_passes(a, &p, 1, f32in, 3, true, dr::kProfLaFwd, st), "segment state launch");
        if (s != DR_OK) return s;
        const dr::LaJoinArgs j{S0, p.seg, p.segdec, (int)nseq, a.nseg, 0, d->Dk * d->Dv};
        s = hip_status(dr::launch_la_join(&j, 1, dr::kProfLaFwd, st), "segment joining launch");
        if (s != DR_OK) return s;
    }
    return hip_status(run_passes(a, &p, 1, f32in, p.out_bf16 ? 2 : 3, false, dr::kProfLaFwd, st),
                      "linear attention launch");
}

dr_status dr_linear_attn_bwd(const dr_linattn_desc* d, const void* q, const void* k, const void* v,
                             const float* log_alpha, const float* S0, const void* dO, const float* dS_final, void* dq,
                             void* dk, void* dv, float* dlog_alpha, float* dS0, void* workspace,
                             size_t workspace_bytes, void* stream) {
    dr_status s = check_la_desc(d, true);
    if (s != DR_OK) return s;
    const size_t nseq = (size_t)seqs(*d), elems = (size_t)d->Dk * d->Dv, state = nseq * elems;
    const hipStream_t st = (hipStream_t)stream;
    const bool tokens = nseq > 0 && d->L > 0;
    if (tokens) {
        if (!q || !k || !v || !dO || !dq || !dk || !dv)
            return fail(DR_ERR_NULL, "q, k, v, dO, dq, dk and dv are required");
        if ((s = check_decay_arg(d->decay, log_alpha)) != DR_OK) return s;
        if ((d->decay == DR_DECAY_NONE) != (dlog_alpha == nullptr))
            return fail(DR_ERR_NULL, "dlog_alpha must be NULL exactly when decay is DR_DECAY_NONE");
    }
    const int od = d->out_dtype;
    const Rows rq{"q", q, d->q, {d->B, d->Hk, d->L}, d->Dk, d->in_dtype};
    const Rows rk{"k", k, d->k, {d->B, d->Hk, d->L}, d->Dk, d->in_dtype};
    const Rows rv{"v", v, d->v, {d->B, d->H, d->L}, d->Dv, d->in_dtype};
    const Rows rdo{"dO", dO, d->o, {d->B, d->H, d->L}, d->Dv, d->in_dtype};
    const Rows rdq{"dq", dq, d->dq, {d->B, d->Hk, d->L}, d->Dk, od};
    const Rows rdk{"dk", dk, d->dk, {d->B, d->Hk, d->L}, d->Dk, od};
    const Rows rdv{"dv", dv, d->dv, {d->B, d->H, d->L}, d->Dv, od};
    const Rows* rows[] = {&rq, &rk, &rv, &rdo, &rdq, &rdk, &rdv};
    for (const Rows* r : rows)
        if ((s = check_strides(*r, true)) != DR_OK) return s;
    for (int i = 4; i < 7; ++i)
        if ((s = check_rows_apart(*rows[i])) != DR_OK) return s;
    const LaLayout w = tokens ? la_layout(*d, true) : LaLayout{};
    const Span ins[] = {rows_span(rq), rows_span(rk), rows_span(rv), rows_span(rdo), {S0, state * 4, "S0"},
                        {dS_final, state * 4, "dS_final"}, {log_alpha, la_elems(*d) * 4, "log_alpha"}};
    const Span outs[] = {rows_span(rdq), rows_span(rdk), rows_span(rdv), {dS0, state * 4, "dS0"},
                         {workspace, w.total, "workspace"}, {dlog_alpha, la_elems(*d) * 4, "dlog_alpha"}};
    if ((s = check_aligned(ins, 6)) != DR_OK || (s = check_aligned(outs, 5)) != DR_OK ||
        (s = check_decay_aligned(d->decay, d->L, log_alpha, "log_alpha")) != DR_OK ||
        (s = check_decay_aligned(d->decay, d->L, dlog_alpha, "dlog_alpha")) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 6, ins, 7)) != DR_OK) return s;
    if ((s = check_workspace(w.total, workspace, workspace_bytes)) != DR_OK) return s;
    const int slot = dr::kProfLaBwd;
    if (!tokens) {
        // no tokens: dS0 = dS_final, and no gradient of a decay
        if (dS0 && state) {
            s = hip_status(dr::launch_la_copy(dS0, dS_final, state, slot, st), "state gradient copy launch");
            if (s != DR_OK) return s;
        }
        if (d->decay == DR_DECAY_HEAD && d->H > 0 && dlog_alpha)
            return hip_status(dr::launch_la_copy(dlog_alpha, nullptr, d->H, slot, st), "decay gradient launch");
        return DR_OK;
    }
    const bool f32in = d->in_dtype == DR_F32, gate = d->decay != DR_DECAY_NONE;
    const int group = d->H / d->Hk;
    char* ws = (char*)workspace;
    const dr::LaArgs a = la_args(*d, log_alpha, w.split);
    const dr::LaTensor tq = tensor(rq, group), tk = tensor(rk, group), tv = tensor(rv, 1), tdo = tensor(rdo, 1);
    const dr::LaTensor none{nullptr, 0, 0, 0, 1};
    float* seg[2] = {(float*)(ws + w.seg[0]), (float*)(ws + w.seg[1])};
    float* dec[2] = {(float*)(ws + w.dec[0]), (float*)(ws + w.dec[1])};
    float* dots[2] = {(float*)(ws + w.dots[0]), (float*)(ws + w.dots[1])};
    float* S_end = gate && dS_final ? (float*)(ws + w.S_end) : nullptr;

    if (a.nseg > 1) {
        // the segments' own states: S forwards, dS backwards
        dr::LaPass p[2] = {};
        p[0].y = tk;
        p[0].z = tv;
        p[1].y = tq;
        p[1].z = tdo;
        p[1].rev = 1;
        for (int i = 0; i < 2; ++i) {
            p[i].x = p[i].w = none;
            p[i].Dx = d->Dk;
            p[i].Dz = d->Dv;
            p[i].seg = seg[i];
            p[i].segdec = dec[i];
        }
        s = hip_status(run_passes(a, p, 2, f32in, 3, true, slot, st), "segment state launch");
        if (s != DR_OK) return s;
        const dr::LaJoinArgs j[2] = {{S0, seg[0], dec[0], (int)nseq, a.nseg, 0, (int)elems},
                                     {dS_final, seg[1], dec[1], (int)nseq, a.nseg, 1, (int)elems}};
        s = hip_status(dr::launch_la_join(j, 2, slot, st), "segment joining launch");
        if (s != DR_OK) return s;
    }

    // dq and dk (contraction over d_v), then dv (over d_k)
    dr::LaPass p[3] = {};
    dr::LaPass& pv = p[2];
    p[0].x = tdo;
    p[0].y = tv;
    p[0].z = tk;
    p[0].w = gate ? tq : none;
    p[0].start = S0;
    p[0].end = S_end;
    p[1].x = tv;
    p[1].y = tdo;
    p[1].z = tq;
    p[1].w = gate ? tk : none;
    p[1].rev = 1;
    p[1].start = dS_final;
    const Rows* rg[2] = {&rdq, &rdk};
    for (int i = 0; i < 2; ++i) {
        p[i].tr = 1;
        p[i].Dx = d->Dv;
        p[i].Dz = d->Dk;
        p[i].seg = seg[i];
        p[i].dots = gate ? dots[i] : nullptr;
        if (group > 1) {
            p[i].out = ws + w.dqk[i];
            p[i].ot = d->Dk;
            p[i].oh = (int64_t)d->L * d->Dk;
            p[i].ob = p[i].oh * d->H;
        } else {
            const dr::LaTensor t = tensor(*rg[i], 1);
            p[i].out = const_cast<void*>(t.p);
            p[i].ob = t.b;
            p[i].oh = t.h;
            p[i].ot = t.t;
            p[i].out_bf16 = od == DR_BF16;
        }
    }
    pv.x = tk;
    pv.y = tq;
    pv.z = tdo;
    pv.w = none;
    pv.rev = 1;
    pv.start = dS_final;
    pv.end = dS0;
    pv.seg = seg[1];
    const dr::LaTensor tdv = tensor(rdv, 1);
    pv.out = dv;
    pv.ob = tdv.b;
    pv.oh = tdv.h;
    pv.ot = tdv.t;
    pv.out_bf16 = od == DR_BF16;
    pv.Dx = d->Dk;
    pv.Dz = d->Dv;
    const int terms = gate || group > 1 || od == DR_F32 ? 3 : 2;
    const bool one = (d->Dk <= 64) == (d->Dv <= 64) && waves_of(d->Dk) == waves_of(d->Dv);
    s = hip_status(run_passes(a, p, one ? 3 : 2, f32in, terms, false, slot, st), "gradient launch");
    if (s != DR_OK) return s;
    if (!one) {
        s = hip_status(run_passes(a, &pv, 1, f32in, od == DR_F32 ? 3 : 2, false, slot, st), "dv launch");
        if (s != DR_OK) return s;
    }

    if (gate) {
        dr::LaGateArgs g{};
        g.dq_dots = dots[0];
        g.dk_dots = dots[1];
        g.segF = seg[0];
        g.segR = seg[1];
        g.la = log_alpha;
        g.S_end = S_end;
        g.dS_end = dS_final;
        g.dla = dlog_alpha;
        g.part = d->decay == DR_DECAY_HEAD ? (double*)(ws + w.part) : nullptr;
        g.B = d->B;
        g.H = d->H;
        g.L = d->L;
        g.nseg = a.nseg;
        g.cps = a.cps;
        g.elems = (int)elems;
        s = hip_status(dr::launch_la_gate(g, slot, st), "decay gradient launch");
        if (s != DR_OK) return s;
    }
    dr::LaFinishArgs f{};
    for (int i = 0; i < 2 && group > 1; ++i) {
        const dr::LaTensor t = tensor(*rg[i], 1);
        f.in[i] = (const float*)(ws + w.dqk[i]);
        f.out[i] = const_cast<void*>(t.p);
        f.ob[i] = t.b;
        f.oh[i] = t.h;
        f.ot[i] = t.t;
    }
    f.out_bf16 = od == DR_BF16;
    f.B = d->B;
    f.Hk = d->Hk;
    f.L = d->L;
    f.D = d->Dk;
    f.group = group;
    f.part = d->decay == DR_DECAY_HEAD ? (const double*)(ws + w.part) : nullptr;
    f.dla_head = dlog_alpha;
    f.H = d->H;
    f.nseg = a.nseg;
    s = hip_status(dr::launch_la_finish(f, slot, st), "backward's last launch");
    if (s != DR_OK) return s;
    return DR_OK;
}

dr_status dr_linear_attn_step(const dr_linattn_step_desc* d, const void* q, const void* k, const void* v,
                              const float* log_alpha, float* S, void* o, void* stream) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    if (d->N < 0 || d->H < 0) return fail(DR_ERR_SHAPE, "negative dimension (N=%d H=%d)", d->N, d->H);
    dr_status s = check_heads(d->H, d->Hk, d->Dk, d->Dv, d->in_dtype, d->out_dtype, d->decay);
    if (s != DR_OK) return s;
    const size_t nst = (size_t)d->N * d->H;
    if (nst * ((d->Dv + 63) / 64) > kMaxGrid) return fail(DR_ERR_UNSUPPORTED, "N*H=%zu too large", nst);
    if (nst == 0) return DR_OK;
    if (!q || !k || !v || !S || !o) return fail(DR_ERR_NULL, "q, k, v, S and o are required");
    if ((s = check_decay_arg(d->decay, log_alpha)) != DR_OK) return s;
    const size_t inb = elem_size(d->in_dtype), nk = (size_t)d->N * d->Hk * d->Dk;
    const size_t nla = d->decay == DR_DECAY_HEAD ? (size_t)d->H : nst;
    const Span ins[] = {{q, nk * inb, "q"}, {k, nk * inb, "k"}, {v, nst * d->Dv * inb, "v"},
                        {log_alpha, nla * 4, "log_alpha"}};
    const Span outs[] = {{o, nst * d->Dv * elem_size(d->out_dtype), "o"}, {S, nst * d->Dk * d->Dv * 4, "S"}};
    if ((s = check_aligned(ins, 3)) != DR_OK || (s = check_aligned(outs, 2)) != DR_OK ||
        (s = check_decay_aligned(d->decay, 0, log_alpha, "log_alpha")) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 2, ins, 4)) != DR_OK) return s;
    const dr::LaStepArgs a{q, k, v, log_alpha, S, o, d->decay == DR_DECAY_HEAD, d->N, d->H, d->H / d->Hk,
                           d->Dk, d->Dv, d->out_dtype == DR_BF16};
    return hip_status(dr::launch_la_step(a, d->in_dtype == DR_F32, dr::kProfLaStep, (hipStream_t)stream),
                      "step kernel launch");
}

}  // extern "C"

// ------------------------------------------------------------ layer norm
namespace {

constexpr int kLnMaxD = 16384;

dr_status check_ln_desc(const dr_layernorm_desc* d) {
    if (!d) return fail(DR_ERR_NULL, "descriptor is NULL");
    if (d->B < 0 || d->H < 0 || d->L < 0)
        return fail(DR_ERR_SHAPE, "negative dimension (B=%d H=%d L=%d)", d->B, d->H, d->L);
    if (d->D < 1 || d->D > kLnMaxD)
        return fail(DR_ERR_UNSUPPORTED, "D=%d: rows of 1 to %d values are supported", d->D, kLnMaxD);
    if (!valid_dtype(d->x_dtype) || !valid_dtype(d->y_dtype) || !valid_dtype(d->dy_dtype))
        return fail(DR_ERR_UNSUPPORTED, "unknown dtype (x %d, y %d, dy %d)", d->x_dtype, d->y_dtype, d->dy_dtype);
    if (d->per_head != 0 && d->per_head != 1) return fail(DR_ERR_UNSUPPORTED, "per_head=%d: 0 or 1", d->per_head);
    if (!(d->eps >= 0.f) || std::isinf(d->eps)) return fail(DR_ERR_UNSUPPORTED, "eps must be finite and not negative");
    if ((double)d->B * d->H * d->L > 2147483647.0 || d->H > (1 << 20))
        return fail(DR_ERR_UNSUPPORTED, "B*H*L=%.0f: at most 2^31 - 1 rows (and 2^20 heads) are supported",
                    (double)d->B * d->H * d->L);
    return DR_OK;
}

// Groups of rows with one weight, and the workgroups of each: no more than stay
// on the chip, so that all walk their rows with the next ones in flight.
// Forward: four per compute unit, two where a lane holds more than eight values
// (of 8191 x 2048 bf16 4: 21.9 us, 8: 25.5, 2: 24.1; of 4096 x 8192 2: 34.3, 4:
// 42.4).  Backward: a workgroup also writes two rows of sums, which a second
// launch joins: four, or two for wider rows (of 65536 x 512 4: 39.8 us, 2: 42.1;
// of 8191 x 2048 2: 30.1, 4: 32.5).
void ln_groups(const dr_layernorm_desc& d, dr::LnArgs& a, bool bwd) {
    a.groups = d.per_head ? d.H : 1;
    a.rows = d.per_head ? (unsigned)d.B * d.L : (unsigned)d.B * d.H * d.L;
    const unsigned pass = (unsigned)dr::ln_pass_rows(d.D);
    const unsigned passes = (a.rows + pass - 1) / pass;
    const unsigned most = d.D <= (bwd ? 512 : 2048) ? 1024 : 512;
    const unsigned want = std::max(1u, (most + a.groups - 1) / a.groups);
    a.blocks = std::max(1u, std::min(want, passes));
}

// Values of a row that its strides allow to be read or written at once: 8 or 2
// where that divides D and every stride, else 1.
int ln_width(const dr_layernorm_desc& d, std::initializer_list<const dr_strides*> strides) {
    long long all = d.D;
    for (const dr_strides* s : strides) {
        if (d.B > 1) all |= s->b;
        if (d.H > 1) all |= s->h;
        if (d.L > 1) all |= s->t;
    }
    return all % 8 == 0 ? 8 : all % 2 == 0 ? 2 : 1;
}

// At width 8 every tensor starts at a multiple of 16 bytes, as everywhere else
// (and so do slices over rows).  Rows of other widths start anywhere, and so may
// the tensors: at whole elements, with one value at a time where a row tensor
// does not start at two.
dr_status check_ln_aligned(int& width, std::initializer_list<const Rows*> rows, const Span* t, int n) {
    dr_status s;
    for (const Rows* r : rows) {
        const size_t elem = elem_size(r->dtype);
        if (width == 8) {
            const Span x{r->p, elem, r->name};
            if ((s = check_aligned(&x, 1)) != DR_OK) return s;
        } else {
            if ((s = check_elements(r->p, elem, r->name)) != DR_OK) return s;
            if ((uintptr_t)r->p % (2 * elem)) width = 1;
        }
    }
    if (width == 8) return check_aligned(t, n);
    for (int i = 0; i < n; ++i)
        if ((s = check_elements(t[i].p, 4, t[i].name)) != DR_OK) return s;
    return DR_OK;
}

dr::LnRows ln_rows(const dr_layernorm_desc& d, const dr_strides& s) {
    return {d.B > 1 ? s.b : 0, d.H > 1 ? s.h : 0, d.L > 1 ? s.t : 0};
}

size_t ln_part_bytes(const dr_layernorm_desc& d) {
    dr::LnArgs a{};
    ln_groups(d, a, true);
    return (size_t)a.groups * a.blocks * 2 * d.D * sizeof(float);
}

}  // namespace

extern "C" {

dr_status dr_layernorm_fwd(const dr_layernorm_desc* d, const void* x, const float* weight, const float* bias, void* y,
                           float* mean, float* rstd, void* stream) {
    dr_status s = check_ln_desc(d);
    if (s != DR_OK) return s;
    const size_t nrow = (size_t)d->B * d->H * d->L;
    if (nrow == 0) return DR_OK;
    if (!x || !y) return fail(DR_ERR_NULL, "x and y are required");
    const Rows rx{"x", x, d->x, {d->B, d->H, d->L}, d->D, d->x_dtype};
    const Rows ry{"y", y, d->y, {d->B, d->H, d->L}, d->D, d->y_dtype};
    if ((s = check_strides(rx, false)) != DR_OK || (s = check_strides(ry, false)) != DR_OK ||
        (s = check_rows_apart(ry)) != DR_OK)
        return s;
    const size_t wb = (size_t)(d->per_head ? d->H : 1) * d->D * 4;
    const Span ins[] = {rows_span(rx), {weight, wb, "weight"}, {bias, wb, "bias"}};
    const Span outs[] = {rows_span(ry), {mean, nrow * 4, "mean"}, {rstd, nrow * 4, "rstd"}};
    int width = ln_width(*d, {&d->x, &d->y});
    if ((s = check_ln_aligned(width, {&rx, &ry}, ins + 1, 2)) != DR_OK ||
        (s = check_ln_aligned(width, {}, outs + 1, 2)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 3, ins, 3)) != DR_OK) return s;
    dr::LnArgs a{};
    a.x = x;
    a.w = weight;
    a.bias = bias;
    a.y = y;
    a.mean_out = mean;
    a.rstd_out = rstd;
    a.sx = ln_rows(*d, d->x);
    a.sy = ln_rows(*d, d->y);
    a.B = d->B;
    a.H = d->H;
    a.L = d->L;
    a.D = d->D;
    a.per_head = d->per_head;
    a.eps = d->eps;
    a.x_f32 = d->x_dtype == DR_F32;
    a.y_f32 = d->y_dtype == DR_F32;
    ln_groups(*d, a, false);
    return hip_status(dr::launch_ln_fwd(a, width, dr::kProfLnFwd, (hipStream_t)stream),
                      "layer norm launch");
}

size_t dr_layernorm_bwd_workspace_bytes(const dr_layernorm_desc* d) {
    if (check_ln_desc(d) != DR_OK || (size_t)d->B * d->H * d->L == 0) return 0;
    return ln_part_bytes(*d);
}

dr_status dr_layernorm_bwd(const dr_layernorm_desc* d, const void* x, const float* weight, const float* mean,
                           const float* rstd, const void* dy, void* dx, float* dweight, float* dbias, void* workspace,
                           size_t workspace_bytes, void* stream) {
    dr_status s = check_ln_desc(d);
    if (s != DR_OK) return s;
    const size_t nrow = (size_t)d->B * d->H * d->L;
    const size_t wn = (size_t)(d->per_head ? d->H : 1) * d->D;
    const hipStream_t st = (hipStream_t)stream;
    const int slot = dr::kProfLnBwd;
    const bool sums = dweight || dbias;
    if (nrow && (!x || !mean || !rstd || !dy || !dx))
        return fail(DR_ERR_NULL, "x, mean, rstd, dy and dx are required");
    const Rows rx{"x", x, d->x, {d->B, d->H, d->L}, d->D, d->x_dtype};
    const Rows rdy{"dy", dy, d->dy, {d->B, d->H, d->L}, d->D, d->dy_dtype};
    const Rows rdx{"dx", dx, d->y, {d->B, d->H, d->L}, d->D, d->y_dtype};
    if ((s = check_strides(rx, false)) != DR_OK || (s = check_strides(rdy, false)) != DR_OK ||
        (s = check_strides(rdx, false)) != DR_OK || (s = check_rows_apart(rdx)) != DR_OK)
        return s;
    const size_t need = nrow && sums ? ln_part_bytes(*d) : 0;
    const Span ins[] = {rows_span(rx), {weight, wn * 4, "weight"}, {mean, nrow * 4, "mean"}, {rstd, nrow * 4, "rstd"},
                        rows_span(rdy)};
    const Span outs[] = {rows_span(rdx), {dweight, wn * 4, "dweight"}, {dbias, wn * 4, "dbias"},
                         {workspace, need, "workspace"}};
    int width = ln_width(*d, {&d->x, &d->dy, &d->y});
    // the statistics are one value per row: those of a slice over rows start anywhere
    if ((s = check_ln_aligned(width, {&rx, &rdy, &rdx}, ins + 1, 1)) != DR_OK ||
        (s = check_ln_aligned(width, {}, outs + 1, 2)) != DR_OK ||
        (s = check_elements(mean, 4, "mean")) != DR_OK || (s = check_elements(rstd, 4, "rstd")) != DR_OK ||
        (s = check_aligned(outs + 3, 1)) != DR_OK)
        return s;
    if ((s = check_disjoint(outs, 4, ins, 5)) != DR_OK) return s;
    if ((s = check_workspace(need, workspace, workspace_bytes)) != DR_OK) return s;
    if (nrow == 0) {
        // no rows: the sums are zero
        for (float* p : {dweight, dbias})
            if (p && wn && (s = hip_status(dr::launch_ln_zero(p, wn, slot, st), "layer norm launch")) != DR_OK) return s;
        return DR_OK;
    }
    dr::LnArgs a{};
    a.x = x;
    a.w = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.dy = dy;
    a.y = dx;
    a.part = sums ? (float*)workspace : nullptr;
    a.dw = dweight;
    a.db = dbias;
    a.sx = ln_rows(*d, d->x);
    a.sdy = ln_rows(*d, d->dy);
    a.sy = ln_rows(*d, d->y);
    a.B = d->B;
    a.H = d->H;
    a.L = d->L;
    a.D = d->D;
    a.per_head = d->per_head;
    a.x_f32 = d->x_dtype == DR_F32;
    a.y_f32 = d->y_dtype == DR_F32;
    a.dy_f32 = d->dy_dtype == DR_F32;
    ln_groups(*d, a, true);
    return hip_status(dr::launch_ln_bwd(a, width, slot, st), "layer norm backward launch");
}

}  // extern "C"
