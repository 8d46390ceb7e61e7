// dr_linattn.h -- argument blocks and launchers of linear attention with a
// decay per head (dr_linattn_abi.hip on the host side, dr_linattn_kernel.h the
// kernels; not part of the public interface).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dr {

constexpr int kLaCols = 16;   // output columns of one wave

// One pass of the operator
//   out_i = sum_{j <= i} e^{u_i - u_j} (x_i . y_j) z_j + e^{u_i} start^T x_i
// over every sequence, i and j running forwards over the tokens, or backwards
// (rev), and u the running sum of log alpha in that order, with the row's own
// term (forwards) or without it (backwards).  The forward of the attention and
// the gradients of q, k and v are all of this form:
//   o:  x, y, z = q, k, v     forwards    start = S0
//   dq:           dO, v, k    forwards    start = S0^T
//   dv:           k, q, dO    backwards   start = dS_final
//   dk:           v, dO, q    backwards   start = dS_final^T
// A state is x's width (Dx) by z's width (Dz).  tr: the stored states ([Dk][Dv])
// are the transpose of the pass's own.
struct LaTensor {
    const void* p;
    int64_t b, h, t;   // strides in elements
    int group;         // state heads per head of this tensor
};

struct LaPass {
    LaTensor x, y, z;
    LaTensor w;          // rows whose dot product with out's rows goes to dots (w.p NULL: none)
    void* out;
    int64_t ob, oh, ot;
    int out_bf16;
    int Dx, Dz;
    int rev, tr;
    const float* start;  // [B*H][Dk][Dv] or NULL (zero)
    float* end;          // the state behind the last token, [B*H][Dk][Dv], or NULL
    // segments (nseg > 1): local states from the state pass, replaced by each
    // segment's start state by the joining pass: [B*H][nseg][Dk][Dv], and the
    // segments' decays [B*H][nseg]
    float* seg;
    float* segdec;
    float* dots;         // [B*H][L]
};

struct LaArgs {
    LaPass pass[3];      // one to three passes in one launch (of one Dx class and tiling)
    int npass;
    const float* la;     // log alpha: [H] (la_head), [B][H][L], or NULL
    int la_head;
    int B, H, L, NC;     // NC: 64-token chunks of a sequence
    int nseg, cps;       // segments, chunks per segment
    int total;           // workgroups
};

// The segment pass's joining step: for every (sequence, element), walk the
// segments in the pass's order and replace each local state by the start state.
struct LaJoinArgs {
    const float* start;
    float* seg;
    const float* segdec;
    int nseq, nseg, rev, elems;
};

// d log alpha from the rows' dot products: within each segment
//   dla_t = <S_end, dS_end> + sum_{s >= t} (q_s . dq_s - k_s . dk_s)
struct LaGateArgs {
    const float* dq_dots;   // [B*H][L]
    const float* dk_dots;
    const float* segF;      // S at the segments' starts, [B*H][nseg][elems]
    const float* segR;      // dS at the segments' ends
    const float* la;        // log alpha: [H] (part) or [B][H][L]
    const float* S_end;     // S behind the last token, dS there (NULL: zero)
    const float* dS_end;
    float* dla;             // [B][H][L], or
    double* part;           // per-head decays: sums over a segment, [B*H][nseg]
    int B, H, L, nseg, cps, elems;
};

struct LaStepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* la;
    float* S;
    void* o;
    int la_head;      // log alpha [H] instead of [N][H]
    int N, H, group, Dk, Dv;
    int out_bf16;
    unsigned total;   // workgroups (launch_la_step sets it)
};

// What is left after the passes of a backward, in one launch: gradients of q and
// k heads shared by `group` state heads (per-state-head gradients [B][H][L][D]
// fp32 summed in head order into [B][H/group][L][D]; in NULL: none), and per-head
// decays' gradients from the partial sums [B*H][nseg] (part NULL: none).
struct LaFinishArgs {
    const float* in[2];
    void* out[2];
    int64_t ob[2], oh[2], ot[2];
    int out_bf16;
    int B, Hk, L, D, group;
    const double* part;
    float* dla_head;
    int H, nseg;
    unsigned blocks;     // workgroups per gradient
};

// terms: bf16 terms per fp32 operand value of the output's products (2 or 3;
// ignored for fp32 inputs); state_only: the state pass
hipError_t launch_la16(const LaArgs& a, int dx, int waves, int terms, bool state_only, int slot, hipStream_t st);
hipError_t launch_la32(const LaArgs& a, int dx, int waves, bool state_only, int slot, hipStream_t st);
hipError_t launch_la_join(const LaJoinArgs* a, int n, int slot, hipStream_t st);
hipError_t launch_la_gate(const LaGateArgs& a, int slot, hipStream_t st);
// dst = src, or zeros (src NULL)
hipError_t launch_la_copy(float* dst, const float* src, size_t n, int slot, hipStream_t st);
hipError_t launch_la_finish(LaFinishArgs a, int slot, hipStream_t st);
hipError_t launch_la_step(LaStepArgs a, bool f32in, int slot, hipStream_t st);

}  // namespace dr
