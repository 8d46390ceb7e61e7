// dr_linattn.hip -- linear attention with a decay per head: the chunked kernel
// for bf16 inputs (dr_linattn_kernel.h), the joining of segment states, the
// gate's gradient, the sum of gradients over heads that share q and k, and the
// one-token step.

#include "dr_linattn_kernel.h"

namespace dr {

hipError_t launch_la16(const LaArgs& a, int dx, int waves, int terms, bool state_only, int slot, hipStream_t st) {
    if (state_only)
        return dx == 64 ? la_launch_w<__bf16, 64, 3, true>(a, waves, slot, st)
                        : la_launch_w<__bf16, 128, 3, true>(a, waves, slot, st);
    if (terms == 2)
        return dx == 64 ? la_launch_w<__bf16, 64, 2, false>(a, waves, slot, st)
                        : la_launch_w<__bf16, 128, 2, false>(a, waves, slot, st);
    return dx == 64 ? la_launch_w<__bf16, 64, 3, false>(a, waves, slot, st)
                    : la_launch_w<__bf16, 128, 3, false>(a, waves, slot, st);
}

// ------------------------------------------------------ joining the segments
struct LaJoin2 {
    LaJoinArgs j[2];
};

// One thread walks four elements of a sequence's state over the segments: the
// state at a segment's start takes the place of the segment's own.  Bound by
// memory: 22 us for the 134 MB of two times 32 sequences of 16 segments (128 x
// 128), 6 TB/s, as the states are still in the last-level cache.
__global__ __launch_bounds__(256) void la_join_kernel(LaJoin2 p) {
    const LaJoinArgs& a = p.j[blockIdx.y];
    const int n4 = a.elems / 4;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)a.nseq * n4) return;
    const size_t seq = i / n4, e = i % n4;
    f32x4 cur = {0.f, 0.f, 0.f, 0.f};
    if (a.start) cur = reinterpret_cast<const f32x4*>(a.start)[seq * n4 + e];
    f32x4* seg = reinterpret_cast<f32x4*>(a.seg) + seq * a.nseg * n4 + e;
    const float* dec = a.segdec + seq * a.nseg;
#pragma unroll 4
    for (int k = 0; k < a.nseg; ++k) {
        const int s = a.rev ? a.nseg - 1 - k : k;
        f32x4 local = {0.f, 0.f, 0.f, 0.f};
        float d = 0.f;
        if (k + 1 < a.nseg) {
            local = seg[(size_t)s * n4];
            d = dec[s];
        }
        seg[(size_t)s * n4] = cur;
#pragma unroll
        for (int j = 0; j < 4; ++j) cur[j] = d * cur[j] + local[j];
    }
}

hipError_t launch_la_join(const LaJoinArgs* a, int n, int slot, hipStream_t st) {
    LaJoin2 p{};
    p.j[0] = a[0];
    p.j[1] = a[n - 1];
    const size_t work = (size_t)a[0].nseq * (a[0].elems / 4);
    return launch_k(slot, la_join_kernel, dim3((unsigned)((work + 255) / 256), n), dim3(256), 0, st, p);
}

// ------------------------------------------------------ the gate's gradient
// dlog_alpha_t = <S_L, dS_L> + sum over s >= t of (q_s . dq_s - k_s . dk_s); the
// same holds from any later state <S, dS> on, so that segments are independent.
// One workgroup per (sequence, segment): <S, dS> at the segment's end, then the
// sums over the tokens behind each token.  The differences are small against
// their terms, so the sums are fp64.  Where alpha is zero its gradient is too,
// exactly.  Bound by reading the states: 22 us for 67 MB (32 sequences of 16
// segments), with their loads and the first tokens' in flight together.
// Sum over the workgroup's 256 threads, in every one of them.
__device__ __forceinline__ double la_block_sum(double x, double* red) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void la_gate_kernel(LaGateArgs a) {
    __shared__ double red[4], waves[4];   // of their own: no barrier lies between their uses
    const int nseq = a.B * a.H;
    const int seq = blockIdx.x % nseq, sg = blockIdx.x / nseq;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float *S = nullptr, *D = nullptr;
    if (sg + 1 < a.nseg) {
        S = a.segF + ((size_t)seq * a.nseg + sg + 1) * a.elems;
        D = a.segR + ((size_t)seq * a.nseg + sg) * a.elems;
    } else if (a.dS_end) {
        S = a.S_end + (size_t)seq * a.elems;
        D = a.dS_end + (size_t)seq * a.elems;
    }
    // 1024 tokens at a time, from the segment's last, four in a row per thread;
    // the first ones are loaded along with the states
    constexpr int kPer = 4, kSweep = 256 * kPer;
    const int t0 = sg * a.cps * 64, t1 = (int)min((int64_t)a.L, (int64_t)t0 + a.cps * 64);
    float fq[kPer], fk[kPer];
    auto load = [&](int hi) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int t = hi - 1 - kPer * tid - e;
            const size_t at = (size_t)seq * a.L + t;
            fq[e] = t >= t0 ? a.dq_dots[at] : 0.f;
            fk[e] = t >= t0 ? a.dk_dots[at] : 0.f;
        }
    };
    load(t1);
    double acc = 0.0;
    if (S)
#pragma unroll 8
        for (int i = tid; i < a.elems / 4; i += 256) {
            const f32x4 s = reinterpret_cast<const f32x4*>(S)[i], d = reinterpret_cast<const f32x4*>(D)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc += (double)s[j] * (double)d[j];
        }
    double carry = la_block_sum(acc, red);
    double total = 0.0;
    for (int hi = t1; hi > t0; hi -= kSweep) {
        // running sums of the thread's tokens, the wave's threads, the waves
        double run[kPer], d = 0.0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) run[e] = d += (double)fq[e] - (double)fk[e];
        const double sum = la_scan(d);
        if (lane == 63) waves[wave] = sum;
        __syncthreads();
        double before = carry + (sum - d);
#pragma unroll
        for (int w = 0; w < 3; ++w)
            if (w < wave) before += waves[w];
        carry += (waves[0] + waves[1]) + (waves[2] + waves[3]);
        __syncthreads();
        load(hi - kSweep);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int t = hi - 1 - kPer * tid - e;
            if (t < t0) continue;
            const double v = before + run[e];
            if (!a.part) a.dla[(size_t)seq * a.L + t] = a.la[(size_t)seq * a.L + t] < kLaZero ? 0.f : (float)v;
            total += v;
        }
    }
    if (a.part) {
        total = la_block_sum(total, red);
        if (tid == 0) a.part[(size_t)seq * a.nseg + sg] = a.la[seq % a.H] < kLaZero ? 0.0 : total;
    }
}

hipError_t launch_la_gate(const LaGateArgs& a, int slot, hipStream_t st) {
    return launch_k(slot, la_gate_kernel, dim3((unsigned)(a.B * a.H * a.nseg)), dim3(256), 0, st, a);
}

__global__ __launch_bounds__(256) void la_copy_kernel(float* dst, const float* src, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
        dst[i] = src ? src[i] : 0.f;
}

hipError_t launch_la_copy(float* dst, const float* src, size_t n, int slot, hipStream_t st) {
    const size_t blocks = (n + 255) / 256;
    return launch_k(slot, la_copy_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, st, dst, src,
                    n);
}

// ------------------------------------------------------ shared heads, per-head decays
// The last launch of a backward: gradients of q and k summed over the state
// heads that share them (fp32, in the heads' order), and per-head decay gradients
// summed over sequences and segments, one wave per head, in a fixed order.  5.6 us
// at B3 H12 Hk4 L1111 d64, most of them the launch; bound by memory where there is
// more: 88 us of 475 at B3 H16 Hk8 L7596, 128 x 64 (373 MB read, 94 written).
__device__ __forceinline__ void la_finish_heads(const LaFinishArgs& a, unsigned block) {
    const int hd = block * 4 + (threadIdx.x >> 6);
    if (hd >= a.H) return;
    double acc = 0.0;
    for (size_t i = threadIdx.x & 63; i < (size_t)a.B * a.nseg; i += 64) {
        const size_t b = i / a.nseg, s = i % a.nseg;
        acc += a.part[(b * a.H + hd) * a.nseg + s];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc += __shfl_xor(acc, d);
    if ((threadIdx.x & 63) == 0) a.dla_head[hd] = (float)acc;
}

__global__ __launch_bounds__(256) void la_finish_heads_kernel(LaFinishArgs a) { la_finish_heads(a, blockIdx.x); }

__global__ __launch_bounds__(256) void la_finish_kernel(LaFinishArgs a) {
    const unsigned which = blockIdx.x / a.blocks;
    if (which >= 2) return la_finish_heads(a, blockIdx.x - 2 * a.blocks);
    const int n4 = a.D / 4;
    const size_t n = (size_t)a.B * a.Hk * a.L * n4;
    for (size_t i = (size_t)(blockIdx.x % a.blocks) * 256 + threadIdx.x; i < n; i += (size_t)a.blocks * 256) {
        const int c = (int)(i % n4);
        size_t r = i / n4;
        const int64_t t = r % a.L;
        r /= a.L;
        const int64_t hk = r % a.Hk, b = r / a.Hk;
        const f32x4* in = reinterpret_cast<const f32x4*>(a.in[which]) +
                          (((size_t)b * a.Hk + hk) * a.group * a.L + t) * n4 + c;
        f32x4 v = in[0];
        for (int g = 1; g < a.group; ++g) v = v + in[(size_t)g * a.L * n4];
        const int64_t at = b * a.ob[which] + hk * a.oh[which] + t * a.ot[which] + 4 * c;
        if (a.out_bf16) *reinterpret_cast<bf16x4*>((__bf16*)a.out[which] + at) = __builtin_convertvector(v, bf16x4);
        else *reinterpret_cast<f32x4*>((float*)a.out[which] + at) = v;
    }
}

hipError_t launch_la_finish(LaFinishArgs a, int slot, hipStream_t st) {
    const size_t n = (size_t)a.B * a.Hk * a.L * (a.D / 4);
    const size_t want = (n + 255) / 256;
    a.blocks = a.in[0] ? (unsigned)(want < 8192 ? want : 8192) : 0;
    const unsigned heads = a.part ? (a.H + 3) / 4 : 0;
    if (a.blocks == 0) {
        if (heads == 0) return hipSuccess;
        return launch_k(slot, la_finish_heads_kernel, dim3(heads), dim3(256), 0, st, a);
    }
    return launch_k(slot, la_finish_kernel, dim3(2 * a.blocks + heads), dim3(256), 0, st, a);
}

// ------------------------------------------------------ one token
// S <- alpha S + k v^T, o = S^T q for N x H states: every state is read once
// and written once, and nothing else is large.  One workgroup takes 64 columns
// of a state; a thread holds four columns of every 16th row, all loaded before
// the first is used.  256 x 16 states of 128 x 128: 96 us, 5.6 TB/s of states (a
// copy of this size reaches 5.2); a single sequence's 16 states 5.2 us, a launch.
// The state's loads and stores are non-temporal, so that they displace nothing.
// Workgroups are counted over two grid dimensions: one of them holds fewer than
// 2^32 threads, 2^24 workgroups, which small states pass (4.3 GB of 8 x 8).
constexpr unsigned kLaStepRow = 1u << 22;   // workgroups of the first dimension

template <bool F32IN>
__global__ __launch_bounds__(256) void la_step_kernel(LaStepArgs a) {
    __shared__ float sq[128], sk[128];
    __shared__ float red[16][64];
    const int nslab = (a.Dv + 63) / 64;
    const unsigned id = blockIdx.y * kLaStepRow + blockIdx.x;   // below 2^31 + 2^22
    if (id >= a.total) return;
    const int sidx = (int)(id / nslab), slab = (int)(id % nslab);
    const int n = sidx / a.H, hd = sidx % a.H;
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
    const int col = slab * 64 + 4 * cg;
    const bool ok = col < a.Dv;
    float* S = a.S + (size_t)sidx * a.Dk * a.Dv + col;
    f32x4 s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = rg + 16 * i;
        if (ok && r < a.Dk) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (size_t)r * a.Dv));
    }
    const size_t qk = ((size_t)n * (a.H / a.group) + hd / a.group) * a.Dk;
    if (tid < a.Dk) sq[tid] = load1<F32IN>(a.q, qk + tid);
    else if (tid >= 128 && tid - 128 < a.Dk) sk[tid - 128] = load1<F32IN>(a.k, qk + tid - 128);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) load_n<F32IN, 4>(a.v, (size_t)sidx * a.Dv + col, v);
    const float al = a.la ? expf(a.la[a.la_head ? hd : sidx]) : 1.f;
    __syncthreads();
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = rg + 16 * i;
            if (r >= a.Dk) continue;
            const float kr = sk[r], qr = sq[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = al * s[i][j] + kr * v[j];
                o[j] += qr * s[i][j];
            }
            __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + (size_t)r * a.Dv));
        }
    }
    *reinterpret_cast<f32x4*>(&red[rg][4 * cg]) = o;
    __syncthreads();
    const int oc = slab * 64 + tid;
    if (tid < 64 && oc < a.Dv) {
        float x = 0.f;
#pragma unroll
        for (int g = 0; g < 16; ++g) x += red[g][tid];
        const size_t at = (size_t)sidx * a.Dv + oc;
        if (a.out_bf16) static_cast<__bf16*>(a.o)[at] = (__bf16)x;
        else static_cast<float*>(a.o)[at] = x;
    }
}

hipError_t launch_la_step(LaStepArgs a, bool f32in, int slot, hipStream_t st) {
    a.total = (unsigned)((size_t)a.N * a.H * ((a.Dv + 63) / 64));   // host: below 2^31
    const dim3 grid(a.total < kLaStepRow ? a.total : kLaStepRow, (a.total + kLaStepRow - 1) / kLaStepRow);
    return f32in ? launch_k(slot, la_step_kernel<true>, grid, dim3(256), 0, st, a)
                 : launch_k(slot, la_step_kernel<false>, grid, dim3(256), 0, st, a);
}

}  // namespace dr
