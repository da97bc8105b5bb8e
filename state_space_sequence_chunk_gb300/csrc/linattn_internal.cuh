// linattn_internal.cuh -- shared declarations of the linear-attention kernels
// (not part of the ABI).
//
// With lam = exp(log_decay[h]) and, per head, a state S [V x K]:
//     S_t = lam S_{t-1} + v_t k_t^T            o_t = scale S_t q_t
// and, backwards, with R_t the gradient of S_t:
//     R_t = scale do_t q_t^T + lam R_{t+1}     (R_L = scale do_L q_L^T + dS_L)
//     dq_t = scale S_t^T do_t    dk_t = R_t^T v_t    dv_t = R_t k_t    dS_0 = lam R_1
// All four are one operator F(a, b; c) over a chain of tokens,
//     X_t = lam X_{t-1} + s_in b_t c_t^T       out_t = s_out a_t^T X_t
// walked forwards (o = F(q, k; v), dq = F(do, v; k)) or backwards
// (dk = F(v, do; q), dv = F(k, q; do)); backwards the state that enters a
// token has not been decayed yet, which only shifts two exponents by one.
// A kernel runs up to three such jobs in one launch.
//
// A chain (sequence, head, 64 columns of c) can be cut into ranges of R tokens
// when there are too few chains to fill the GPU: a first launch sums every
// range's own b c^T (from a zero state), a scan turns those into the state at
// each range's start, and the main launch then runs the ranges independently.
#pragma once

#include "ssd_internal.cuh"

namespace ssd {

constexpr int kLaCols = 64;       // columns of c (and of the output) per chain

struct LaGeom {
    const int* cu;       // first token of each sequence [nseq + 1], or NULL: equal lengths L
    int nseq, H;
    int T, L;            // tokens in all; tokens of a sequence when cu is NULL
    int R;               // tokens per range
    int split;           // ranges run independently, from the states in `agg`
    int range_cap;       // grid size in ranges (an upper bound of their number)
    const float* a;      // log decay [H]
};

struct LaJob {
    const void *A, *B, *C;       // [T, heads, DK], [T, heads, DK], [T, heads, DV]
    int64_t sA, sB, sC;          // elements from one token to the next
    int dA, dB, dC;              // head h of the chain reads head h / d of the operand
    int hA, hB, hC;              // heads of the operand
    int DK, DV;
    void* out;                   // [T, H, DV] in the operands' type, or fp32 if out_f32
    int out_f32;
    int rev;
    float s_in, s_out;
    int sk, sv;                  // element strides of X's rows (DK) and columns (DV) in a stored state
    const float* init;           // [nseq, H, DK x DV], or NULL
    float* fin;                  // likewise, or NULL
    float* agg;                  // [range_cap, H, DK x DV] when split
};

struct LaParams {
    LaGeom g;
    LaJob job[3];
    int njobs;
};

// Where a range lies.  seq == nseq: tokens past the last sequence (their
// outputs are zero); seq < 0: no such range.
struct LaRange {
    int seq, r, n;       // sequence, range within it, ranges of the sequence
    int t0, len;         // first token and tokens of the range
    int slen;            // tokens of the whole sequence
};

#ifdef __CUDACC__
__device__ __forceinline__ void la_bounds(const LaGeom& g, int s, int& lo, int& hi) {
    // clamped, so that no content of cu leads out of the tensors
    if (g.cu != nullptr) {
        lo = min(max(g.cu[s], 0), g.T);
        hi = s < g.nseq ? min(max(g.cu[s + 1], lo), g.T) : g.T;
    } else {
        lo = s * g.L;
        hi = s < g.nseq ? lo + g.L : lo;
    }
}
__device__ __forceinline__ int la_count(const LaGeom& g, int s, int lo, int hi) {
    const int len = hi - lo, n = len / g.R + (len % g.R != 0);
    return s < g.nseq && n == 0 ? 1 : n;   // an empty sequence still passes its state on
}
// Range number `idx` in the order of the sequences; executed by one whole warp.
__device__ __forceinline__ LaRange la_find(const LaGeom& g, int idx) {
    const int lane = threadIdx.x & 31;
    LaRange res;
    res.seq = -1;
    res.r = res.n = res.t0 = res.len = res.slen = 0;
    int base = 0;
    for (int s0 = 0; s0 <= g.nseq; s0 += 32) {
        const int s = s0 + lane;
        int lo = 0, hi = 0, n = 0;
        if (s <= g.nseq) {
            la_bounds(g, s, lo, hi);
            n = la_count(g, s, lo, hi);
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const int first = base + inc - n;
        const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && idx >= first && idx < first + n);
        if (hit != 0u) {
            const int src = __ffs(hit) - 1;
            const int r = idx - __shfl_sync(0xffffffffu, first, src);
            lo = __shfl_sync(0xffffffffu, lo, src);
            hi = __shfl_sync(0xffffffffu, hi, src);
            res.seq = s0 + src;
            res.r = r;
            res.n = __shfl_sync(0xffffffffu, n, src);
            res.t0 = lo + r * g.R;
            res.len = min(g.R, hi - res.t0);
            res.slen = hi - lo;
            return res;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return res;
}

// log2 of the head's decay: 0 or less.  -inf (no memory) becomes a finite value
// whose every power but the 0th is 0; a NaN stays one.
__device__ __forceinline__ float la_log2_decay(const float* a, int h) {
    float v = a[h] * kLog2e;
    if (v > 0.f) v = 0.f;
    if (v < -1e30f) v = -1e30f;
    return v;
}
// lam^n as a sum hi + lo of two floats.  A chain multiplies its state by the
// same power hundreds of times, so that the rounding of a single float would add
// up; near 1, where memories are long, the power is 1 + expm1.
__device__ __forceinline__ void la_decay_pow(const float* a, int h, int n, float& hi, float& lo) {
    float e = a[h] * (float)n;
    if (e > 0.f) e = 0.f;
    if (e > -0.7f) {
        hi = 1.f;
        lo = expm1f(e);
    } else {
        hi = expf(e);   // also for a NaN
        lo = 0.f;
    }
}
#endif

// Launchers.  `mode` 0: the main pass; 1: the ranges' own sums into agg.  fp32
// operands on the CUDA cores, bf16 ones on the tensor cores.
cudaError_t launch_linattn_simt(const LaParams& p, int mode, cudaStream_t stream);
cudaError_t launch_linattn_tc(const LaParams& p, int mode, cudaStream_t stream);
// agg -> the state at each range's start, in place.
cudaError_t launch_linattn_scan(const LaParams& p, cudaStream_t stream);
// out[t, g, :] = sum over the group's heads of part[t, h, :], rounded to `dtype`; two of them.
cudaError_t launch_linattn_group_sum(const float* const part[2], void* out0, void* out1, int64_t T, int G,
                                     int hpg, int D, int dtype, cudaStream_t stream);
cudaError_t launch_linattn_step(const ssd_linattn_dims& d, int64_t qs, int64_t ks, int64_t vs,
                                const void* q, const void* k, const void* v, const float* a,
                                float scale, const int* slots, float* cache, int64_t nslots,
                                void* o, cudaStream_t stream);

}  // namespace ssd
