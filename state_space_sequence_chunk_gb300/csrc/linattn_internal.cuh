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
    int range_cap;       // how far the numbers of ranges go
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
    float* agg;                  // [la_slots, H, DK x DV] when split
};

struct LaParams {
    LaGeom g;
    LaJob job[3];
    int njobs;
};

// Where a range lies.  seq == nseq: tokens past the last sequence (their
// outputs are zero); seq < 0: no such range.
struct LaRange {
    int seq, first, last;   // sequence; whether the range is its first and its last
    int t0, len;            // first token and tokens of the range
    int slot;               // where its state is in agg, if its sequence is cut
};
// Slots of agg: j for the range that begins at row j R, T / R + 1 + j for one that
// begins a sequence and ends there.  So they do not grow with the sequences.
__host__ __device__ inline int64_t la_slots(int64_t T, int64_t R) { return 2 * (T / R + 1); }

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
// Range number `idx`; executed by one whole warp.  Sequences are cut at multiples of R
// of the packed rows: numbers 0 .. nseq are the ranges that begin a sequence (or the rows of none), nseq +
// 1 + j the one that begins at row j R inside one.  So a range is found in a search of
// cu at most, in steps of 32 (a count over all sequences before it made 16384
// sequences of one token take 266 ms).
__device__ __forceinline__ LaRange la_find(const LaGeom& g, int idx) {
    LaRange r;
    r.seq = -1;
    r.first = r.last = 1;
    r.t0 = r.len = r.slot = 0;
    int lo, hi;
    if (idx <= g.nseq) {
        la_bounds(g, idx, lo, hi);
        const int end = g.split ? min(hi, (lo / g.R + 1) * g.R) : hi;
        if (idx == g.nseq && lo == hi) return r;
        r.seq = idx;
        r.last = end == hi;
        r.t0 = lo;
        r.len = end - lo;
        r.slot = g.T / g.R + 2 + lo / g.R;
    } else {
        const int lane = threadIdx.x & 31, x = (idx - g.nseq - 1) * g.R;
        if (x >= g.T) return r;
        // cu[0 .. at) <= x, and n entries to look at
        int at = g.cu != nullptr ? 0 : x / g.L + 1, n = g.cu != nullptr ? g.nseq + 1 : 0;
        while (n > 0) {
            const int step = (n + 31) / 32, o = lane * step;
            const int c = __popc(__ballot_sync(0xffffffffu, o < n && g.cu[at + min(o, n - 1)] <= x));
            if (c == 0) break;
            at += (c - 1) * step + 1;
            n = min(step - 1, n - (c - 1) * step - 1);
        }
        if (at == 0) return r;
        la_bounds(g, at - 1, lo, hi);
        if (lo >= x || hi <= x) return r;   // a sequence begins here, or no content of cu says where
        r.seq = at - 1;
        r.slot = idx - g.nseq - 1;
        r.first = 0;
        r.t0 = x;
        r.len = min(g.R, hi - x);
        r.last = x + r.len == hi;
    }
    return r;
}

// f(row, piece) for every piece of `rows` rows of `pieces` each (16 at most), shared out
// among `nthreads`.  Rows and pieces are counted apart: rows of no sequence can be 2^30,
// and their pieces do not fit 32 bits.
template <typename F>
__host__ __device__ __forceinline__ void la_zero_rows(int rows, int pieces, int thread, int nthreads, const F& f) {
    const int step = nthreads / pieces, t = thread / pieces;
    if (t >= step) return;
    for (int row = t; row < rows; row += step) f(row, thread - t * pieces);
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
