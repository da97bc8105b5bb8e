// selscan.cuh -- shared declarations of the selective-scan kernels (not part of the ABI).
//
// Per channel d with N states, for the tokens t of a sequence in order:
//     delta_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias)
//     h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
//     y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
// Unlike the SSD's, the decay differs for every state of every channel, so no
// matrix product evaluates it: each (token, channel, state) takes one exponential
// and four multiply-adds' worth of fp32.  An SM does 32 exponentials and 128
// multiply-adds a clock, so both pipes are the bound at once, at 4 clocks for 32
// elements a quarter-SM.
//
// A sequence is walked by one warp for each 32 / lanes-a-channel channels.  Where
// that leaves SMs idle it is cut into ranges of R tokens: a first launch walks each
// range from a zero state and keeps its end and its sum of delta (the range
// multiplies a state by exp(A sum delta)), a scan makes the states at the ranges'
// starts, and the main launch walks the ranges independently.
#pragma once

#include "approx.cuh"

namespace ssd {

struct ScanGeom {
    const int* cu;       // first token of each sequence [nseq + 1], or NULL: equal lengths L
    int nseq, T, L;
    int R;               // tokens of a range; above T: no sequence is cut
    int items;           // ranges of sequences: T / R + nseq at most
};

struct ScanParams {
    ScanGeom g;
    int D, N, G, cpg;    // channels, states, groups, channels of a group
    int softplus;
    int vecB, vecC;      // rows of B (C) can be read in vectors of four
    const void *x, *dt, *z, *B, *C;
    int64_t xs, dts, zs, Bs, Cs;     // elements from one row to the next
    const float *A, *Dk, *bias;
    const float* init;   // [nseq, D, N] or NULL
    float* fin;          // likewise
    float* states;       // [T / kScanChunk + nseq, D, N]: before each kScanChunk-th token, or NULL
    void* y;
    float *agg, *aggd;   // [items, D, N] and [items, D] where sequences are cut
    // gradient
    const void* dout;
    const float* dfin;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dinit;
    float* part;         // [tiles of a group, T, G, 2, N]: the terms of dB and dC
    float *partA, *partD; // [slots, D, N] and [slots, 2, D]: the terms of dA, of dD and dbias
    int slots, per_slot; // items / per_slot slots, each with the terms of per_slot items
};

constexpr int kScanChunk = SSD_SELSCAN_CHUNK;   // tokens between two stored states

// What an item of a launch is: rows t0 .. t0 + len of sequence seq.
struct ScanItem {
    int seq, t0, len, first, last;
    int row0;            // number of the sequence's first stored state
    int done;            // tokens of the sequence before t0
};

#ifdef __CUDACC__
__device__ __forceinline__ void scan_bounds(const ScanGeom& g, int s, int& lo, int& hi) {
    // clamped, so that no content of cu leads out of the tensors
    if (g.cu != nullptr) {
        lo = min(max(g.cu[s], 0), g.T);
        hi = min(max(g.cu[s + 1], lo), g.T);
    } else {
        lo = s * g.L;
        hi = lo + g.L;
    }
}
__device__ __forceinline__ int scan_base(const ScanGeom& g, int s) {
    const int lo = g.cu != nullptr ? min(max(g.cu[s], 0), g.T) : s * g.L;
    return lo / g.R + s;
}
// Item i: sequence s's ranges are numbered from cu[s] / R + s on, which leaves room
// for all of them.  Found in steps of 32; executed by a whole warp.  False: no such range.
__device__ __forceinline__ bool scan_find(const ScanGeom& g, int i, ScanItem& it) {
    int s = i;
    if (g.R <= g.T) {
        const int lane = threadIdx.x & 31;
        int at = 0, n = g.nseq;          // the last s with base(s) <= i is in at .. at + n - 1
        while (n > 1) {
            const int step = (n + 31) / 32, o = lane * step;
            const int c = __popc(__ballot_sync(0xffffffffu, o < n && scan_base(g, at + min(o, n - 1)) <= i));
            const int k = max(c, 1) - 1;
            at += k * step;
            n = min(step, n - k * step);
        }
        s = at;
    } else if (g.nseq <= 32 && g.nseq > 1) {
        // whole sequences, longest first: a long one that begins last would keep the GPU waiting
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = 0, rank = 0;
        if (lane < g.nseq) scan_bounds(g, lane, lo, hi);
        for (int j = 0; j < g.nseq; ++j) {
            const int len = __shfl_sync(0xffffffffu, hi - lo, j);
            rank += len > hi - lo || (len == hi - lo && j < lane);
        }
        s = __ffs(__ballot_sync(0xffffffffu, lane < g.nseq && rank == i)) - 1;
    }
    int lo, hi;
    scan_bounds(g, s, lo, hi);
    const int64_t off = g.R <= g.T ? (int64_t)(i - scan_base(g, s)) * g.R : 0;
    if (off < 0 || (off > 0 && off >= hi - lo)) return false;
    it.seq = s;
    it.done = (int)off;
    it.t0 = lo + (int)off;
    it.len = min(g.R, hi - it.t0);
    it.first = off == 0;
    it.last = it.t0 + it.len == hi;
    it.row0 = lo / kScanChunk + s;
    return true;
}

// log(1 + e) for e in [0, 1], from log(1 + e) = 2 atanh(e / (2 + e)): the quotient is at
// most 1/3, and atanh(s) / s is fitted by a polynomial in s^2 (Chebyshev interpolation on
// [0, 1/9], off by 8e-9).  Small e keep their relative precision, which log(1 + e) loses.
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * rcp(2.f + e), u = s * s;
    float q = fmaf(u, 0.14078889787197113f, 0.13982579112052917f);
    q = fmaf(u, q, 0.20012298226356506f);
    q = fmaf(u, q, 0.3333316147327423f);
    return 2.f * fmaf(u * s, q, s);
}
__device__ __forceinline__ f32x2 log1p_unit2(f32x2 e) {
    float a, b;
    unpair(add2(e, both(2.f)), a, b);
    const f32x2 s = mul2(e, pair(rcp(a), rcp(b))), u = mul2(s, s);
    f32x2 q = fma2(u, both(0.14078889787197113f), both(0.13982579112052917f));
    q = fma2(u, q, both(0.20012298226356506f));
    q = fma2(u, q, both(0.3333316147327423f));
    return fma2(mul2(u, s), q, s);            // half of it
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)); a NaN stays one.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1p_unit(exp_neg_abs(v)); }
__device__ __forceinline__ f32x2 softplus2(float a, float b) {
    const f32x2 l = log1p_unit2(exp_neg_abs2(a, b));
    return fma2(both(2.f), l, pair(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
// its derivative, 1 / (1 + exp(-v))
__device__ __forceinline__ float softplus_grad(float v) { return sigmoid<true>(v); }
// z sigmoid(z) of two numbers
template <bool EXACT> __device__ __forceinline__ f32x2 silu2(f32x2 z) { return mul2(z, sigmoid2<EXACT>(z)); }

// A log2(e), so that the decays are base-2 exponentials; -inf (no memory) becomes a finite
// value whose every power but the 0th is 0.
__device__ __forceinline__ float scan_rate(float a) {
    const float v = a * kLog2e;
    return v < -1e37f ? -1e37f : v;
}

// One step of a butterfly: of M values a lane keeps the half that its bit names, summed
// with its partner's.
template <int M> __device__ __forceinline__ void halve(float* v, int lane, int bit) {
    if (M > 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
            const float keep = up ? v[i + M / 2] : v[i], send = up ? v[i] : v[i + M / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
    }
}

// The fast exponential is a little low on average (half its last place is 6e-8): for 2^-x by
// 5.5e-9 of it while x is below 0.002, then by more up to 2.45e-8 at 0.01 (measured over steps spread
// by half their size, x from 1e-5 to 1).  A state that remembers a thousand tokens is
// multiplied a thousand times, and would be off by 5e-6 to 1e-5, always to the same side.  So every 16
// tokens a state gets back what it lost on average, c of it, from the sum of its 16 exponents
// X = |A| log2(e) sum of delta: c = min(5.5e-4 X, 16 * 2.75e-9 + 2.3e-6 X, 16 * 2.45e-8, 16 * 2.45e-8 / (0.35 + 1.6 X)),
// which is 0 where nothing decays.  (2.75e-9 instead of 5.5e-9 because so small a share of h is rounded to a whole
// last place of it, more often up than down.)  The last is for states that forget: what is left of older tokens
// has lost 16 times, but is little of the state.  It is fitted so that a state is as much too large behind the 16th token as
// it is too small before it.  Inputs of either sign, 2400 tokens in one piece, decays of e^-d a token, d = 0.001,
// 0.01, 0.02, 0.04, 0.1, 1: states off on average by 3e-7, 2e-7, 1e-7, 9e-8, 3e-8, -1e-8 behind a 16th token and by 3e-7,
// 1e-8, -8e-8, -6e-8, -6e-8, 0 behind an 8th (without c -2.5e-6, -1.2e-6, -6.5e-7, -2.2e-7, -7e-8, -1e-8 everywhere;
// without the last 3e-7, 2e-7, 2e-7, 3e-7, 3e-7, 4e-7 behind a 16th), their gradients about the same; 5 to 6 % of the
// forward pass's time, 3 of the gradient's.  What is left are the single roundings, whose directions differ.
constexpr int kMakeUp = 16;
template <int M> __device__ __forceinline__ void make_up(f32x2 (&h)[M], const f32x2 (&a2)[M], float sum) {
    constexpr float kMost = kMakeUp * 2.45e-8f;          // c in units of this
    const f32x2 s1 = both(-5.5e-4f / kMost * sum), s2 = both(-2.3e-6f / kMost * sum), s3 = both(-1.6f * sum);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float a, b, c, d, e, f;
        unpair(mul2(a2[i], s1), a, b);
        unpair(fma2(a2[i], s2, both(kMakeUp * 2.75e-9f / kMost)), c, d);
        unpair(fma2(a2[i], s3, both(0.35f)), e, f);
        a = __saturatef(fminf(fminf(a, c), rcp(e)));
        b = __saturatef(fminf(fminf(b, d), rcp(f)));
        h[i] = fma2(h[i], mul2(pair(a, b), both(kMost)), h[i]);
    }
}

// Four consecutive states of a row of B or C from n on, 0 beyond N: as loaded, and as floats.
template <typename T> struct Raw4;
template <> struct Raw4<float> { float4 v; };
template <> struct Raw4<__nv_bfloat16> { uint2 v; };
__device__ __forceinline__ void fetch(Raw4<float>& r, const float* p, int n, int N, bool vec) {
    if (vec) r.v = n < N ? __ldg(reinterpret_cast<const float4*>(p + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
    else r.v = make_float4(n < N ? __ldg(p + n) : 0.f, n + 1 < N ? __ldg(p + n + 1) : 0.f,
                           n + 2 < N ? __ldg(p + n + 2) : 0.f, n + 3 < N ? __ldg(p + n + 3) : 0.f);
}
__device__ __forceinline__ void fetch(Raw4<__nv_bfloat16>& r, const __nv_bfloat16* p, int n, int N, bool vec) {
    if (vec) {
        r.v = n < N ? __ldg(reinterpret_cast<const uint2*>(p + n)) : make_uint2(0u, 0u);
    } else {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = n + i < N ? (uint32_t)__ldg(q + n + i) : 0u;
        r.v = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
    }
}
__device__ __forceinline__ float4 widen(const Raw4<float>& r) { return r.v; }
__device__ __forceinline__ float4 widen(const Raw4<__nv_bfloat16>& r) {
    return make_float4(__uint_as_float(r.v.x << 16), __uint_as_float(r.v.x & 0xFFFF0000u),
                       __uint_as_float(r.v.y << 16), __uint_as_float(r.v.y & 0xFFFF0000u));
}
#endif

// Launchers.  kScanSums: the ranges' own ends into agg and aggd; kScanRevSums: the same
// backwards, of the gradient that leaves each at its start.
enum ScanMode { kScanMain = 0, kScanSums = 1, kScanRevSums = 2 };
cudaError_t launch_selscan_fwd(const ScanParams& p, int dtype, ScanMode mode, cudaStream_t stream);
// agg -> the state at each range's start, in place (rev: the gradient entering each range's end).
cudaError_t launch_selscan_ranges(const ScanParams& p, int rev, cudaStream_t stream);

// The gradient's main pass and the sums of its terms; channels of a tile of `part`.
int selscan_bwd_channels(int N);
cudaError_t launch_selscan_bwd(const ScanParams& p, int dtype, cudaStream_t stream);

struct ScanStep {
    int D, N, G, cpg, softplus;
    int vecB, vecC;      // as in ScanParams
    int64_t batch, nslots;
    const void *x, *dt, *z, *B, *C;
    int64_t xs, dts, zs, Bs, Cs;
    const float *A, *Dk, *bias;
    const int* slots;
    float* cache;
    void* y;
};
cudaError_t launch_selscan_step(const ScanStep& p, int dtype, cudaStream_t stream);

}  // namespace ssd
