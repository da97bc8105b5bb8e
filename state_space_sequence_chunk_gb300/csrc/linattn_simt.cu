// linattn_simt.cu -- linear attention on the CUDA cores (fp32 operands), and the
// small kernels shared with the tensor-core form: the scan over ranges and the sum
// over the heads of a group.
//
// Per chunk of 64 tokens with i, j its rows (forwards; backwards the exponents
// are mirrored):
//     P = s_in (A B^T) o lam^{i-j} [i >= j]
//     out = s_out (P C + lam^{i+1} o (A X))
//     X <- lam^n X + s_in B^T (lam^{n-1-j} o C)
// in packed fp32 FMAs on shared-memory tiles: 256 threads, each with a 4 x 4 block of
// P, of the output and of X (two of X for DK > 64).  fp32 operands need it: a TF32
// product keeps 11 bits of them.  B is kept twice, transposed for P and by rows, times
// its decays, for X: read transposed there, X's product took 10000 to 14000 cycles of
// a chunk, and takes 3500.  Bound by instruction issue: a 64 x 64 x 64 product is 15
// instructions for each of 64 steps, 4 warps on a scheduler (two CTAs on an SM): 3840
// cycles, measured 3400 to 4500; the tiles' loads are another 4000 to 5000 of a chunk's
// 20000.  67.5 us for 2 x 2048 tokens, 8 heads of 64 x 64, in three launches of about 18
// (the ranges' own sums), 8 (scan) and 42 us, chained so that each one's set-up overlaps
// the end of the one before (2 us); with its gradient 217 to 219 us.  Ranges go down to 128 tokens here: two
// chunks each keep 256 CTAs busy, two on an SM.
#include "f32x2.cuh"
#include "linattn_internal.cuh"
#include "sm100_ptx.cuh"

namespace ssd {
namespace {

constexpr int kC = 64;            // tokens per chunk
constexpr int kPitch = kC + 4;    // floats per row of a tile with kC columns
constexpr int kThreads = 256;

// Tiles by the head sizes of the call, so that two CTAs share an SM for DK <= 64.
struct Smem {
    float *X, *Cv;            // state [k][v]; C [j][v]
    float* Bw;                // s_in lam^{n-1-j} o B [j][k], rows of dk + 4
    float *At, *Bt, *Pt;      // A and B transposed [k][i]; P transposed [j][i] (main pass only)
    float* lamp;              // lam^0 .. lam^64
    LaRange* rg;
    __device__ Smem(float* base, int dk, bool agg) {
        X = base;
        Cv = X + dk * kPitch;
        Bw = Cv + kC * kPitch;
        At = Bw + kC * (dk + 4);
        Bt = At + (agg ? 0 : dk * kPitch);
        Pt = Bt + (agg ? 0 : dk * kPitch);
        lamp = Pt + (agg ? 0 : kC * kPitch);
        rg = reinterpret_cast<LaRange*>(lamp + kC + 4);
    }
    static size_t bytes(int dk, bool agg) {
        return ((size_t)(agg ? 1 : 3) * dk * kPitch + (size_t)kC * (dk + 4) + (agg ? 1 : 2) * kC * kPitch + kC + 4) * 4 +
               sizeof(LaRange);
    }
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }

// a 4 x 4 block, in pairs along its rows
struct Acc {
    f32x2 v[4][2];
    __device__ __forceinline__ Acc() {
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x][0] = v[x][1] = 0ull;
    }
    __device__ __forceinline__ void fma(const float4& a, const float4& b) {
        const float av[4] = {a.x, a.y, a.z, a.w};
        const f32x2 b0 = pair(b.x, b.y), b1 = pair(b.z, b.w);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const f32x2 a2 = pair(av[x], av[x]);
            v[x][0] = fma2(a2, b0, v[x][0]);
            v[x][1] = fma2(a2, b1, v[x][1]);
        }
    }
    // rows from or up to the y-th alone: what is not added may be an infinity or a NaN
    __device__ __forceinline__ void fma_part(const float4& a, const float4& b, int y, bool up_to) {
        const float av[4] = {a.x, a.y, a.z, a.w};
        const f32x2 b0 = pair(b.x, b.y), b1 = pair(b.z, b.w);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (up_to ? x > y : x < y) continue;
            const f32x2 a2 = pair(av[x], av[x]);
            v[x][0] = fma2(a2, b0, v[x][0]);
            v[x][1] = fma2(a2, b1, v[x][1]);
        }
    }
    __device__ __forceinline__ void row(int x, float (&f)[4]) const {
        unpair(v[x][0], f[0], f[1]);
        unpair(v[x][1], f[2], f[3]);
    }
};

template <bool kAgg>
__global__ void __launch_bounds__(kThreads, 2) linattn_simt(const __grid_constant__ LaParams p) {
    extern __shared__ __align__(16) float raw[];
    const LaGeom& g = p.g;
    const LaJob& jb = p.job[blockIdx.z];
    const Smem s(raw, jb.DK, kAgg);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int nvb = (jb.DV + kLaCols - 1) / kLaCols;
    const int h = blockIdx.y / nvb, v0 = (blockIdx.y - h * nvb) * kLaCols;
    if (h >= g.H) return;
    if (kAgg) grid_launch_dependents();
    if (tid < 32) {
        const LaRange r = la_find(g, blockIdx.x);
        if (tid == 0) *s.rg = r;
    }
    const float a2 = la_log2_decay(g.a, h);
    if (tid <= kC) s.lamp[tid] = exp2f(a2 * (float)tid);
    __syncthreads();
    const LaRange rg = *s.rg;
    if (rg.seq < 0) return;
    const int nv = min(kLaCols, jb.DV - v0);
    if (rg.seq == g.nseq) {               // tokens of no sequence: zeros
        if (kAgg) return;
        la_zero_rows(rg.len, nv / 4, tid, kThreads, [&](int t, int v) {
            st4(static_cast<float*>(jb.out) + ((int64_t)(rg.t0 + t) * g.H + h) * jb.DV + v0 + 4 * v,
                make_float4(0.f, 0.f, 0.f, 0.f));
        });
        return;
    }
    const bool cut = g.split && !(rg.first && rg.last);
    const bool last = jb.rev ? rg.first : rg.last;
    if (kAgg && (!cut || last)) return;
    const int64_t elems = (int64_t)jb.DK * jb.DV;
    const int64_t so = ((int64_t)rg.seq * g.H + h) * elems;
    if (!kAgg) grid_dependency_wait();
    float* ag = cut ? jb.agg + ((int64_t)rg.slot * g.H + h) * elems : nullptr;
    const float* in = kAgg ? nullptr : (cut ? ag : (jb.init ? jb.init + so : nullptr));
    // neighbouring threads along whichever of the stored state's axes is contiguous
    const bool kfirst = jb.sk == 1;
    const auto each = [&](const auto& f) {   // every (k, v) of the state's block
        for (int m = 0; m < (kfirst ? jb.DK : kLaCols); m += 64) {
            const int fast = m + (tid & 63);
#pragma unroll 8
            for (int slow = tid >> 6; slow < (kfirst ? kLaCols : jb.DK); slow += kThreads / 64)
                if (!kfirst || fast < jb.DK) f(kfirst ? fast : slow, kfirst ? slow : fast);
        }
    };
    each([&](int k, int v) {
        s.X[k * kPitch + v] = in && v < nv ? in[(int64_t)k * jb.sk + (int64_t)(v0 + v) * jb.sv] : 0.f;
    });
    const float* Ap = static_cast<const float*>(jb.A) + (int64_t)(h / jb.dA) * jb.DK;
    const float* Bp = static_cast<const float*>(jb.B) + (int64_t)(h / jb.dB) * jb.DK;
    const float* Cp = static_cast<const float*>(jb.C) + (int64_t)(h / jb.dC) * jb.DV + v0;
    const int nch = (rg.len + kC - 1) / kC;
    float cf_hi, cf_lo;
    la_decay_pow(g.a, h, kC, cf_hi, cf_lo);
    for (int ci = 0; ci < nch; ++ci) {
        const int c = jb.rev ? nch - 1 - ci : ci;
        const int t0 = rg.t0 + c * kC, n = min(kC, rg.len - c * kC);
        if (ci > 0) __syncthreads();
        {
            // every load of a tile before its first store; rows past n are zero,
            // whatever memory holds there
            const int row = tid & (kC - 1);
            const bool in_n = row < n;
            const float w = in_n ? s.lamp[jb.rev ? row + 1 : n - 1 - row] * jb.s_in : 0.f;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 cv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = (tid >> 4) + 16 * e, v = (tid & 15) * 4;
                cv[e] = r < n && v < nv ? __ldg(reinterpret_cast<const float4*>(Cp + (int64_t)(t0 + r) * jb.sC + v)) : zero;
            }
            for (int d0 = (tid / kC) * 4; d0 < jb.DK; d0 += 64) {
                float4 a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = d0 + 16 * e;
                    const bool ok = in_n && d < jb.DK;
                    b[e] = ok ? __ldg(reinterpret_cast<const float4*>(Bp + (int64_t)(t0 + row) * jb.sB + d)) : zero;
                    if (!kAgg) a[e] = ok ? __ldg(reinterpret_cast<const float4*>(Ap + (int64_t)(t0 + row) * jb.sA + d)) : zero;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = d0 + 16 * e;
                    if (d >= jb.DK) break;
                    st4(s.Bw + row * (jb.DK + 4) + d, make_float4(b[e].x * w, b[e].y * w, b[e].z * w, b[e].w * w));
                    if (!kAgg) {
                        const float av[4] = {a[e].x, a[e].y, a[e].z, a[e].w}, bv[4] = {b[e].x, b[e].y, b[e].z, b[e].w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            s.At[(d + x) * kPitch + row] = av[x];
                            s.Bt[(d + x) * kPitch + row] = bv[x];
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) st4(s.Cv + ((tid >> 4) + 16 * e) * kPitch + (tid & 15) * 4, cv[e]);
        }
        __syncthreads();
        if (!kAgg) {
            {
                Acc acc;
#pragma unroll 4
                for (int k = 0; k < jb.DK; ++k)
                    acc.fma(ld4(s.Bt + k * kPitch + tx * 4), ld4(s.At + k * kPitch + ty * 4));
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int j = tx * 4 + y;
                    float f[4];
                    acc.row(y, f);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int i = ty * 4 + x, d = jb.rev ? j - i : i - j;
                        f[x] = d >= 0 && j < n ? f[x] * (s.lamp[d] * jb.s_in) : 0.f;
                    }
                    st4(s.Pt + j * kPitch + ty * 4, make_float4(f[0], f[1], f[2], f[3]));
                }
            }
            Acc o1, o2;
#pragma unroll 4
            for (int k = 0; k < jb.DK; ++k)
                o1.fma(ld4(s.At + k * kPitch + ty * 4), ld4(s.X + k * kPitch + tx * 4));
            __syncthreads();
            // the rows of C that a row of out may see, and no others: 0 times an infinity
            // or a NaN of a later token would be one
            if (!jb.rev)
#pragma unroll 4
                for (int j = 0; j < ty * 4; ++j)
                    o2.fma(ld4(s.Pt + j * kPitch + ty * 4), ld4(s.Cv + j * kPitch + tx * 4));
#pragma unroll
            for (int y = 0; y < 4; ++y)
                o2.fma_part(ld4(s.Pt + (ty * 4 + y) * kPitch + ty * 4), ld4(s.Cv + (ty * 4 + y) * kPitch + tx * 4), y,
                            jb.rev != 0);
            if (jb.rev)
#pragma unroll 4
                for (int j = ty * 4 + 4; j < kC; ++j)
                    o2.fma(ld4(s.Pt + j * kPitch + ty * 4), ld4(s.Cv + j * kPitch + tx * 4));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = ty * 4 + x;
                if (i >= n || tx * 4 >= nv) continue;
                const float f = s.lamp[jb.rev ? n - 1 - i : i + 1];
                float r1[4], r2[4];
                o1.row(x, r1);
                o2.row(x, r2);
                const int64_t at = ((int64_t)(t0 + i) * g.H + h) * jb.DV + v0 + tx * 4;
                st4(static_cast<float*>(jb.out) + at,
                    make_float4(jb.s_out * fmaf(f, r1[0], r2[0]), jb.s_out * fmaf(f, r1[1], r2[1]),
                                jb.s_out * fmaf(f, r1[2], r2[2]), jb.s_out * fmaf(f, r1[3], r2[3])));
            }
        }
        // X <- lam^n X + (w o B)^T C; every thread reads and writes its own 4 x 4 (two
        // of them for DK > 64)
        float hi = cf_hi, lo = cf_lo;
        if (n < kC) la_decay_pow(g.a, h, n, hi, lo);
        for (int k0 = ty * 4; k0 < jb.DK; k0 += 64) {
            Acc u;
#pragma unroll 4
            for (int j = 0; j < kC; ++j)
                u.fma(ld4(s.Bw + j * (jb.DK + 4) + k0), ld4(s.Cv + j * kPitch + tx * 4));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float f[4];
                u.row(x, f);
                float* X = s.X + (k0 + x) * kPitch + tx * 4;
                float4 q = ld4(X);
                q.x = fmaf(q.x, hi, fmaf(q.x, lo, f[0]));
                q.y = fmaf(q.y, hi, fmaf(q.y, lo, f[1]));
                q.z = fmaf(q.z, hi, fmaf(q.z, lo, f[2]));
                q.w = fmaf(q.w, hi, fmaf(q.w, lo, f[3]));
                st4(X, q);
            }
        }
    }
    __syncthreads();
    float* outst = kAgg ? ag : (last && jb.fin ? jb.fin + so : nullptr);
    if (outst == nullptr) return;
    each([&](int k, int v) {
        if (v < nv) outst[(int64_t)k * jb.sk + (int64_t)(v0 + v) * jb.sv] = s.X[k * kPitch + v];
    });
}

// One thread per state element of (sequence, head): walks the sequence's
// ranges, leaving in agg the state at each range's start.
__global__ void __launch_bounds__(256) linattn_scan(const __grid_constant__ LaParams p, int eblocks) {
    const LaGeom& g = p.g;
    const LaJob& jb = p.job[blockIdx.z];
    const int seq = blockIdx.x / eblocks, eb = blockIdx.x - seq * eblocks, h = blockIdx.y;
    grid_launch_dependents();
    int lo, hi;
    la_bounds(g, seq, lo, hi);
    const int n = hi > lo ? (hi - 1) / g.R - lo / g.R + 1 : 1, first = (lo / g.R + 1) * g.R - lo;
    grid_dependency_wait();
    if (n <= 1) return;
    const int elems = jb.DK * jb.DV;
    const int e = (eb * 256 + threadIdx.x) * 4;
    if (e >= elems) return;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (jb.init) S = *reinterpret_cast<const float4*>(jb.init + ((int64_t)seq * g.H + h) * elems + e);
    float b_hi, b_lo, f_hi, f_lo, t_hi, t_lo;   // over the first range, a whole one, the last
    la_decay_pow(g.a, h, first, b_hi, b_lo);
    la_decay_pow(g.a, h, g.R, f_hi, f_lo);
    la_decay_pow(g.a, h, hi - lo - first - (n - 2) * g.R, t_hi, t_lo);
    const auto state = [&](int r) {
        const int id = r == 0 ? g.T / g.R + 2 + lo / g.R : lo / g.R + r;
        return reinterpret_cast<float4*>(jb.agg + ((int64_t)id * g.H + h) * elems + e);
    };
    // eight ranges' sums in flight: the walk is all latency
    for (int i0 = 0; i0 < n; i0 += 8) {
        float4 u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int i = i0 + q, r = jb.rev ? n - 1 - i : i;
            if (i < n - 1)
                u[q] = *state(r);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int i = i0 + q, r = jb.rev ? n - 1 - i : i;
            if (i >= n) break;
            *state(r) = S;
            if (i == n - 1) break;   // the last range's pass writes the final state
            const float d_hi = r == n - 1 ? t_hi : r == 0 ? b_hi : f_hi, d_lo = r == n - 1 ? t_lo : r == 0 ? b_lo : f_lo;
            S.x = fmaf(S.x, d_hi, fmaf(S.x, d_lo, u[q].x));
            S.y = fmaf(S.y, d_hi, fmaf(S.y, d_lo, u[q].y));
            S.z = fmaf(S.z, d_hi, fmaf(S.z, d_lo, u[q].z));
            S.w = fmaf(S.w, d_hi, fmaf(S.w, d_lo, u[q].w));
        }
    }
}

// Both gradients of shared heads in one launch (blockIdx.y): small ones are all
// launch latency.
template <typename T>
__global__ void __launch_bounds__(256) linattn_group_sum(const float* __restrict__ part0, const float* __restrict__ part1,
                                                         T* __restrict__ out0, T* __restrict__ out1, int64_t n4,
                                                         int hpg, int d4) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const int64_t row = i / d4;   // (token, group)
    const int col = (int)(i - row * d4);
    const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? part1 : part0) + row * hpg * d4 + col;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < hpg; ++x) {
        const float4 v = src[(int64_t)x * d4];
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    T* dst = (blockIdx.y ? out1 : out0) + 4 * i;
    if constexpr (sizeof(T) == 2) {
        union { __nv_bfloat162 h[2]; uint2 u; } w;
        w.h[0] = __floats2bfloat162_rn(a.x, a.y);
        w.h[1] = __floats2bfloat162_rn(a.z, a.w);
        *reinterpret_cast<uint2*>(dst) = w.u;
    } else {
        *reinterpret_cast<float4*>(dst) = a;
    }
}

template <bool kAgg>
cudaError_t go(const LaParams& p, cudaStream_t stream) {
    int nvb = 1, dk = 0;
    for (int j = 0; j < p.njobs; ++j) {
        const int n = (p.job[j].DV + kLaCols - 1) / kLaCols;
        nvb = n > nvb ? n : nvb;
        dk = p.job[j].DK > dk ? p.job[j].DK : dk;
    }
    const size_t bytes = Smem::bytes(dk, kAgg);
    auto k = linattn_simt<kAgg>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    return launch_chained(k, dim3((unsigned)p.g.range_cap, (unsigned)(p.g.H * nvb), (unsigned)p.njobs), dim3(kThreads), bytes,
                          stream, !kAgg && p.g.split, p);
}

}  // namespace

cudaError_t launch_linattn_simt(const LaParams& p, int mode, cudaStream_t stream) {
    return mode ? go<true>(p, stream) : go<false>(p, stream);
}

cudaError_t launch_linattn_scan(const LaParams& p, cudaStream_t stream) {
    const int elems = p.job[0].DK * p.job[0].DV;   // the same product for every job
    const int eblocks = (elems / 4 + 255) / 256;
    return launch_chained(linattn_scan, dim3((unsigned)(p.g.nseq * eblocks), (unsigned)p.g.H, (unsigned)p.njobs), dim3(256), 0,
                          stream, true, p, eblocks);
}

cudaError_t launch_linattn_group_sum(const float* const part[2], void* out0, void* out1, int64_t T, int G,
                                     int hpg, int D, int dtype, cudaStream_t stream) {
    const int64_t n4 = T * G * (D / 4);
    const dim3 grid((unsigned)((n4 + 255) / 256), 2);
    if (dtype == SSD_BF16)
        linattn_group_sum<__nv_bfloat16><<<grid, 256, 0, stream>>>(part[0], part[1], (__nv_bfloat16*)out0,
                                                                   (__nv_bfloat16*)out1, n4, hpg, D / 4);
    else
        linattn_group_sum<float><<<grid, 256, 0, stream>>>(part[0], part[1], (float*)out0, (float*)out1, n4, hpg, D / 4);
    return cudaGetLastError();
}

}  // namespace ssd
