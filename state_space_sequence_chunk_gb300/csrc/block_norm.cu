// block_norm.cu -- the norms before and after a block, fused with the block's
// gate and residual scale, and their gradient.
//
// Per row (token) of width D, with a(z) the gate (SiLU, sigmoid or none) and
// the block's output y normalised in `ngroups` groups of its columns:
//     yh = y rsqrt(mean_g(y^2) + eps)
//     r' = r + alpha o w_post o a(z) o yh          (residual stream after the block)
//     n  = w_pre o r' rsqrt(mean(r'^2) + eps)      (input of the next block)
// Gradient, with dr' and dn given, rh = r' rsqrt(...), e = w_pre o dn:
//     g   = dr' + rsqrt(...) (e - rh mean(e o rh))                     = dr
//     u   = g o alpha o w_post o a(z);   dy = rsqrt_g (u - yh mean_g(u o yh))
//     dz  = g o alpha o w_post o yh o a'(z)
//     dw_pre = sum_t dn o rh;   E = sum_t g o a(z) o yh;
//     dw_post = alpha o E;      dalpha = w_post o E
// r' is recomputed from r, y and z in fp32, so that the gradient reads no
// rounded copy of it.
//
// Both directions are bound by HBM: 5 and 8 tensors of the input's size.  A row
// stays in registers between its reductions and is read once.  Columns are
// held as vectors of eight; a thread keeps the same columns for all its rows,
// so the weights (and the gradient's column sums) stay in registers too.  CTAs
// are persistent over the rows; each leaves one partial column sum, and a
// second kernel adds those in a fixed order.
#include "block_norm.cuh"

namespace ssd {
namespace {

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xFFFF0000u);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    unpack2(v.x, f[0], f[1]); unpack2(v.y, f[2], f[3]);
    unpack2(v.z, f[4], f[5]); unpack2(v.w, f[6], f[7]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]),
                                              pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's threads.  kWarp: the row is one warp.  Else the CTA; `buf`
// (32 floats) must not be reused until a barrier later than this one.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if (kWarp) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? buf[lane] : 0.f);
}

// Per-group sums of part[i] (one per vector of eight columns) for each of this
// thread's vectors.  Three forms: one group (a row sum), groups of 8, 16 .. 256
// columns that lie within a warp's consecutive vectors (shuffles), and any
// other (through shared memory: grp[] holds a float for each vector, then
// behind it one for each group).
template <int NV, bool kWarp>
__device__ __forceinline__ void group_sum(const NormParams& p, float (&part)[NV], float* buf, float* grp,
                                          int first, int stride) {
    if (p.ngroups == 1) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) v += part[i];
        v = row_sum<kWarp>(v, buf);
#pragma unroll
        for (int i = 0; i < NV; ++i) part[i] = v;
        return;
    }
    if (p.gvecs <= 32 && (p.gvecs & (p.gvecs - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            for (int o = 1; o < p.gvecs; o <<= 1) part[i] += __shfl_xor_sync(0xffffffffu, part[i], o);
        return;
    }
    const int lane = threadIdx.x & 31, warp = kWarp ? 0 : threadIdx.x >> 5,
              nw = kWarp ? 1 : blockDim.x >> 5;
    float* sums = grp + p.vecs;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (first + i * stride < p.vecs) grp[first + i * stride] = part[i];
    if (kWarp) __syncwarp(); else __syncthreads();
    for (int g = warp; g < p.ngroups; g += nw) {
        float v = 0.f;
        for (int j = lane; j < p.gvecs; j += 32) v += grp[g * p.gvecs + j];
        v = warp_sum(v);
        if (lane == 0) sums[g] = v;
    }
    if (kWarp) __syncwarp(); else __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) part[i] = sums[j / p.gvecs];
    }
    if (kWarp) __syncwarp(); else __syncthreads();
}

// the gate and, for the gradient, its derivative
template <bool kGrad>
__device__ __forceinline__ void gate_of(int kind, float z, float& a, float& da) {
    if (kind == SSD_GATE_NONE) {
        a = 1.f;
        da = 0.f;
        return;
    }
    const float s = 1.f / (1.f + expf(-z));
    if (kind == SSD_GATE_SILU) {
        a = z * s;
        if (kGrad) da = s * (1.f + z * (1.f - s));
    } else {
        a = s;
        if (kGrad) da = s * (1.f - s);
    }
}

template <typename T, typename R, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : NV == 1 ? 256 : 512) block_norm_fwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int rpb = kWarp ? blockDim.x >> 5 : 1, sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    float cw[NV][8], wp[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
#pragma unroll
        for (int e = 0; e < 8; ++e) cw[i][e] = wp[i][e] = 1.f;
        if (j < p.vecs) {
            float t[8];
            load8(p.w_pre + 8 * j, wp[i]);
            if (p.w_post) load8(p.w_post + 8 * j, cw[i]);
            if (p.alpha) {
                load8(p.alpha + 8 * j, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) cw[i][e] *= t[e];
            }
        }
    }
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    // the last reduction's buffer alternates: a row may have no other barrier
    float* buf = sm + 32;
    for (int64_t row = (int64_t)blockIdx.x * rpb + sub; row < p.T; row += (int64_t)gridDim.x * rpb) {
        const R* r = static_cast<const R*>(p.r) + row * p.D;
        const T* y = static_cast<const T*>(p.y) + row * p.ys;
        const T* z = static_cast<const T*>(p.z) + row * p.zs;
        float yv[NV][8], zv[NV][8], rv[NV][8], part[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
#pragma unroll
            for (int e = 0; e < 8; ++e) yv[i][e] = zv[i][e] = rv[i][e] = 0.f;
            if (j < p.vecs) {
                load8(y + 8 * j, yv[i]);
                if (p.gate != SSD_GATE_NONE) load8(z + 8 * j, zv[i]);
                load8(r + 8 * j, rv[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            part[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) part[i] = fmaf(yv[i][e], yv[i][e], part[i]);
        }
        group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            const float rs = rsqrtf(part[i] * inv_gw + p.eps);
            if (j < p.vecs && p.rstd_post && j % p.gvecs == 0)
                p.rstd_post[row * p.ngroups + j / p.gvecs] = rs;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a, da;
                gate_of<false>(p.gate, zv[i][e], a, da);
                rv[i][e] = fmaf(cw[i][e] * a, yv[i][e] * rs, rv[i][e]);
                if (j < p.vecs) sq = fmaf(rv[i][e], rv[i][e], sq);
            }
            if (j < p.vecs) store8(static_cast<R*>(p.r_out) + row * p.D + 8 * j, rv[i]);
        }
        const float q = rsqrtf(row_sum<kWarp>(sq, buf) * inv_d + p.eps);
        buf = buf == sm + 32 ? sm + 64 : sm + 32;
        if (p.rstd_pre && first == 0) p.rstd_pre[row] = q;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
#pragma unroll
                for (int e = 0; e < 8; ++e) rv[i][e] *= q * wp[i][e];
                store8(static_cast<T*>(p.n) + row * p.D + 8 * j, rv[i]);
            }
        }
    }
}

template <typename T, typename R, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : NV == 1 ? 256 : 512) block_norm_bwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int rpb = kWarp ? blockDim.x >> 5 : 1, sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    float cw[NV][8], wp[NV][8], se[NV][8], sf[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cw[i][e] = wp[i][e] = 1.f;
            se[i][e] = sf[i][e] = 0.f;
        }
        if (j < p.vecs) {
            float t[8];
            load8(p.w_pre + 8 * j, wp[i]);
            if (p.w_post) load8(p.w_post + 8 * j, cw[i]);
            if (p.alpha) {
                load8(p.alpha + 8 * j, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) cw[i][e] *= t[e];
            }
        }
    }
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    // the last reduction's buffer alternates: a row may have no other barrier
    float* buf = sm + 32;
    for (int64_t row = (int64_t)blockIdx.x * rpb + sub; row < p.T; row += (int64_t)gridDim.x * rpb) {
        const float q = p.rstd_pre[row];
        float yv[NV][8], zv[NV][8], rv[NV][8], dn[NV][8], gr[NV][8], rs[NV], part[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            rs[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) yv[i][e] = zv[i][e] = rv[i][e] = dn[i][e] = gr[i][e] = 0.f;
            if (j < p.vecs) {
                load8(static_cast<const T*>(p.y) + row * p.ys + 8 * j, yv[i]);
                if (p.gate != SSD_GATE_NONE) load8(static_cast<const T*>(p.z) + row * p.zs + 8 * j, zv[i]);
                load8(static_cast<const R*>(p.r) + row * p.D + 8 * j, rv[i]);
                load8(static_cast<const T*>(p.dn) + row * p.D + 8 * j, dn[i]);
                load8(static_cast<const R*>(p.dr_out) + row * p.D + 8 * j, gr[i]);
                rs[i] = p.rstd_post[row * p.ngroups + j / p.gvecs];
            }
        }
        // rv becomes rh; the mean of e o rh over the row
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a, da;
                gate_of<false>(p.gate, zv[i][e], a, da);
                yv[i][e] *= rs[i];                                    // yh
                rv[i][e] = fmaf(cw[i][e] * a, yv[i][e], rv[i][e]) * q;
                sf[i][e] = fmaf(dn[i][e], rv[i][e], sf[i][e]);
                dot = fmaf(wp[i][e] * dn[i][e], rv[i][e], dot);
            }
        dot = row_sum<kWarp>(dot, buf) * inv_d;
        buf = buf == sm + 32 ? sm + 64 : sm + 32;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            part[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a, da;
                gate_of<true>(p.gate, zv[i][e], a, da);
                const float g = fmaf(q, fmaf(wp[i][e], dn[i][e], -rv[i][e] * dot), gr[i][e]);
                gr[i][e] = g;
                se[i][e] = fmaf(g * a, yv[i][e], se[i][e]);
                dn[i][e] = g * cw[i][e] * a;                          // u
                zv[i][e] = g * cw[i][e] * yv[i][e] * da;              // dz
                part[i] = fmaf(dn[i][e], yv[i][e], part[i]);
            }
            if (j < p.vecs) {
                store8(static_cast<R*>(p.dr) + row * p.D + 8 * j, gr[i]);
                if (p.gate != SSD_GATE_NONE) store8(static_cast<T*>(p.dz) + row * p.D + 8 * j, zv[i]);
            }
        }
        group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                const float m = part[i] * inv_gw;
#pragma unroll
                for (int e = 0; e < 8; ++e) dn[i][e] = rs[i] * fmaf(-yv[i][e], m, dn[i][e]);
                store8(static_cast<T*>(p.dy) + row * p.D + 8 * j, dn[i]);
            }
        }
    }
    float* pe = p.partial + ((int64_t)blockIdx.x * rpb + sub) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
            store8(pe + 8 * j, se[i]);
            store8(pe + p.D + 8 * j, sf[i]);
        }
    }
}

// Column sums of the partials: 32 columns and 8 strided runs of them per CTA.
__global__ void __launch_bounds__(256) block_norm_reduce(const __grid_constant__ NormParams p, int nparts) {
    __shared__ float sh[2][8][33];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float e = 0.f, f = 0.f;
    if (c < p.D)
        for (int i = w; i < nparts; i += 8) {
            e += p.partial[(int64_t)i * 2 * p.D + c];
            f += p.partial[(int64_t)i * 2 * p.D + p.D + c];
        }
    sh[0][w][x] = e;
    sh[1][w][x] = f;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    e = f = 0.f;
    for (int i = 0; i < 8; ++i) {
        e += sh[0][i][x];
        f += sh[1][i][x];
    }
    if (p.dw_post) p.dw_post[c] = (p.alpha ? p.alpha[c] : 1.f) * e;
    if (p.dalpha) p.dalpha[c] = (p.w_post ? p.w_post[c] : 1.f) * e;
    p.dw_pre[c] = f;
}

struct Cut {
    int nv, threads;
    bool warp;
};
// Vectors per thread and threads per row: rows of up to 512 columns take one
// warp each (four to a CTA), longer ones a CTA.
Cut cut_of(int vecs) {
    if (vecs <= 64) return {vecs <= 32 ? 1 : 2, 128, true};
    const int nv = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
    const int per = (vecs + nv - 1) / nv;
    return {nv, (per + 31) / 32 * 32, false};
}

size_t shared_bytes(const NormParams& p, const Cut& c) {
    return (96 + (size_t)p.grp_floats * (c.warp ? c.threads / 32 : 1)) * 4;
}

template <typename T, typename R>
cudaError_t go(NormParams& p, bool backward, int grid, cudaStream_t stream) {
    const Cut c = cut_of(p.vecs);
    void (*k)(NormParams) = nullptr;
    if (backward)
        k = c.warp ? (c.nv == 1 ? block_norm_bwd<T, R, 1, true> : block_norm_bwd<T, R, 2, true>)
          : c.nv == 1 ? block_norm_bwd<T, R, 1, false>
          : c.nv == 2 ? block_norm_bwd<T, R, 2, false> : block_norm_bwd<T, R, 4, false>;
    else
        k = c.warp ? (c.nv == 1 ? block_norm_fwd<T, R, 1, true> : block_norm_fwd<T, R, 2, true>)
          : c.nv == 1 ? block_norm_fwd<T, R, 1, false>
          : c.nv == 2 ? block_norm_fwd<T, R, 2, false> : block_norm_fwd<T, R, 4, false>;
    k<<<grid, c.threads, shared_bytes(p, c), stream>>>(p);
    return cudaGetLastError();
}

cudaError_t dispatch(NormParams& p, int dtype, int rdtype, bool backward, int grid, cudaStream_t st) {
    if (dtype == SSD_BF16)
        return rdtype == SSD_BF16 ? go<__nv_bfloat16, __nv_bfloat16>(p, backward, grid, st)
                                  : go<__nv_bfloat16, float>(p, backward, grid, st);
    return go<float, float>(p, backward, grid, st);
}

}  // namespace

int block_norm_grid(int64_t T, int vecs, bool backward, int sms) {
    const Cut c = cut_of(vecs);
    const int rpb = c.warp ? c.threads / 32 : 1;
    // CTAs that fit an SM by threads and (for the gradient's larger register
    // footprint) half of that
    int per = 2048 / c.threads;
    if (backward) per = per > 1 ? per / 2 : 1;
    if (per > 16) per = 16;
    const int64_t rows = (T + rpb - 1) / rpb, full = (int64_t)sms * per;
    return (int)(rows < full ? rows : full);
}

int block_norm_parts(int64_t T, int vecs, int sms) {
    const Cut c = cut_of(vecs);
    return block_norm_grid(T, vecs, true, sms) * (c.warp ? c.threads / 32 : 1);
}

cudaError_t launch_block_norm_fwd(NormParams& p, int dtype, int rdtype, int sms, cudaStream_t st) {
    return dispatch(p, dtype, rdtype, false, block_norm_grid(p.T, p.vecs, false, sms), st);
}

cudaError_t launch_block_norm_bwd(NormParams& p, int dtype, int rdtype, int sms, cudaStream_t st) {
    const int grid = p.T > 0 ? block_norm_grid(p.T, p.vecs, true, sms) : 0;
    if (grid > 0) {
        const cudaError_t e = dispatch(p, dtype, rdtype, true, grid, st);
        if (e != cudaSuccess) return e;
    }
    const int parts = grid > 0 ? block_norm_parts(p.T, p.vecs, sms) : 0;
    block_norm_reduce<<<(p.D + 31) / 32, 256, 0, st>>>(p, parts);
    return cudaGetLastError();
}

}  // namespace ssd
