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
// is read once and stays in registers, as it was loaded (bf16 pairs), between
// its reductions; columns are held as vectors of eight.  The weights are read
// where they are used: 12 bytes a column from L1, against 10 to 32 bytes of HBM
// traffic, and the registers they would take hold more rows in flight instead.
// Forwards, a CTA (or, for rows of up to 512 columns, a warp) runs one row.
// Backwards, CTAs are persistent: a thread keeps the same columns for all its
// rows, loads the next row while it computes one, and adds its columns' sums in
// shared memory; each CTA leaves one partial sum, and a second kernel adds those
// in a fixed order.
#include "block_norm.cuh"

namespace ssd {
namespace {

// Eight elements as loaded.
template <typename T> struct Raw;
template <> struct Raw<float> { float4 a, b; };
template <> struct Raw<__nv_bfloat16> { uint4 a; };
__device__ __forceinline__ void zero(Raw<float>& r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void zero(Raw<__nv_bfloat16>& r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void load(Raw<float>& r, const float* p) {
    r.a = __ldg(reinterpret_cast<const float4*>(p));
    r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void load(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p) {
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&f)[8]) {
    unpack2(r.a.x, f[0], f[1]); unpack2(r.a.y, f[2], f[3]);
    unpack2(r.a.z, f[4], f[5]); unpack2(r.a.w, f[6], f[7]);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    Raw<float> r;
    load(r, p);
    unpack(r, f);
}
// alpha o w_post of eight columns
__device__ __forceinline__ void scale8(const NormParams& p, int j, float (&cw)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cw[e] = 1.f;
    if (p.w_post) load8(p.w_post + 8 * j, cw);
    if (p.alpha) {
        float t[8];
        load8(p.alpha + 8 * j, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) cw[e] *= t[e];
    }
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

// sigmoid(z).  Beside bf16 inputs the fast exponential and division serve (errors
// of a few 2^-23 of the value, and of z 2^-24 in the exponent); fp32 inputs get
// the exact ones.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-z));
    return 1.f / (1.f + expf(-z));
}
// Gate and derivative from z and s = sigmoid(z).
__device__ __forceinline__ float gate_of(int kind, float z, float s) {
    return kind == SSD_GATE_NONE ? 1.f : kind == SSD_GATE_SILU ? z * s : s;
}
__device__ __forceinline__ float dgate_of(int kind, float z, float s) {
    return kind == SSD_GATE_NONE ? 0.f : kind == SSD_GATE_SILU ? s * (1.f + z * (1.f - s)) : s * (1.f - s);
}

template <typename T, typename R, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : 512) block_norm_fwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    const int64_t row = kWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + sub : (int64_t)blockIdx.x;
    if (row >= p.T) return;   // a whole row's threads
    Raw<T> y[NV], z[NV];
    Raw<R> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        zero(y[i]);
        zero(z[i]);
        zero(r[i]);
        if (j < p.vecs) {
            load(y[i], static_cast<const T*>(p.y) + row * p.ys + 8 * j);
            if (p.gate != SSD_GATE_NONE) load(z[i], static_cast<const T*>(p.z) + row * p.zs + 8 * j);
            load(r[i], static_cast<const R*>(p.r) + row * p.D + 8 * j);
        }
    }
    float part[NV], rp[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack(y[i], f);
        part[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) part[i] = fmaf(f[e], f[e], part[i]);
    }
    group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
            const float rs = rsqrtf(part[i] * inv_gw + p.eps);
            if (p.rstd_post && j % p.gvecs == 0) p.rstd_post[row * p.ngroups + j / p.gvecs] = rs;
            float cw[8], yf[8], zf[8];
            scale8(p, j, cw);
            unpack(y[i], yf);
            unpack(z[i], zf);
            unpack(r[i], rp[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = gate_of(p.gate, zf[e], sigmoid<T>(zf[e]));
                rp[i][e] = fmaf(cw[e] * a, yf[e] * rs, rp[i][e]);
                sq = fmaf(rp[i][e], rp[i][e], sq);
            }
            store8(static_cast<R*>(p.r_out) + row * p.D + 8 * j, rp[i]);
        }
    }
    const float q = rsqrtf(row_sum<kWarp>(sq, sm + 32) * inv_d + p.eps);
    if (p.rstd_pre && first == 0) p.rstd_pre[row] = q;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
            float wp[8];
            load8(p.w_pre + 8 * j, wp);
#pragma unroll
            for (int e = 0; e < 8; ++e) rp[i][e] *= q * wp[e];
            store8(static_cast<T*>(p.n) + row * p.D + 8 * j, rp[i]);
        }
    }
}

// One row of the gradient's inputs, as loaded.
template <typename T, typename R, int NV>
struct Row {
    Raw<T> y[NV], z[NV], dn[NV];
    Raw<R> r[NV], g[NV];
    float rs[NV], q;
    __device__ __forceinline__ void fetch(const NormParams& p, int64_t row, int first, int stride) {
        q = __ldg(p.rstd_pre + row);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                load(y[i], static_cast<const T*>(p.y) + row * p.ys + 8 * j);
                if (p.gate != SSD_GATE_NONE) load(z[i], static_cast<const T*>(p.z) + row * p.zs + 8 * j);
                load(r[i], static_cast<const R*>(p.r) + row * p.D + 8 * j);
                load(dn[i], static_cast<const T*>(p.dn) + row * p.D + 8 * j);
                load(g[i], static_cast<const R*>(p.dr_out) + row * p.D + 8 * j);
                rs[i] = __ldg(p.rstd_post + row * p.ngroups + j / p.gvecs);
            }
        }
    }
    __device__ __forceinline__ void clear() {
        q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            zero(y[i]); zero(z[i]); zero(dn[i]); zero(r[i]); zero(g[i]);
            rs[i] = 0.f;
        }
    }
};

// Registers: kPrefetch holds two rows.  `acc` in shared memory: per vector four
// float4 a thread (E's eight columns, then w_pre's), strided by the block.
template <typename T, typename R, int NV, bool kWarp, bool kPrefetch>
__global__ void __launch_bounds__(kWarp ? 128 : 640) block_norm_bwd(const __grid_constant__ NormParams p) {
    extern __shared__ float sm[];
    const int first = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
    const int rpb = kWarp ? blockDim.x >> 5 : 1, sub = kWarp ? threadIdx.x >> 5 : 0;
    float* grp = sm + 96 + (kWarp ? sub * p.grp_floats : 0);
    float4* acc = reinterpret_cast<float4*>(sm + 96 + ((p.grp_floats * rpb + 3) & ~3)) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) acc[i * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add8 = [&](int at, const float (&f)[8]) {
        float4 a = acc[at * blockDim.x], b = acc[(at + 1) * blockDim.x];
        a.x += f[0]; a.y += f[1]; a.z += f[2]; a.w += f[3];
        b.x += f[4]; b.y += f[5]; b.z += f[6]; b.w += f[7];
        acc[at * blockDim.x] = a;
        acc[(at + 1) * blockDim.x] = b;
    };
    const float inv_gw = 1.f / (float)(8 * p.gvecs), inv_d = 1.f / (float)(8 * p.vecs);
    const int64_t step = (int64_t)gridDim.x * rpb;
    // the last reduction's buffer alternates: a row may have no other barrier
    float* buf = sm + 32;
    Row<T, R, NV> cur, nxt;
    cur.clear();
    if (kPrefetch) nxt.clear();
    int64_t row = (int64_t)blockIdx.x * rpb + sub;
    if (kPrefetch && row < p.T) cur.fetch(p, row, first, stride);
    for (; row < p.T; row += step) {
        if (!kPrefetch) cur.fetch(p, row, first, stride);
        else if (row + step < p.T) nxt.fetch(p, row + step, first, stride);
        // rh = r' rsqrt; the mean of e o rh over the row
        float dot = 0.f, u[NV][8], sg[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                float cw[8], wp[8], yf[8], zf[8], dnf[8], t[8];
                scale8(p, j, cw);
                load8(p.w_pre + 8 * j, wp);
                unpack(cur.y[i], yf);
                unpack(cur.z[i], zf);
                unpack(cur.r[i], u[i]);
                unpack(cur.dn[i], dnf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sg[i][e] = sigmoid<T>(zf[e]);
                    const float a = gate_of(p.gate, zf[e], sg[i][e]);
                    u[i][e] = fmaf(cw[e] * a, yf[e] * cur.rs[i], u[i][e]) * cur.q;
                    t[e] = dnf[e] * u[i][e];
                    dot = fmaf(wp[e], t[e], dot);
                }
                add8(4 * i + 2, t);
            }
        }
        dot = row_sum<kWarp>(dot, buf) * inv_d;
        buf = buf == sm + 32 ? sm + 64 : sm + 32;
        float part[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            part[i] = 0.f;
            if (j < p.vecs) {
                float cw[8], wp[8], yf[8], zf[8], dnf[8], gf[8], t[8];
                scale8(p, j, cw);
                load8(p.w_pre + 8 * j, wp);
                unpack(cur.y[i], yf);
                unpack(cur.z[i], zf);
                unpack(cur.dn[i], dnf);
                unpack(cur.g[i], gf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = gate_of(p.gate, zf[e], sg[i][e]);
                    const float yh = yf[e] * cur.rs[i];
                    gf[e] = fmaf(cur.q, fmaf(wp[e], dnf[e], -u[i][e] * dot), gf[e]);
                    t[e] = gf[e] * a * yh;
                    u[i][e] = gf[e] * cw[e] * a;
                    zf[e] = gf[e] * cw[e] * yh * dgate_of(p.gate, zf[e], sg[i][e]);
                    part[i] = fmaf(u[i][e], yh, part[i]);
                }
                add8(4 * i, t);
                store8(static_cast<R*>(p.dr) + row * p.D + 8 * j, gf);
                if (p.gate != SSD_GATE_NONE) store8(static_cast<T*>(p.dz) + row * p.D + 8 * j, zf);
            }
        }
        group_sum<NV, kWarp>(p, part, sm, grp, first, stride);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = first + i * stride;
            if (j < p.vecs) {
                const float m = part[i] * inv_gw;
                float yf[8];
                unpack(cur.y[i], yf);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[i][e] = cur.rs[i] * fmaf(-yf[e] * cur.rs[i], m, u[i][e]);
                store8(static_cast<T*>(p.dy) + row * p.D + 8 * j, u[i]);
            }
        }
        if (kPrefetch) cur = nxt;
    }
    float* pe = p.partial + ((int64_t)blockIdx.x * rpb + sub) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = first + i * stride;
        if (j < p.vecs) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                reinterpret_cast<float4*>(pe + (x >> 1) * p.D + 8 * j)[x & 1] = acc[(4 * i + x) * blockDim.x];
        }
    }
}

// Column sums of the partials: a CTA has 32 columns of E (blockIdx.y 0) or of
// w_pre's sums, and 16 strided runs of the partials, joined in a fixed order.
__global__ void __launch_bounds__(512) block_norm_reduce(const __grid_constant__ NormParams p, int nparts) {
    __shared__ float sh[16][33];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float v = 0.f;
    if (c < p.D) {
        const float* src = p.partial + (int64_t)blockIdx.y * p.D + c;
#pragma unroll 8
        for (int i = w; i < nparts; i += 16) v += src[(int64_t)i * 2 * p.D];
    }
    sh[w][x] = v;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += sh[i][x];
    if (blockIdx.y == 1) {
        p.dw_pre[c] = v;
    } else {
        if (p.dw_post) p.dw_post[c] = (p.alpha ? p.alpha[c] : 1.f) * v;
        if (p.dalpha) p.dalpha[c] = (p.w_post ? p.w_post[c] : 1.f) * v;
    }
}

struct Cut {
    int nv, threads;
    bool warp;
};
// Vectors per thread and threads per row: rows of up to 512 columns take one
// warp each (four to a CTA), longer ones a CTA.  Backwards fewer vectors fit a
// thread's registers.
Cut cut_of(int vecs, bool backward) {
    if (vecs <= 64) return {vecs <= 32 ? 1 : 2, 128, true};
    const int nv = backward ? (vecs <= 640 ? 1 : vecs <= 1280 ? 2 : 4) : vecs <= 128 ? 1 : vecs <= 1024 ? 2 : 4;
    const int per = (vecs + nv - 1) / nv;
    return {nv, (per + 31) / 32 * 32, false};
}

size_t shared_bytes(const NormParams& p, const Cut& c, bool backward) {
    const int rpb = c.warp ? c.threads / 32 : 1;
    const size_t grp = 96 + ((size_t)p.grp_floats * rpb + 3) / 4 * 4;
    return (grp + (backward ? (size_t)16 * c.nv * c.threads : 0)) * 4;
}

template <typename T, typename R>
cudaError_t go(NormParams& p, bool backward, int64_t grid, cudaStream_t stream) {
    const Cut c = cut_of(p.vecs, backward);
    const size_t bytes = shared_bytes(p, c, backward);
    void (*k)(NormParams) = nullptr;
    if (backward)
        // two rows at once where they fit the registers
        k = c.warp ? (c.nv == 1 ? block_norm_bwd<T, R, 1, true, sizeof(T) == 2> : block_norm_bwd<T, R, 2, true, false>)
          : c.nv == 1 ? block_norm_bwd<T, R, 1, false, sizeof(T) == 2>
          : c.nv == 2 ? block_norm_bwd<T, R, 2, false, false> : block_norm_bwd<T, R, 4, false, false>;
    else
        k = c.warp ? (c.nv == 1 ? block_norm_fwd<T, R, 1, true> : block_norm_fwd<T, R, 2, true>)
          : c.nv == 1 ? block_norm_fwd<T, R, 1, false>
          : c.nv == 2 ? block_norm_fwd<T, R, 2, false> : block_norm_fwd<T, R, 4, false>;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)grid, c.threads, bytes, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t dispatch(NormParams& p, int dtype, int rdtype, bool backward, int64_t grid, cudaStream_t st) {
    if (dtype == SSD_BF16)
        return rdtype == SSD_BF16 ? go<__nv_bfloat16, __nv_bfloat16>(p, backward, grid, st)
                                  : go<__nv_bfloat16, float>(p, backward, grid, st);
    return go<float, float>(p, backward, grid, st);
}

}  // namespace

int block_norm_grid(int64_t T, int vecs, int sms) {
    const Cut c = cut_of(vecs, true);
    const int rpb = c.warp ? c.threads / 32 : 1;
    const int per = 640 / c.threads;   // by registers
    const int64_t rows = (T + rpb - 1) / rpb, full = (int64_t)sms * per;
    return (int)(rows < full ? rows : full);
}

int block_norm_parts(int64_t T, int vecs, int sms) {
    const Cut c = cut_of(vecs, true);
    return block_norm_grid(T, vecs, sms) * (c.warp ? c.threads / 32 : 1);
}

cudaError_t launch_block_norm_fwd(NormParams& p, int dtype, int rdtype, cudaStream_t st) {
    const Cut c = cut_of(p.vecs, false);
    const int rpb = c.warp ? c.threads / 32 : 1;
    return dispatch(p, dtype, rdtype, false, (p.T + rpb - 1) / rpb, st);
}

cudaError_t launch_block_norm_bwd(NormParams& p, int dtype, int rdtype, int sms, cudaStream_t st) {
    const int grid = p.T > 0 ? block_norm_grid(p.T, p.vecs, sms) : 0;
    if (grid > 0) {
        const cudaError_t e = dispatch(p, dtype, rdtype, true, grid, st);
        if (e != cudaSuccess) return e;
    }
    const int parts = grid > 0 ? block_norm_parts(p.T, p.vecs, sms) : 0;
    block_norm_reduce<<<dim3((unsigned)(p.D + 31) / 32, 2), 512, 0, st>>>(p, parts);
    return cudaGetLastError();
}

}  // namespace ssd
