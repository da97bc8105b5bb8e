// linattn_tc.cu -- linear attention with a decay for each head on the tcgen05
// tensor cores (bf16 operands, fp32 accumulation and state).
//
// One chain is (range of a sequence, head, 64 columns of c), walked in chunks of
// 128 tokens.  With i, j the rows of a chunk (counted from its end when the walk
// is backwards), n its tokens and X the state before it:
//     W   = A B^T                                   128 x 128 x DK
//     P   = s_in W o lam^{i-j} [i >= j]             (bf16, tensor memory)
//     out = s_out (lam^{i+1} o (A X) + P C)         128 x 64 x DK, 128 x 64 x 128
//     U   = B^T (s_in lam^{n-1-j} o C)              DK x 64 x 128
//     X   <- lam^n X + U
// (backwards X and U have decayed one step less and one more).  No factor is above 1:
// lam^{i-j} is taken as a power up to the column's block of 32 times one within it, and
// the rows of A X get theirs in the accumulator, before P C is added to it.  So products
// and states of any size that fp32 holds come through, however fast the head forgets.
// (Row and column factors about the chunk's middle, lam^{i-64} and lam^{64-j}, save that
// pass over the accumulator, but reach 2^+-60 for a head with lam = 1/2: a product or a
// state beyond 2^67 overflowed, one below 2^-66 was lost.  They were 2 % faster for the
// packed prompt below, 5 % for the training step, and 5 % slower for the long prompt.)
// Every operand is read once per chain from HBM (a and b once per 64 columns of
// c, from L2 the second time) and no state leaves the chip between chunks.
//
// Precision.  P and the copy of X that multiplies A are rounded to bf16, as operands of
// products whose result is rounded to bf16 (P to 16 bits for a chunk of few tokens): o is
// off by 0.0023 where its own rounding makes 0.0017.  (Both operands in two bf16 terms
// bring 0.0017.  Their products fit into the tensor pipe's pauses, but cutting them and the
// second tile for X took the packed prompt below from 154 to 193 us.)  X itself must not
// be rounded: it is kept in fp32 registers and U is exact to fp32: C's scaled rows are cut into three
// bf16 terms of 8 bits each, multiplied side by side (N = 192) into separate
// accumulators and added from the smallest up.  X <- lam^n X + U runs on the
// CUDA cores, where it is rounded to nearest (how the tensor core's accumulator
// rounds is not documented, and a chain adds it up over hundreds of chunks).
//
// Persistent CTAs of 30 warps, one per SM:
//   0-7   P: tensor memory -> decay, mask -> tensor memory (bf16, in place; two
//         warpgroups, half of the columns each)
//   8-15  C's scaled terms (a thread owns half of a token's row); zeroes the rows
//         of a ragged chunk that belong to other tokens, whatever they hold, and takes
//         infinities and NaN out of the C tile
//   16-23 X in registers (a thread owns 32 columns of a row): bf16 copy for A X,
//         update with U, stored states
//   24-27 out (a thread owns a token row): the rows' decay of A X, then the stores
//   28    TMA, two stages of A and B tiles (64 KB each), three C tiles; the next item
//   29    MMA issue: U(c)'s first half, W(c + 1), A X(c), U(c)'s second half, P C(c)
// The roles' loops are kept short (packed fp32 arithmetic, little unrolling): six
// codes run side by side on each scheduler, and fully unrolled they spent most of
// their time on instruction fetches.
//
// A chunk takes about 4000 cycles of an SM: 1900 of products and 3000 of shared-memory
// traffic (400 KB) side by side, and between them a chain that bounds it (terms, half of U,
// terms, half of U, state, and the issuing warp's fetches at each turn of its loop).
// 16384 packed tokens, 32 heads of 128 x 128: 154 us, 57 % of the copy rate on the bytes
// that must move; one sequence of 65536, 24 heads of 128 x 64 with shared q and k: 266 us
// in three launches (79, 10 and 177); a training step of 16384 tokens, 16 heads of
// 128 x 128: 317 us.
#include <cuda.h>
#include <string.h>

#include <atomic>

#include "f32x2.cuh"
#include "linattn_internal.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace ssd {
namespace {

// The number of the last launch in which a bounded wait gave up, or 0: by it the other
// waits of that launch learn to give up too, and no later launch is taken for it.
__device__ unsigned int g_la_error;
// Test hook (ssd_debug_withhold_handoffs): nonzero makes the TMA warps load nothing, so
// that the first waits run out.
__device__ unsigned int g_la_withhold;

constexpr int kC = 128;                       // tokens per chunk
constexpr int kRow = 128;                     // bytes of a tile row (64 columns)
constexpr int kAtom = kC * kRow;              // 16 KB: 128 rows of 64 columns
constexpr int kThreads = 960;
constexpr int kTmaWarp = 28, kMmaWarp = 29;
constexpr int kTerms = 3;
constexpr int kTerm = kAtom / 2;              // a term of 64 tokens
// What the two passes keep: stages of A and B, C tiles, buffers for a half's terms
// (with one, the halves take turns), accumulators for U.  The pass over the ranges'
// own sums has no A, W and out.
template <bool kAgg> struct Cfg {
    static constexpr int kCs = kAgg ? 4 : 3;
    static constexpr int kSt = kAgg ? 3 : 2;
    static constexpr int kTb = kAgg ? 2 : 1;
    static constexpr int kUb = kAgg ? 2 : 1;
    static constexpr int kB = kAgg ? 0 : 2 * kAtom;      // a stage: A (2 atoms), B (2)
    static constexpr int kStage = kB + 2 * kAtom;
    static constexpr int kSmem = kSt * kStage + kCs * kAtom + kTb * kTerms * kTerm + (kAgg ? 0 : kAtom + 1024) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};
// tensor memory columns
constexpr uint32_t kW = 0;                    // W / P, two buffers of 128
constexpr uint32_t kO = 256, kUMain = 320;    // out; U's three terms

struct TcParams {
    LaParams p;
    int nvb;
    unsigned int launch;       // number of the launch, not 0
    unsigned int* host_err;
};
struct TcMaps {
    CUtensorMap m[3][4];   // job, operand (A, B, C, out)
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// Shared memory by its 32-bit address: through generic pointers these accesses
// take the path of global loads.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void bar_p() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// mbar_wait (the same bounds) in as few instructions as it takes: the roles' loops
// share the instruction cache, and there are two dozen waits in them.  A thread whose
// wait gave up is gone: it waits for nothing more, walks its item to the end, whatever
// that computes, and leaves.  (Leaving after a chunk took a vote in every chunk of every
// role: the long prompt took 5 % more.)
struct Watch {
    unsigned int launch;
    uint32_t slow;   // cycles after which a wait looks at the launch's error word; 0: gone
    __device__ __forceinline__ bool gone() const { return slow == 0u; }
};
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, Watch& w) {
    if (mbar_try_wait(bar, parity)) return;
    const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        const uint32_t dt = (uint32_t)clock() - t0;
        if (dt > w.slow) {
            volatile unsigned int* e = &g_la_error;
            if (*e == w.launch || dt > (uint32_t)kWaitLimitCycles) {
                *e = w.launch;
                w.slow = 0u;
                return;
            }
        }
    }
}
// Whether `v` holds for any of a named barrier's threads, which wait for one another:
// the warps of a role that uses one leave together.
template <int kId, int kThr>
__device__ __forceinline__ bool any_of(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)v), "n"(kId), "n"(kThr) : "memory");
    return r != 0u;
}

// After a wait that gave up: time for the copies and products in flight to end
// before the CTA's shared and tensor memory are given back.
__device__ __noinline__ void settle() {
    const uint32_t t0 = (uint32_t)clock();
    while ((uint32_t)clock() - t0 < (uint32_t)kWaitSlowCycles) {}
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Whether the first barrier's phase completes before the second's (or within 64 looks).
__device__ __forceinline__ bool first_of(uint32_t a, uint32_t a_parity, uint32_t b, uint32_t b_parity) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        if (mbar_test(a, a_parity)) return true;
        if (mbar_test(b, b_parity)) break;
    }
    return false;
}

// A chunk of so few tokens leaves the second half of P's contraction free: it holds
// P's second terms there (and P is then good to 16 bits), for tokens whose output is
// a sum of a few products, or of one.
__device__ __forceinline__ bool few(int n) { return n <= 64; }
// P of such a chunk, a row to a thread.  Not inlined: the roles' loops share the
// instruction cache (in line, a training step of 16384 tokens takes 334 us, not 317).
__device__ __noinline__ void few_p(uint32_t base, int row, int n, float a2, float s_in, int rev) {
#pragma unroll 1
    for (int j0 = 0; j0 < 64; j0 += 8) {
        uint32_t v[8], hi[4], lo[4];
        __syncwarp();
        tmem_ld_x8(base + j0, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float r[2], l[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = j0 + e + y, d = rev ? j - row : row - j;
                const float w = exp2f(a2 * (float)max(d, 0)) * s_in;
                r[y] = d >= 0 && j < n ? __uint_as_float(v[e + y]) * w : 0.f;
            }
            hi[e / 2] = pack2(r[0], r[1]);
            l[0] = r[0] - lo16(hi[e / 2]);
            l[1] = r[1] - hi16(hi[e / 2]);
            // an infinity or a NaN is the first term's alone
            lo[e / 2] = pack2(fabsf(l[0]) < INFINITY ? l[0] : 0.f, fabsf(l[1]) < INFINITY ? l[1] : 0.f);
        }
        __syncwarp();
        tmem_st_x4(base + j0 / 2, hi);
        tmem_st_x4(base + j0 / 2 + 64, lo);
    }
    tmem_wait_st();
}
// Infinities and NaN in C.  The products above P's diagonal are 0 times C's later rows, and
// would hand such a value to the rows before it.  It is taken out of the C tile, and the
// first row (counted in the walk's direction) that had one is kept for each column: from
// there on the column's results become NaN.  U, and with it the state, takes the value.
struct Spoilt {
    uint32_t first, any;   // of a C tile: int [64], and whether there is one
};
__device__ __forceinline__ bool spoils(uint32_t v) { return (v & 0x7F80u) == 0x7F80u; }   // a bf16
__device__ __noinline__ void take_out(uint32_t row_at, int row, int ch0, int place, Spoilt sp) {
#pragma unroll 1
    for (int v = ch0 * 8; v < ch0 * 8 + 32; ++v) {
        const uint32_t at = row_at + (((v >> 3) ^ (row & 7)) << 4) + 2 * (v & 7);
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
        if (spoils(x)) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0) : "memory");
            asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(sp.first + 4 * v), "r"(place) : "memory");
        }
    }
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(sp.any), "r"(1) : "memory");
}
// The out role's part, on the accumulator of a row; one warp.
__device__ __noinline__ void spoil(uint32_t acc, int place, Spoilt sp) {
#pragma unroll 1
    for (int v = 0; v < 64; v += 8) {
        uint32_t p[8];
        __syncwarp();
        tmem_ld_x8(acc + v, p);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (place >= __float_as_int(lds32(sp.first + 4 * (v + e)))) p[e] = 0x7FFFFFFFu;
        tmem_st_x8(acc + v, p);
    }
    tmem_wait_st();
}
// 2^(a2 n), with the product's rounding put back: n a2 can be as large as kSpan,
// where a rounding of the exponent would be one of the result's last bits.
__device__ __forceinline__ float la_exp2(float a2, int n) {
    const float p = a2 * (float)n, e = fmaf(a2, (float)n, -p);
    const float r = exp2f(p);
    return fmaf(r, e * 0.6931471805599453f, r);
}

// Items are handed out by the hardware: the grid has one CTA for each, and a
// running CTA takes the index of one that has not started, which is then not
// launched (cluster launch control).  Ranges differ in length, so a fixed share
// of them for each CTA left SMs idle.
__device__ __forceinline__ void request_item(uint32_t slot, uint32_t bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
        ::"r"(slot), "r"(bar) : "memory");
}
// The answer in `slot`: a CTA's index, or -1 when none is left.
__device__ __forceinline__ int granted_item(uint32_t slot) {
    int x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%1];\n\tmov.b32 %0, -1;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x) : "r"(slot) : "memory");
    return x;
}

// One item: 64 columns of one job, of one head, of one range.  The TMA warp
// works it out, a chunk or more before the others need it, and leaves it in
// shared memory: found by every role for itself, each change of item cost the
// time of two or three chunks.
struct Item {
    int seq, ridx, t0, len;        // sequence (nseq: rows of none), range (its slot of agg), its rows
    int job, h, v0, nch;           // nch < 0: no more items
    int cut, last;
    float a2, hi, lo;              // log2 of the decay; the decay over a chunk
    int pad[3];
};
static_assert(sizeof(Item) == 64, "two slots of 64 bytes");

// The idx-th longest sequence, when none is cut and there are fewer than 32 (rows of
// no sequence come last): the SMs then end together, also where a long sequence
// stands behind short ones (355 -> 317 us for a training step on six sequences of 1477
// to 3868 tokens, 16 heads of 128 x 128).  One warp.
__device__ __forceinline__ LaRange longest(const LaGeom& g, int idx) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = 0, key = -1;
    if (lane <= g.nseq) {
        la_bounds(g, lane, lo, hi);
        if (lane < g.nseq) key = hi - lo;
    }
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o <= g.nseq; ++o) {
        const int k = __shfl_sync(0xffffffffu, key, o);
        rank += k > key || (k == key && o < lane) ? 1 : 0;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, lane <= g.nseq && rank == idx)) - 1;
    LaRange r;
    r.seq = -1;
    r.first = r.last = 1;
    r.t0 = r.len = r.slot = 0;
    if (src < 0) return r;
    lo = __shfl_sync(0xffffffffu, lo, src);
    hi = __shfl_sync(0xffffffffu, hi, src);
    if (src == g.nseq && lo == hi) return r;
    r.seq = src;
    r.t0 = lo;
    r.len = hi - lo;
    return r;
}

template <bool kAgg>
__device__ __forceinline__ void decode_item(const TcParams& tp, int it, Item* slot) {
    Item r;
    const int vb = it % tp.nvb;
    int x = it / tp.nvb;
    r.job = x % tp.p.njobs;
    x /= tp.p.njobs;
    r.h = x % tp.p.g.H;
    r.ridx = x / tp.p.g.H;
    const float a = tp.p.g.a[r.h];
    const LaRange rg = !tp.p.g.split && tp.p.g.nseq < 32 ? longest(tp.p.g, r.ridx) : la_find(tp.p.g, r.ridx);
    r.seq = rg.seq;
    r.ridx = rg.slot;
    r.t0 = rg.t0;
    r.len = rg.len;
    r.v0 = vb * kLaCols;
    const LaJob& jb = tp.p.job[r.job];
    r.cut = tp.p.g.split && !(rg.first && rg.last);
    r.last = jb.rev ? rg.first : rg.last;
    const bool none = rg.seq < 0 || r.v0 >= jb.DV || (kAgg && (!r.cut || r.last || rg.seq == tp.p.g.nseq));
    r.nch = none || rg.seq == tp.p.g.nseq ? 0 : (rg.len + kC - 1) / kC;
    if (none) r.seq = -1;
    r.a2 = la_log2_decay(&a, 0);
    la_decay_pow(&a, 0, kC, r.hi, r.lo);
    r.pad[0] = r.pad[1] = r.pad[2] = 0;
    const int lane = threadIdx.x & 31;
    if (lane == 0) *slot = r;
    // the state that the item starts from, to L2
    if (!kAgg && !none && rg.seq != tp.p.g.nseq) {
        const int64_t elems = (int64_t)jb.DK * jb.DV;
        const float* in = r.cut ? jb.agg + ((int64_t)r.ridx * tp.p.g.H + r.h) * elems
                                : (jb.init ? jb.init + ((int64_t)rg.seq * tp.p.g.H + r.h) * elems : nullptr);
        const int nv = min(kLaCols, jb.DV - r.v0);
        const int rows = jb.sk == 1 ? nv : jb.DK, width = jb.sk == 1 ? jb.DK : nv, pitch = jb.sk == 1 ? jb.sv : jb.sk;
        if (in != nullptr) {
            in += (int64_t)r.v0 * jb.sv;
            const int lines = (width + 31) / 32;
            for (int e = lane; e < rows * lines; e += 32)
                prefetch_l2(in + (int64_t)(e / lines) * pitch + (e % lines) * 32);
        }
    }
    __syncwarp();
}

// One lane of a converged warp.  The compiler knows such a branch to be uniform
// and keeps what it computes in uniform registers: an MMA then takes 3
// instructions to issue, in a branch of lane 0 it takes 8 and more (and some 200
// cycles, which bound the kernel).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0u;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// Up to 8 products of 16 along the contraction, overwriting d.  An operand is
// K-major (two 64-wide tiles side by side) or MN-major (rows of the contraction).
template <bool kAK, bool kBK>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t a, uint64_t b, int steps, uint32_t idesc) {
    const auto one = [&](int kk) {
        const uint32_t ok = (uint32_t)((kk / 4) * kAtom + (kk % 4) * 32) >> 4, om = (uint32_t)(kk * 16 * kRow) >> 4;
        mma_f16_ss(d, a + (kAK ? ok : om), b + (kBK ? ok : om), idesc, kk > 0 ? 1u : 0u);
    };
    if (steps == 8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) one(kk);
    } else {
#pragma unroll 1
        for (int kk = 0; kk < steps; ++kk) one(kk);
    }
}

// kPart: some job's outputs are fp32, for a sum over a group's heads.  (Without what the
// others need the code is shorter, which every call feels.)
template <bool kAgg, bool kPart>
__global__ void __launch_bounds__(kThreads, 1)
linattn_tc(const __grid_constant__ TcParams tp, const __grid_constant__ TcMaps maps) {
    // aligned by declaration, not by arithmetic: its addresses are then constants
    // and cost no registers
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) {
            g_la_error = tp.launch;
            report_timeout_to_host(&g_la_error, tp.host_err);
        }
        return;
    }
    constexpr int kB = Cfg<kAgg>::kB, kStage = Cfg<kAgg>::kStage, kCs = Cfg<kAgg>::kCs, kTb = Cfg<kAgg>::kTb, kSt = Cfg<kAgg>::kSt, kUb = Cfg<kAgg>::kUb;
    constexpr uint32_t kU = kAgg ? 0 : kUMain;
    uint8_t* ctile = smem + kSt * kStage;
    uint8_t* terms = ctile + kCs * kAtom;
    uint8_t* xs = terms + kTb * kTerms * kTerm;
    uint64_t* bars = reinterpret_cast<uint64_t*>(xs + (kAgg ? 0 : kAtom));
    uint64_t* b_fab = bars;           // [3] stage's A and B loaded (tx)
    uint64_t* b_eab = bars + 33;      // [3] A and B read by every product (commit)
    uint64_t* b_fc = bars + 4;        // [4] C tile loaded (tx)
    uint64_t* b_ec = bars + 8;        // [4] C read by every product, and out stored from it
    uint64_t* b_wdone = bars + 12;    // [2] W computed (commit)
    uint64_t* b_pready = bars + 14;   // [2] P written (256)
    uint64_t* b_vready = bars + 16;   // [2] terms of a half of the tokens written (128)
    uint64_t* b_udone = bars + 18;    // [2] U's half computed, its terms read (commit)
    uint64_t* b_ux = bars + 20;       // [2] U computed (commit)
    uint64_t* b_ufree = bars + 22;    // [2] U read (256)
    uint64_t* b_sready = bars + 24;   // bf16 X written (256)
    uint64_t* b_xdone = bars + 25;    // A X computed: the bf16 X may change (commit)
    uint64_t* b_odone = bars + 26;    // out computed (commit)
    uint64_t* b_ofree = bars + 27;    // out read (128)
    uint64_t* b_scaled = bars + 118;  // A X has its rows' decay (128)
    uint64_t* b_answer = bars + 28;   // answer to an item request (tx)
    uint64_t* b_iready = bars + 29;   // [2] item decoded (1)
    uint64_t* b_ifree = bars + 31;    // [2] item read (every other warp that walks items)
    uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 3);
    const uint32_t answer = smem_u32(bars + 36);    // 16 bytes
    Item* items = reinterpret_cast<Item*>(bars + 38);   // [2]
    const uint32_t ptab = smem_u32(bars + 54);      // [128] fp32: column factors of P
    // of C tile s: the rows from which its columns are spoilt, and whether any is
    const auto spoilt = [&](int s) { return Spoilt{smem_u32(bars + 128) + 256 * s, smem_u32(bars + 128) + 768 + 4 * s}; };

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(b_wdone + s), 1);
            mbar_init(smem_u32(b_pready + s), 256);
            mbar_init(smem_u32(b_vready + s), 128);
            mbar_init(smem_u32(b_udone + s), 1);
            mbar_init(smem_u32(b_ux + s), 1);
            mbar_init(smem_u32(b_ufree + s), 256);
            mbar_init(smem_u32(b_iready + s), 1);
            mbar_init(smem_u32(b_ifree + s), kAgg ? 17 : kThreads / 32 - 1);
        }
        for (int s = 0; s < kSt; ++s) {
            mbar_init(smem_u32(b_fab + s), 1);
            mbar_init(smem_u32(b_eab + s), 1);
        }
        for (int s = 0; s < kCs; ++s) {
            mbar_init(smem_u32(b_fc + s), 1);
            mbar_init(smem_u32(b_ec + s), 1);
        }
        mbar_init(smem_u32(b_answer), 1);
        mbar_init(smem_u32(b_sready), 256);
        mbar_init(smem_u32(b_scaled), 128);
        mbar_init(smem_u32(b_xdone), 1);
        mbar_init(smem_u32(b_odone), 1);
        mbar_init(smem_u32(b_ofree), 128);
        fence_mbar_init();
    }
    if (!kAgg && threadIdx.x < 195) reinterpret_cast<int*>(bars + 128)[threadIdx.x] = threadIdx.x < 192 ? kC : 0;
    if (warp == kMmaWarp) tmem_alloc(smem_u32(holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *holder, 0);
    Watch err = {tp.launch, (uint32_t)kWaitSlowCycles};
    const LaGeom& g = tp.p.g;
    // every role walks the same items and counts chunks in c: barrier phases
    // follow from the count alone
    int c = 0, k_item = 0;
    auto read_item = [&](Item& im) {
        const int slot = k_item & 1;
        wait_on(smem_u32(b_iready + slot), (k_item >> 1) & 1, err);
        const uint32_t at = smem_u32(items) + slot * 64;
        const uint4 q0 = lds128(at), q1 = lds128(at + 16), q2 = lds128(at + 32);
        im.seq = q0.x; im.ridx = q0.y; im.t0 = q0.z; im.len = q0.w;
        im.job = q1.x; im.h = q1.y; im.v0 = q1.z; im.nch = q1.w;
        im.cut = q2.x; im.last = q2.y; im.a2 = __uint_as_float(q2.z); im.hi = __uint_as_float(q2.w);
        im.lo = lds32(at + 48);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(b_ifree + slot));
        ++k_item;
        return im.nch >= 0 && !__any_sync(0xffffffffu, err.gone());
    };
    Item im;

    if (warp == kTmaWarp) {
        const volatile unsigned int* failed = &g_la_error;
        const unsigned int failed0 = *failed, held = *const_cast<const volatile unsigned int*>(&g_la_withhold);
        if (failed0 != tp.launch) decode_item<kAgg>(tp, blockIdx.x, items);
        else if (lane == 0) items[0].nch = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(b_iready));
#pragma unroll 1
        for (;; ++k_item) {
            const uint32_t at = smem_u32(items) + (k_item & 1) * 64;
            const uint4 q0 = lds128(at), q1 = lds128(at + 16);
            const int t0 = uniform(q0.z), nch = uniform(q1.w), h = uniform(q1.y), v0 = uniform(q1.z);
            if (nch < 0) break;
            const int loads = held ? 0 : nch;
            const unsigned int failed1 = *failed;
            const int jn = uniform(q1.x);
            const LaJob& jb = tp.p.job[jn];
            const CUtensorMap* m = maps.m[jn];
            const int ka = (jb.DK + 63) / 64, ha = h / jb.dA, hb = h / jb.dB, hc = h / jb.dC, rev = jb.rev;
            if (elect_one()) {   // the next item, while this one runs
                mbar_arrive_expect_tx(smem_u32(b_answer), 16);
                request_item(answer, smem_u32(b_answer));
            }
            // the first chunk's loads, then the next item's decoding, then the rest
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                if (elect_one()) {
                    // C tiles are three deep and go one chunk ahead of A and B: their
                    // scaled terms take the longest to prepare
#pragma unroll 1
                    for (int x = part == 0 ? -1 : 1; x < (part == 0 ? min(loads, 1) : loads); ++x) {
                        const int cc = c + x, s = kSt == 2 ? cc & 1 : cc % kSt;
                        if (x >= 0) {
                            const int t = t0 + (rev ? nch - 1 - x : x) * kC;
                            const uint32_t st = smem_u32(smem) + s * kStage, fab = smem_u32(b_fab + s);
                            wait_on(smem_u32(b_eab + s), ((cc / kSt) & 1) ^ 1, err);
                            if (err.gone()) break;
                            mbar_arrive_expect_tx(fab, (kAgg ? 1 : 2) * ka * kAtom);
                            for (int a = 0; a < ka; ++a) {
                                if (!kAgg) tma_load_3d(st + a * kAtom, m + 0, fab, a * 64, ha, t);
                                tma_load_3d(st + kB + a * kAtom, m + 1, fab, a * 64, hb, t);
                            }
                        }
                        if (x + 1 < loads) {
                            const int t = t0 + (rev ? nch - 2 - x : x + 1) * kC, c1 = cc + 1, s3 = c1 % kCs;
                            const uint32_t fc = smem_u32(b_fc) + 8 * s3;
                            wait_on(smem_u32(b_ec) + 8 * s3, ((c1 / kCs) & 1) ^ 1, err);
                            if (err.gone()) break;
                            mbar_arrive_expect_tx(fc, kAtom);
                            tma_load_3d(smem_u32(ctile) + s3 * kAtom, m + 2, fc, v0, hc, t);
                        }
                    }
                }
                __syncwarp();
                if (part == 0) {
                    const int slot = (k_item + 1) & 1;
                    wait_on(smem_u32(b_answer), k_item & 1, err);
                    const int it = uniform(granted_item(answer));
                    fence_proxy_async_smem();
                    wait_on(smem_u32(b_ifree + slot), (((k_item + 1) >> 1) & 1) ^ 1, err);
                    if (__any_sync(0xffffffffu, err.gone())) break;
                    if (it >= 0 && failed1 != tp.launch) decode_item<kAgg>(tp, it, items + slot);
                    else if (lane == 0) items[slot].nch = -1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(b_iready + slot));
                }
            }
            if (__any_sync(0xffffffffu, err.gone())) break;
            c += nch;
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kIdW = make_idesc(1, 128, 128, 0, 0);
        constexpr uint32_t kIdO = make_idesc(1, 128, 64, 0, 1);
        constexpr uint32_t kIdU = make_idesc(1, 128, 64 * kTerms, 1, 1);
        bool ahead = false;   // the item's first W has been issued with the item before it
#pragma unroll 1
        while (read_item(im)) {
            const int nch = uniform(im.nch), ks = uniform(tp.p.job[im.job].DK / 16);
            // x = -1: the W of the item's first chunk
            const int x0 = kAgg || ahead ? 0 : -1;
            ahead = false;
            // the item's only chunk that may be of few tokens
            const int few_x = uniform(!few(im.len - (nch - 1) * kC) ? -1 : tp.p.job[im.job].rev ? 0 : nch - 1);
            if (elect_one()) {
#pragma unroll 1
                for (int x = x0; x < nch; ++x) {
                    const int cc = c + x, s = cc & 1, use = cc >> 1, sb = kSt == 2 ? s : cc % kSt;
                    const uint32_t st = smem_u32(smem) + sb * kStage;
                    const int s1 = s ^ 1, use1 = (cc + 1) >> 1;
                    const uint32_t st1 = smem_u32(smem) + s1 * kStage;
                    bool w_due = !kAgg && x + 1 < nch;
                    int ks_w = ks;
                    const auto w_product = [&]() {
                        w_due = false;
                        wait_on(smem_u32(b_fab + s1), use1 & 1, err);
                        tc_fence_after();
                        mma_steps<true, true>(tmem + kW + s1 * 128, smem_desc_sw128(st1, 16, 8 * kRow),
                                              smem_desc_sw128(st1 + kB, 16, 8 * kRow), ks_w, kIdW);
                        mma_commit(smem_u32(b_wdone + s1));
                    };
                    const auto u_half = [&](int half) {
                        const uint64_t ad = smem_desc_sw128(st + kB + half * kTerm, kAtom, 8 * kRow);
                        const uint64_t bd = smem_desc_sw128(
                            smem_u32(terms) + (kTb == 2 ? half * kTerms * kTerm : 0), kTerm, 8 * kRow);
                        const uint32_t ud = tmem + kU + (kUb == 2 ? (cc & 1) * 64 * kTerms : 0);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t o = (uint32_t)(kk * 16 * kRow) >> 4;
                            mma_f16_ss(ud, ad + o, bd + o, kIdU, half + kk > 0 ? 1u : 0u);
                        }
                    };
                    const auto x_product = [&]() {   // out = A X
                        wait_on(smem_u32(b_sready), cc & 1, err);
                        tc_fence_after();
                        mma_steps<true, false>(tmem + kO, smem_desc_sw128(st, 16, 8 * kRow),
                                               smem_desc_sw128(smem_u32(xs), 8 * kRow, 8 * kRow), ks, kIdO);
                        mma_commit(smem_u32(b_xdone));
                    };
                    if (x >= 0) {
                        if (kAgg) wait_on(smem_u32(b_fab + sb), (cc / kSt) & 1, err);
                        // U = B^T (scaled C), its three terms side by side: B is read once
                        wait_on(smem_u32(b_vready), cc & 1, err);
                        if (kUb == 2) wait_on(smem_u32(b_ufree + s), (use & 1) ^ 1, err);
                        else wait_on(smem_u32(b_ufree), (cc & 1) ^ 1, err);
                        tc_fence_after();
                        u_half(0);
                        mma_commit(smem_u32(b_udone));
                        if (!kAgg) {
                            // the last out is read: its accumulator is free
                            wait_on(smem_u32(b_ofree), (cc & 1) ^ 1, err);
                            if (x + 1 == nch && mbar_test(smem_u32(b_iready + (k_item & 1)), (k_item >> 1) & 1)) {
                                // the first W of the next item, if that is known by now
                                const uint4 q1 = lds128(smem_u32(items) + (k_item & 1) * 64 + 16);
                                if ((int)q1.w > 0) {
                                    w_due = ahead = true;
                                    ks_w = tp.p.job[q1.x].DK / 16;
                                }
                            }
                            // W of the next chunk, if its tiles are there before the other half's
                            // terms: P is then built a chunk ahead, and the tensor pipe has work
                            // while the terms are written.  (After U: 334 us instead of 317 for the
                            // training step of 16384 tokens, 16 heads of 128 x 128; waited for: 336,
                            // and the packed prompt of 32 heads, whose tiles come from HBM, in 165
                            // instead of 154.)
                            if (w_due && first_of(smem_u32(b_fab + s1), use1 & 1, smem_u32(b_vready + 1), cc & 1)) w_product();
                            // A X too: the out role gives its rows their decay meanwhile.  (Before
                            // W, looked for but not waited for, or after U: 1 to 3 % more.)
                            x_product();
                        }
                        wait_on(smem_u32(b_vready + 1), cc & 1, err);
                        tc_fence_after();
                        u_half(1);
                        mma_commit(smem_u32(b_udone + 1));
                        mma_commit(smem_u32(b_ux + (kUb == 2 ? s : 0)));
                        mma_commit(smem_u32(b_eab + sb));
                        if (kAgg) {
                            mma_commit(smem_u32(b_ec) + 8 * (cc % kCs));
                        } else {
                            // out += P C
                            wait_on(smem_u32(b_fc) + 8 * (cc % kCs), (cc / kCs) & 1, err);
                            wait_on(smem_u32(b_pready + s), use & 1, err);
                            wait_on(smem_u32(b_scaled), cc & 1, err);
                            tc_fence_after();
                            const uint64_t bd = smem_desc_sw128(smem_u32(ctile) + (cc % kCs) * kAtom, 8 * kRow, 8 * kRow);
                            const uint32_t pa = tmem + kW + s * 128, pb = pa + 32;
                            // the second half of the contraction: tokens 64 .. 127, or for a
                            // chunk of few tokens their second terms
                            const uint64_t be = bd - (x == few_x ? (uint64_t)((64 * kRow) >> 4) : 0);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_f16_ts(tmem + kO, (kk < 4 ? pa : pb) + kk * 8, (kk < 4 ? bd : be) + (uint64_t)((kk * 16 * kRow) >> 4),
                                           kIdO, 1u);
                            mma_commit(smem_u32(b_odone));
                        }
                    }
                    if (w_due) w_product();
                    if (err.gone()) break;
                }
            }
            __syncwarp();
            if (__any_sync(0xffffffffu, err.gone())) break;
            ahead = __any_sync(0xffffffffu, ahead);
            c += nch;
        }
    } else if (!kAgg && warp < 8) {
        // ===================== P =====================
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
#pragma unroll 1
        for (;;) {
            const bool item = read_item(im);
            if (any_of<1, 256>(!item)) break;   // and the table's last readers are done
            if (im.nch == 0) continue;
            const LaJob& jb = tp.p.job[im.job];
            const float a2 = im.a2;
            // s_in lam^j for j < 32 and, from there on, s_in lam^{31-j}
            if (warp < 2) sts32(ptab + 4 * row, exp2f(a2 * (float)(row < 32 ? row : 63 - row)) * jb.s_in);
            bar_p();
            const uint32_t vt = jb.rev ? ptab : ptab + 32 * 4;
#pragma unroll 1
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = c & 1, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.len - ci * kC);
                wait_on(smem_u32(b_wdone + s), (c >> 1) & 1, err);
                tc_fence_after();
                const uint32_t base = tmem + lane_off + kW + s * 128;
                if (few(n)) {
                    if (warp < 4 && quad * 32 < n) few_p(base, row, n, a2, jb.s_in, jb.rev);
                    tc_fence_before();
                    mbar_arrive(smem_u32(b_pready + s));
                    continue;
                }
                // 16 columns at a time, in place: each half's packed columns lie
                // within its own and behind its reads
                const int b0 = warp < 4 ? 0 : 4, b1 = b0 + 4;
#pragma unroll 1
                for (int b = b0; b < b1; ++b) {
                    const int rel = jb.rev ? (b >> 1) - quad : quad - (b >> 1);
                    uint32_t o[8];
                    if (rel < 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = 0u;
                    } else {
                        const int j0 = b * 16;
                        uint32_t v[16];
                        __syncwarp();
                        tmem_ld_x16(base + j0, v);
                        if (rel > 0) {
                            const uint32_t ct = vt + 4 * (j0 & 31);
                            // lam^{i-j} as a row factor times a column factor, both <= 1
                            const float u = exp2f(a2 * (float)(jb.rev ? (j0 & ~31) - row : row - (j0 & ~31) - 31));
                            const f32x2 u2 = pair(u, u);
                            tmem_wait_ld();
#pragma unroll
                            for (int e4 = 0; e4 < 4; ++e4) {
                                const uint4 t = lds128(ct + 16 * e4);
                                o[2 * e4] = pack2(mul2(pair(v[4 * e4], v[4 * e4 + 1]), mul2(pair(t.x, t.y), u2)));
                                o[2 * e4 + 1] = pack2(mul2(pair(v[4 * e4 + 2], v[4 * e4 + 3]), mul2(pair(t.z, t.w), u2)));
                            }
                        } else {
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int d = (j0 & 31) + 2 * e - lane;   // above the diagonal: masked below
                                o[e] = pack2(mul2(pair(v[2 * e], v[2 * e + 1]),
                                                  pair(lds32(ptab + 4 * ((jb.rev ? d : -d) & 31)),
                                                       lds32(ptab + 4 * ((jb.rev ? d + 1 : -d - 1) & 31)))));
                            }
                        }
                        // a select, never a product, drops what is above the diagonal
                        // or (backwards) past the chunk's tokens: columns lo .. hi stay
                        if (rel == 0 || (n < kC && jb.rev)) {
                            const int lo = (jb.rev && rel == 0 ? row : 0) - j0;
                            const int hi = (jb.rev ? n - 1 : rel == 0 ? row : kC) - j0;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                if (2 * e < lo || 2 * e > hi) o[e] &= 0xFFFF0000u;
                                if (2 * e + 1 < lo || 2 * e + 1 > hi) o[e] &= 0x0000FFFFu;
                            }
                        }
                    }
                    __syncwarp();
                    tmem_st_x8(base + b * 8 + (b0 == 4 ? 32 : 0), o);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(b_pready + s));
            }
        }
    } else if (warp >= 8 && warp < 16) {
        // ===================== scaled terms of C =====================
        // a warpgroup has half of the tokens, a thread half of a token's columns
        const int half = warp >= 12, row = half * 64 + (threadIdx.x & 63), ch0 = threadIdx.x & 64 ? 4 : 0;
#pragma unroll 1
        while (read_item(im)) {
            const LaJob& jb = tp.p.job[im.job];
            const float a2 = im.a2;
#pragma unroll 1
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int s = kSt == 2 ? c & 1 : c % kSt, ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.len - ci * kC);
                const float w = la_exp2(a2, jb.rev ? row + 1 : max(n - 1 - row, 0)) * jb.s_in;
                const f32x2 w2 = pair(w, w);
                wait_on(smem_u32(b_fc) + 8 * (c % kCs), (c / kCs) & 1, err);
                const uint32_t st = smem_u32(smem) + s * kStage, tm = smem_u32(terms) + half * (kTb == 2 ? (kTerms - 1) * kTerm : -kTerm);
                const uint32_t ct = smem_u32(ctile) + (c % kCs) * kAtom;
                // the terms of this thread's 32 columns are ready in registers when the
                // last U lets go of their tiles; a row of other tokens gives zeros
                uint32_t t[4][kTerms][4], most = 0u;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint4 q = lds128(ct + row * kRow + (((ch0 + ch) ^ (row & 7)) << 4));
                    if (row >= n) q = make_uint4(0u, 0u, 0u, 0u);   // a row of other tokens
                    const uint32_t in[4] = {q.x, q.y, q.z, q.w};
                    if (!kAgg) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)   // the largest magnitudes, a NaN above all
                            asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(in[e]));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // 24 bits as three times 8, cut off rather than rounded: the
                        // three add up to the product exactly
                        f32x2 r = mul2(pair(lo16(in[e]), hi16(in[e])), w2);
#pragma unroll
                        for (int y = 0; y < kTerms; ++y) {
                            float a, b;
                            unpair(r, a, b);
                            t[ch][y][e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                            if (y + 1 < kTerms)
                                r = add2(r, pair(-hi16(__float_as_uint(a)), -hi16(__float_as_uint(b))));
                        }
                    }
                }
                if (!kAgg && (spoils(most) || spoils(most >> 16)))
                    take_out(ct + row * kRow, row, ch0, jb.rev ? kC - 1 - row : row, spoilt(c % kCs));
                if (n < kC) {
                    wait_on(smem_u32(b_fab + s), (c / kSt) & 1, err);
                    if (row >= n) {   // nothing of such a row may reach a product
#pragma unroll 1
                        for (int ch = ch0; ch < ch0 + 4; ++ch) {
                            const int at = row * kRow + (ch << 4);
                            sts128(st + kB + at, 0u, 0u, 0u, 0u);
                            sts128(st + kB + kAtom + at, 0u, 0u, 0u, 0u);
                            sts128(ct + at, 0u, 0u, 0u, 0u);
                        }
                    }
                }
                if (kTb == 2) {
                    if (c > 0) wait_on(smem_u32(b_udone + half), (c - 1) & 1, err);
                } else if (half) {   // the halves take turns in the same tiles
                    wait_on(smem_u32(b_udone), c & 1, err);
                } else if (c > 0) {
                    wait_on(smem_u32(b_udone + 1), (c - 1) & 1, err);
                }
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int y = 0; y < kTerms; ++y)
                        sts128(tm + y * kTerm + row * kRow + (((ch0 + ch) ^ (row & 7)) << 4),
                               t[ch][y][0], t[ch][y][1], t[ch][y][2], t[ch][y][3]);
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(b_vready + half));
            }
        }
    } else if (warp >= 16 && warp < 24) {
        // ===================== X =====================
        const int k = (warp & 3) * 32 + lane;           // X's row = tensor-memory lane
        const int vc = warp < 20 ? 0 : 32;              // X's columns: 32 a thread
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
#pragma unroll 1
        while (read_item(im)) {
            if (im.seq < 0 || im.seq == g.nseq) continue;
            const LaJob& jb = tp.p.job[im.job];
            const int nv = min(kLaCols, jb.DV - im.v0) - vc;
            const int64_t elems = (int64_t)jb.DK * jb.DV;
            const int64_t at = (int64_t)k * jb.sk + (int64_t)(im.v0 + vc) * jb.sv;
            const int64_t so = ((int64_t)im.seq * g.H + im.h) * elems + at;
            float* ag = im.cut ? jb.agg + ((int64_t)im.ridx * g.H + im.h) * elems + at : nullptr;
            const float* in = kAgg ? nullptr : (im.cut ? ag : (jb.init ? jb.init + so : nullptr));
            f32x2 X[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) {   // nv is a multiple of 16
                const bool ok = in != nullptr && k < jb.DK && 2 * v < nv;
                X[v] = pair(ok ? in[(int64_t)(2 * v) * jb.sv] : 0.f, ok ? in[(int64_t)(2 * v + 1) * jb.sv] : 0.f);
            }
#pragma unroll 1
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.len - ci * kC);
                if (!kAgg) {
                    if (c > 0) wait_on(smem_u32(b_xdone), (c - 1) & 1, err);
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
                        sts128(smem_u32(xs) + k * kRow + (((vc / 8 + ch) ^ (k & 7)) << 4),
                               pack2(X[4 * ch]), pack2(X[4 * ch + 1]), pack2(X[4 * ch + 2]), pack2(X[4 * ch + 3]));
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(b_sready));
                }
                float hi = im.hi, lo = im.lo;
                if (n < kC) la_decay_pow(g.a, im.h, n, hi, lo);
                if (kUb == 2) wait_on(smem_u32(b_ux + (c & 1)), (c >> 1) & 1, err);
                else wait_on(smem_u32(b_ux), c & 1, err);
                tc_fence_after();
                const uint32_t ub = tmem + lane_off + kU + vc + (kUb == 2 ? (c & 1) * 64 * kTerms : 0);
                const f32x2 hi2 = pair(hi, hi), lo2 = pair(lo, lo);
#pragma unroll
                for (int q = 0; q < 8; ++q) {   // 4 columns of the three terms
                    uint32_t u0[4], u1[4], u2[4];
                    __syncwarp();
                    tmem_ld_x4(ub + q * 4, u0);
                    tmem_ld_x4(ub + 64 + q * 4, u1);
                    tmem_ld_x4(ub + 128 + q * 4, u2);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const f32x2 u = add2(pair(u0[2 * e], u0[2 * e + 1]),
                                             add2(pair(u1[2 * e], u1[2 * e + 1]), pair(u2[2 * e], u2[2 * e + 1])));
                        f32x2& X2 = X[q * 2 + e];
                        X2 = fma2(X2, hi2, fma2(X2, lo2, u));
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(b_ufree + (kUb == 2 ? (c & 1) : 0)));
            }
            float* outst = kAgg ? ag : (im.last && jb.fin ? jb.fin + so : nullptr);
            if (outst != nullptr && k < jb.DK) {
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    float x0, x1;
                    unpair(X[v], x0, x1);
                    if (2 * v < nv) {   // nv is a multiple of 16
                        outst[(int64_t)(2 * v) * jb.sv] = x0;
                        outst[(int64_t)(2 * v + 1) * jb.sv] = x1;
                    }
                }
            }
            __syncwarp();
        }
    } else if (!kAgg && warp >= 24) {
        // ===================== out =====================
        const int i = (warp - 24) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp - 24) * 32) << 16;
#pragma unroll 1
        for (;;) {
            const bool item = read_item(im);
            if (any_of<2, 128>(!item)) break;
            const LaJob& jb = tp.p.job[im.job];
            const int nv = min(kLaCols, jb.DV - im.v0);
            const bool f32o = kPart && jb.out_f32;
            const int64_t os = (int64_t)g.H * jb.DV, oh = (int64_t)im.h * jb.DV + im.v0;
            if (im.seq == g.nseq) {                   // tokens of no sequence: zeros
                la_zero_rows(im.len, nv / 16, i, 128, [&](int t, int v) {
                    const int64_t e = (int64_t)(im.t0 + t) * os + oh + v * 16;
                    uint4* d = f32o ? reinterpret_cast<uint4*>(static_cast<float*>(jb.out) + e)
                                          : reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(jb.out) + e);
                    for (int q = 0; q < (f32o ? 4 : 2); ++q) d[q] = make_uint4(0u, 0u, 0u, 0u);
                });
            }
            const float a2 = im.a2;
            const f32x2 f2 = pair(jb.s_out, jb.s_out);
#pragma unroll 1
            for (int x = 0; x < im.nch; ++x, ++c) {
                const int ci = jb.rev ? im.nch - 1 - x : x;
                const int n = min(kC, im.len - ci * kC);
                const int64_t e0 = (int64_t)(im.t0 + ci * kC + i) * os + oh;
                // A X in place: each row its decay, before P C is added
                const float d = exp2f(a2 * (float)(jb.rev ? max(n - 1 - i, 0) : i + 1));
                const f32x2 d2 = pair(d, d);
                wait_on(smem_u32(b_xdone), c & 1, err);
                tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < 64; b += 16) {
                    uint32_t p[16];
                    __syncwarp();
                    tmem_ld_x16(tmem + lane_off + kO + b, p);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const f32x2 r = mul2(d2, pair(p[2 * e], p[2 * e + 1]));
                        p[2 * e] = (uint32_t)r;
                        p[2 * e + 1] = (uint32_t)(r >> 32);
                    }
                    tmem_st_x16(tmem + lane_off + kO + b, p);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(b_scaled));
                wait_on(smem_u32(b_odone), c & 1, err);
                tc_fence_after();
                const Spoilt sp = spoilt(c % kCs);
                if (__float_as_int(lds32(sp.any)) != 0) spoil(tmem + lane_off + kO, jb.rev ? kC - 1 - i : i, sp);
                // A full chunk's bf16 rows go out by TMA from the chunk's C tile, which
                // nothing reads any more: stored from registers, a row to a thread, they
                // took a fifth of the shared-memory and L1 data path that bounds the
                // kernel.  The rows behind a ragged chunk's belong to others, so that
                // one is stored row by row.
                const bool tile = n == kC;
                const uint32_t ct = smem_u32(ctile) + (c % kCs) * kAtom;
                if (tile) {
                    // the next chunk's product waits for the accumulator: it is given up
                    // as soon as its second half is in registers
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t p[32];
                        __syncwarp();
                        tmem_ld_x32(tmem + lane_off + kO + hf * 32, p);
                        tmem_wait_ld();
                        if (hf == 1) {
                            tc_fence_before();
                            mbar_arrive(smem_u32(b_ofree));
                        }
                        if (f32o) {   // 32 columns fill the tile: in two turns
                            if (hf == 1) asm volatile("bar.sync 2, 128;" ::: "memory");
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const f32x2 r0 = mul2(f2, pair(p[4 * q], p[4 * q + 1]));
                                const f32x2 r1 = mul2(f2, pair(p[4 * q + 2], p[4 * q + 3]));
                                sts128(ct + i * kRow + ((q ^ (i & 7)) << 4), (uint32_t)r0, (uint32_t)(r0 >> 32),
                                       (uint32_t)r1, (uint32_t)(r1 >> 32));
                            }
                            if (hf == 0) {
                                fence_proxy_async_smem();
                                asm volatile("bar.sync 2, 128;" ::: "memory");
                                if (warp == 24 && lane == 0) {
                                    tma_store_3d(maps.m[im.job] + 3, ct, im.v0, im.h, im.t0 + ci * kC);
                                    bulk_commit_group();
                                    bulk_wait_group_read0();
                                }
                                __syncwarp();
                            }
                            continue;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) w[y] = pack2(mul2(f2, pair(p[8 * q + 2 * y], p[8 * q + 2 * y + 1])));
                            sts128(ct + i * kRow + (((4 * hf + q) ^ (i & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        uint32_t p[16];
                        f32x2 r[8];
                        __syncwarp();
                        tmem_ld_x16(tmem + lane_off + kO + b * 16, p);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = mul2(f2, pair(p[2 * e], p[2 * e + 1]));
                        if (b == 3) {
                            tc_fence_before();
                            mbar_arrive(smem_u32(b_ofree));
                        }
                        if (i >= n || b * 16 >= nv) continue;
                        if (f32o) {
                            ulonglong2* d = reinterpret_cast<ulonglong2*>(static_cast<float*>(jb.out) + e0 + b * 16);
#pragma unroll
                            for (int y = 0; y < 4; ++y) d[y] = make_ulonglong2(r[2 * y], r[2 * y + 1]);
                        } else {
                            uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(jb.out) + e0 + b * 16);
                            d[0] = make_uint4(pack2(r[0]), pack2(r[1]), pack2(r[2]), pack2(r[3]));
                            d[1] = make_uint4(pack2(r[4]), pack2(r[5]), pack2(r[6]), pack2(r[7]));
                        }
                    }
                }
                if (tile) fence_proxy_async_smem();
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (warp == 24 && lane == 0) {
                    if (tile) {
                        // columns past DV are cut off, but a tile may not start there
                        const int v1 = im.v0 + (f32o ? 32 : 0);
                        if (v1 < jb.DV) {
                            tma_store_3d(maps.m[im.job] + 3, ct, v1, im.h, im.t0 + ci * kC);
                            bulk_commit_group();
                            bulk_wait_group_read0();
                        }
                    }
                    if (__float_as_int(lds32(sp.any)) != 0) {   // the tile's next chunk starts anew
                        for (int v = 0; v < 64; ++v) sts32(sp.first + 4 * v, __int_as_float(kC));
                        sts32(sp.any, __int_as_float(0));
                    }
                    mbar_arrive(smem_u32(b_ec) + 8 * (c % kCs));
                }
                __syncwarp();
            }
        }
        if (warp == 24 && lane == 0) bulk_wait_group0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        if (lane == 0) {
            if (*const_cast<const volatile unsigned int*>(&g_la_error) == tp.launch) settle();
            report_timeout_to_host(&g_la_error, tp.host_err);
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

bool encode(CUtensorMap* m, const void* base, int D, int heads, int64_t stride, int T, bool f32 = false) {
    const uint64_t es = f32 ? 4 : 2;
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)T};
    const uint64_t str[2] = {(uint64_t)D * es, (uint64_t)stride * es};
    const uint32_t box[3] = {f32 ? 32u : 64u, 1, kC};   // rows of 128 bytes
    return encode_tmap(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                       str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_linattn_tc(const LaParams& p, int mode, cudaStream_t stream) {
    TcParams tp;
    TcMaps maps;
    tp.p = p;
    tp.nvb = 1;
    memset(&maps, 0, sizeof(maps));
    bool part = false;
    for (int j = 0; j < p.njobs; ++j) {
        const LaJob& b = p.job[j];
        const int n = (b.DV + kLaCols - 1) / kLaCols;
        tp.nvb = n > tp.nvb ? n : tp.nvb;
        part = part || b.out_f32;
        if (p.g.T > 0 && (!encode(&maps.m[j][0], b.A, b.DK, b.hA, b.sA, p.g.T) ||
                          !encode(&maps.m[j][1], b.B, b.DK, b.hB, b.sB, p.g.T) ||
                          !encode(&maps.m[j][2], b.C, b.DV, b.hC, b.sC, p.g.T) ||
                          !encode(&maps.m[j][3], b.out, b.DV, p.g.H, (int64_t)p.g.H * b.DV, p.g.T, b.out_f32 != 0)))
            return cudaErrorInvalidValue;
    }
    const int64_t items = (int64_t)p.g.range_cap * p.g.H * p.njobs * tp.nvb;
    if (items >= (1LL << 31)) return cudaErrorInvalidValue;
    static std::atomic<unsigned int> launches{0};
    do tp.launch = ++launches; while (tp.launch == 0u);
    tp.host_err = host_timeout_word();
    auto k = mode ? linattn_tc<true, false>
           : part ? linattn_tc<false, true> : linattn_tc<false, false>;
    const int smem = mode ? Cfg<true>::kSmem : Cfg<false>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)items, kThreads, smem, stream>>>(tp, maps);
    return cudaGetLastError();
}

cudaError_t set_linattn_withhold(unsigned int on) {
    return cudaMemcpyToSymbol(g_la_withhold, &on, sizeof(on));
}

unsigned int take_linattn_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_la_error, sizeof(v)) != cudaSuccess) return ~0u;
    cudaMemcpyToSymbol(g_la_error, &zero, sizeof(zero));
    return v;
}

}  // namespace ssd
