// NF4 LoRA linears for a handful of tokens (1 to LSN_DECODE_MAX_T):
//   y[t, n] = sum_b a[n, b] sum_{k in block b} level[code[n, k]] x[t, k] + s sum_j u[t, j] B[n, j],   u = x A^T,
// straight from the packed codes: every code is read once and no bf16 copy of
// W is made.  Calls of many rounds take two kernels: lsn_decode_prep_kernel
// makes u and lays x out for the tensor cores, lsn_decode_kernel streams the
// codes.  Calls of few take one, lsn_decode_small_kernel.
//
// Decoding.  A byte is a pair of codes and an entry of a 256-entry table of
// pairs of fp16 levels in shared memory: a byte permute and a 4-byte load for
// two weights (by permutes of a table in registers it takes 5.5 instructions,
// and those issue at half the rate of others).  The pair is an A register of
// mma.sync m16n8k16: with at most 16 columns the warp-level instruction, 0.475
// a clock and SM, costs a sixth of the lookups' time, and a tcgen05 tile would
// stand nearly empty.  The levels are rounded to fp16, 1.8e-4 of a weight on
// average, which is little beside the rounding of y to bf16 (y's error against 64
// bits is 1.667e-3, with exact levels 1.657e-3).  A second fp16 for what the first
// leaves out, in 8-byte entries and with twice the MMAs, took 54 us where this
// takes 40 (8B layer, one token), and 63 against 49 (8 tokens).
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.cuh"

namespace lsn {

namespace {

constexpr int kPrepThreads = 512;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kPrepCtas = 8;       // CTAs (one cluster) that share the contraction of a slice of one projection's u
constexpr int kSliceBlocks = kPrepCtas * kPrepWarps;       // a block of 64 a warp; longer rows are cut into
constexpr int kMaxSlices = 4;                              // up to so many slices, then warps take more blocks
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32;          // output rows of a warp's tile: two 16-row MMA operands
constexpr int kStageBlocks = 4;    // blocks of 64 codes in a stage: 128 bytes of each row
constexpr int kStageBytes = kRows * kStageBlocks * 32;
constexpr int kDepth = 2;          // stages of a warp in flight
constexpr int kMaxGrid = 148;

// Shared memory, in addresses of the shared window: the lookup table at 64 KB,
// so that an entry's address is its 16 low bits or-ed with a constant; the
// rings of the first 7 warps below it, the others' and the rest above.
constexpr uint32_t kTableAt = 0x10000, kTableEnd = 0x20000;
constexpr uint32_t kRingBytes = kDepth * kStageBytes;                  // of a warp
constexpr int kRingsBelow = 7;
constexpr uint32_t kBelowAt = kTableAt - kRingsBelow * kRingBytes;     // also the highest start of the block's memory
constexpr uint32_t kAmAt = kTableEnd + (kWarps - kRingsBelow) * kRingBytes;
constexpr uint32_t kBarAt = kAmAt + kWarps * kRows * kStageBlocks * 4;
constexpr uint32_t kSmem = kBarAt + kWarps * kDepth * 8 - 1024;        // the window's first KB is the system's

struct PrepProj {
    const uint16_t* x;
    const uint16_t* A;      // NULL: adapter off
    float* u;               // [slices, T, r]
    __half* xf;             // [K/64, 2, TP, 32] fp16, or NULL when another projection lays the same x out
    float* xs;              // [K/64, TP] scale of each fp16 block
    int nb;                 // K / 64
    int slices;
};
struct PrepArgs {
    PrepProj p[LSN_LAYER_MAX_PROJ];
    int* counters;          // zeroed for lsn_decode_kernel
    int n_counters;
    int T, r;
};

// The work of a projection in CTA steps: a step is one stage (4 blocks along
// K) for each of the CTA's 16 warps, G row groups of 32 rows times W = 16 / G
// stages along K.  Tiles of G row groups take `steps` steps each.
struct DecodeProj {
    const uint8_t* q;
    const float* s2;
    const float* offset;
    const __half* xf;
    const float* xs;
    const float* u;         // NULL: adapter off
    int slices;             // of u
    const uint16_t* B;
    uint16_t* y;
    int nb, N;
    int log_g;              // G = 1 << log_g
    int steps, tiles, stages;   // stages: along K
    int counter0;           // its first counter
    int q_align;            // rows of q start on multiples of 16, 4, 2 or 1 bytes
};
struct DecodeArgs {
    CUtensorMap map[LSN_LAYER_MAX_PROJ];
    int step0[LSN_LAYER_MAX_PROJ];      // first step of each projection (beyond the last: INT_MAX)
    float level[16];
    DecodeProj p[LSN_LAYER_MAX_PROJ];
    int* err;
    int* counters;          // one per row group and warp share of it
    float* part;            // [grid, 2][16 warps][8 NT][32] partial sums
    int n, T, r;
    int per, rem;           // steps of a CTA
    float scale;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Has the line at p brought into the L2.
__device__ __forceinline__ void l2_hint(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float bf16_f(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

// The four registers of 16 consecutive bf16 (32 bytes) split over two 16-byte loads.
struct X16 {
    uint4 a, b;
    __device__ uint32_t w(int i) const {
        return i < 4 ? (i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : a.w)
                     : (i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w);
    }
};
__device__ __forceinline__ X16 load16(const uint16_t* p, bool on) {
    X16 v{};
    if (on) {
        v.a = *reinterpret_cast<const uint4*>(p);
        v.b = *reinterpret_cast<const uint4*>(p + 8);
    }
    return v;
}

// One block of 64 x values of one token, 16 per lane of a quad, as fp16 times
// a power of two of the block's own, which it returns the inverse of: bf16 has
// 8 significant bits and fp16 11, and the power of two puts the largest finite
// value into [2^14, 2^15): a value down to 2^-31 of the largest is kept exactly,
// a smaller one to half of fp16's last step 2^-24, 2^-39 of the largest, below
// what an fp32 sum keeps.  Infinities and NaN stay what they are.  A block's sum
// takes its absmax before this scale: the other way round a block of the largest
// inputs would leave fp32's range.
__device__ __forceinline__ float half_x(const X16& v, uint32_t (&h)[8]) {
    uint32_t top = 0;
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v.w(i) & 0x7fff7fffu;
        const uint32_t lo = w & 0xffffu, hi = w >> 16;
        if (lo < 0x7f80u) top = max(top, lo);
        if (hi < 0x7f80u) top = max(top, hi);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(14 - e) for the largest value's exponent e, kept within what fp32 holds as a normal number
    const int e = min(max((int)(top >> 7) - 127, -112), 127);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v.w(i);
        const __half2 p = __floats2half2_rn(bf16_f(w & 0xffffu) * up, __uint_as_float(w & 0xffff0000u) * up);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}

// u = x A^T for 16 rows of A (blockIdx.y) of one projection (blockIdx.z), the
// blocks of 64 along K shared out over the cluster's CTAs and their warps,
// and x laid out for lsn_decode_kernel.  Sums in fp32: MMA accumulators, then
// the warps in order, then the cluster's CTAs in order, then (add_adapter)
// the slices.  Bound by latency: one round of loads for each warp, which is
// why rows of more than 128 blocks take more clusters (72B down, 8 tokens:
// 59.0 us with one, 57.1 with four).
template <int TP>
__global__ void __launch_bounds__(kPrepThreads) lsn_decode_prep_kernel(const __grid_constant__ PrepArgs args) {
    constexpr int NT = (TP + 7) / 8;
    __shared__ float part[kPrepWarps][16][8 * NT];
    __shared__ float sums[kPrepCtas][16 * 8 * NT];       // of CTA 0: every CTA's sums
    const int slice = blockIdx.x / kPrepCtas, slices = args.p[blockIdx.z].slices;
    const bool dots = args.p[blockIdx.z].A != nullptr && slice < slices;       // the same for the whole cluster
    if (dots) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");    // started: waited for before writing to CTA 0
    {   // a warp's first block of A, into the L2: a hint that reads nothing, so it need not wait (0.5B layer, one
        // token, after such a call: 13.3 -> 12.4 us)
        const PrepProj& p = args.p[blockIdx.z];
        const int lane = threadIdx.x & 31, b = blockIdx.x * kPrepWarps + (threadIdx.x >> 5), j = blockIdx.y * 16 + lane;
        if (dots && lane < 16 && j < args.r && b < p.nb)
            l2_hint(p.A + (int64_t)j * p.nb * 64 + (int64_t)b * 64);
    }
    pdl_wait();
    pdl_launch_dependents();
    for (int i = ((blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * kPrepThreads + threadIdx.x; i < args.n_counters;
         i += gridDim.z * gridDim.y * gridDim.x * kPrepThreads)
        args.counters[i] = 0;
    const PrepProj& p = args.p[blockIdx.z];
    const int T = args.T, r = args.r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int j0 = blockIdx.y * 16;
    const bool lays = p.xf != nullptr && blockIdx.y == 0 && slice < slices;
    const int64_t K = (int64_t)p.nb * 64;
    float acc[NT][4] = {};
    if (lays || dots) {
        #pragma unroll 2
        for (int b = blockIdx.x * kPrepWarps + warp; b < p.nb; b += slices * kSliceBlocks) {
            const int64_t k = (int64_t)b * 64 + 16 * t4;
            X16 xv[NT];
            #pragma unroll
            for (int i = 0; i < NT; ++i) xv[i] = load16(p.x + (int64_t)(g + 8 * i) * K + k, g + 8 * i < T);
            if (dots) {
                const X16 a0 = load16(p.A + (int64_t)(j0 + g) * K + k, true);
                const X16 a1 = load16(p.A + (int64_t)(j0 + 8 + g) * K + k, j0 + 8 < r);
                #pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t a[4] = {a0.w(2 * m), a1.w(2 * m), a0.w(2 * m + 1), a1.w(2 * m + 1)};
                    #pragma unroll
                    for (int i = 0; i < NT; ++i) mma_bf16(acc[i], a, xv[i].w(2 * m), xv[i].w(2 * m + 1));
                }
            }
            if (lays) {
                #pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int t = g + 8 * i;
                    // absent tokens (all zeros) take part in the shuffles and leave a scale that multiplies zeros
                    uint32_t h[8];
                    const float scale = half_x(xv[i], h);
                    if (t < T) {
                        __half* const d = p.xf + ((int64_t)b * 2 * TP + t) * 32 + 8 * t4;
                        *reinterpret_cast<uint4*>(d) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(d + TP * 32) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    if (t < TP && t4 == 0) p.xs[(int64_t)b * TP + t] = scale;
                }
            }
        }
    }
    if (!dots) return;      // the whole cluster: no CTA waits for it
    #pragma unroll
    for (int i = 0; i < NT; ++i) {
        part[warp][g][8 * i + 2 * t4] = acc[i][0];
        part[warp][g][8 * i + 2 * t4 + 1] = acc[i][1];
        part[warp][g + 8][8 * i + 2 * t4] = acc[i][2];
        part[warp][g + 8][8 * i + 2 * t4 + 1] = acc[i][3];
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // each CTA's sums go into CTA 0's shared memory; it alone waits for them
    const uint32_t rank = cluster_ctarank();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kPrepThreads) {
        float s = 0.f;
        #pragma unroll
        for (int w = 0; w < kPrepWarps; ++w) s += (&part[w][0][0])[i];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&sums[rank][i]), 0)), "f"(s) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kPrepThreads) {
        const int j = j0 + i / (8 * NT), t = i % (8 * NT);
        if (j >= r || t >= T) continue;
        float s = 0.f;
        #pragma unroll
        for (int c = 0; c < kPrepCtas; ++c) s += sums[c][i];
        p.u[((int64_t)slice * T + t) * r + j] = s;
    }
}

extern __shared__ __align__(1024) uint8_t smem_raw[];

// First step of CTA c, and the CTA that has step s: the first `rem` CTAs take
// one step more than the others' `per`.
__device__ __forceinline__ int first_step(const DecodeArgs& a, int c) { return c * a.per + min(c, a.rem); }
__device__ __forceinline__ int cta_of(const DecodeArgs& a, int s) {
    const unsigned cut = (unsigned)a.rem * (unsigned)(a.per + 1);
    return (unsigned)s < cut ? (unsigned)s / (unsigned)(a.per + 1) : a.rem + ((unsigned)s - cut) / (unsigned)a.per;
}

// A warp's walk over its stages of the CTA's steps: the projection and tile
// it is in, and within the tile one stage every W.
struct Walk {
    int left;            // steps of the CTA still to come, this tile's included
    int here;            // of those, steps of this tile
    int p, tile;
    int ks, dks;         // this step's stage, and the distance to the next step's
    int stages;          // stages of this tile's rows for this warp (0: it has no rows here)
    int rg;

    __device__ __forceinline__ void enter(const DecodeArgs& a, int warp, int step) {
        const DecodeProj& q = a.p[p];
        const int lg = q.log_g;
        rg = (tile << lg) + (warp & ((1 << lg) - 1));
        dks = kWarps >> lg;
        ks = step * dks + (warp >> lg);
        stages = rg * kRows < q.N ? q.stages : 0;
        here = min(left, q.steps - step);
    }
    __device__ void start(const DecodeArgs& a, int warp, int s0, int s1) {
        left = s1 - s0;
        p = 0;
        #pragma unroll
        for (int i = 1; i < LSN_LAYER_MAX_PROJ; ++i) p += s0 >= a.step0[i];
        const int local = s0 - a.step0[p];
        tile = local / a.p[p].steps;
        enter(a, warp, local - tile * a.p[p].steps);
    }
    __device__ __forceinline__ void next_tile(const DecodeArgs& a, int warp) {
        if (++tile == a.p[p].tiles) {
            tile = 0;
            ++p;
        }
        enter(a, warp, 0);
    }
};

// The same for the loads, with the lane's row of the second-level codes.  Rows
// that start on 16 bytes and are walked one stage after the other are read 16
// codes, four stages, at a time, a load ahead: four bytes a stage from 512 rows
// are as many requests as the codes themselves.
struct LoadWalk : Walk {
    const uint8_t* q;
    const float* s2;
    uint32_t at0;        // number of the row's first block (< 2^32: checked at launch)
    int nb, align;
    uint4 now, next;     // align 16: the codes of the four stages that ks is in, and of the next four

    __device__ __forceinline__ uint4 codes16(int first_stage) const {
        return first_stage * kStageBlocks < nb ? *reinterpret_cast<const uint4*>(q + first_stage * kStageBlocks) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void rows(const DecodeArgs& a, int lane) {
        const DecodeProj& d = a.p[p];
        nb = d.nb;
        align = d.q_align == 16 && dks > 1 ? 4 : d.q_align;
        at0 = (uint32_t)(rg * kRows + lane) * (uint32_t)nb;
        q = d.q + at0;
        s2 = d.s2;
        if (align == 16 && stages > 0) {
            now = codes16(ks & ~3);
            next = codes16((ks & ~3) + 4);
        }
    }
};

// absmax = offset + table[q] s2 with table[q] = (q - 127) / 127, [255] = 0, of
// the four blocks of a stage; blocks from `cut` on belong to the next group's s2.
struct AmRaw {
    uint32_t q;
    float s2a, s2b;
    int cut;
};
__device__ __forceinline__ AmRaw load_am(LoadWalk& w, int ks) {
    AmRaw r;
    const int b0 = ks * kStageBlocks;
    const uint32_t at = w.at0 + (uint32_t)b0;
    const uint8_t* q = w.q + b0;
    r.cut = kStageBlocks;
    r.s2a = r.s2b = w.s2[at >> 8];
    if (w.align == 16) {
        const int i = ks & 3;
        r.q = i == 0 ? w.now.x : i == 1 ? w.now.y : i == 2 ? w.now.z : w.now.w;
        if (i == 3) {
            w.now = w.next;
            w.next = w.codes16(ks + 5);
        }
        return r;
    }
    if (w.align == 4) {                         // nb % 4 == 0: four blocks, all of one group
        r.q = *reinterpret_cast<const uint32_t*>(q);
        return r;
    }
    const int n = min(kStageBlocks, w.nb - b0);
    if (w.align == 2) {                         // nb % 2 == 0: n is 2 or 4
        r.q = *reinterpret_cast<const uint16_t*>(q);
        if (n > 2) r.q |= (uint32_t)*reinterpret_cast<const uint16_t*>(q + 2) << 16;
    } else {
        r.q = q[0];
        if (n > 1) r.q |= (uint32_t)q[1] << 8;
        if (n > 2) r.q |= (uint32_t)q[2] << 16;
        if (n > 3) r.q |= (uint32_t)q[3] << 24;
    }
    r.cut = 256 - (int)(at & 255u);
    if (r.cut < n) r.s2b = w.s2[(at >> 8) + 1];
    return r;
}
__device__ __forceinline__ float4 absmax4(const AmRaw& r, float offset) {
    uint32_t q = r.q;
    if (((q & 0x7f7f7f7fu) + 0x01010101u) & q & 0x80808080u) {  // a byte is 255: it stands for 0, as 127 does
        const uint32_t ff = __vcmpeq4(q, 0xffffffffu);
        q = (q & ~ff) | (0x7f7f7f7fu & ff);
    }
    const float ka = r.s2a * (1.f / 127.f), kb = r.s2b * (1.f / 127.f);
    const float oa = offset - r.s2a, ob = offset - r.s2b;
    float4 v;
    v.x = fmaf((float)(q & 255u), ka, oa);
    v.y = fmaf((float)((q >> 8) & 255u), r.cut > 1 ? ka : kb, r.cut > 1 ? oa : ob);
    v.z = fmaf((float)((q >> 16) & 255u), r.cut > 2 ? ka : kb, r.cut > 2 ? oa : ob);
    v.w = fmaf((float)(q >> 24), r.cut > 3 ? ka : kb, r.cut > 3 ? oa : ob);
    return v;
}

// Shared memory by its 32-bit address.
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float ldsf(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void stsf(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void stsf4(uint32_t a, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// The table's entry for byte I of w, in this lane's copy: its address is
// kTableAt | byte << 8 | lane * 4, one byte permute.
template <int I>
__device__ __forceinline__ uint32_t lookup(uint32_t w, uint32_t lane4) {
    uint32_t v;
    asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(prmt(w, lane4, 0x7604u | (uint32_t)I << 4)));
    return v;
}
// The four A registers of an MMA: bytes k and k + 1 of a word of the rows 0-7 (u) and 8-15 (v).
template <int K>
__device__ __forceinline__ void operand(uint32_t (&a)[4], uint32_t u, uint32_t v, uint32_t lane4) {
    a[0] = lookup<K>(u, lane4);
    a[1] = lookup<K>(v, lane4);
    a[2] = lookup<K + 1>(u, lane4);
    a[3] = lookup<K + 1>(v, lane4);
}

// Row of MMA operand row g (0..7) within 8 where lanes read 8 bytes: the lanes of half a warp take even
// (odd) rows, whose 16-byte pieces the 128-byte swizzle puts into different banks.
__device__ __forceinline__ int row_of(int g) { return g < 4 ? 2 * g : 2 * g - 7; }

// The adapter's term of a warp's tile, s u B^T, added to its sums.  TP == 2:
// the lanes of a quad, whose sums are added up afterwards, take a quarter of
// the rank each; otherwise each lane has its own tokens.
template <int TP, int NT>
__device__ __forceinline__ void add_adapter(const DecodeArgs& a, const DecodeProj& p, int row, int t4, float (&acc)[2][NT][4]) {
    const int r = a.r, T = a.T;
    if constexpr (TP == 2) {
        for (int j = 2 * t4; j < r; j += 8) {
            uint32_t b[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const uint32_t*>(p.B + (int64_t)(row + 8 * i) * r + j);
            #pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t >= T) break;
                float2 u = *reinterpret_cast<const float2*>(p.u + t * r + j);
                for (int k = 1; k < p.slices; ++k) {
                    const float2 v = *reinterpret_cast<const float2*>(p.u + (k * T + t) * r + j);
                    u.x += v.x;
                    u.y += v.y;
                }
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = fmaf(u.x, __uint_as_float(b[i] << 16), u.y * __uint_as_float(b[i] & 0xffff0000u));
                    acc[i / 2][0][2 * (i & 1) + t] = fmaf(a.scale, d, acc[i / 2][0][2 * (i & 1) + t]);
                }
            }
        }
    } else {
        for (int j = 0; j < r; j += 4) {
            uint2 b[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const uint2*>(p.B + (int64_t)(row + 8 * i) * r + j);
            #pragma unroll
            for (int k = 0; k < 2 * NT; ++k) {
                const int t = 8 * (k / 2) + 2 * t4 + (k & 1);
                if (t >= T) continue;
                float4 u = *reinterpret_cast<const float4*>(p.u + t * r + j);
                for (int n = 1; n < p.slices; ++n) {
                    const float4 v = *reinterpret_cast<const float4*>(p.u + (n * T + t) * r + j);
                    u.x += v.x;
                    u.y += v.y;
                    u.z += v.z;
                    u.w += v.w;
                }
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float d = u.x * __uint_as_float(b[i].x << 16);
                    d = fmaf(u.y, __uint_as_float(b[i].x & 0xffff0000u), d);
                    d = fmaf(u.z, __uint_as_float(b[i].y << 16), d);
                    d = fmaf(u.w, __uint_as_float(b[i].y & 0xffff0000u), d);
                    float& s = acc[i / 2][k / 2][2 * (i & 1) + (k & 1)];
                    s = fmaf(a.scale, d, s);
                }
            }
        }
    }
}

// Persistent: every CTA takes an equal, contiguous share of the steps of all
// projections.  Each warp streams its own stages (32 rows x 128 bytes) through
// a ring of TMA copies, looks every pair of codes up in the table and
// multiplies on the tensor cores; nothing is shared between the warps until a
// tile's sums are complete.  A tile cut between CTAs is added up by the CTA
// that finishes it last, in the order of the CTAs.
//
// Bound by instruction issue and the table's loads, with about 10 us of launch,
// preparation and joins: 8B layer in a CUDA graph (floor 17.8 us), one token
// 39.8 us, 8 tokens 48.9, 16 tokens 66.6; 72B down, 8 tokens 57 to 64 us by
// machine (floor 19.6).  Stages shared by the CTA, filled and scaled by producer warps, took
// 48-55 us where this took 46 (the absmax values of 512 rows kept them behind).
//
// TP is the padded token count.  8 or 16: the MMA's columns are tokens, and
// each block of 64 is scaled by its absmax after its four MMAs.  2: a column
// is (block of the stage, token), B being zero in the columns of other blocks;
// a stage's 16 MMAs then accumulate into one set of sums, scaled together at
// its end, each lane its own block.
template <int TP>
__global__ void __launch_bounds__(kThreads, 1) lsn_decode_kernel(const __grid_constant__ DecodeArgs args) {
    // entry e of the table: the levels of byte e's two codes (high nibble
    // first) as fp16, once for each lane (256 bytes apart), so that a warp's
    // lookups never meet in a bank.  The second 128 bytes of an entry hold
    // sums on their way between warps.
    constexpr int NT = (TP + 7) / 8;
    constexpr int Q = 8 * NT;           // sums per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    uint8_t* const window = smem_raw - smem_u32(smem_raw);              // address 0 of the shared window
    const uint32_t ring = (warp < kRingsBelow ? kBelowAt + warp * kRingBytes : kTableEnd + (warp - kRingsBelow) * kRingBytes);
    const uint32_t am_sh = kAmAt + warp * kRows * kStageBlocks * 4;
    uint64_t* const full = reinterpret_cast<uint64_t*>(window + kBarAt) + warp * kDepth;
    if (smem_u32(smem_raw) < 1024 || smem_u32(smem_raw) > kBelowAt) {   // the layout does not fit this window
        if (threadIdx.x == 0) atomicExch(args.err, 2);
        return;
    }
    const int T = args.T;
    const int begin = first_step(args, blockIdx.x), end = first_step(args, blockIdx.x + 1);
    const int rowp = row_of(g);

    if (lane == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();

    // the codes and their scales are not written by the kernel before this one
    // on the stream, which itself began after everything older was complete:
    // they are read ahead of pdl_wait
    LoadWalk ld;
    ld.start(args, warp, begin, end);
    ld.rows(args, lane);
    AmRaw raw[kDepth];
    int issued = 0;
    auto load_next = [&](AmRaw& out) {
        while (ld.left > 0) {
            if (ld.here == 0) {
                ld.next_tile(args, warp);
                ld.rows(args, lane);
            }
            const int ks = ld.ks;
            --ld.left;
            --ld.here;
            ld.ks += ld.dks;
            if (ks >= ld.stages) continue;
            if (lane == 0) {
                uint64_t* bar = &full[issued % kDepth];
                mbar_arrive_expect_tx(bar, kStageBytes);
                tma_load_2d(window + ring + (issued % kDepth) * kStageBytes, &args.map[ld.p], ks * 64, ld.rg * kRows, bar);
            }
            out = load_am(ld, ks);
            ++issued;
            return;
        }
    };
    #pragma unroll
    for (int i = 0; i < kDepth; ++i) load_next(raw[i]);

    {   // warp w makes entries 16 w .. 16 w + 15: the high code's level is its own
        const float lv = args.level[lane & 15], hi = __shfl_sync(0xffffffffu, lv, warp);
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __half2 h = __floats2half2_rn(hi, __shfl_sync(0xffffffffu, lv, i));
            *reinterpret_cast<__half2*>(window + kTableAt + (warp * 16 + i) * 256 + lane * 4) = h;
        }
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t lane4 = kTableAt | lane * 4;
    // this lane's first piece of a row in a stage, in the 128-byte swizzle.
    // the 8 bytes that are t4's of block 0 (block j: xor 32 j)
    const uint32_t piece = rowp * 128 + ((t4 >> 1) ^ rowp) * 16 + (t4 & 1) * 8;

    int used = 0;
    bool dead = false;
    Walk cur;
    cur.start(args, warp, begin, end);
    while (cur.left > 0) {
        const DecodeProj& p = args.p[cur.p];
        const int tile = cur.tile, tile_first = args.step0[cur.p] + tile * p.steps;
        const int nb = p.nb, G = 1 << p.log_g, W = kWarps >> p.log_g;
        const int grp = warp & (G - 1), share = warp >> p.log_g;
        const int rg = cur.rg;
        const bool mine = rg * kRows < p.N;
        const float offset = *p.offset;
        float acc[2][NT][4] = {};
        if (p.u != nullptr && mine)             // read at the tile's end
            l2_hint(p.B + (int64_t)(rg * kRows + lane) * args.r);
        const char* const xf = reinterpret_cast<const char*>(p.xf) + (TP == 2 ? (g >> 1) * (TP * 128) + (g & 1) * 64 : g * 64) + t4 * 16;
        const char* const xsp = reinterpret_cast<const char*>(p.xs) + t4 * 8;
        for (int n = cur.here; n > 0; --n) {
            const int ks = cur.ks;
            cur.ks += cur.dks;
            if (ks >= cur.stages) continue;
            const int slot = used % kDepth;
            const int b0 = ks * kStageBlocks;
            const char* xb = xf + (size_t)b0 * (TP * 128);
            const char* xsb = xsp + (size_t)b0 * (TP * 4);
            uint4 xa2 = make_uint4(0, 0, 0, 0), xc2 = xa2;
            float2 xs2 = make_float2(0.f, 0.f);
            if constexpr (TP == 2) {            // ahead of the wait
                if ((g & 1) < T && b0 + (g >> 1) < nb) {
                    xa2 = *reinterpret_cast<const uint4*>(xb);
                    xc2 = *reinterpret_cast<const uint4*>(xb + TP * 64);
                }
                if (b0 + t4 < nb) xs2 = *reinterpret_cast<const float2*>(xsb);
            }
            if (!dead && !__all_sync(0xffffffffu, mbar_try_wait(&full[slot], (used / kDepth) & 1))) {
                if (__any_sync(0xffffffffu, !mbar_wait(&full[slot], (used / kDepth) & 1, nullptr))) {
                    dead = true;                // keep walking, so that the CTA's barriers stay whole
                    if (lane == 0) atomicExch(args.err, 1);
                }
            }
            if (dead) continue;
            ++used;
            stsf4(am_sh + lane * 16, absmax4(raw[0], offset));
            const uint32_t st = ring + slot * kStageBytes;
            if constexpr (TP == 2) {
                // the stage's codes, all into registers: the slot is free again before the arithmetic begins
                uint2 cw[kStageBlocks][4];
                #pragma unroll
                for (int j = 0; j < kStageBlocks; ++j)
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) cw[j][i] = lds64(st + (piece ^ (32 * j)) + i * 1024);
                __syncwarp();
                #pragma unroll
                for (int i = 0; i + 1 < kDepth; ++i) raw[i] = raw[i + 1];
                load_next(raw[kDepth - 1]);
                float c[2][4] = {}, e[2][4] = {};       // two chains of MMAs each
                #pragma unroll
                for (int j = 0; j < kStageBlocks; ++j) {
                    const uint32_t on = (g >> 1) == j ? 0xffffffffu : 0u;
                    const uint32_t bx[8] = {xa2.x & on, xa2.y & on, xa2.z & on, xa2.w & on, xc2.x & on, xc2.y & on, xc2.z & on, xc2.w & on};
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 u = cw[j][2 * h], v = cw[j][2 * h + 1];
                        uint32_t a[4];
                        operand<0>(a, u.x, v.x, lane4);
                        mma_f16(c[h], a, bx[0], bx[1]);
                        operand<2>(a, u.x, v.x, lane4);
                        mma_f16(e[h], a, bx[2], bx[3]);
                        operand<0>(a, u.y, v.y, lane4);
                        mma_f16(e[h], a, bx[4], bx[5]);
                        operand<2>(a, u.y, v.y, lane4);
                        mma_f16(c[h], a, bx[6], bx[7]);
                    }
                }
                #pragma unroll
                for (int h = 0; h < 2; ++h)
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) c[h][i] += e[h][i];
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float lo = ldsf(am_sh + (16 * h + rowp) * 16 + t4 * 4), hi = ldsf(am_sh + (16 * h + 8 + rowp) * 16 + t4 * 4);
                    acc[h][0][0] = fmaf(c[h][0] * lo, xs2.x, acc[h][0][0]);
                    acc[h][0][1] = fmaf(c[h][1] * lo, xs2.y, acc[h][0][1]);
                    acc[h][0][2] = fmaf(c[h][2] * hi, xs2.x, acc[h][0][2]);
                    acc[h][0][3] = fmaf(c[h][3] * hi, xs2.y, acc[h][0][3]);
                }
            } else {
                // a rolled loop: unrolled, or with the next block's x read ahead, registers spill and moves
                // add up (8B layer, 8 tokens: 54 and 51 us against 50)
                __syncwarp();                   // am_sh is written
                const int nj = min(kStageBlocks, nb - b0);
                #pragma unroll 1
                for (int j = 0; j < nj; ++j) {
                    uint4 xa[NT], xc[NT];
                    float2 xs[NT];
                    #pragma unroll
                    for (int i = 0; i < NT; ++i) {  // lane (g, t4): a quarter of token g
                        xa[i] = xc[i] = make_uint4(0, 0, 0, 0);
                        if (g + 8 * i < T) {
                            xa[i] = *reinterpret_cast<const uint4*>(xb + i * 512);
                            xc[i] = *reinterpret_cast<const uint4*>(xb + i * 512 + TP * 64);
                        }
                        xs[i] = *reinterpret_cast<const float2*>(xsb + i * 32);
                    }
                    xb += TP * 128;
                    xsb += TP * 4;
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 u = lds64(st + (piece ^ (32 * j)) + h * 2048), v = lds64(st + (piece ^ (32 * j)) + h * 2048 + 1024);
                        const float lo = ldsf(am_sh + (16 * h + rowp) * 16 + j * 4), hi = ldsf(am_sh + (16 * h + 8 + rowp) * 16 + j * 4);
                        float c[NT][4] = {};
                        uint32_t a[4];
                        operand<0>(a, u.x, v.x, lane4);
                        #pragma unroll
                        for (int i = 0; i < NT; ++i) mma_f16(c[i], a, xa[i].x, xa[i].y);
                        operand<2>(a, u.x, v.x, lane4);
                        #pragma unroll
                        for (int i = 0; i < NT; ++i) mma_f16(c[i], a, xa[i].z, xa[i].w);
                        operand<0>(a, u.y, v.y, lane4);
                        #pragma unroll
                        for (int i = 0; i < NT; ++i) mma_f16(c[i], a, xc[i].x, xc[i].y);
                        operand<2>(a, u.y, v.y, lane4);
                        #pragma unroll
                        for (int i = 0; i < NT; ++i) mma_f16(c[i], a, xc[i].z, xc[i].w);
                        #pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            acc[h][i][0] = fmaf(c[i][0] * lo, xs[i].x, acc[h][i][0]);
                            acc[h][i][1] = fmaf(c[i][1] * lo, xs[i].y, acc[h][i][1]);
                            acc[h][i][2] = fmaf(c[i][2] * hi, xs[i].x, acc[h][i][2]);
                            acc[h][i][3] = fmaf(c[i][3] * hi, xs[i].y, acc[h][i][3]);
                        }
                    }
                }
                __syncwarp();                   // every lane has read the slot
                #pragma unroll
                for (int i = 0; i + 1 < kDepth; ++i) raw[i] = raw[i + 1];
                load_next(raw[kDepth - 1]);
            }
            __syncwarp();                       // every lane has read am_sh
        }
        const int seg_begin = end - cur.left;
        if (p.u != nullptr && mine && seg_begin == tile_first && share == 0) add_adapter<TP, NT>(args, p, rg * kRows + rowp, t4, acc);
        if constexpr (TP == 2) {                // the columns of a token: the stage's blocks, one per lane of a quad
            #pragma unroll
            for (int q = 0; q < Q; ++q) {
                float& v = acc[q / 4][0][q % 4];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
            }
        }

        // the segment's sums: value q of lane (g, t4) is row
        // 16 (q / 4 NT) + 8 (q / 2 % 2) + rowp, token 8 (q / 4 % NT) + 2 t4 + q % 2
        float v[Q];
        #pragma unroll
        for (int q = 0; q < Q; ++q) v[q] = acc[q / (4 * NT)][(q / 4) % NT][q % 4];
        if (W > 1) {                            // the W warps of a row group: each ends up with every W-th value
            #pragma unroll
            for (int q = 0; q < Q; ++q) stsf((warp * Q + q) * 256 + 128 + lane4, v[q]);
            __syncthreads();
            #pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (q % W != share) continue;
                float s = 0.f;
                for (int w = 0; w < W; ++w) s += ldsf(((grp + w * G) * Q + q) * 256 + 128 + lane4);
                v[q] = s;
            }
            __syncthreads();
        }
        const int first = cta_of(args, tile_first), last = cta_of(args, tile_first + p.steps - 1);
        bool write = mine;
        if (first != last && mine && share < Q) {
            float* const part = args.part;
            const int slot = 2 * blockIdx.x + (seg_begin == begin ? 0 : 1);
            #pragma unroll
            for (int q = 0; q < Q; ++q)
                if (q % W == share) __stcg(&part[((int64_t)(slot * kWarps + grp) * Q + q) * 32 + lane], v[q]);
            __syncwarp();
            int done = 0;
            int* const counter = args.counters + p.counter0 + rg * W + share;
            if (lane == 0) asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(done) : "l"(counter) : "memory");
            done = __shfl_sync(0xffffffffu, done, 0);
            __syncwarp();
            write = done == last - first;
            if (write) {
                #pragma unroll
                for (int q = 0; q < Q; ++q) v[q] = 0.f;
                #pragma unroll 4
                for (int c = first; c <= last; ++c) {
                    const int at = 2 * c + (c > first || first_step(args, c) == tile_first ? 0 : 1);
                    #pragma unroll
                    for (int q = 0; q < Q; ++q)
                        if (q % W == share) v[q] += __ldcg(&part[((int64_t)(at * kWarps + grp) * Q + q) * 32 + lane]);
                }
            }
        }
        if (write && !dead) {
            #pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (q % W != share) continue;
                const int row = rg * kRows + 16 * (q / (4 * NT)) + 8 * ((q / 2) & 1) + rowp, t = 8 * ((q / 4) % NT) + 2 * t4 + (q & 1);
                if (t < T && (TP > 2 || t4 == 0)) p.y[(int64_t)t * p.N + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v[q]));
            }
        }
        cur.left -= cur.here;
        if (cur.left > 0) cur.next_tile(args, warp);
    }
    if (dead)                                   // copies still on their way must land before the CTA ends
        for (; used < issued; ++used) mbar_wait(&full[used % kDepth], (used / kDepth) & 1, nullptr);
}

// ------------------------------------------------- small calls, one launch --

// Taken while its rounds (CTAs over SMs, times 1024 codes of a row at a time)
// are few.  Measured in a graph, this launch against the two: 512 x 512, one
// token, 2.7 and 8.0 us; 4096 x 1024, 16 tokens, 7.2 and 14.9; 4096 x 4096, one
// token, 9.0 and 10.9 (rank 64: 14.0 and 12.3); 8192 x 2048, 8 tokens, 12.2
// and 12.0; the seven 0.5B projections, one token, 18.6 and 12.4.
constexpr int64_t kSmallRounds = 4;

// absmax = offset + table[q] s2 with table[q] = (q - 127) / 127, [255] = 0
__device__ __forceinline__ float absmax_of(uint32_t q, float s2, float offset) {
    return fmaf(((float)(q == 255u ? 127u : q) - 127.f) * (1.f / 127.f), s2, offset);
}

// One 32-row tile over the whole of K per CTA: each warp takes every 16th block
// of 64, laying x out in its registers and, ahead of the codes' arithmetic,
// multiplying its blocks of x with A for u.  A is read once per tile, four
// times the codes' bytes at rank 16, from the L2: that pays while a call is
// bound by its launches and latencies.
struct SmallProj {
    const uint8_t* packed;
    const uint8_t* q;
    const float* s2;
    const float* offset;
    const uint16_t* x;
    const uint16_t* A;      // NULL: adapter off
    const uint16_t* B;
    uint16_t* y;
    int nb, N;
};
struct SmallArgs {
    int tile0[LSN_LAYER_MAX_PROJ];      // first tile of each projection (beyond the last: INT_MAX)
    float level[16];
    int T, r;
    float scale;
    SmallProj p[LSN_LAYER_MAX_PROJ];
};
constexpr int kSmallThreads = 512;
constexpr int kAhead = 2;               // blocks of a warp whose codes are in flight

template <int NT>
constexpr int small_smem(int groups) {  // table, partial sums of y and, for each 16 ranks, of u
    return 65536 + kWarps * kRows * 8 * NT * 4 + groups * kWarps * 16 * 8 * NT * 4;
}

template <int NT>
__global__ void __launch_bounds__(kSmallThreads, 1) lsn_decode_small_kernel(const __grid_constant__ SmallArgs args) {
    float* const part = reinterpret_cast<float*>(smem_raw + 65536);                 // [warp][row][token]
    float* const upart = part + kWarps * kRows * 8 * NT;                            // [rank group][warp][rank][token]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int T = args.T, r = args.r;
    int pi = 0;
    #pragma unroll
    for (int i = 1; i < LSN_LAYER_MAX_PROJ; ++i) pi += (int)blockIdx.x >= args.tile0[i];
    const SmallProj& p = args.p[pi];
    const int n0 = ((int)blockIdx.x - args.tile0[pi]) * kRows;
    const int nb = p.nb;
    const int64_t K = (int64_t)nb * 64;
    {
        const float lv = args.level[lane & 15], hi = __shfl_sync(0xffffffffu, lv, warp);
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __half2 h = __floats2half2_rn(hi, __shfl_sync(0xffffffffu, lv, i));
            *reinterpret_cast<__half2*>(smem_raw + (warp * 16 + i) * 256 + lane * 4) = h;
        }
    }
    // the tile's codes, into the L2: hints that read nothing, so they need not wait (9.7 -> 9.0 us)
    for (int64_t i = (int64_t)threadIdx.x * 128; i < (int64_t)kRows * nb * 32; i += kSmallThreads * 128)
        l2_hint(p.packed + (int64_t)n0 * nb * 32 + i);
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    struct Codes {
        uint2 w[4];
        uint32_t q[4];
        float s2[4];
    };
    auto load = [&](Codes& c, int b) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t blk = (int64_t)(n0 + 8 * i + g) * nb + b;
            c.w[i] = __ldcs(reinterpret_cast<const uint2*>(p.packed + blk * 32 + t4 * 8));
            c.q[i] = p.q[blk];
            c.s2[i] = p.s2[blk >> 8];
        }
    };
    Codes ahead[kAhead];
    #pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (warp + k * kWarps < nb) load(ahead[k], warp + k * kWarps);
    const float offset = *p.offset;

    if (p.A != nullptr) {
        for (int j0 = 0; j0 < r; j0 += 16) {
            float acc[NT][4] = {};
            #pragma unroll 2
            for (int b = warp; b < nb; b += kWarps) {
                const int64_t k = (int64_t)b * 64 + 16 * t4;
                const X16 a0 = load16(p.A + (int64_t)(j0 + g) * K + k, true);
                const X16 a1 = load16(p.A + (int64_t)(j0 + 8 + g) * K + k, j0 + 8 < r);
                X16 xv[NT];
                #pragma unroll
                for (int i = 0; i < NT; ++i) xv[i] = load16(p.x + (int64_t)(g + 8 * i) * K + k, g + 8 * i < T);
                #pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t a[4] = {a0.w(2 * m), a1.w(2 * m), a0.w(2 * m + 1), a1.w(2 * m + 1)};
                    #pragma unroll
                    for (int i = 0; i < NT; ++i) mma_bf16(acc[i], a, xv[i].w(2 * m), xv[i].w(2 * m + 1));
                }
            }
            float* const d = upart + ((j0 / 16 * kWarps + warp) * 16 + g) * 8 * NT + 2 * t4;
            #pragma unroll
            for (int i = 0; i < NT; ++i) {
                *reinterpret_cast<float2*>(d + 8 * i) = make_float2(acc[i][0], acc[i][1]);
                *reinterpret_cast<float2*>(d + 8 * 8 * NT + 8 * i) = make_float2(acc[i][2], acc[i][3]);
            }
        }
    }

    const uint32_t lane4 = lane * 4, table = smem_u32(smem_raw);
    float acc[2][NT][4] = {};
    for (int b0 = warp; b0 < nb; b0 += kAhead * kWarps) {
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int b = b0 + k * kWarps;
            if (b >= nb) break;
            uint32_t xh[NT][8];
            float2 xs[NT];
            #pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float s = half_x(load16(p.x + (int64_t)(g + 8 * i) * K + (int64_t)b * 64 + 16 * t4, g + 8 * i < T), xh[i]);
                // lane (g, t4) holds token g's scale and needs those of tokens 2 t4 and 2 t4 + 1
                xs[i].x = __shfl_sync(0xffffffffu, s, 8 * t4);
                xs[i].y = __shfl_sync(0xffffffffu, s, 8 * t4 + 4);
            }
            const Codes c = ahead[k];
            if (b + kAhead * kWarps < nb) load(ahead[k], b + kAhead * kWarps);
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                float d[NT][4] = {};
                #pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t u = m < 2 ? c.w[2 * h].x : c.w[2 * h].y, v = m < 2 ? c.w[2 * h + 1].x : c.w[2 * h + 1].y;
                    uint32_t a[4];
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t at = table + prmt((e & 1) ? v : u, lane4, 0x7604u | (uint32_t)(((2 * m) & 3) + (e >> 1)) << 4);
                        asm("ld.shared.b32 %0, [%1];" : "=r"(a[e]) : "r"(at));
                    }
                    #pragma unroll
                    for (int i = 0; i < NT; ++i) mma_f16(d[i], a, xh[i][2 * m], xh[i][2 * m + 1]);
                }
                const float lo = absmax_of(c.q[2 * h], c.s2[2 * h], offset), hi = absmax_of(c.q[2 * h + 1], c.s2[2 * h + 1], offset);
                #pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[h][i][0] = fmaf(d[i][0] * lo, xs[i].x, acc[h][i][0]);
                    acc[h][i][1] = fmaf(d[i][1] * lo, xs[i].y, acc[h][i][1]);
                    acc[h][i][2] = fmaf(d[i][2] * hi, xs[i].x, acc[h][i][2]);
                    acc[h][i][3] = fmaf(d[i][3] * hi, xs[i].y, acc[h][i][3]);
                }
            }
        }
    }
    #pragma unroll
    for (int h = 0; h < 2; ++h)
        #pragma unroll
        for (int i = 0; i < NT; ++i) {
            float* const d = part + (warp * kRows + 16 * h + g) * 8 * NT + 8 * i + 2 * t4;
            *reinterpret_cast<float2*>(d) = make_float2(acc[h][i][0], acc[h][i][1]);
            *reinterpret_cast<float2*>(d + 8 * 8 * NT) = make_float2(acc[h][i][2], acc[h][i][3]);
        }
    __syncthreads();
    if (p.A != nullptr) {                       // u: the warps' sums in order, left in the first warp's place
        for (int o = threadIdx.x; o < r * 8 * NT; o += kSmallThreads) {
            float* const d = upart + (o / (128 * NT) * kWarps * 128 * NT) + o % (128 * NT);
            float s = 0.f;
            #pragma unroll
            for (int w = 0; w < kWarps; ++w) s += d[w * 128 * NT];
            d[0] = s;
        }
        __syncthreads();
    }
    for (int o = threadIdx.x; o < kRows * T; o += kSmallThreads) {
        const int t = o / kRows, row = o % kRows;
        float s = 0.f;
        #pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[(w * kRows + row) * 8 * NT + t];
        if (p.A != nullptr) {
            const uint4* B = reinterpret_cast<const uint4*>(p.B + (int64_t)(n0 + row) * r);
            float d = 0.f;
            for (int j = 0; j < r; j += 8) {
                const uint4 v = B[j / 8];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                const float* u = upart + (j / 16 * kWarps * 16 + j % 16) * 8 * NT + t;
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d = fmaf(u[2 * e * 8 * NT], bf16_f(w[e] & 0xffffu), d);
                    d = fmaf(u[(2 * e + 1) * 8 * NT], __uint_as_float(w[e] & 0xffff0000u), d);
                }
            }
            s = fmaf(args.scale, d, s);
        }
        p.y[(int64_t)t * p.N + n0 + row] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
}

// The largest shared memory size a kernel may take, set once per device.
template <class F>
lsn_status allow_smem(std::atomic<uint64_t>& ready, F kernel, int bytes) {
    int dev = 0;
    LSN_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        LSN_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        if (dev < 64) ready.fetch_or(1ull << dev);
    }
    return LSN_OK;
}

template <int NT>
lsn_status launch_small(const SmallArgs& a, int tiles, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    lsn_status s = allow_smem(ready, lsn_decode_small_kernel<NT>, small_smem<NT>(4));
    if (s != LSN_OK) return s;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = small_smem<NT>((a.r + 15) / 16);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = pdl_attr(at);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, lsn_decode_small_kernel<NT>, a));
    return LSN_OK;
}

template <int TP>
lsn_status launch_tp(const PrepArgs& pa, const DecodeArgs& da, int grid, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    lsn_status s = allow_smem(ready, lsn_decode_kernel<TP>, kSmem);
    if (s != LSN_OK) return s;
    int slices = 1;
    for (int i = 0; i < da.n; ++i) slices = std::max(slices, pa.p[i].slices);
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kPrepCtas * slices), (unsigned)((pa.r + 15) / 16), (unsigned)da.n);
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kPrepCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1 + pdl_attr(&at[1]);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, lsn_decode_prep_kernel<TP>, pa));
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = pdl_attr(&at[0]);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, lsn_decode_kernel<TP>, da));
    return LSN_OK;
}

// How a projection is cut into steps (T tokens): the warps of a CTA share out
// G row groups and W = 16 / G stages along K.
struct Cut {
    int log_g, steps, tiles;
};
Cut cut_of(int64_t N, int64_t K, int64_t per_cta) {
    const int64_t stages = ceil_div(K / 64, kStageBlocks), groups = N / kRows;
    int lg = per_cta < 2 ? 0 : 4;
    while (lg < 4 && (kWarps >> lg) > stages) ++lg;
    Cut c;
    c.log_g = lg;
    c.steps = (int)ceil_div(stages, kWarps >> lg);
    c.tiles = (int)ceil_div(groups, 1 << lg);
    return c;
}

// Workspace: the status word (256 bytes), then the counters, the partial sums
// and per projection u, the fp16 x and its block scales.
struct DecodeWs {
    int* err;
    int* counters;
    float* part;
    float* u[LSN_LAYER_MAX_PROJ];
    __half* xf[LSN_LAYER_MAX_PROJ];
    float* xs[LSN_LAYER_MAX_PROJ];
    size_t total;
};
int pad_tokens(int64_t T) { return T <= 2 ? 2 : T <= 8 ? 8 : 16; }
DecodeWs carve_decode(void* ws, int n, const lsn_lora_proj* p, int64_t T, int r) {
    DecodeWs w{};
    size_t off = 0;
    char* b = reinterpret_cast<char*>(ws);
    auto take = [&](size_t bytes) { char* q = b ? b + off : nullptr; off += round_up(bytes, 256); return q; };
    w.err = reinterpret_cast<int*>(take(256));
    size_t counters = 0;
    for (int i = 0; i < n; ++i) counters += (size_t)(p[i].W.rows / kRows + kWarps) * kWarps;
    w.counters = reinterpret_cast<int*>(take(counters * 4));
    w.part = reinterpret_cast<float*>(take((size_t)kMaxGrid * 2 * kWarps * kRows * LSN_DECODE_MAX_T * 4));
    for (int i = 0; i < n; ++i) {
        const size_t K = (size_t)p[i].W.cols;
        w.u[i] = reinterpret_cast<float*>(take((size_t)kMaxSlices * T * r * 4));
        w.xf[i] = reinterpret_cast<__half*>(take((size_t)pad_tokens(T) * K * 2));
        w.xs[i] = reinterpret_cast<float*>(take(K / 64 * LSN_DECODE_MAX_T * 4));
    }
    w.total = off;
    return w;
}

}  // namespace

int decode_kernels(int n, const lsn_lora_proj* p, int64_t T, int r) {
    int64_t tiles = 0, k = 0;
    bool on = false;
    for (int i = 0; i < n; ++i) {
        tiles += p[i].W.rows / kRows;
        k = std::max(k, p[i].W.cols);
        on = on || p[i].A != nullptr;
    }
    // larger ranks read more of A, more than 8 tokens do twice the arithmetic
    const int64_t rounds = ceil_div(tiles, kMaxGrid) * ceil_div(k, 64 * kWarps) * (on && r > 16 ? 2 : 1) * (T > 8 ? 2 : 1);
    return rounds <= kSmallRounds ? 1 : 2;
}

size_t decode_ws_bytes(int n, const lsn_lora_proj* p, int64_t T, int r) { return carve_decode(nullptr, n, p, T, r).total; }

lsn_status launch_decode(int n, const lsn_lora_proj* p, int T, int r, float scale, void* ws, cudaStream_t st) {
    if (decode_kernels(n, p, T, r) == 1) {
        SmallArgs a;
        a.T = T;
        a.r = r;
        a.scale = scale;
        std::copy(nf4_tables().level, nf4_tables().level + 16, a.level);
        std::fill(a.tile0, a.tile0 + LSN_LAYER_MAX_PROJ, INT32_MAX);
        int tile = 0;
        for (int i = 0; i < n; ++i) {
            const lsn_nf4_weight& f = p[i].W.nf4;
            a.p[i] = SmallProj{f.packed, f.absmax_q, f.absmax_s2, f.offset, p[i].x, p[i].A, p[i].B, p[i].y, (int)(p[i].W.cols / 64), (int)p[i].W.rows};
            a.tile0[i] = tile;
            tile += (int)(p[i].W.rows / kRows);
        }
        return T <= 8 ? launch_small<1>(a, tile, st) : launch_small<2>(a, tile, st);
    }
    const DecodeWs w = carve_decode(ws, n, p, T, r);
    PrepArgs pa{};
    DecodeArgs da;
    pa.T = da.T = T;
    pa.r = da.r = r;
    da.n = n;
    da.scale = scale;
    da.err = w.err;
    da.part = w.part;
    pa.counters = da.counters = w.counters;
    std::copy(nf4_tables().level, nf4_tables().level + 16, da.level);
    int64_t total = 0, counters = 0, work = 0;
    std::fill(da.step0, da.step0 + LSN_LAYER_MAX_PROJ, INT32_MAX);
    for (int i = 0; i < n; ++i) work += p[i].W.rows / kRows * ceil_div(p[i].W.cols / 64, kStageBlocks);
    const int64_t per_cta = work / (kWarps * kMaxGrid);
    for (int i = 0; i < n; ++i) {
        const lsn_lora_proj& q = p[i];
        int lead = 0;                       // the first projection that reads the same x
        while (p[lead].x != q.x || p[lead].W.cols != q.W.cols) ++lead;
        const bool off = q.A == nullptr;
        const int nb = (int)(q.W.cols / 64);
        const int slices = (int)std::min<int64_t>(ceil_div(nb, kSliceBlocks), kMaxSlices);
        pa.p[i] = PrepProj{q.x, q.A, w.u[i], lead == i ? w.xf[i] : nullptr, w.xs[i], nb, slices};
        const lsn_nf4_weight& f = q.W.nf4;
        const Cut c = cut_of(q.W.rows, q.W.cols, per_cta);
        const uintptr_t qa = reinterpret_cast<uintptr_t>(f.absmax_q) | (uintptr_t)nb;
        da.p[i] = DecodeProj{f.absmax_q, f.absmax_s2, f.offset, w.xf[lead], w.xs[lead], off ? nullptr : w.u[i], slices, q.B, q.y, nb, (int)q.W.rows,
                             c.log_g, c.steps, c.tiles, (int)ceil_div(nb, kStageBlocks), (int)counters, qa % 16 == 0 ? 16 : qa % 4 == 0 ? 4 : qa % 2 == 0 ? 2 : 1};
        da.step0[i] = (int)total;
        // the packed codes as 16-bit elements: rows of K / 4, boxes of 64 x 32
        lsn_status s = make_tmap_2d(&da.map[i], f.packed, q.W.cols / 4, q.W.rows, q.W.cols / 4, 64, kRows, false);
        if (s != LSN_OK) return s;
        total += (int64_t)c.steps * c.tiles;
        counters += (int64_t)c.tiles * kWarps;
        if (total > INT32_MAX / 2 || counters > INT32_MAX || q.W.rows * nb > (int64_t)UINT32_MAX) return fail(LSN_ERR_UNSUPPORTED, "lora_layer_decode: weights too large");
    }
    const int grid = (int)std::min<int64_t>({total, sm_count(), kMaxGrid});
    da.per = (int)(total / grid);
    da.rem = (int)(total % grid);
    pa.n_counters = (int)counters;
    return T <= 2 ? launch_tp<2>(pa, da, grid, st) : T <= 8 ? launch_tp<8>(pa, da, grid, st) : launch_tp<16>(pa, da, grid, st);
}

}  // namespace lsn
