// NF4 LoRA linears for a handful of tokens (1 to LSN_DECODE_MAX_T):
//   y[t, n] = sum_b a[n, b] sum_{k in block b} level[code[n, k]] x[t, k] + s sum_j u[t, j] B[n, j],   u = x A^T,
// straight from the packed codes: every code is read once and no bf16 copy of
// W is made.  Two kernels: lsn_decode_prep_kernel makes u and lays x out for
// the tensor cores, lsn_decode_kernel streams the codes.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace lsn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kPrepCtas = 8;       // CTAs (one cluster) that share the contraction of one projection's u
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32;          // output rows of a tile: two 16-row MMA operands per warp
constexpr int kTableBytes = 65536;

struct PrepProj {
    const uint16_t* x;
    const uint16_t* A;      // NULL: adapter off
    float* u;               // [T, r]
    __half* xf;             // [K/64, T, 64] fp16, or NULL when another projection lays the same x out
    float* xs;              // [K/64, 8 NT] scale of each fp16 block
    int nb;                 // K / 64
};
struct PrepArgs {
    PrepProj p[LSN_LAYER_MAX_PROJ];
    int T, r;
};

struct DecodeProj {
    const uint8_t* packed;
    const uint8_t* q;
    const float* s2;
    const float* offset;
    const __half* xf;
    const float* xs;
    const float* u;         // NULL: adapter off
    const uint16_t* B;
    uint16_t* y;
    int nb, N;
    int tile0;              // number of this projection's first tile
};
struct DecodeArgs {
    DecodeProj p[LSN_LAYER_MAX_PROJ];
    float level[16];
    int n, T, r, tiles;
    float scale;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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
// a power of two of the block's own: bf16 has 8 significant bits and fp16 11,
// so a value down to 2^-28 of the block's largest is kept exactly or to
// 2^-24 of 2^-14 of the largest, below what an fp32 sum keeps; the power of
// two puts the largest finite value into [2^14, 2^15).  Infinities and NaN
// stay what they are.
__device__ __forceinline__ void lay_out_x(const X16& v, bool on, __half* dst, float* xs, int t4) {
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
    uint32_t h[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v.w(i);
        const __half2 p = __floats2half2_rn(bf16_f(w & 0xffffu) * up, __uint_as_float(w & 0xffff0000u) * up);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    if (on) {
        uint4* d = reinterpret_cast<uint4*>(dst);
        d[0] = make_uint4(h[0], h[1], h[2], h[3]);
        d[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
    if (t4 == 0) *xs = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}

// u = x A^T for 16 rows of A (blockIdx.y) of one projection (blockIdx.z), the
// blocks of 64 along K shared out over the cluster's CTAs and their warps,
// and x laid out for lsn_decode_kernel.  Sums in fp32: MMA accumulators, then
// the warps in order, then the cluster's CTAs in order.
template <int NT>
__global__ void __launch_bounds__(kPrepThreads) lsn_decode_prep_kernel(const __grid_constant__ PrepArgs args) {
    __shared__ float part[kPrepWarps][16][8 * NT];
    __shared__ float mine[16][8 * NT];
    pdl_wait();
    pdl_launch_dependents();
    const PrepProj& p = args.p[blockIdx.z];
    const int T = args.T, r = args.r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int j0 = blockIdx.y * 16;
    const bool lays = p.xf != nullptr && blockIdx.y == 0;
    const bool dots = p.A != nullptr;
    const int64_t K = (int64_t)p.nb * 64;
    float acc[NT][4] = {};
    if (lays || dots) {
        for (int b = blockIdx.x * kPrepWarps + warp; b < p.nb; b += kPrepCtas * kPrepWarps) {
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
                    lay_out_x(xv[i], t < T, p.xf + ((int64_t)b * T + t) * 64 + 16 * t4, p.xs + (int64_t)b * 8 * NT + t, t4);
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
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kPrepThreads) {
        float s = 0.f;
        #pragma unroll
        for (int w = 0; w < kPrepWarps; ++w) s += (&part[w][0][0])[i];
        (&mine[0][0])[i] = s;
    }
    cluster_sync_all();
    if (cluster_ctarank() == 0) {
        for (int i = threadIdx.x; i < 16 * 8 * NT; i += kPrepThreads) {
            const int j = j0 + i / (8 * NT), t = i % (8 * NT);
            if (j >= r || t >= T) continue;
            float s = 0.f;
            #pragma unroll
            for (int c = 0; c < kPrepCtas; ++c) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&mine[0][0] + i), c)) : "memory");
                s += v;
            }
            p.u[(int64_t)t * r + j] = s;
        }
    }
    cluster_sync_all();     // the partial sums stay readable until CTA 0 has them
}

extern __shared__ __align__(1024) uint8_t smem_raw[];

// One 32-row tile of one projection at a time: each warp takes every 16th
// block of 64 along K of all 32 rows, so a warp's x registers serve two MMA
// row groups; the warps' partial sums meet in shared memory.
template <int NT>
__global__ void __launch_bounds__(kThreads, 1) lsn_decode_kernel(const __grid_constant__ DecodeArgs args) {
    // entry e of the table: the levels of byte e's two codes (high nibble
    // first) as fp16, once for each lane (256 bytes apart), so that a warp's
    // lookups never meet in a bank and an entry's address is a byte permute
    float* const part = reinterpret_cast<float*>(smem_raw + kTableBytes);   // [warp][row][token]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int T = args.T, r = args.r;
    for (int e = warp; e < 256; e += kWarps) {
        const __half2 h = __floats2half2_rn(args.level[e >> 4], args.level[e & 15]);
        *reinterpret_cast<__half2*>(smem_raw + e * 256 + lane * 4) = h;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t lane4 = lane * 4;

    int pi = 0;
    for (int tile = blockIdx.x; tile < args.tiles; tile += gridDim.x) {
        while (pi + 1 < args.n && tile >= args.p[pi + 1].tile0) ++pi;
        const DecodeProj& p = args.p[pi];
        const int n0 = (tile - p.tile0) * kRows;
        const int nb = p.nb;
        const float offset = *p.offset;
        float acc[2][NT][4] = {};
        for (int b = warp; b < nb; b += kWarps) {
            uint2 cw[4];
            float am[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t blk = (int64_t)(n0 + 8 * i + g) * nb + b;
                cw[i] = __ldcs(reinterpret_cast<const uint2*>(p.packed + blk * 32 + t4 * 8));
                // absmax = fp32(fp32(table[q] s2) + offset), the codec's own roundings
                const int q = p.q[blk];
                am[i] = __fadd_rn(__fmul_rn(__fdiv_rn((float)(q < 255 ? q - 127 : 0), 127.f), p.s2[blk >> 8]), offset);
            }
            X16 xv[NT];
            float2 xs[NT];
            #pragma unroll
            for (int i = 0; i < NT; ++i) {
                xv[i] = load16(reinterpret_cast<const uint16_t*>(p.xf) + ((int64_t)b * T + g + 8 * i) * 64 + 16 * t4, g + 8 * i < T);
                xs[i] = *reinterpret_cast<const float2*>(p.xs + (int64_t)b * 8 * NT + 8 * i + 2 * t4);
            }
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                float c[NT][4] = {};
                #pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t w0 = m < 2 ? cw[2 * h].x : cw[2 * h].y, w1 = m < 2 ? cw[2 * h + 1].x : cw[2 * h + 1].y;
                    const int j = (2 * m) & 3;
                    uint32_t a[4];
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at = prmt((q & 1) ? w1 : w0, lane4, 0x5504u | (uint32_t)(j + (q >> 1)) << 4);
                        a[q] = *reinterpret_cast<const uint32_t*>(smem_raw + at);
                    }
                    #pragma unroll
                    for (int i = 0; i < NT; ++i) mma_f16(c[i], a, xv[i].w(2 * m), xv[i].w(2 * m + 1));
                }
                #pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[h][i][0] += c[i][0] * xs[i].x * am[2 * h];
                    acc[h][i][1] += c[i][1] * xs[i].y * am[2 * h];
                    acc[h][i][2] += c[i][2] * xs[i].x * am[2 * h + 1];
                    acc[h][i][3] += c[i][3] * xs[i].y * am[2 * h + 1];
                }
            }
        }
        #pragma unroll
        for (int h = 0; h < 2; ++h)
            #pragma unroll
            for (int i = 0; i < NT; ++i) {
                float* d = part + ((warp * kRows + 16 * h + g) * 8 * NT + 8 * i + 2 * t4);
                *reinterpret_cast<float2*>(d) = make_float2(acc[h][i][0], acc[h][i][1]);
                *reinterpret_cast<float2*>(d + 8 * 8 * NT) = make_float2(acc[h][i][2], acc[h][i][3]);
            }
        __syncthreads();
        for (int o = threadIdx.x; o < kRows * T; o += kThreads) {
            const int t = o / kRows, row = o % kRows;
            float s = 0.f;
            #pragma unroll
            for (int w = 0; w < kWarps; ++w) s += part[(w * kRows + row) * 8 * NT + t];
            if (p.u != nullptr) {
                const uint4* B = reinterpret_cast<const uint4*>(p.B + (int64_t)(n0 + row) * r);
                const float* u = p.u + (int64_t)t * r;
                float d = 0.f;
                for (int j = 0; j < r; j += 8) {
                    const uint4 v = B[j / 8];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        d = fmaf(u[j + 2 * q], bf16_f(w[q] & 0xffffu), d);
                        d = fmaf(u[j + 2 * q + 1], __uint_as_float(w[q] & 0xffff0000u), d);
                    }
                }
                s = fmaf(args.scale, d, s);
            }
            p.y[(int64_t)t * p.N + n0 + row] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
        }
        __syncthreads();
    }
}

template <int NT>
lsn_status launch_nt(const PrepArgs& pa, const DecodeArgs& da, cudaStream_t st) {
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPrepCtas, (unsigned)((pa.r + 15) / 16), (unsigned)da.n);
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kPrepCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1 + pdl_attr(&at[1]);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, lsn_decode_prep_kernel<NT>, pa));
    const int smem = kTableBytes + kWarps * kRows * 8 * NT * 4;
    LSN_CUDA_TRY(cudaFuncSetAttribute(lsn_decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3((unsigned)std::min(da.tiles, sm_count()));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = pdl_attr(&at[0]);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, lsn_decode_kernel<NT>, da));
    return LSN_OK;
}

}  // namespace

// Workspace: 256 bytes reserved, then per projection u, the fp16 x and its block scales.
namespace {
struct DecodeWs {
    float* u[LSN_LAYER_MAX_PROJ];
    __half* xf[LSN_LAYER_MAX_PROJ];
    float* xs[LSN_LAYER_MAX_PROJ];
    size_t total;
};
DecodeWs carve_decode(void* ws, int n, const lsn_lora_proj* p, int64_t T, int r) {
    DecodeWs w{};
    size_t off = 256;
    char* b = reinterpret_cast<char*>(ws);
    auto take = [&](size_t bytes) { char* q = b ? b + off : nullptr; off += round_up(bytes, 256); return q; };
    for (int i = 0; i < n; ++i) {
        const size_t K = (size_t)p[i].W.cols;
        w.u[i] = reinterpret_cast<float*>(take((size_t)T * r * 4));
        w.xf[i] = reinterpret_cast<__half*>(take((size_t)T * K * 2));
        w.xs[i] = reinterpret_cast<float*>(take(K / 64 * LSN_DECODE_MAX_T * 4));
    }
    w.total = off;
    return w;
}
}  // namespace

size_t decode_ws_bytes(int n, const lsn_lora_proj* p, int64_t T, int r) { return carve_decode(nullptr, n, p, T, r).total; }

lsn_status launch_decode(int n, const lsn_lora_proj* p, int T, int r, float scale, void* ws, cudaStream_t st) {
    const DecodeWs w = carve_decode(ws, n, p, T, r);
    PrepArgs pa{};
    DecodeArgs da{};
    pa.T = da.T = T;
    pa.r = da.r = r;
    da.n = n;
    da.scale = scale;
    std::copy(nf4_tables().level, nf4_tables().level + 16, da.level);
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        const lsn_lora_proj& q = p[i];
        int lead = 0;                       // the first projection that reads the same x
        while (p[lead].x != q.x || p[lead].W.cols != q.W.cols) ++lead;
        const bool off = q.A == nullptr;
        pa.p[i] = PrepProj{q.x, q.A, w.u[i], lead == i ? w.xf[i] : nullptr, w.xs[i], (int)(q.W.cols / 64)};
        const lsn_nf4_weight& f = q.W.nf4;
        da.p[i] = DecodeProj{f.packed, f.absmax_q, f.absmax_s2, f.offset, w.xf[lead], w.xs[lead], off ? nullptr : w.u[i], q.B, q.y,
                             (int)(q.W.cols / 64), (int)q.W.rows, (int)tiles};
        tiles += q.W.rows / kRows;
        if (tiles > INT32_MAX) return fail(LSN_ERR_UNSUPPORTED, "lora_layer_decode: too many rows");
    }
    da.tiles = (int)tiles;
    return T <= 8 ? launch_nt<1>(pa, da, st) : launch_nt<2>(pa, da, st);
}

}  // namespace lsn
