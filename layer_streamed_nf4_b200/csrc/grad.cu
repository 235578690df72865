// The global norm of many gradient tensors and their clipping:
//   norm = sqrt(sum over tensors and elements of g^2),   dst = g min(1, max_norm / norm).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "timing.cuh"

namespace lsn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTensors = 1024;          // of one launch (28 bytes of kernel parameters each)
constexpr int kFewTensors = 16;            // launches of up to so many take a small parameter block
constexpr int kChunkBytes = 16384;         // one CTA's piece of a tensor at a time
constexpr int kMaxCtas = 2048;             // partial sums per launch

// Tensors of one launch; tensor i covers chunks chunk0[i] .. chunk0[i + 1].
template <int MAX>
struct GradArgs {
    int n, chunks;
    int chunk0[MAX];
    const void* src[MAX];
    void* dst[MAX];
    uint64_t numel[MAX];                   // bit 63: bf16
};
static_assert(sizeof(GradArgs<kMaxTensors>) + 64 <= 32764, "kernel parameters");

// Head of the workspace: the scale for the clip kernel, which multiplies by
// both numbers in turn (pre is 1, or a power of two that keeps a scale below
// fp32's normal range from losing bits), the count of finished CTAs (zero
// between calls), then one fp64 partial sum per CTA and launch.
struct GradWs {
    float pre, factor;
    int done;
    double part[1];
};
constexpr float kPre = 0x1p-100f;
constexpr size_t kWsHead = 256;

template <int MAX>
__device__ __forceinline__ int tensor_of(const GradArgs<MAX>& a, int chunk) {
    int lo = 0, hi = a.n - 1;              // the last tensor whose first chunk is <= chunk
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (a.chunk0[m] <= chunk) lo = m; else hi = m - 1;
    }
    return lo;
}

// A chunk is 16-byte words of src's own alignment: element e of the tensor is
// element e + mis of the words that start at src - mis.
struct Chunk {
    const char* base;      // 16-byte aligned start of the chunk
    int lo, hi;            // its elements' bounds within the tensor, in elements from base
    bool bf16;
};
template <int MAX>
__device__ __forceinline__ Chunk chunk_of(const GradArgs<MAX>& a, int i, int chunk) {
    const uint64_t nm = a.numel[i];
    Chunk c;
    c.bf16 = nm >> 63;
    const int es = c.bf16 ? 2 : 4;
    const int64_t numel = (int64_t)(nm & ~(1ull << 63));
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.src[i]);
    const int mis = (int)(p & 15) / es;
    const int64_t at = (int64_t)(chunk - a.chunk0[i]) * (kChunkBytes / es);
    c.base = reinterpret_cast<const char*>(p - (p & 15)) + at * es;
    c.lo = at == 0 ? mis : 0;
    const int64_t left = numel + mis - at;
    c.hi = (int)(left < kChunkBytes / es ? left : kChunkBytes / es);
    return c;
}

// The words w0 .. w1 of a chunk lie within the tensor whole; the n elements
// outside of them, before and after, are its edges.
constexpr int kWords = kChunkBytes / 16 / kThreads;     // of a thread
struct Edges {
    int w0, w1, n;
    __device__ __forceinline__ int at(int j, const Chunk& c, int per) const {
        const int before = w0 * per - c.lo;
        return w1 == w0 || j < before ? c.lo + j : w1 * per + j - before;
    }
};
__device__ __forceinline__ Edges edges_of(const Chunk& c, int per) {
    Edges e;
    e.w0 = (c.lo + per - 1) / per;
    e.w1 = max(c.hi / per, e.w0);
    e.n = c.hi - c.lo - (e.w1 - e.w0) * per;
    return e;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sum of squares of up to 8 values: fp32 within a 16-byte word, fp64 above,
// and in fp64 from the start where a square would leave fp32's normal range.
__device__ __forceinline__ double squares4(float a, float b, float c, float d) {
    const float s = fmaf(a, a, fmaf(b, b, fmaf(c, c, d * d)));
    if (s < 3e38f && s > 1e-30f) return (double)s;
    return (double)a * a + (double)b * b + (double)c * c + (double)d * d;
}

__device__ __forceinline__ double squares_of(const uint4& v, bool bf16) {
    if (bf16)
        return squares4(lo_bf16(v.x), hi_bf16(v.x), lo_bf16(v.y), hi_bf16(v.y)) + squares4(lo_bf16(v.z), hi_bf16(v.z), lo_bf16(v.w), hi_bf16(v.w));
    return squares4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
struct Scale {
    float pre, factor;
    __device__ __forceinline__ float operator()(float g) const { return g * pre * factor; }
};
__device__ __forceinline__ uint4 scaled(uint4 v, Scale f, bool bf16) {
    if (bf16) {
        v.x = pack_bf16x2(f(lo_bf16(v.x)), f(hi_bf16(v.x)));
        v.y = pack_bf16x2(f(lo_bf16(v.y)), f(hi_bf16(v.y)));
        v.z = pack_bf16x2(f(lo_bf16(v.z)), f(hi_bf16(v.z)));
        v.w = pack_bf16x2(f(lo_bf16(v.w)), f(hi_bf16(v.w)));
    } else {
        v.x = __float_as_uint(f(__uint_as_float(v.x)));
        v.y = __float_as_uint(f(__uint_as_float(v.y)));
        v.z = __float_as_uint(f(__uint_as_float(v.z)));
        v.w = __float_as_uint(f(__uint_as_float(v.w)));
    }
    return v;
}

__device__ double block_sum(double v, double* sh) {
    #pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = threadIdx.x < kThreads / 32 ? sh[threadIdx.x] : 0.0;
    if (threadIdx.x < 32) {
        #pragma unroll
        for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;               // the sum, in thread 0
}

// Partial sums of one launch's tensors; with `last`, the last CTA to finish
// adds those of every launch (`parts` in all, in order) and writes the norm.
// Bound by reading where tensors are large; where they are small, by latency:
// all words of a chunk, a tensor's first and last included, are in flight at
// once (norm and scaling of 300 odd tensors, 23 MB: 16.9 us; one after the
// other in the first and last chunks, 18.9).
template <int MAX>
__global__ void __launch_bounds__(kThreads) lsn_grad_norm_kernel(const __grid_constant__ GradArgs<MAX> a, GradWs* ws, int part0, int parts, bool last,
                                                                 float max_norm, float* norm) {
    __shared__ double sh[kThreads / 32];
    __shared__ int is_last;
    pdl_wait();
    pdl_launch_dependents();
    double sum = 0.0;
    for (int ch = blockIdx.x; ch < a.chunks; ch += gridDim.x) {
        const Chunk c = chunk_of(a, tensor_of(a, ch), ch);
        const int es = c.bf16 ? 2 : 4, per = 16 / es;
        if (c.lo == 0 && c.hi == kChunkBytes / es) {                    // a whole chunk: a thread's words all in flight
            uint4 v[kWords];
            #pragma unroll
            for (int u = 0; u < kWords; ++u) v[u] = reinterpret_cast<const uint4*>(c.base)[threadIdx.x + u * kThreads];
            #pragma unroll
            for (int u = 0; u < kWords; ++u) sum += squares_of(v[u], c.bf16);
            continue;
        }
        const Edges g = edges_of(c, per);
        if ((int)threadIdx.x < g.n) {
            const int k = g.at(threadIdx.x, c, per);
            const double x = c.bf16 ? (double)lo_bf16(reinterpret_cast<const uint16_t*>(c.base)[k]) : (double)reinterpret_cast<const float*>(c.base)[k];
            sum += x * x;
        }
        const uint4* const p = reinterpret_cast<const uint4*>(c.base) + g.w0 + threadIdx.x;
        const int left = g.w1 - g.w0 - (int)threadIdx.x;
        uint4 v[kWords];
        #pragma unroll
        for (int u = 0; u < kWords; ++u)
            if (u * kThreads < left) v[u] = p[u * kThreads];
        #pragma unroll
        for (int u = 0; u < kWords; ++u)
            if (u * kThreads < left) sum += squares_of(v[u], c.bf16);
    }
    sum = block_sum(sum, sh);
    if (threadIdx.x == 0) {
        ws->part[part0 + blockIdx.x] = sum;
        is_last = 0;
        if (last) {
            __threadfence();
            is_last = atomicAdd(&ws->done, 1) == (int)gridDim.x - 1;
            __threadfence();
        }
    }
    __syncthreads();
    if (!is_last) return;
    double t = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) t += __ldcg(&ws->part[i]);
    t = block_sum(t, sh);
    if (threadIdx.x == 0) {
        const double nrm = sqrt(t);
        *norm = (float)nrm;
        // over the largest norm: scale; a norm that is no number, or infinite as fp32 reports it, leaves the gradients
        // as they are
        const double f = nrm > (double)max_norm && (float)nrm < INFINITY ? (double)max_norm / nrm : 1.0;
        ws->pre = f < kPre ? kPre : 1.f;
        ws->factor = (float)(f < kPre ? f / kPre : f);
        ws->done = 0;
    }
}

// The last chunks first: they are what the norm read last and the L2 still
// holds.  The first one is looked up before pdl_wait: it depends on nothing the
// norm writes.  Bound by reading and writing: norm and scaling of 168 MB take 80
// to 82 us together, 78 at the copy rate.
template <int MAX>
__global__ void __launch_bounds__(kThreads) lsn_grad_scale_kernel(const __grid_constant__ GradArgs<MAX> a, const GradWs* ws) {
    int ch = a.chunks - 1 - (int)blockIdx.x, i = 0;
    Chunk c;
    auto find = [&] {
        if (ch < 0) return;
        i = tensor_of(a, ch);
        c = chunk_of(a, i, ch);
    };
    find();
    pdl_wait();
    pdl_launch_dependents();
    const Scale f{ws->pre, ws->factor};
    for (; ch >= 0; ch -= (int)gridDim.x, find()) {
        char* const dst = reinterpret_cast<char*>(a.dst[i]) + (c.base - reinterpret_cast<const char*>(a.src[i]));
        if (f.pre == 1.f && f.factor == 1.f && dst == c.base) continue;
        const int es = c.bf16 ? 2 : 4, per = 16 / es;
        const bool wide = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
        if (wide && c.lo == 0 && c.hi == kChunkBytes / es) {            // a whole chunk: a thread's words all in flight
            uint4 v[kWords];
            #pragma unroll
            for (int u = 0; u < kWords; ++u) v[u] = __ldcs(reinterpret_cast<const uint4*>(c.base) + threadIdx.x + u * kThreads);
            #pragma unroll
            for (int u = 0; u < kWords; ++u) __stcs(reinterpret_cast<uint4*>(dst) + threadIdx.x + u * kThreads, scaled(v[u], f, c.bf16));
            continue;
        }
        const Edges g = wide ? edges_of(c, per) : Edges{0, 0, c.hi - c.lo};     // dst lies otherwise: one by one
        for (int j = threadIdx.x; j < g.n; j += kThreads) {
            const int k = g.at(j, c, per);
            if (c.bf16)
                reinterpret_cast<uint16_t*>(dst)[k] = __bfloat16_as_ushort(__float2bfloat16_rn(f(lo_bf16(reinterpret_cast<const uint16_t*>(c.base)[k]))));
            else
                reinterpret_cast<float*>(dst)[k] = f(reinterpret_cast<const float*>(c.base)[k]);
        }
        const uint4* const p = reinterpret_cast<const uint4*>(c.base) + g.w0 + threadIdx.x;
        uint4* const q = reinterpret_cast<uint4*>(dst) + g.w0 + threadIdx.x;
        const int left = g.w1 - g.w0 - (int)threadIdx.x;
        uint4 v[kWords];
        #pragma unroll
        for (int u = 0; u < kWords; ++u)
            if (u * kThreads < left) v[u] = __ldcs(p + u * kThreads);
        #pragma unroll
        for (int u = 0; u < kWords; ++u)
            if (u * kThreads < left) __stcs(q + u * kThreads, scaled(v[u], f, c.bf16));
    }
}

int64_t chunks_of(const lsn_grad& t) {
    const int es = t.dtype == LSN_DT_BF16 ? 2 : 4;
    const int64_t mis = (int64_t)(reinterpret_cast<uintptr_t>(t.src) & 15) / es;
    return t.numel == 0 ? 0 : ceil_div(t.numel + mis, kChunkBytes / es);
}

// The next tensors of t[*i ..], up to kMaxTensors, as one launch's arguments;
// those that go on where the one before ends (the tensors of one flat buffer)
// count as one.  *i becomes the first tensor left over.
void fill(GradArgs<kMaxTensors>& a, const lsn_grad* t, int n, int* i, bool clip) {
    a.n = a.chunks = 0;
    for (; *i < n; ++*i) {
        lsn_grad r = t[*i];
        if (r.numel == 0) continue;
        if (a.n == kMaxTensors) return;
        const int64_t es = r.dtype == LSN_DT_BF16 ? 2 : 4;
        for (; *i + 1 < n; ++*i) {
            const lsn_grad& q = t[*i + 1];
            if (q.numel != 0 && (q.dtype != r.dtype || q.src != reinterpret_cast<const char*>(r.src) + es * r.numel ||
                                 (clip && q.dst != reinterpret_cast<char*>(r.dst) + es * r.numel)))
                break;
            r.numel += q.numel;
        }
        a.src[a.n] = r.src;
        a.dst[a.n] = r.dst;
        a.numel[a.n] = (uint64_t)r.numel | (r.dtype == LSN_DT_BF16 ? 1ull << 63 : 0);
        a.chunk0[a.n++] = a.chunks;
        a.chunks += (int)chunks_of(r);
    }
}

template <class... P, class... A>
lsn_status launch(void (*kernel)(P...), int grid, cudaStream_t st, A&&... args) {
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = pdl_attr(at);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return LSN_OK;
}

size_t ws_bytes_of(int n) { return kWsHead + 8 * (size_t)kMaxCtas * (size_t)std::max<int64_t>(1, ceil_div(n, kMaxTensors)); }

lsn_status grad_call(int n, const lsn_grad* t, bool clip, float max_norm, float* norm, void* ws, size_t ws_bytes, lsn_stream_t stream,
                     const char* who) {
    const std::string f(who);
    LSN_CHECK_ARG(n >= 0, f + ": n must be >= 0");
    LSN_CHECK_ARG(n == 0 || t != nullptr, f + ": tensor array is NULL");
    LSN_CHECK_ARG(!clip || (max_norm > 0.f && std::isfinite(max_norm)), f + ": max_norm must be positive and finite");
    LSN_CHECK_ARG(norm != nullptr && (reinterpret_cast<uintptr_t>(norm) & 3) == 0, f + ": norm must be a 4-byte aligned device pointer");
    LSN_CHECK_ARG(ws != nullptr && aligned16(ws), f + ": workspace must be a 16-byte aligned device pointer");
    LSN_CHECK_ARG(ws_bytes >= ws_bytes_of(n), f + ": workspace too small (need " + std::to_string(ws_bytes_of(n)) + " bytes)");
    int64_t chunks = 0;
    double bytes = 0.0;
    auto fi = [&](int i, const char* what) { return f + ": tensor " + std::to_string(i) + what; };
    for (int i = 0; i < n; ++i) {
        LSN_CHECK_ARG(t[i].numel >= 0 && t[i].numel <= (int64_t)1 << 42, fi(i, ": numel out of range"));
        LSN_CHECK_ARG(t[i].dtype == LSN_DT_BF16 || t[i].dtype == LSN_DT_F32, fi(i, ": unknown type"));
        const uintptr_t es = t[i].dtype == LSN_DT_BF16 ? 2 : 4;
        if (t[i].numel == 0) continue;
        LSN_CHECK_ARG(t[i].src != nullptr && (reinterpret_cast<uintptr_t>(t[i].src) % es) == 0, fi(i, ": src must be aligned to its type"));
        if (clip) {
            LSN_CHECK_ARG(t[i].dst != nullptr && (reinterpret_cast<uintptr_t>(t[i].dst) % es) == 0, fi(i, ": dst must be aligned to its type"));
            const uintptr_t a = reinterpret_cast<uintptr_t>(t[i].src), b = reinterpret_cast<uintptr_t>(t[i].dst), k = es * (uintptr_t)t[i].numel;
            LSN_CHECK_ARG(a == b || a + k <= b || b + k <= a, fi(i, ": dst overlaps src in part"));
        }
        chunks += chunks_of(t[i]);
        bytes += (double)es * (double)t[i].numel * (clip ? 2.0 : 1.0);
    }
    LSN_CHECK_ARG(chunks <= INT32_MAX, f + ": too many elements");
    lsn_status s = check_device();
    if (s != LSN_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    TimingScope ts(LSN_K_GRAD, bytes, st, clip ? 2 : 1);
    GradArgs<kMaxTensors> a;
    GradArgs<kFewTensors> few;
    a.n = a.chunks = 0;
    auto grid_of = [&] { return std::max(1, std::min({a.chunks, 8 * sm_count(), kMaxCtas})); };
    auto is_few = [&] {                     // a small copy of the arguments, when they fit one
        if (a.n > kFewTensors) return false;
        few.n = a.n;
        few.chunks = a.chunks;
        std::copy(a.chunk0, a.chunk0 + a.n, few.chunk0);
        std::copy(a.src, a.src + a.n, few.src);
        std::copy(a.dst, a.dst + a.n, few.dst);
        std::copy(a.numel, a.numel + a.n, few.numel);
        return true;
    };
    int parts = 0, i = 0, launches = 0;
    do {
        fill(a, t, n, &i, clip);
        const int grid = grid_of();
        s = is_few() ? launch(lsn_grad_norm_kernel<kFewTensors>, grid, st, few, (GradWs*)ws, parts, parts + grid, i >= n, max_norm, norm)
                     : launch(lsn_grad_norm_kernel<kMaxTensors>, grid, st, a, (GradWs*)ws, parts, parts + grid, i >= n, max_norm, norm);
        if (s != LSN_OK) return s;
        parts += grid;
        ++launches;
    } while (i < n);
    if (!clip) return LSN_OK;
    i = 0;
    do {
        if (launches > 1) fill(a, t, n, &i, clip);
        else i = n;
        const int grid = grid_of();
        s = is_few() ? launch(lsn_grad_scale_kernel<kFewTensors>, grid, st, few, (const GradWs*)ws)
                     : launch(lsn_grad_scale_kernel<kMaxTensors>, grid, st, a, (const GradWs*)ws);
        if (s != LSN_OK) return s;
    } while (i < n);
    return LSN_OK;
}

}  // namespace

}  // namespace lsn

using namespace lsn;

extern "C" {

size_t lsn_grad_ws_bytes(int n) { return n < 0 ? 0 : ws_bytes_of(n); }

lsn_status grad_norm(int n, const lsn_grad* t, float* norm, void* ws, size_t ws_bytes, lsn_stream_t stream) {
    NvtxRange nvtx("grad_norm");
    return grad_call(n, t, false, 1.f, norm, ws, ws_bytes, stream, "grad_norm");
}

lsn_status grad_clip(int n, const lsn_grad* t, float max_norm, float* norm, void* ws, size_t ws_bytes, lsn_stream_t stream) {
    NvtxRange nvtx("grad_clip");
    return grad_call(n, t, true, max_norm, norm, ws, ws_bytes, stream, "grad_clip");
}

}  // extern "C"
