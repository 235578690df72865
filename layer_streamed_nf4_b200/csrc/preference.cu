// Sequence log-probabilities and the preference loss, from logits:
//   lse_t = log sum_v exp l[t, v],   logp_i = sum over scored t of sequence i of (l[t, y_t] - lse_t),
//   the loss of each pair of sequences from its difference of log ratios, and
//   dl[t, v] = c_t ([v = y_t] - exp(l[t, v] - lse_t)),   c_t = dloss/dlogp of t's sequence.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "timing.cuh"

namespace lsn {

namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 148 * 8;             // that run at the same time
constexpr int kFinThreads = 512;           // of the finishing kernel: half of them for each sequence of a pair
constexpr size_t kWsHead = 256;

// Pieces a row is cut into, from the shape alone: enough that every SM has
// work, in pieces of 4096 logits at least; and up to four times as many pieces
// as CTAs run at once, for an even end, in pieces of 16384 at least (1021 rows
// of 32000 in 5 pieces each took 19 us, in 2 pieces 12.5).
int row_splits(int64_t T, int64_t V) {
    if (T <= 0) return 1;
    return (int)std::max<int64_t>({1, std::min(ceil_div(kCtas, T), V / 4096), std::min(ceil_div(4 * kCtas, T), V / 16384)});
}

// The workspace behind its head: a row's pieces, its target's logit, its gradient's factor.
struct Scratch {
    float2* part;                          // [T, splits] maximum and sum
    float* ly;                             // [T]
    float* coef;                           // [T]
    size_t total;
};
Scratch carve(void* ws, int64_t T, int64_t V) {
    Scratch w;
    char* b = reinterpret_cast<char*>(ws);
    size_t off = kWsHead;
    auto take = [&](size_t bytes) { char* q = b ? b + off : nullptr; off += round_up(bytes, 256); return q; };
    w.part = reinterpret_cast<float2*>(take((size_t)T * row_splits(T, V) * sizeof(float2)));
    w.ly = reinterpret_cast<float*>(take((size_t)T * 4));
    w.coef = reinterpret_cast<float*>(take((size_t)T * 4));
    w.total = off;
    return w;
}

struct Ws {
    int done;                              // finished CTAs of the last kernel that counts (zero between calls)
};

struct Rows {
    const void* logits;
    int64_t ld;
    int T, V, n_seq, splits, average;
    const int32_t* targets;
    const int32_t* start;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);      // 1.9e-8: what fp32's log2 e leaves out

// 2^t for t <= 1/2, within about an ulp either way: ex2.approx is 5.0e-8 low on
// average, which adds up where a sum is scaled several times.  The series of
// exp(f ln 2) for |f| <= 1/2 to the 7th power (the 8th is below 5.3e-9).
__device__ __forceinline__ float exp2_even(float t) {
    t = fmaxf(t, -127.f);                   // and what is below 2^-126 counts as 0
    const float n = rintf(t), f = (t - n) * 0.6931471805599453f;
    float p = 1.f / 5040.f;
    p = fmaf(p, f, 1.f / 720.f);
    p = fmaf(p, f, 1.f / 120.f);
    p = fmaf(p, f, 1.f / 24.f);
    p = fmaf(p, f, 1.f / 6.f);
    p = fmaf(p, f, 0.5f);
    p = fmaf(p, f, 1.f);
    p = fmaf(p, f, 1.f);
    return n < -126.f ? 0.f : p * __int_as_float(((int)n + 127) << 23);
}
// exp(x) for a difference x <= 0 of two numbers
__device__ __forceinline__ float exp_even(float x) { return exp2_even(fmaf(x, kLog2e, x * kLog2eRest)); }
// Maxima below it take one multiply-add a logit: the rounding of their product with
// log2 e, which is left in the sum until the end, is at most 2^-8 there.  (From 2^31
// on it leaves exp2's range.)
constexpr float kSmallMax = 65536.f;

template <class E> struct Words;           // 16-byte words of a row: how many values, and unpacking
template <> struct Words<uint16_t> {
    static constexpr int per = 8;
    static __device__ __forceinline__ void get(const uint4& w, float (&v)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }     // -infinity
    template <int U>
    static __device__ __forceinline__ float largest(const uint4 (&x)[U]) {  // two at a time
        __nv_bfloat162 m = __floats2bfloat162_rn(-INFINITY, -INFINITY);
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            #pragma unroll
            for (int i = 0; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        }
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ void set(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    // the exponential behind a gradient: off by 2^-22 and 2^-23 of its argument here, far below bf16's step
    static __device__ __forceinline__ float exp(float x) { return ex2(x * kLog2e); }
};
template <> struct Words<float> {
    static constexpr int per = 4;
    static __device__ __forceinline__ void get(const uint4& w, float (&v)[4]) {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    template <int U>
    static __device__ __forceinline__ float largest(const uint4 (&x)[U]) {
        float m = -INFINITY;
        #pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(x[u].x), __uint_as_float(x[u].y))), fmaxf(__uint_as_float(x[u].z), __uint_as_float(x[u].w)));
        return m;
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ void set(float* p, float v) { *p = v; }
    static __device__ __forceinline__ float exp(float x) { return expf(x); }        // 2 ulp for every argument
};

// Whether row t's target is counted: in the vocabulary, inside the sequences.
__device__ __forceinline__ bool scored(const Rows& r, int t, int y) {
    return y >= 0 && y < r.V && t >= r.start[0] && t < r.start[r.n_seq];
}

// The sum s of exp(x - m) about another maximum `at` >= m.  m = -infinity stands
// for "no finite value yet"; NaN stays NaN.
__device__ __forceinline__ float about(float m, float s, float at) { return s * exp_even(m - (at == -INFINITY ? 0.f : at)); }

// The 16-byte words of a row that can be taken whole, counted from `row`
// rounded down to 16 bytes (word w holds elements w per - mis ..): all full
// ones, less `skip` at either end; the rest of the row is its edge, less than
// 4 words.  Piece `split` takes words w0 .. w1.
struct Piece {
    int w0, w1, mis, head, tail;           // edge: elements below head and from tail on
};
template <class E>
__device__ __forceinline__ Piece piece_of(const void* row, int V, int split, int splits, int skip) {
    constexpr int per = Words<E>::per;
    Piece p;
    p.mis = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(E);
    const int first = (p.mis ? 1 : 0) + skip, end = (V + p.mis) / per - skip;
    const int n = max(end - first, 0);
    p.w0 = first + (int)((int64_t)n * split / splits);
    p.w1 = first + (int)((int64_t)n * (split + 1) / splits);
    p.head = n > 0 ? first * per - p.mis : V;
    p.tail = n > 0 ? end * per - p.mis : V;
    return p;
}

// (m, s) of one piece of one row per CTA, and the target's logit.  Each thread
// keeps four 16-byte loads in flight; maxima of bf16 are taken two at a time.
// A thread's sum is scaled once to the CTA's maximum, and evenly (exp2_even): at
// every join by ex2.approx it came out 1.0 to 1.3e-7 low, token after token,
// now 1.5e-8 (1000 tokens of a 152k vocabulary: their sum off by 1e-5).
// Bound by DRAM and, nearly as much, the special-function unit (one exp2 a
// logit): 2048 x 151936 bf16, three quarters scored, 77 us, 6.1 TB/s.  With
// exp2((x - m) log2 e) in two instructions it took 94 us, with the words behind
// a piece's end computed like others 81 (3 pieces of 6.2 rounds took 7 each);
// two products or sums in one instruction (f32x2) changed nothing.  CTAs are
// handed out as others finish: rows that are not scored cost nothing.
template <class E>
__global__ void __launch_bounds__(kThreads) lsn_seq_stats_kernel(const __grid_constant__ Rows r, float2* part, float* ly) {
    constexpr int per = Words<E>::per;
    constexpr int U = 4;
    __shared__ float2 sh[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int t = (int)(blockIdx.x / (unsigned)r.splits), split = (int)(blockIdx.x % (unsigned)r.splits);
    const int y = r.targets[t];
    if (!scored(r, t, y)) return;
    const E* row = reinterpret_cast<const E*>(r.logits) + (int64_t)t * r.ld;
    const Piece p = piece_of<E>(row, r.V, split, r.splits, 0);
    const uint4* words = reinterpret_cast<const uint4*>(row - p.mis);
    // s: the sum of exp2(x log2 e - c), c about m log2 e, for a small m; of exp2((x - m) log2 e) for a large one
    float m = -INFINITY, c = -INFINITY, s = 0.f;
    for (int w = p.w0 + threadIdx.x; w < p.w1; w += U * kThreads) {
        uint4 x[U];
        #pragma unroll
        for (int u = 0; u < U; ++u) x[u] = w + u * kThreads < p.w1 ? words[w + u * kThreads] : Words<E>::none();
        const int first = w - (int)(threadIdx.x & 31);      // of the warp's words; those past the end are -infinity
        const float old = m, top = fmaxf(m, Words<E>::template largest<U>(x));
        m = top;
        if (fabsf(top) < kSmallMax) {
            // c is a number like any other: what its rounding leaves out is put right at the end
            const float c1 = top * kLog2e;
            if (c1 != c) s *= exp2_even(fabsf(old) < kSmallMax ? c - c1 : fmaf(old, kLog2e, -c1));
            c = c1;
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u > 0 && first + u * kThreads >= p.w1) break;
                float v[per];
                Words<E>::get(x[u], v);
                #pragma unroll
                for (int i = 0; i < per; ++i) s += ex2(fmaf(v[i], kLog2e, -c1));
            }
        } else {                                        // masks of any size, infinities, nothing yet
            const float at = top == -INFINITY ? 0.f : top;
            if (top != old) s *= fabsf(old) < kSmallMax ? exp2_even(-fmaf(at, kLog2e, -c)) : exp_even(old - at);
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[per];
                Words<E>::get(x[u], v);
                #pragma unroll
                for (int i = 0; i < per; ++i) s += ex2((v[i] - at) * kLog2e);
            }
        }
    }
    if (fabsf(m) < kSmallMax) s *= exp2_even(-fmaf(m, kLog2e, -c));
    if (split == 0) {
        if (threadIdx.x == 0) ly[t] = Words<E>::one(row + y);
        const int edge = p.head + r.V - p.tail;
        if ((int)threadIdx.x < edge) {
            const int e = (int)threadIdx.x < p.head ? (int)threadIdx.x : p.tail + (int)threadIdx.x - p.head;
            const float x = Words<E>::one(row + e);
            const float top = fmaxf(m, x);
            s = about(m, s, top) + about(x, x == -INFINITY ? 0.f : x - x + 1.f, top);     // NaN and +infinity give NaN
            m = top;
        }
    }
    float top = m;
    #pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    s = about(m, s, top);
    #pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(top, s);
    __syncthreads();
    if (threadIdx.x < 32) {                             // the warps', by the lanes of the first
        const float2 w = threadIdx.x < kThreads / 32 ? sh[threadIdx.x] : make_float2(-INFINITY, 0.f);
        top = w.x;
        #pragma unroll
        for (int o = kThreads / 64; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        s = about(w.x, w.y, top);
        #pragma unroll
        for (int o = kThreads / 64; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) part[blockIdx.x] = make_float2(top, s);
    }
}

struct Finish {
    const float2* part;
    const float* ly;
    float* coef;                           // NULL: no gradient follows in this call
    float* lse;
    double* logp;
    int32_t* count;
    // the loss (pairs of sequences), when wanted
    int pairs, kind;
    float beta, smooth, grad_scale;
    const double* ref;
    float* reward;
    float* loss;
    float* mean;
    float* dlogp;
    Ws* ws;
};

// Loss and its derivative with respect to the difference h of the log ratios.
__device__ __forceinline__ void pair_loss(const Finish& f, double h, double* loss, double* d) {
    const double b = f.beta, e = f.smooth, z = b * h;
    if (f.kind == LSN_PREF_SIGMOID) {
        // softplus(v) = max(v, 0) + log(1 + t) and sigmoid(v) = 1 / (1 + t), or t / (1 + t) for v < 0, with t = exp(-|v|)
        const double t = exp(-fabs(z)), rest = log1p(t), large = 1.0 / (1.0 + t), small = t * large;
        // (without smoothing the second term is left out, not multiplied by 0: it may be infinite)
        *loss = (1.0 - e) * ((z < 0.0 ? -z : 0.0) + rest) + (e > 0.0 ? e * ((z > 0.0 ? z : 0.0) + rest) : 0.0);
        *d = b * (z >= 0.0 ? e * large - (1.0 - e) * small : e * small - (1.0 - e) * large);
    } else if (f.kind == LSN_PREF_HINGE) {
        const bool nan = z != z;
        *loss = nan ? z : fmax(1.0 - z, 0.0);
        *d = nan ? z : 1.0 - z > 0.0 ? -b : 0.0;
    } else {
        const double q = h - 0.5 / b;
        *loss = q * q;
        *d = 2.0 * q;
    }
}

// One CTA per two sequences (a pair, when there is a loss), half of it for
// each: the rows' pieces joined into lse, the sequences' sums in fp64 (hundreds
// of terms that later cancel against the reference's), the loss, its gradients
// and, for the gradient kernel of the same call, every row's factor; the last
// CTA to finish adds the losses up in order.  Bound by its chain of loads, of
// which those of the caller's tensors come before pdl_wait: the statistics
// kernel does not write them and itself began after everything older was
// complete (without it, T = 0, they wait like the rest).
__global__ void __launch_bounds__(kFinThreads) lsn_seq_finish_kernel(const __grid_constant__ Rows r, const __grid_constant__ Finish f) {
    constexpr int kHalf = kFinThreads / 2;
    __shared__ double sums[kFinThreads / 32];
    __shared__ int counts[kFinThreads / 32];
    __shared__ double lp[2];
    __shared__ float c_row[2];
    __shared__ int is_last;
    if (r.T == 0) pdl_wait();
    const int half = threadIdx.x / kHalf, tid = threadIdx.x % kHalf, warp = threadIdx.x >> 5;
    const int q = 2 * blockIdx.x + half;
    const bool have = q < r.n_seq;
    const int a = have ? max(r.start[q], 0) : 0, b = have ? min(r.start[q + 1], r.T) : 0;
    const double ref0 = f.ref ? f.ref[2 * blockIdx.x] : 0.0, ref1 = f.ref ? f.ref[2 * blockIdx.x + 1] : 0.0;     // (pairs only)
    // eight lanes to a row that has many pieces (37 x 151936 scored, 32 pieces: 9.7 us, with one lane 13.3; 2 to 4
    // pieces are one round of loads for one lane)
    const int lg = r.splits > 4 ? 3 : 0, lane0 = tid & ((1 << lg) - 1), t1 = a + (tid >> lg);
    const bool on0 = a + tid < b && scored(r, a + tid, r.targets[a + tid]);
    const bool on1 = lg == 0 ? on0 : t1 < b && scored(r, t1, r.targets[t1]);
    if (r.T > 0) pdl_wait();
    pdl_launch_dependents();
    double sum = 0.0;
    int n = 0;
    for (int t0 = a; t0 < b; t0 += kHalf >> lg) {       // the same rounds for a whole warp
        const int t = t0 + (tid >> lg);
        const bool on = t0 == a ? on1 : t < b && scored(r, t, r.targets[t]);
        const float2* const part = f.part + (int64_t)t * r.splits;
        const int end = on ? r.splits : 0;
        float m = -INFINITY;
        double s = 0.0;
        for (int i0 = lane0; i0 < end; i0 += 4 << lg) { // four pieces in flight
            float2 p[4];
            float top = m;
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + (k << lg);
                p[k] = i < end ? part[i] : make_float2(-INFINITY, 0.f);
                top = fmaxf(top, p[k].x);
            }
            s *= (double)about(m, 1.f, top);
            #pragma unroll
            for (int k = 0; k < 4; ++k) s += (double)about(p[k].x, p[k].y, top);
            m = top;
        }
        if (lg > 0) {
            float top = m;
            for (int o = (1 << lg) >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            s *= (double)about(m, 1.f, top);
            m = top;
            for (int o = (1 << lg) >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        if (t >= b || lane0 != 0) continue;
        float l = 0.f;
        if (on) {
            const double ls = log(s);
            l = (float)((double)m + ls);
            sum += ((double)f.ly[t] - (double)m) - ls;
            ++n;
        }
        f.lse[t] = l;
    }
    #pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if ((threadIdx.x & 31) == 0) {
        sums[warp] = sum;
        counts[warp] = n;
    }
    __syncthreads();
    if (tid == 0) {
        sum = 0.0;
        n = 0;
        for (int w = 0; w < kHalf / 32; ++w) {
            sum += sums[half * (kHalf / 32) + w];
            n += counts[half * (kHalf / 32) + w];
        }
        if (r.average) sum /= (double)max(n, 1);
        lp[half] = sum;
        counts[half * (kHalf / 32)] = max(n, 1);
        if (have) {
            f.logp[q] = sum;
            if (f.count) f.count[q] = n;
        }
    }
    // rows in no sequence
    if (blockIdx.x == 0) {
        for (int t = threadIdx.x; t < min(r.start[0], r.T); t += kFinThreads) {
            f.lse[t] = 0.f;
            if (f.coef) f.coef[t] = 0.f;
        }
        for (int t = max(r.start[r.n_seq], 0) + threadIdx.x; t < r.T; t += kFinThreads) {
            f.lse[t] = 0.f;
            if (f.coef) f.coef[t] = 0.f;
        }
    }
    if (f.pairs == 0) return;
    __syncthreads();
    const int i = blockIdx.x;
    if (threadIdx.x == 0) {
        const double ra = lp[0] - ref0, rb = lp[1] - ref1;
        double loss, d;
        pair_loss(f, ra - rb, &loss, &d);
        d *= (double)f.grad_scale / f.pairs;
        c_row[0] = (float)d;
        c_row[1] = (float)-d;
        if (f.reward) {
            f.reward[2 * i] = (float)(f.beta * ra);
            f.reward[2 * i + 1] = (float)(f.beta * rb);
        }
        f.loss[i] = (float)loss;
        f.dlogp[2 * i] = (float)d;
        f.dlogp[2 * i + 1] = (float)-d;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int before = -1;
        if (f.mean != nullptr) asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(before) : "l"(&f.ws->done) : "memory");
        is_last = before == f.pairs - 1;
    }
    if (f.coef) {
        float c = c_row[half];
        if (r.average) c /= (float)counts[half * (kHalf / 32)];
        for (int t = a + tid; t < b; t += kHalf) f.coef[t] = (t == a + tid ? on0 : scored(r, t, r.targets[t])) ? c : 0.f;
    }
    if (f.mean == nullptr) return;
    __syncthreads();
    if (!is_last) return;
    double s = 0.0;
    for (int i = threadIdx.x; i < f.pairs; i += kFinThreads) s += (double)__ldcg(&f.loss[i]);
    #pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int w = 0; w < kFinThreads / 32; ++w) s += sums[w];
        *f.mean = (float)(s / f.pairs);
        f.ws->done = 0;
    }
}

// The sequence of row t: the last one that starts at or before t.
__device__ __forceinline__ int seq_of(const Rows& r, int t) {
    int lo = 0, hi = r.n_seq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (r.start[m] <= t) lo = m; else hi = m - 1;
    }
    return lo;
}

// 16 bytes from byte offset o (0 < o < 16, even) of two neighbouring words.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int o) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (o & 8) {
        #pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (o & 4) {
        #pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (o & 2) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row whose lse is so far from zero that fp32 holds too little of it (rows of
// which a mask leaves nothing, say): its maximum and sum once more from the
// logits, dl = c ([v = y] - exp(l - m) / s), by one CTA, so that it may be in
// place.  Not inlined: it is rare, and its registers would be the common path's.
constexpr float kFarLse = 4096.f;          // 2^-13 of a probability
template <class E>
__device__ __noinline__ void far_row(const E* row, E* out, int V, int y, float c) {
    __shared__ float sh[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY, s = 0.f;
    for (int v = threadIdx.x; v < V; v += kThreads) m = fmaxf(m, Words<E>::one(row + v));
    #pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sh[warp] = m;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sh[w]);
    for (int v = threadIdx.x; v < V; v += kThreads) s += expf(Words<E>::one(row + v) - m);
    #pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane == 0) sh[warp] = s;
    __syncthreads();                        // every thread has read the row
    s = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
    const float f = -c / s;
    for (int v = threadIdx.x; v < V; v += kThreads) Words<E>::set(out + v, fmaf(f, expf(Words<E>::one(row + v) - m), v == y ? c : 0.f));
}

// dl = c ([v = y] - exp(l - lse)), zero in rows that are not scored.  One piece
// of a row per CTA, the last rows first: they are what the statistics kernel
// read last and the L2 still holds (2048 x 151936 bf16: 4 us of 269 for the
// whole loss).  Bound by reading the logits and writing their gradient: 171 us
// there, 6.4 TB/s.  Where a row of logits and its row of gradients lie
// differently against 16 bytes, words are put together from two neighbours.
// Behind the finishing kernel (coef) the first logits are asked for before
// pdl_wait, into the L2 (into registers the kernel's loop came out slower: 274
// us where this takes 255).
template <class E>
__global__ void __launch_bounds__(kThreads) lsn_seq_grad_kernel(const __grid_constant__ Rows r, const float* lse, const float* dlogp,
                                                                const int32_t* count, const float* coef, E* dl, int64_t ld_d) {
    constexpr int per = Words<E>::per;
    constexpr int U = 4;
    if (coef == nullptr) pdl_wait();
    const unsigned item = gridDim.x - 1 - blockIdx.x;
    const int t = (int)(item / (unsigned)r.splits), split = (int)(item % (unsigned)r.splits);
    const int y = r.targets[t];
    const E* row = reinterpret_cast<const E*>(r.logits) + (int64_t)t * r.ld;
    E* out = dl + (int64_t)t * ld_d;
    const bool on = scored(r, t, y);
    const int o = (int)((reinterpret_cast<uintptr_t>(row) - reinterpret_cast<uintptr_t>(out)) & 15);   // 0: they lie alike
    const Piece p = piece_of<E>(out, r.V, split, r.splits, o ? 1 : 0);
    // with the out row's words: word w's elements start o bytes into word w of `words`
    const uint4* words = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row - p.mis) & ~(uintptr_t)15);
    uint4* outs = reinterpret_cast<uint4*>(out - p.mis);
    if (on && threadIdx.x < U * kThreads / 8 && p.w0 + 8 * (int)threadIdx.x < p.w1)      // a line each
        asm volatile("prefetch.global.L2 [%0];" ::"l"(words + p.w0 + 8 * threadIdx.x));
    if (coef != nullptr) pdl_wait();
    pdl_launch_dependents();
    float c = 0.f;
    if (on) {
        if (coef != nullptr) {
            c = coef[t];
        } else {
            const int q = seq_of(r, t);
            c = dlogp[q];
            if (r.average) c /= (float)max(count[q], 1);
        }
    }
    const float nc = -c, L = on ? lse[t] : 0.f;
    if (fabsf(L) >= kFarLse && fabsf(L) < INFINITY) {
        if (split == 0) far_row<E>(row, out, r.V, y, c);
        return;
    }
    if (!on) {
        for (int w = p.w0 + threadIdx.x; w < p.w1; w += kThreads) __stcs(&outs[w], make_uint4(0, 0, 0, 0));
    } else {
        for (int w = p.w0 + threadIdx.x; w < p.w1; w += U * kThreads) {
            uint4 x[U];
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = w + u * kThreads;
                if (k < p.w1) x[u] = o ? shifted(words[k], words[k + 1], o) : words[k];
            }
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = w + u * kThreads;
                if (k >= p.w1) break;
                float v[per];
                Words<E>::get(x[u], v);
                #pragma unroll
                for (int i = 0; i < per; ++i) v[i] = nc * Words<E>::exp(v[i] - L);
                const int at = y + p.mis - k * per;                 // the target's place in this word, in one word of the row
                if ((unsigned)at < (unsigned)per) {
                    #pragma unroll
                    for (int i = 0; i < per; ++i) v[i] += i == at ? c : 0.f;
                }
                __stcs(&outs[k], Words<E>::put(v));
            }
        }
    }
    if (split == 0) {
        const int edge = p.head + r.V - p.tail;
        if ((int)threadIdx.x < edge) {
            const int e = (int)threadIdx.x < p.head ? (int)threadIdx.x : p.tail + (int)threadIdx.x - p.head;
            Words<E>::set(out + e, on ? nc * Words<E>::exp(Words<E>::one(row + e) - L) + (e == y ? c : 0.f) : 0.f);
        }
    }
}

template <class... P, class... A>
lsn_status launch(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t st, A&&... args) {
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, grid));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = pdl_attr(at);
    LSN_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return LSN_OK;
}

size_t ws_bytes_of(int64_t T, int64_t V) { return carve(nullptr, T, V).total; }

bool off_by(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

lsn_status check_in(const lsn_seq_logits* in, const std::string& f) {
    LSN_CHECK_ARG(in != nullptr, f + ": logits descriptor is NULL");
    LSN_CHECK_ARG(in->T >= 0 && in->T <= (int64_t)1 << 30, f + ": T out of range");
    LSN_CHECK_ARG(in->V >= 1 && in->V <= (int64_t)1 << 30, f + ": V out of range");
    LSN_CHECK_ARG(in->ld >= in->V && in->ld <= (int64_t)1 << 31, f + ": ld must be at least V");
    LSN_CHECK_ARG(in->dtype == LSN_DT_BF16 || in->dtype == LSN_DT_F32, f + ": unknown type of the logits");
    LSN_CHECK_ARG(in->n_seq >= 1 && in->n_seq <= 1 << 24, f + ": n_seq out of range");
    LSN_CHECK_ARG((in->logits && in->targets) || in->T == 0, f + ": NULL tensor");
    LSN_CHECK_ARG(in->seq_start != nullptr, f + ": seq_start is NULL");
    LSN_CHECK_ARG(!off_by(in->logits, in->dtype == LSN_DT_BF16 ? 2 : 4), f + ": logits must be aligned to their type");
    LSN_CHECK_ARG(!off_by(in->targets, 4) && !off_by(in->seq_start, 4), f + ": targets and seq_start must be 4-byte aligned");
    return LSN_OK;
}

lsn_status check_ws(const lsn_seq_logits* in, void* ws, size_t ws_bytes, const std::string& f) {
    LSN_CHECK_ARG(ws != nullptr && aligned16(ws), f + ": workspace must be a 16-byte aligned device pointer");
    const size_t need = ws_bytes_of(in->T, in->V);
    LSN_CHECK_ARG(ws_bytes >= need, f + ": workspace too small (need " + std::to_string(need) + " bytes)");
    return LSN_OK;
}

lsn_status check_grad(const lsn_seq_logits* in, const float* lse, const float* dlogp, const int32_t* count, const void* dlogits, int64_t ld_d,
                      const std::string& f) {
    const size_t es = in->dtype == LSN_DT_BF16 ? 2 : 4;
    LSN_CHECK_ARG((lse && dlogits) || in->T == 0, f + ": NULL tensor");
    LSN_CHECK_ARG(dlogp != nullptr, f + ": dlogp is NULL");
    LSN_CHECK_ARG(count || !in->average, f + ": count is needed for averaged log-probabilities");
    LSN_CHECK_ARG(ld_d >= in->V && ld_d <= (int64_t)1 << 31, f + ": ld of dlogits must be at least V");
    LSN_CHECK_ARG(!off_by(dlogits, es), f + ": dlogits must be aligned to its type");
    if (in->T > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(in->logits), b = reinterpret_cast<uintptr_t>(dlogits);
        const uintptr_t na = es * ((uintptr_t)(in->T - 1) * (uintptr_t)in->ld + (uintptr_t)in->V);
        const uintptr_t nb = es * ((uintptr_t)(in->T - 1) * (uintptr_t)ld_d + (uintptr_t)in->V);
        LSN_CHECK_ARG((a == b && ld_d == in->ld) || a + na <= b || b + nb <= a, f + ": dlogits may be the logits themselves or lie apart from them");
    }
    return LSN_OK;
}

Rows rows_of(const lsn_seq_logits* in) {
    return Rows{in->logits, in->ld, (int)in->T, (int)in->V, in->n_seq, row_splits(in->T, in->V), in->average != 0, in->targets, in->seq_start};
}

lsn_status fwd(const lsn_seq_logits* in, Finish f, bool grad, void* ws, cudaStream_t st) {
    const Rows r = rows_of(in);
    const Scratch w = carve(ws, in->T, in->V);
    f.ws = reinterpret_cast<Ws*>(ws);
    f.part = w.part;
    f.ly = w.ly;
    f.coef = grad ? w.coef : nullptr;
    const bool bf16 = in->dtype == LSN_DT_BF16;
    TimingScope ts(LSN_K_SEQ_LOGP, (bf16 ? 2.0 : 4.0) * (double)in->T * (double)in->V + 8.0 * (double)in->T, st, r.T > 0 ? 2 : 1);
    if (r.T > 0) {
        const int64_t items = (int64_t)r.T * r.splits;
        lsn_status s = bf16 ? launch(lsn_seq_stats_kernel<uint16_t>, items, kThreads, st, r, w.part, w.ly)
                            : launch(lsn_seq_stats_kernel<float>, items, kThreads, st, r, w.part, w.ly);
        if (s != LSN_OK) return s;
    }
    return launch(lsn_seq_finish_kernel, ceil_div(r.n_seq, 2), kFinThreads, st, r, f);
}

lsn_status bwd(const lsn_seq_logits* in, const float* lse, const float* dlogp, const int32_t* count, const float* coef, void* dlogits, int64_t ld_d,
               cudaStream_t st) {
    const Rows r = rows_of(in);
    const int64_t items = (int64_t)r.T * r.splits;
    const bool bf16 = in->dtype == LSN_DT_BF16;
    TimingScope ts(LSN_K_SEQ_GRAD, (bf16 ? 4.0 : 8.0) * (double)in->T * (double)in->V, st, 1);
    return bf16 ? launch(lsn_seq_grad_kernel<uint16_t>, items, kThreads, st, r, lse, dlogp, count, coef, (uint16_t*)dlogits, ld_d)
                : launch(lsn_seq_grad_kernel<float>, items, kThreads, st, r, lse, dlogp, count, coef, (float*)dlogits, ld_d);
}

lsn_status check_loss(const lsn_seq_logits* in, const double* ref, const lsn_preference* p, float* lse, double* logp, int32_t* count, float* reward,
                      float* loss, float* mean, float* dlogp, const std::string& f) {
    LSN_CHECK_ARG(p != nullptr, f + ": loss descriptor is NULL");
    LSN_CHECK_ARG(p->kind == LSN_PREF_SIGMOID || p->kind == LSN_PREF_HINGE || p->kind == LSN_PREF_SQUARED, f + ": unknown loss");
    LSN_CHECK_ARG(p->beta > 0.f && std::isfinite(p->beta), f + ": beta must be positive and finite");
    LSN_CHECK_ARG(p->label_smoothing >= 0.f && p->label_smoothing <= 0.5f, f + ": label_smoothing must be in [0, 0.5]");
    LSN_CHECK_ARG(p->label_smoothing == 0.f || p->kind == LSN_PREF_SIGMOID, f + ": label_smoothing belongs to the sigmoid loss");
    LSN_CHECK_ARG(std::isfinite(p->grad_scale), f + ": grad_scale must be finite");
    LSN_CHECK_ARG(in->n_seq % 2 == 0, f + ": sequences come in pairs, one at least");
    LSN_CHECK_ARG((lse || in->T == 0) && logp && loss && dlogp, f + ": NULL tensor");
    LSN_CHECK_ARG(!off_by(lse, 4) && !off_by(logp, 8) && !off_by(ref, 8) && !off_by(count, 4) && !off_by(reward, 4) && !off_by(loss, 4) &&
                      !off_by(mean, 4) && !off_by(dlogp, 4), f + ": tensors must be aligned to their types");
    return LSN_OK;
}

Finish finish_of(const lsn_seq_logits* in, const double* ref, const lsn_preference* p, float* lse, double* logp, int32_t* count, float* reward, float* loss,
                 float* mean, float* dlogp) {
    Finish f{};
    f.lse = lse;
    f.logp = logp;
    f.count = count;
    f.pairs = in->n_seq / 2;
    f.kind = p->kind;
    f.beta = p->beta;
    f.smooth = p->label_smoothing;
    f.grad_scale = p->grad_scale;
    f.ref = ref;
    f.reward = reward;
    f.loss = loss;
    f.mean = mean;
    f.dlogp = dlogp;
    return f;
}

}  // namespace

}  // namespace lsn

using namespace lsn;

extern "C" {

size_t lsn_seq_logp_ws_bytes(const lsn_seq_logits* in) {
    if (in == nullptr || in->T < 0 || in->T > (int64_t)1 << 30 || in->V < 1 || in->V > (int64_t)1 << 30) return 0;
    return ws_bytes_of(in->T, in->V);
}

lsn_status seq_logp_fwd(const lsn_seq_logits* in, float* lse, double* logp, int32_t* count, void* ws, size_t ws_bytes, lsn_stream_t stream) {
    NvtxRange nvtx("seq_logp_fwd");
    lsn_status s = check_in(in, "seq_logp_fwd");
    if (s != LSN_OK) return s;
    LSN_CHECK_ARG((lse || in->T == 0) && logp, "seq_logp_fwd: NULL tensor");
    LSN_CHECK_ARG(!off_by(lse, 4) && !off_by(logp, 8) && !off_by(count, 4), "seq_logp_fwd: tensors must be aligned to their types");
    if ((s = check_ws(in, ws, ws_bytes, "seq_logp_fwd")) != LSN_OK) return s;
    if ((s = check_device()) != LSN_OK) return s;
    Finish f{};
    f.lse = lse;
    f.logp = logp;
    f.count = count;
    return fwd(in, f, false, ws, reinterpret_cast<cudaStream_t>(stream));
}

lsn_status seq_logp_bwd(const lsn_seq_logits* in, const float* lse, const float* dlogp, const int32_t* count, void* dlogits, int64_t ld_d,
                        lsn_stream_t stream) {
    NvtxRange nvtx("seq_logp_bwd");
    lsn_status s = check_in(in, "seq_logp_bwd");
    if (s != LSN_OK) return s;
    if (in->T == 0) return LSN_OK;
    if ((s = check_grad(in, lse, dlogp, count, dlogits, ld_d, "seq_logp_bwd")) != LSN_OK) return s;
    LSN_CHECK_ARG(!off_by(lse, 4) && !off_by(dlogp, 4) && !off_by(count, 4), "seq_logp_bwd: tensors must be aligned to their types");
    if ((s = check_device()) != LSN_OK) return s;
    return bwd(in, lse, dlogp, count, nullptr, dlogits, ld_d, reinterpret_cast<cudaStream_t>(stream));
}

lsn_status preference_loss_fwd(const lsn_seq_logits* in, const double* ref_logp, const lsn_preference* p, float* lse, double* logp, int32_t* count,
                               float* reward, float* loss, float* mean_loss, float* dlogp, void* ws, size_t ws_bytes, lsn_stream_t stream) {
    NvtxRange nvtx("preference_loss_fwd");
    lsn_status s = check_in(in, "preference_loss_fwd");
    if (s != LSN_OK) return s;
    if ((s = check_loss(in, ref_logp, p, lse, logp, count, reward, loss, mean_loss, dlogp, "preference_loss_fwd")) != LSN_OK) return s;
    if ((s = check_ws(in, ws, ws_bytes, "preference_loss_fwd")) != LSN_OK) return s;
    if ((s = check_device()) != LSN_OK) return s;
    return fwd(in, finish_of(in, ref_logp, p, lse, logp, count, reward, loss, mean_loss, dlogp), false, ws, reinterpret_cast<cudaStream_t>(stream));
}

lsn_status preference_loss_fwd_bwd(const lsn_seq_logits* in, const double* ref_logp, const lsn_preference* p, float* lse, double* logp, int32_t* count,
                                   float* reward, float* loss, float* mean_loss, float* dlogp, void* dlogits, int64_t ld_d, void* ws, size_t ws_bytes,
                                   lsn_stream_t stream) {
    NvtxRange nvtx("preference_loss_fwd_bwd");
    const char* who = "preference_loss_fwd_bwd";
    lsn_status s = check_in(in, who);
    if (s != LSN_OK) return s;
    if ((s = check_loss(in, ref_logp, p, lse, logp, count, reward, loss, mean_loss, dlogp, who)) != LSN_OK) return s;
    if ((s = check_grad(in, lse, dlogp, count, dlogits, ld_d, who)) != LSN_OK) return s;
    if ((s = check_ws(in, ws, ws_bytes, who)) != LSN_OK) return s;
    if ((s = check_device()) != LSN_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = fwd(in, finish_of(in, ref_logp, p, lse, logp, count, reward, loss, mean_loss, dlogp), true, ws, st)) != LSN_OK) return s;
    if (in->T == 0) return LSN_OK;
    return bwd(in, lse, dlogp, count, carve(ws, in->T, in->V).coef, dlogits, ld_d, st);
}

}  // extern "C"
