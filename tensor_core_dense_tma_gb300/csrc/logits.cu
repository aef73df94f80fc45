// logits.cu -- operators on the rows of a logits matrix (include/logits.h):
// token log-probabilities with entropy and top alternatives, distillation
// from a teacher's top logits, and the gradients of both.
//
// Mathematics.  With c = log2(e) / temperature and a running maximum m of the
// row's logits z, one pass keeps
//     S = sum 2^u,   U = sum u 2^u,   u = (z - m) c <= 0,
// and a larger maximum m' turns them into S' = 2^d S, U' = 2^d (U + d S) with
// d = (m - m') c.  Then log2 S and m give everything else:
//     lse = m / temperature + ln 2 log2 S,   entropy = ln 2 (log2 S - U / S),
//     log2 p_j = (z_j - m) c - log2 S.
// z - m is formed before the scaling, so rows of the type's lowest value
// cancel exactly instead of overflowing.  m starts at the lowest finite
// number, not at -inf, and u is cut off at -200 (2^-200 is 0 in fp32): a
// masked logit of -inf then adds 0 to both sums without a test, and a NaN
// still reaches them (max.NaN).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "logits.h"
#include "ptx_sm103.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;               // 16-byte loads in flight per thread
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 2048;        // kMaxCluster lists of LOGITS_MAX_TOP fit too
constexpr int kSlack = 64;               // buckets more than wanted that are not worth telling ties apart
constexpr int kStashVectors = 9;         // 16-byte vectors of a thread kept on chip with three CTAs an SM
constexpr int kStashMost = 26;           // and with one
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxExtent = 0x7FFFFFFF - 4096;

// operator and outputs of an instantiation
constexpr int kLogprobs = 0, kDistill = 1;

struct Args {
    const void* z;
    int64_t ld;
    int32_t V;
    int cluster, stash;           // CTAs of a row; vectors of a thread kept in shared memory
    float c, inv_t, t;            // log2(e) / temperature, 1 / temperature, temperature
    const int64_t* tokens;        // [T], or teacher tokens [T][ldt]
    // log-probabilities
    int top;
    const float* g;
    const float* h;
    float* logprob;
    float* entropy;
    float* top_logprob;
    int64_t* top_token;
    // distillation
    int K;
    int64_t ldt;
    const void* teacher;
    int teacher_type;
    const float* w;
    float* loss;
    // both
    float* lse;
    void* dz;
    int64_t ldd;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max that keeps a NaN of x
__device__ __forceinline__ float max_nan(float x, float lo) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
    return y;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t at) { return __uint_as_float(ld_cluster_u32(at)); }

// Element types: kPer elements in a 16-byte vector.
template <typename E>
struct Ele;

template <>
struct Ele<float> {
    static constexpr int kPer = 4;
    static constexpr uint32_t kNegInf = 0xFF800000u;
    __device__ static float load(const float* p) { return *p; }
    template <int N>
    __device__ static float max_of(const uint4 (&q)[N]) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(q[k].x), __uint_as_float(q[k].y)),
                               fmaxf(__uint_as_float(q[k].z), __uint_as_float(q[k].w))));
        return m;
    }
    __device__ static void unpack(const uint4& v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    __device__ static float round(float x) { return x; }
};

template <>
struct Ele<__half> {
    static constexpr int kPer = 8;
    static constexpr uint32_t kNegInf = 0xFC00FC00u;
    template <int N>
    __device__ static float max_of(const uint4 (&q)[N]) {
        uint32_t none = kNegInf;
        __half2 m = *reinterpret_cast<const __half2*>(&none);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const __half2* h = reinterpret_cast<const __half2*>(&q[k]);
            m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        }
        return fmaxf(__half2float(__low2half(m)), __half2float(__high2half(m)));
    }
    __device__ static float load(const __half* p) { return __half2float(*p); }
    __device__ static void unpack(const uint4& v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __half round(float x) { return __float2half_rn(x); }
};

template <>
struct Ele<__nv_bfloat16> {
    static constexpr int kPer = 8;
    static constexpr uint32_t kNegInf = 0xFF80FF80u;
    template <int N>
    __device__ static float max_of(const uint4 (&q)[N]) {
        uint32_t none = kNegInf;
        __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&none);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q[k]);
            m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        }
        return fmaxf(__bfloat162float(__low2bfloat16(m)), __bfloat162float(__high2bfloat16(m)));
    }
    __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ static void unpack(const uint4& v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};

// A row as 16-byte vectors: vector v holds the elements v * kPer - head ..
// + kPer - 1, head the elements between the 16-byte boundary at or below the
// row's start and the start.  Vectors lo..hi-1 lie inside the row and are
// read whole; the (at most two) others are read element by element, so
// nothing outside the row is touched whatever the row's alignment.
template <typename E>
struct Row {
    static constexpr int kPer = Ele<E>::kPer;
    const char* base;    // 16-byte boundary at or below the row's start
    int head, V, lo, hi, nv;

    __device__ Row(const void* z, int64_t offset, int V_) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(z) + static_cast<uintptr_t>(offset) * sizeof(E);
        base = reinterpret_cast<const char*>(a & ~uintptr_t(15));
        head = static_cast<int>((a & 15) / sizeof(E));
        V = V_;
        lo = head ? 1 : 0;
        hi = static_cast<int>((static_cast<int64_t>(head) + V) / kPer);
        nv = static_cast<int>((static_cast<int64_t>(head) + V + kPer - 1) / kPer);
    }
    __device__ const E* element(int j) const { return reinterpret_cast<const E*>(base) + head + j; }
    __device__ int first(int v) const { return v * kPer - head; }    // V < 2^31 - 4096: no overflow
    __device__ uint4 load_whole(int v) const {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(base + static_cast<int64_t>(v) * 16)
                     : "memory");
        return r;
    }
    // vector v's bits, -inf outside the row and from vector `end` on
    __device__ uint4 load_any(int v, int end) const {
        if (v >= lo && v < hi && v < end) return load_whole(v);
        uint4 r = make_uint4(Ele<E>::kNegInf, Ele<E>::kNegInf, Ele<E>::kNegInf, Ele<E>::kNegInf);
        if (v < end) {
            float x[kPer];
            load(v, x);
            r = Ele<E>::pack(x);     // exact: the values are of type E
        }
        return r;
    }
    // elements of vector v as fp32, -inf outside the row
    __device__ void load(int v, float (&x)[kPer]) const {
        if (v >= lo && v < hi) {
            Ele<E>::unpack(load_whole(v), x);
            return;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = first(v) + e;
            x[e] = (j >= 0 && j < V) ? Ele<E>::load(element(j)) : -INFINITY;
        }
    }
};

// Running statistics of a set of logits.
struct Stats {
    float m, S, U;
};

__device__ __forceinline__ Stats empty_stats() { return {-FLT_MAX, 0.f, 0.f}; }

// d is cut off so that an empty side (m = -FLT_MAX, S = U = 0) stays 0.
__device__ __forceinline__ void raise_max(Stats& s, float m, float c) {
    const float d = max_nan((s.m - m) * c, -1e4f);
    const float f = ex2(d);
    s.U = f * fmaf(d, s.S, s.U);
    s.S *= f;
    s.m = m;
}

__device__ __forceinline__ Stats join(Stats a, Stats b, float c) {
    const float m = fmaxf(a.m, b.m);
    raise_max(a, m, c);
    raise_max(b, m, c);
    return {m, a.S + b.S, a.U + b.U};
}

template <bool ENTROPY>
__device__ __forceinline__ void add(Stats& s, float x, float c) {
    const float u = max_nan((x - s.m) * c, -200.f);
    const float e = ex2(u);
    s.S += e;
    if constexpr (ENTROPY) s.U = fmaf(e, u, s.U);
}

__device__ __forceinline__ Stats warp_join(Stats s, float c) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Stats r;
        r.m = __shfl_xor_sync(~0u, s.m, o);
        r.S = __shfl_xor_sync(~0u, s.S, o);
        r.U = __shfl_xor_sync(~0u, s.U, o);
        s = join(s, r, c);
    }
    return s;
}

// log p of a logit z.  Not ln 2 times the base-2 logarithm: scaled by c, a
// finite z near the type's lowest value would overflow to -inf.
__device__ __forceinline__ float log_p(float z, float m, float log2_S, float inv_t) {
    return fmaf(z - m, inv_t, -kLn2 * log2_S);
}

// Order of alternatives: larger logit first, equal ones by the lowest token.
// key = the logit's bits as an ordered integer above the complemented token;
// 0 for what is no alternative (-inf, NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);    // -0 and +0 are equal
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ uint64_t make_key(float x, int j) {
    const uint32_t o = ordered(x);
    return o ? (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~j) : 0ull;
}

__device__ __forceinline__ float teacher_value(const void* p, int type, int64_t at) {
    if (type == GEMM_F32) return static_cast<const float*>(p)[at];
    if (type == GEMM_F16) return __half2float(static_cast<const __half*>(p)[at]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

// What a CTA of a row tells the others: its statistics, and its part of a
// distillation loss, sum P_k (log P_k - (z_k - m) / temperature) and sum P_k
// over the tokens in its segment.
struct Exchange {
    Stats s;
    float A, P;
};

// The keys of a segment's largest logits, in descending order.
struct TopState {
    uint64_t list[LOGITS_MAX_TOP];
    uint64_t cand[kCandidates];
    int bucket[kThreads];
    int buckets, found;
    int count;
};

// `count` = the number of keys in list[0..n-1], the rest 0.
//
// Each thread's logits are a bucket, of which `key` is the largest one's
// ordered value and `batch` the index of its first batch of vectors with it.
// The n-th largest of the bucket maxima is no larger than the n-th largest
// logit (n buckets hold one each that reaches it), so what reaches it is all
// that can be among the n: only the n buckets whose maximum does have to be
// read again, and of 512 buckets of random order few hold two.  It is found
// bit by bit, each a count over the block.  Equal maxima (a mask of the type's
// lowest value) are told apart by their tokens in the same way, or there would
// be as many buckets as there are ties.
template <typename E>
__device__ void select_top(TopState& t, const Row<E>& row, int v0, int v1, uint32_t key, int batch, int n) {
    constexpr int kPer = Ele<E>::kPer;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) t.buckets = t.found = 0;
    for (int i = tid; i < n; i += kThreads) t.list[i] = 0;
    uint32_t thr = 0;
    int reach = kThreads;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = thr | (1u << bit);
        const int cnt = __syncthreads_count(key >= c);
        if (cnt >= n) {
            thr = c;
            reach = cnt;
            if (cnt == n) break;
        }
    }
    int limit = INT_MAX, mine = 0;     // tokens with the threshold's value count up to `limit`
    if (thr == 0) {
        thr = 1;                       // fewer than n buckets hold anything
    } else if (reach > n + kSlack) {
        mine = INT_MAX;
        if (key == thr) {
            for (int k = kUnroll - 1; k >= 0; --k) {
                const int v = v0 + (batch * kUnroll + k) * kThreads + tid;
                if (v >= v1) continue;
                float x[kPer];
                row.load(v, x);
#pragma unroll
                for (int e = kPer - 1; e >= 0; --e)
                    if (ordered(x[e]) == thr) mine = row.first(v) + e;
            }
        }
        const int need = n - __syncthreads_count(key > thr);
        limit = 0;
        for (int bit = 30; bit >= 0; --bit) {
            const int c = limit | (1 << bit);
            if (__syncthreads_count(mine < c) < need) limit = c;
        }
    }
    if (key > thr || (key == thr && mine <= limit)) t.bucket[atomicAdd(&t.buckets, 1)] = tid;
    __syncthreads();
    for (int b = warp; b < t.buckets; b += kWarps) {
        for (int v = v0 + t.bucket[b] + lane * kThreads; v < v1; v += 32 * kThreads) {
            float x[kPer];
            row.load(v, x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t o = ordered(x[e]);
                const int j = row.first(v) + e;
                if (o > thr || (o == thr && j <= limit)) {
                    const int at = atomicAdd(&t.found, 1);
                    if (at < kCandidates) t.cand[at] = (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~j);
                }
            }
        }
    }
    __syncthreads();
    const int found = t.found;
    if (found <= kCandidates) {
        // a key's place is the number of larger ones
        for (int i = tid; i < found; i += kThreads) {
            const uint64_t k = t.cand[i];
            int place = 0;
            for (int o = 0; o < found; ++o) place += t.cand[o] > k;
            if (place < n) t.list[place] = k;
        }
        if (tid == 0) t.count = found < n ? found : n;
        __syncthreads();
        return;
    }
    // Large logits crowded into few buckets: the largest key below the last
    // one found, n times over the segment.
    uint64_t last = ~0ull;
    int count = 0;
    for (; count < n; ++count) {
        uint64_t best = 0;
        for (int v = v0 + tid; v < v1; v += kThreads) {
            float x[kPer];
            row.load(v, x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint64_t k = make_key(x[e], row.first(v) + e);
                if (k < last && k > best) best = k;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(~0u, best, o);
            if (k > best) best = k;
        }
        if (lane == 0) t.cand[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            if (t.cand[w] > best) best = t.cand[w];
        __syncthreads();
        if (!best) break;
        if (tid == 0) t.list[count] = best;
        last = best;
    }
    if (tid == 0) t.count = count;
    __syncthreads();
}

// A row is computed by a cluster of a.cluster CTAs, each of which takes a
// segment of its 16-byte vectors: one pass for the statistics, exchanged
// through distributed shared memory, and (GRAD) a second one that writes the
// gradient from the copy of the segment kept in shared memory (each thread
// reads back its own vectors; what exceeds the copy is read again).
template <typename E, int OP, bool GRAD, bool TOP>
__global__ void __launch_bounds__(kThreads, GRAD ? 3 : 2) rows_kernel(const Args a) {
    constexpr int kPer = Ele<E>::kPer;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Stats warp_stats[kWarps];
    __shared__ Exchange own, all;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row_index = blockIdx.x / a.cluster;
    const int rank = static_cast<int>(blockIdx.x % a.cluster);
    const Row<E> row(a.z, row_index * a.ld, a.V);
    const int per = (row.nv + a.cluster - 1) / a.cluster;
    const int v0 = rank * per, v1 = min(row.nv, v0 + per);
    auto in_segment = [&](int j) {
        const int v = static_cast<int>((static_cast<int64_t>(j) + row.head) / kPer);
        return v >= v0 && v < v1;
    };

    // the given token, or the teacher's: P_k, its log, and the student's logits there
    int token = -1;
    float z_token = 0.f;
    uint4* stash = reinterpret_cast<uint4*>(dyn);
    float* P = reinterpret_cast<float*>(stash + a.stash * kThreads);
    float* logP = P + a.K;
    float* zt = logP + a.K;
    int* tok = reinterpret_cast<int*>(zt + a.K);    // -1: padding, or (for the loss) another CTA's
    if constexpr (OP == kLogprobs) {
        if (a.tokens) {
            const int64_t y = a.tokens[row_index];
            if (y >= 0 && y < a.V) {
                token = static_cast<int>(y);
                z_token = Ele<E>::load(row.element(token));
            }
        }
    } else {
        // softmax over the real entries, by every warp alike
        const int64_t at = row_index * a.ldt;
        float m = -FLT_MAX, total = 0.f;
        for (int k = lane; k < a.K; k += 32) {
            const int64_t y = a.tokens[at + k];
            if (y >= 0 && y < a.V) m = fmaxf(m, teacher_value(a.teacher, a.teacher_type, at + k));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        for (int k = lane; k < a.K; k += 32) {
            const int64_t y = a.tokens[at + k];
            if (y >= 0 && y < a.V) total += ex2((teacher_value(a.teacher, a.teacher_type, at + k) - m) * a.c);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
        const float log2_total = lg2(total);
        for (int k = tid; k < a.K; k += kThreads) {
            const int64_t y = a.tokens[at + k];
            const bool real = y >= 0 && y < a.V && in_segment(static_cast<int>(y));
            tok[k] = real ? static_cast<int>(y) : -1;
            const float l = real ? (teacher_value(a.teacher, a.teacher_type, at + k) - m) * a.c - log2_total : -INFINITY;
            P[k] = real && total != 0.f ? ex2(l) : 0.f;
            logP[k] = l * kLn2;
            zt[k] = real ? Ele<E>::load(row.element(static_cast<int>(y))) : 0.f;
        }
    }

    // statistics
    constexpr bool kEntropy = OP == kLogprobs;
    Stats s = empty_stats();
    float bucket_max = -INFINITY;
    int bucket_batch = 0;
    const int whole_end = min(row.hi, v1);
    for (int b = 0, v = v0 + tid; v < v1; ++b, v += kUnroll * kThreads) {
        uint4 q[kUnroll];
        if (v >= row.lo && v + (kUnroll - 1) * kThreads < whole_end) {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) q[k] = row.load_whole(v + k * kThreads);
        } else {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) q[k] = row.load_any(v + k * kThreads, v1);
        }
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (b * kUnroll + k < a.stash) stash[(b * kUnroll + k) * kThreads + tid] = q[k];
        }
        const float m = Ele<E>::template max_of<kUnroll>(q);
        if constexpr (TOP) {
            if (m > bucket_max) bucket_max = m, bucket_batch = b;
        }
        if (m > s.m) raise_max(s, m, a.c);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            float x[kPer];
            Ele<E>::unpack(q[k], x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) add<kEntropy>(s, x[e], a.c);
        }
    }
    s = warp_join(s, a.c);
    if (lane == 0) warp_stats[warp] = s;
    __syncthreads();
    if (warp == 0) {
        s = warp_stats[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s = join(s, warp_stats[w], a.c);
        float A = 0.f, p = 0.f;
        if constexpr (OP == kDistill) {
            for (int k = lane; k < a.K; k += 32)
                if (!(P[k] <= 0.f)) {
                    A = fmaf(P[k], logP[k] - (zt[k] - s.m) * a.inv_t, A);
                    p += P[k];
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                A += __shfl_xor_sync(~0u, A, o);
                p += __shfl_xor_sync(~0u, p, o);
            }
        }
        if (lane == 0) own = {s, A, p};
    }
    TopState* top = reinterpret_cast<TopState*>(dyn);
    if constexpr (TOP) select_top(*top, row, v0, v1, ordered(bucket_max), bucket_batch, a.top);
    float log2_S = 0.f;
    bool nothing = false;
    __syncwarp();
    if (a.cluster > 1) tcdt::cluster_sync_all();
    // the row's statistics, joined in the order of its segments by every CTA's first warp
    if (warp == 0) {
        Exchange x{empty_stats(), 0.f, 0.f};
        if (a.cluster == 1) {
            __syncwarp();
            x = own;
        } else if (lane < a.cluster) {
            const uint32_t at = tcdt::map_to_cta(tcdt::smem_addr(&own), lane);
            x.s.m = ld_cluster_f32(at), x.s.S = ld_cluster_f32(at + 4), x.s.U = ld_cluster_f32(at + 8);
            x.A = ld_cluster_f32(at + 12), x.P = ld_cluster_f32(at + 16);
        }
        if (a.cluster == 1) {
            s = x.s;
        } else {
            s = empty_stats();
            for (int r = 0; r < a.cluster; ++r) {
                Stats o;
                o.m = __shfl_sync(~0u, x.s.m, r);
                o.S = __shfl_sync(~0u, x.s.S, r);
                o.U = __shfl_sync(~0u, x.s.U, r);
                s = join(s, o, a.c);
            }
        }
        nothing = s.S == 0.f;
        log2_S = lg2(s.S);
        float l = 0.f, p = 0.f;
        if constexpr (OP == kDistill) {
            for (int r = 0; r < a.cluster; ++r) {
                const float A = a.cluster == 1 ? x.A : __shfl_sync(~0u, x.A, r);
                const float Pr = a.cluster == 1 ? x.P : __shfl_sync(~0u, x.P, r);
                const float mr = a.cluster == 1 ? x.s.m : __shfl_sync(~0u, x.s.m, r);
                // a part without teacher tokens has no maximum to shift by
                if (!(Pr <= 0.f)) l += nothing ? A : fmaf(Pr, fmaf(s.m - mr, a.inv_t, kLn2 * log2_S), A);
                p += Pr;
            }
        }
        if (lane == 0) all = {s, l, p};
    }
    __syncthreads();
    s = all.s;
    nothing = s.S == 0.f;
    log2_S = lg2(s.S);
    const float entropy = nothing ? 0.f : kLn2 * (log2_S - s.U / s.S);
    if (rank == 0 && tid == 0) {
        if (a.lse) a.lse[row_index] = nothing ? -INFINITY : fmaf(s.m, a.inv_t, kLn2 * log2_S);
        if constexpr (OP == kLogprobs) {
            if (a.logprob)
                a.logprob[row_index] =
                    token < 0 ? 0.f : nothing ? -INFINITY : log_p(z_token, s.m, log2_S, a.inv_t);
            if (a.entropy) a.entropy[row_index] = entropy;
        } else {
            a.loss[row_index] = a.t * a.t * all.A;
        }
    }

    if constexpr (GRAD) {
        // p_j (ga + gb log2 p_j), and the given tokens' terms put in at the end
        float ga, gb = 0.f, g_token;
        if constexpr (OP == kLogprobs) {
            const float g = token >= 0 && a.g ? a.g[row_index] : 0.f, h = a.h ? a.h[row_index] : 0.f;
            ga = -a.inv_t * fmaf(h, entropy, g);
            gb = -a.inv_t * h * kLn2;
            g_token = a.inv_t * g;
        } else {
            g_token = a.w[row_index] * a.t;
            ga = g_token * all.P;
        }
        E* out = static_cast<E*>(a.dz) + row_index * a.ldd;
        const bool whole = (reinterpret_cast<uintptr_t>(out) & 15) == static_cast<uintptr_t>(row.head) * sizeof(E);
        for (int i = 0, v = v0 + tid; v < v1; ++i, v += kThreads) {
            float x[kPer];
            if (i < a.stash) Ele<E>::unpack(stash[i * kThreads + tid], x);
            else row.load(v, x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float l = max_nan((x[e] - s.m) * a.c - log2_S, -200.f);
                x[e] = nothing ? 0.f : ex2(l) * fmaf(gb, l, ga);
            }
            if (whole && v >= row.lo && v < row.hi) {
                *reinterpret_cast<uint4*>(out + row.first(v)) = Ele<E>::pack(x);
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const int j = row.first(v) + e;
                    if (j >= 0 && j < a.V) out[j] = Ele<E>::round(x[e]);
                }
            }
        }
        __syncthreads();
        if constexpr (OP == kLogprobs) {
            if (tid == 0 && token >= 0 && !nothing && in_segment(token)) {
                const float l = max_nan((z_token - s.m) * a.c - log2_S, -200.f);
                out[token] = Ele<E>::round(fmaf(ex2(l), fmaf(gb, l, ga), g_token));
            }
        } else {
            for (int k = tid; k < a.K; k += kThreads) {
                if (tok[k] < 0 || nothing) continue;
                float p = 0.f;    // a token given twice: each of its entries writes the same sum
                for (int i = 0; i < a.K; ++i)
                    if (tok[i] == tok[k]) p += P[i];
                const float l = max_nan((zt[k] - s.m) * a.c - log2_S, -200.f);
                out[tok[k]] = Ele<E>::round(fmaf(ga, ex2(l), -g_token * p));
            }
        }
    }

    if constexpr (TOP) {
        if (rank == 0) {
            // the segments' lists side by side; a key's place is its place in its own list and the
            // number of larger keys in each of the others
            const int n = a.top, lists = a.cluster;
            int total = 0;
            for (int r = 0; r < lists; ++r)
                total += lists == 1 ? top->count
                                    : static_cast<int>(ld_cluster_u32(
                                          tcdt::map_to_cta(tcdt::smem_addr(&top->count), static_cast<uint32_t>(r))));
            const uint64_t* keys = top->list;
            if (lists > 1) {
                for (int i = tid; i < lists * n; i += kThreads) {
                    const uint32_t at =
                        tcdt::map_to_cta(tcdt::smem_addr(&top->list[i % n]), static_cast<uint32_t>(i / n));
                    top->cand[i] = static_cast<uint64_t>(ld_cluster_u32(at + 4)) << 32 | ld_cluster_u32(at);
                }
                __syncthreads();
                keys = top->cand;
            }
            for (int i = tid; i < lists * n; i += kThreads) {
                const uint64_t k = keys[i];
                if (!k) continue;
                int place = i % n;
                for (int r = 0; r < lists; ++r) {
                    if (r == i / n) continue;
                    int lo = 0, hi = n;    // keys[r * n + 0 .. lo - 1] are larger, from hi on none is
                    while (lo < hi) {
                        const int mid = (lo + hi) / 2;
                        if (keys[r * n + mid] > k) lo = mid + 1;
                        else hi = mid;
                    }
                    place += lo;
                }
                if (place < n) {
                    const float z = from_ordered(static_cast<uint32_t>(k >> 32));
                    a.top_logprob[row_index * n + place] = log_p(z, s.m, log2_S, a.inv_t);
                    a.top_token[row_index * n + place] = static_cast<int64_t>(~static_cast<uint32_t>(k));
                }
            }
            for (int i = total + tid; i < n; i += kThreads) {
                a.top_logprob[row_index * n + i] = -INFINITY;
                a.top_token[row_index * n + i] = -1;
            }
        }
    }
    // nobody leaves while its shared memory may still be read
    __syncwarp();
    if (a.cluster > 1) tcdt::cluster_sync_all();
}

bool float_type(gemm_dtype_t d) { return d == GEMM_F32 || d == GEMM_F16 || d == GEMM_BF16; }
uintptr_t bytes_of(gemm_dtype_t d) { return d == GEMM_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

gemm_status_t check_rows(gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld, float temperature) {
    if (!float_type(dtype) || T < 0 || V < 0 || ld < V) return GEMM_ERR_INVALID_ARG;
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(kLog2e / temperature))
        return GEMM_ERR_INVALID_ARG;
    if (T > kMaxExtent || V > kMaxExtent || ld > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (T > 0 && V > 0 && !logits) return GEMM_ERR_INVALID_ARG;
    if (!aligned(logits, bytes_of(dtype))) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

gemm_status_t check_gradient(gemm_dtype_t dtype, const void* dlogits, int64_t T, int64_t V, int64_t ldd) {
    if (ldd < V) return GEMM_ERR_INVALID_ARG;
    if (ldd > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (T > 0 && V > 0 && !dlogits) return GEMM_ERR_INVALID_ARG;
    return aligned(dlogits, bytes_of(dtype)) ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

// Makes `device` current, once checked to be the kind the kernels are built
// for, and restores the previous one.
struct OnDevice {
    int prev = -1;
    gemm_status_t status = GEMM_OK;
    explicit OnDevice(int device) {
        int count = 0, major = 0, minor = 0;
        if (device < 0) {
            status = GEMM_ERR_INVALID_ARG;
        } else if (cudaGetDeviceCount(&count) != cudaSuccess || count <= 0) {
            status = GEMM_ERR_NO_DEVICE;
        } else if (device >= count) {
            status = GEMM_ERR_INVALID_ARG;
        } else if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
                   cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess) {
            status = GEMM_ERR_CUDA;
        } else if (major != 10 || minor != 3) {
            status = GEMM_ERR_NO_DEVICE;
        } else if (cudaGetDevice(&prev) != cudaSuccess || (prev != device && cudaSetDevice(device) != cudaSuccess)) {
            status = GEMM_ERR_CUDA;
        } else if (prev == device) {
            prev = -1;
        }
        if (status != GEMM_OK) cudaGetLastError();
    }
    ~OnDevice() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// CTAs of a row.  A gradient keeps the row on chip: as many CTAs as it takes
// for kStashVectors vectors a thread.  Beyond that rows are split only while
// there are fewer CTAs than two an SM and every thread of a CTA still has
// loads for a batch.
int cluster_of(int64_t T, int64_t vectors, bool grad, int sms) {
    int c = 1;
    if (grad)
        while (c < kMaxCluster && (vectors + c - 1) / c > static_cast<int64_t>(kStashVectors) * kThreads) c *= 2;
    while (c < kMaxCluster && T * c * 2 <= 2 * sms && vectors / (2 * c) >= kThreads) c *= 2;
    return c;
}

template <typename E, int OP, bool GRAD, bool TOP>
gemm_status_t launch(Args a, int64_t T, int device, cudaStream_t stream) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return GEMM_ERR_CUDA;
    const int64_t vectors = a.V / Ele<E>::kPer + 2;
    a.cluster = cluster_of(T, vectors, GRAD, sms);
    const int64_t each = ((vectors + a.cluster - 1) / a.cluster + kThreads - 1) / kThreads;
    a.stash = GRAD ? static_cast<int>(each < kStashMost ? each : kStashMost) : 0;
    const size_t dyn = TOP ? sizeof(TopState)
                           : static_cast<size_t>(a.stash) * kThreads * 16 +
                                 (OP == kDistill ? static_cast<size_t>(a.K) * 16 : 0);
    auto kernel = rows_kernel<E, OP, GRAD, TOP>;
    if (T * a.cluster > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    if (dyn > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dyn)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(T * a.cluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

template <int OP, bool GRAD, bool TOP>
gemm_status_t launch_type(int device, gemm_dtype_t dtype, const Args& a, int64_t T, void* stream) {
    if (T == 0) return GEMM_OK;
    const OnDevice on(device);
    if (on.status != GEMM_OK) return on.status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GEMM_F32) return launch<float, OP, GRAD, TOP>(a, T, device, s);
    if (dtype == GEMM_F16) return launch<__half, OP, GRAD, TOP>(a, T, device, s);
    return launch<__nv_bfloat16, OP, GRAD, TOP>(a, T, device, s);
}

void fill_rows(Args& a, const void* logits, int64_t V, int64_t ld, float temperature) {
    a.z = logits;
    a.V = static_cast<int32_t>(V);
    a.ld = ld;
    a.t = temperature;
    a.inv_t = 1.0f / temperature;
    a.c = kLog2e / temperature;
}

gemm_status_t check_distill(gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld, int64_t K,
                            const int64_t* teacher_tokens, gemm_dtype_t teacher_dtype, const void* teacher_logits,
                            int64_t ldt, float temperature, const float* loss, const float* lse) {
    const gemm_status_t st = check_rows(dtype, logits, T, V, ld, temperature);
    if (st != GEMM_OK) return st;
    if (K < 0 || K > LOGITS_MAX_TEACHER || ldt < K || !float_type(teacher_dtype)) return GEMM_ERR_INVALID_ARG;
    if (ldt > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (T > 0 && (!loss || (K > 0 && (!teacher_tokens || !teacher_logits)))) return GEMM_ERR_INVALID_ARG;
    if (!aligned(teacher_tokens, 8) || !aligned(teacher_logits, bytes_of(teacher_dtype)) || !aligned(loss, 4) ||
        !aligned(lse, 4))
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

void fill_distill(Args& a, int64_t K, const int64_t* teacher_tokens, gemm_dtype_t teacher_dtype,
                  const void* teacher_logits, int64_t ldt, float* loss, float* lse) {
    a.K = static_cast<int>(K);
    a.tokens = teacher_tokens;
    a.teacher = teacher_logits;
    a.teacher_type = teacher_dtype;
    a.ldt = ldt;
    a.loss = loss;
    a.lse = lse;
}

}  // namespace

extern "C" {

gemm_status_t logits_logprobs(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                              const int64_t* tokens, float temperature, int top, float* logprob, float* entropy,
                              float* lse, float* top_logprob, int64_t* top_token, void* stream) {
    const gemm_status_t st = check_rows(dtype, logits, T, V, ld, temperature);
    if (st != GEMM_OK) return st;
    if (top < 0 || top > LOGITS_MAX_TOP) return GEMM_ERR_INVALID_ARG;
    if (T > 0 && top > 0 && (!top_logprob || !top_token)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(tokens, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
        !aligned(top_logprob, 4) || !aligned(top_token, 8))
        return GEMM_ERR_MISALIGNED;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    a.tokens = tokens;
    a.top = top;
    a.logprob = tokens ? logprob : nullptr;
    a.entropy = entropy;
    a.lse = lse;
    a.top_logprob = top_logprob;
    a.top_token = top_token;
    return top > 0 ? launch_type<kLogprobs, false, true>(device, dtype, a, T, stream)
                   : launch_type<kLogprobs, false, false>(device, dtype, a, T, stream);
}

gemm_status_t logits_logprobs_grad(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V,
                                   int64_t ld, const int64_t* tokens, float temperature, const float* g,
                                   const float* h, float* logprob, float* entropy, float* lse, void* dlogits,
                                   int64_t ldd, void* stream) {
    gemm_status_t st = check_rows(dtype, logits, T, V, ld, temperature);
    if (st == GEMM_OK) st = check_gradient(dtype, dlogits, T, V, ldd);
    if (st != GEMM_OK) return st;
    if (T > 0 && g && !tokens) return GEMM_ERR_INVALID_ARG;
    if (!aligned(tokens, 8) || !aligned(g, 4) || !aligned(h, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(lse, 4))
        return GEMM_ERR_MISALIGNED;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    a.tokens = tokens;
    a.g = g;
    a.h = h;
    a.logprob = tokens ? logprob : nullptr;
    a.entropy = entropy;
    a.lse = lse;
    a.dz = dlogits;
    a.ldd = ldd;
    return launch_type<kLogprobs, true, false>(device, dtype, a, T, stream);
}

gemm_status_t logits_distill(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                             int64_t K, const int64_t* teacher_tokens, gemm_dtype_t teacher_dtype,
                             const void* teacher_logits, int64_t ldt, float temperature, float* loss, float* lse,
                             void* stream) {
    const gemm_status_t st = check_distill(dtype, logits, T, V, ld, K, teacher_tokens, teacher_dtype, teacher_logits,
                                           ldt, temperature, loss, lse);
    if (st != GEMM_OK) return st;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_distill(a, K, teacher_tokens, teacher_dtype, teacher_logits, ldt, loss, lse);
    return launch_type<kDistill, false, false>(device, dtype, a, T, stream);
}

gemm_status_t logits_distill_grad(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V,
                                  int64_t ld, int64_t K, const int64_t* teacher_tokens, gemm_dtype_t teacher_dtype,
                                  const void* teacher_logits, int64_t ldt, float temperature, const float* w,
                                  float* loss, float* lse, void* dlogits, int64_t ldd, void* stream) {
    gemm_status_t st = check_distill(dtype, logits, T, V, ld, K, teacher_tokens, teacher_dtype, teacher_logits, ldt,
                                     temperature, loss, lse);
    if (st == GEMM_OK) st = check_gradient(dtype, dlogits, T, V, ldd);
    if (st != GEMM_OK) return st;
    if (T > 0 && !w) return GEMM_ERR_INVALID_ARG;
    if (!aligned(w, 4)) return GEMM_ERR_MISALIGNED;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_distill(a, K, teacher_tokens, teacher_dtype, teacher_logits, ldt, loss, lse);
    a.w = w;
    a.dz = dlogits;
    a.ldd = ldd;
    return launch_type<kDistill, true, false>(device, dtype, a, T, stream);
}

}  // extern "C"
