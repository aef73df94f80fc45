// logits.cu -- operators on the rows of a logits matrix (include/logits.h):
// token log-probabilities with entropy and top alternatives, distillation
// from a teacher's top logits, a clipped policy loss, a preference loss of paired
// sequences, and the gradients of the four.
//
// Mathematics.  With c = log2(e) / temperature and a running maximum m of the
// row's logits z, one pass keeps
//     S = sum 2^u,   U = sum u 2^u,   u = (z - m) c <= 0,
// and a larger maximum m' turns them into S' = 2^d S, U' = 2^d (U + d S) with
// d = (m - m') c.  Then log2 S and m give everything else:
//     lse = m / temperature + ln 2 log2 S,   entropy = ln 2 (log2 S - U / S),
//     log2 p_j = (z_j - m) c - log2 S.
// z - m is formed before the scaling: it is exact near the maximum, where p
// is large, and rows of the type's lowest value cancel instead of overflowing
// (z c - m c in one multiply-add saved nothing that showed).  m starts at the
// lowest finite number, not at -inf: a masked logit of -inf then adds
// 2^-inf = 0 without a test.  Where u or log2 p is also a factor it is cut off
// at -200 (2^-200 is 0 in fp32, and 0 times -200 is 0, where 0 times -inf is
// not); a NaN still reaches the sums (max.NaN).  S = 0 means that every logit
// is -inf.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "logits.h"
#include "ptx_sm103.cuh"

namespace {

constexpr int kThreads = 256;            // that compute; one more warp starts the copies
// CTAs an SM (4096 x 131072 bf16 with gradient: 3 CTAs 372 us, 4 CTAs 408, 5 CTAs
// 531; 64 alternatives: 4 CTAs 287 us, 3 CTAs 334, 5 CTAs 353 in an earlier form).
constexpr int ctas_of(bool grad) { return grad ? 3 : 4; }
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 1024 / kThreads; // 16-byte vectors of a thread in a chunk
constexpr int kChunk = kUnroll * kThreads;   // vectors of an asynchronous copy: 16 KB
constexpr int kSlotsMost = 12;           // of the ring
constexpr int kBlock = kThreads + 32;
// A copy is waited for this long, other CTAs' statistics twice as long (a CTA that
// gave up on a copy still brings its own), a slot of the ring three times.
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;        // kMaxCluster lists of LOGITS_MAX_TOP fit too
constexpr int kSlack = 64;               // buckets more than wanted that are not worth telling ties apart
constexpr int64_t kInFlight = 64 << 20, kInFlightWhole = 80 << 20;   // bytes of logits that a gradient works on at once
constexpr int64_t kSharedOfSm = 228 * 1024;
constexpr int kDynamicMost = 225 * 1024;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxExtent = 0x7FFFFFFF - 4096;

// operator and outputs of an instantiation
constexpr int kLogprobs = 0, kDistill = 1, kPolicy = 2, kScore = 3;   // kScore: the rows of a preference loss

struct __align__(16) RowState {
    float m, log2_S, g, unused;       // log2_S is +inf where the row's gradient is 0 whatever g is
};

struct Args {
    const void* z;
    int64_t ld;
    int32_t V;
    int64_t T;
    int cluster, rows, slots;     // CTAs of a row, rows of a CTA, chunks of the ring
    int per;                      // vectors of a segment
    float c, inv_t, t;            // log2(e) / temperature, 1 / temperature, temperature
    float c_rest;                 // what c lacks, as a part of it (see log_sum)
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
    const float* w;      // and of a policy loss
    float* loss;
    // policy loss: e^(logprob - old) is clipped to lo..hi
    const float* old_logprob;
    const float* advantage;
    const float* ref_logprob;
    float* kl;
    float lo, hi, kl_coef, bonus;
    // preference loss: (maximum, log2 S, gradient of the loss for logprob) of each row
    RowState* state;
    // all
    float* lse;
    void* dz;
    int64_t ldd;
#ifdef TCDT_FAULT_INJECTION
    // test builds only: the limit above; in CTAs of rank fi_rank of a row (-1: all) the copy that is not
    // started, the chunk that the warps of a mask do not wait for, and whether statistics are kept back
    uint64_t fi_limit_ns;
    int64_t fi_skip_copy, fi_late_chunk;
    uint32_t fi_late_warps;
    int fi_silent, fi_rank;
    __device__ bool fi_here(int rank) const { return fi_rank < 0 || fi_rank == rank; }
    __device__ uint64_t limit_ns() const { return fi_limit_ns; }
#else
    __device__ static constexpr uint64_t limit_ns() { return kWaitLimitNs; }
#endif
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

// Asynchronous copy of whole 16-byte units into shared memory, counted on an mbarrier.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Waits for a phase of a barrier; false once the limit has passed.
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    if (tcdt::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tcdt::globaltimer_ns();
    while (!tcdt::mbar_try_wait(bar, parity))
        if (tcdt::globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

// The same for a slot of the ring, given up as soon as a computing thread has
// given up on a copy (the slot may then never be given back).
__device__ __forceinline__ bool wait_slot(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* gave_up) {
    if (tcdt::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tcdt::globaltimer_ns();
    while (!tcdt::mbar_try_wait(bar, parity))
        if (*gave_up || tcdt::globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

// Two 32-bit values as a register pair.
__device__ __forceinline__ uint64_t bit_pair(uint32_t x, uint32_t y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x), "r"(y));
    return v;
}

// Barriers of the computing threads.
__device__ __forceinline__ void sync_threads() { tcdt::named_bar_sync(1, kThreads); }
__device__ __forceinline__ int sync_count(bool p) {
    int n;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.popc.aligned.u32 %0, 1, %2, q;\n\t}"
                 : "=r"(n)
                 : "r"(p ? 1u : 0u), "n"(kThreads)
                 : "memory");
    return n;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// wait_limited for arrivals from other CTAs of the cluster.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    if (tcdt::mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = tcdt::globaltimer_ns();
    while (!tcdt::mbar_try_wait_cluster(bar, parity))
        if (tcdt::globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

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
    __device__ static void pairs(const uint4& v, uint64_t (&x)[2]) {
        x[0] = bit_pair(v.x, v.y), x[1] = bit_pair(v.z, v.w);
    }
    __device__ static uint4 pack_pairs(const uint64_t (&x)[2]) {
        uint4 r;
        asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(x[0]));
        asm("mov.b64 {%0, %1}, %2;" : "=r"(r.z), "=r"(r.w) : "l"(x[1]));
        return r;
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
    __device__ static void pairs(const uint4& v, uint64_t (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 a, b;\n\t.reg .f32 l, h;\n\tmov.b32 {a, b}, %1;\n\t"
                "cvt.f32.f16 l, a;\n\tcvt.f32.f16 h, b;\n\tmov.b64 %0, {l, h};\n\t}"
                : "=l"(x[i])
                : "r"(w[i]));
    }
    __device__ static uint4 pack_pairs(const uint64_t (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .f32 l, h;\n\tmov.b64 {l, h}, %1;\n\tcvt.rn.f16x2.f32 %0, h, l;\n\t}" : "=r"(w[i]) : "l"(x[i]));
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
    __device__ static void pairs(const uint4& v, uint64_t (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = bit_pair(w[i] << 16, w[i] & 0xFFFF0000u);
    }
    __device__ static uint4 pack_pairs(const uint64_t (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .f32 l, h;\n\tmov.b64 {l, h}, %1;\n\tcvt.rn.bf16x2.f32 %0, h, l;\n\t}" : "=r"(w[i]) : "l"(x[i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};

// A CTA's part of a row: `n` of the 16-byte vectors that lie whole between
// the 16-byte boundaries of the row, and, with the row's first and last CTA,
// the fewer than kPer elements before the first and after the last boundary
// (thread i has the i-th of each).  Nothing outside the row is touched,
// whatever its alignment.
template <typename E>
struct Segment {
    static constexpr int kPer = Ele<E>::kPer;
    const E* row;
    const uint4* vec;       // the segment's first vector
    int head, tail;         // elements before the first and from the last boundary on, where they are this CTA's
    int first, after;       // token of vec's first element; of the first one of the tail
    int n;

    __device__ __forceinline__ Segment(const void* z, int64_t offset, int V, int rank, int cluster, int per) {
        row = static_cast<const E*>(z) + offset;
        const int skip = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<int>(sizeof(E));
        const int lead = min(skip, V);
        const int whole = static_cast<int>(static_cast<unsigned>(V - lead) / kPer);
        const int v0 = min(rank * per, whole);
        n = min(per, whole - v0);
        first = lead + v0 * kPer;
        vec = reinterpret_cast<const uint4*>(row + first);
        after = lead + whole * kPer;
        head = rank == 0 ? lead : 0;
        tail = rank == cluster - 1 ? V - after : 0;
    }
    __device__ __forceinline__ int chunks() const { return static_cast<int>(static_cast<unsigned>(n + kChunk - 1) / kChunk); }
    __device__ __forceinline__ bool holds(int j) const {
        return (j >= first && j < first + n * kPer) || j < head || (tail > 0 && j >= after);
    }
    __device__ __forceinline__ uint4 load(int v) const {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(vec + v)
                     : "memory");
        return r;
    }
};

// Running statistics of a set of logits.
struct Stats {
    float m, S, U;
};

__device__ __forceinline__ Stats empty_stats() { return {-FLT_MAX, 0.f, 0.f}; }

// d is cut off so that an empty side (S = U = 0) stays 0.
__device__ __forceinline__ void raise_max(Stats& s, float m, float c) {
    const float d = max_nan((s.m - m) * c, -1e4f);
    const float f = ex2(d);
    s.U = f * fmaf(d, s.S, s.U);
    s.S *= f;
    s.m = m;
}

// What ex2.approx lacks on average, relatively: measured over all floats of a range, 4.95e-8 to
// 5.06e-8 in each of -10 .. -9 to -2 .. -1, 2.5e-8 in -1 .. -1/2, 2.0e-8 in -1/4 .. 0, nothing at 0.
constexpr float kEx2Lacks = 5.0e-8f;

// raise_max for a sum that is joined with others.  Every value goes through several exponentials on its
// way into the row's sum, its own and those that scale it to the maximum of the warp, the block and the
// cluster, all off to one side: what the factor lacks (and `more`) is put back, before the products are
// rounded (afterwards, below half a unit, it would be lost); in U too, which the entropy divides by S.
__device__ __forceinline__ void raise_joined(Stats& s, float m, float c, float more) {
    const float S = s.S, d = max_nan((s.m - m) * c, -1e4f), f = ex2(d);
    const float U = fmaf(d, S, s.U), lacks = fmaf(fminf(-d, 1.f), kEx2Lacks, more);
    s.U = fmaf(U, f, U * f * lacks);
    s.S = fmaf(S, f, S * f * lacks);
    s.m = m;
}

// Two floats in a register pair, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t a) {
    uint64_t v;
    asm("{\n\t.reg .f32 l, h;\n\tmov.b64 {l, h}, %1;\n\tex2.approx.ftz.f32 l, l;\n\tex2.approx.ftz.f32 h, h;\n\t"
        "mov.b64 %0, {l, h};\n\t}"
        : "=l"(v)
        : "l"(a));
    return v;
}
// max_nan of both
__device__ __forceinline__ uint64_t max_nan2(uint64_t a, float lo) {
    uint64_t v;
    asm("{\n\t.reg .f32 l, h;\n\tmov.b64 {l, h}, %1;\n\tmax.NaN.f32 l, l, %2;\n\tmax.NaN.f32 h, h, %2;\n\t"
        "mov.b64 %0, {l, h};\n\t}"
        : "=l"(v)
        : "l"(a), "f"(lo));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// Of all lanes of a warp, for all of them: the maximum first (one
// instruction), so that each lane's sums are scaled once and then added.
__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

__device__ __forceinline__ float warp_sum(float x, int width) {
    for (int o = width / 2; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

template <bool ENTROPY>
__device__ __forceinline__ Stats warp_join(Stats s, int width, float c, float more = 0.f) {
    // (of a distillation's sums no one adds up thousands)
    if constexpr (ENTROPY) raise_joined(s, warp_max(s.m), c, more);
    else raise_max(s, warp_max(s.m), c);
    s.S = warp_sum(s.S, width);
    if constexpr (ENTROPY) s.U = warp_sum(s.U, width);
    return s;
}

// The logarithm of a row's sum S of e^((z - m) / t), in two parts.  Callers add up thousands of
// log-probabilities, where an error to one side adds up and one to either side does not:
//  * lg2.approx is off by up to 2^-22 to one side for long stretches.  So S = 2^e f, f in
//    3/4 .. 3/2, and ln 2 is split after Cody and Waite: e times its first 12 bits is
//    exact, logf(f) and what is left are below 0.41, where a unit is 2^-25;
//  * c = log2(e) / t, rounded to fp32, is a part c_rest too small, the same in every
//    exponent: S lacks c_rest ln 2 times U, the sum of 2^u u.
struct LogSum {
    float hi, lo;
};
constexpr float kLn2First = 2839.f / 4096.f, kLn2Rest = static_cast<float>(0.6931471805599453 - 2839.0 / 4096.0);

__device__ __forceinline__ LogSum log_sum(float S, float U, float c_rest) {
    const int bits = __float_as_int(S), e = (bits - 0x3F400000) >> 23;
    const float f = __int_as_float(bits - e * (1 << 23)), n = static_cast<float>(e);
    return {n * kLn2First, logf(f) + fmaf(n, kLn2Rest, c_rest * kLn2 * __fdividef(U, S)) + (S - S)};      // a NaN stays one
}

// log p of a logit z.  Not ln 2 times the base-2 logarithm: scaled by c, a
// finite z near the type's lowest value would overflow to -inf.
__device__ __forceinline__ float log_p(float z, float m, const LogSum& l, float t, float inv_t) {
    const float d = z - m, q = d * inv_t;
    // what q lacks (inv_t's own rounding is the same in all rows); the logarithm is put together first,
    // as its last bits differ from row to row and those of 16-bit logits over t hardly do
    const float rest = isinf(q) ? 0.f : fmaf(-q, t, d) * inv_t;
    return q - (l.hi + (l.lo - rest));
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

// The policy operator (4096 x 131072 bf16 with gradient 388 us, 0.83 of the copy rate; 2048 x 65537
// without entropy bonus, a quarter of the rows unread, 84, with the bonus's arithmetic 88).
// Policy loss of a row without its entropy bonus, its KL term and the loss's
// derivative with respect to the log-probability.  With d = ref - logprob the
// KL term is e^d - 1 - d >= 0, from expm1: for small d it is d^2 / 2, of which
// e^d in fp32 would keep nothing.  A NaN is not lost in the minimum.
struct PolicyLoss {
    float loss, kl, slope, logprob;
};

__device__ __forceinline__ PolicyLoss policy_loss(const Args& a, float logprob, float A, float old, float ref) {
    const float x = logprob - old, ratio = expf(x);
    const float bounded = fminf(fmaxf(ratio, a.lo), a.hi) * A;
    float free = ratio * A;
    if (ratio == INFINITY && x != INFINITY) {      // beyond fp32, which the product need not be
        const float half = expf(0.5f * x);
        free = A == 0.f ? 0.f : half * A * half;
    }
    PolicyLoss l{-bounded, 0.f, 0.f, logprob};
    if (!(free > bounded)) l.loss = l.slope = -free;
    if (a.ref_logprob) {
        const float d = ref - logprob, e = expm1f(d);
        l.kl = e == INFINITY ? e : e - d;
        if (a.kl_coef != 0.f) l.loss = fmaf(a.kl_coef, l.kl, l.loss), l.slope = fmaf(-a.kl_coef, e, l.slope);
    }
    return l;
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
    uint32_t key[kThreads];
    int narrow[kThreads], wide[kThreads], batch[kThreads];
    int narrows, wides, found;
    int count;                           // of keys in the list
    uint32_t thr;
    int reach;
};

// Into t.list[0..n-1] and t.count; the rest of the list is 0.
//
// Each thread's logits are a bucket, of which `key` is the largest one's
// ordered value and `batch` the first chunk of vectors that has it (kInHead,
// kInTail: the thread's element before or after the vectors).
// The n-th largest of the bucket maxima is no larger than the n-th largest
// logit (n buckets hold one each that reaches it), so what reaches it is all
// that can be among the n: only the buckets whose maximum does have to be read
// again, and most of them (the narrow ones, whose second best chunk does not
// reach it) in that chunk only.  It is found bit by bit, by one warp that holds
// all the maxima.  Equal maxima (a mask of
// the type's lowest value) are told apart by their tokens in the same way, or
// there would be as many buckets as there are ties.
constexpr uint32_t kOrderedLowest = 0x00800000u;     // ordered(-FLT_MAX)
constexpr int kInHead = -1, kInTail = INT_MAX;

template <typename E>
__device__ __forceinline__ void select_top(TopState& t, const Segment<E>& seg, uint32_t key, int batch, float second,
                                           int n) {
    constexpr int kPer = Ele<E>::kPer;
    uint64_t* list = t.list;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) t.narrows = t.wides = t.found = 0;
    for (int i = tid; i < n; i += kThreads) list[i] = 0;
    t.key[tid] = key;
    sync_threads();
    if (warp == 0) {
        uint32_t k[kThreads / 32];
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) k[i] = t.key[i * 32 + lane];
        uint32_t thr = 0;
        int reach = kThreads;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t c = thr | (1u << bit);
            int cnt = 0;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) cnt += k[i] >= c;
            cnt = __reduce_add_sync(~0u, cnt);
            if (cnt >= n) {
                thr = c;
                reach = cnt;
                if (cnt == n) break;
            }
        }
        if (lane == 0) t.thr = thr, t.reach = reach;
    }
    sync_threads();
    uint32_t thr = t.thr;
    const int reach = t.reach;
    int limit = INT_MAX, mine = 0;     // tokens with the threshold's value count up to `limit`
    if (thr == 0) {
        thr = 1;                       // fewer than n buckets hold anything
    } else if (reach > n + kSlack) {
        mine = INT_MAX;
        if (key == thr) {
            if (batch == kInHead) mine = tid;
            else if (batch == kInTail) mine = seg.after + tid;
            else
                for (int k = kUnroll - 1; k >= 0; --k) {
                    const int v = (batch * kUnroll + k) * kThreads + tid;
                    if (v >= seg.n) continue;
                    float x[kPer];
                    Ele<E>::unpack(seg.load(v), x);
#pragma unroll
                    for (int e = kPer - 1; e >= 0; --e)
                        if (ordered(x[e]) == thr) mine = seg.first + v * kPer + e;
                }
        }
        const int need = n - sync_count(key > thr);
        limit = 0;
        for (int bit = 30; bit >= 0; --bit) {
            const int c = limit | (1 << bit);
            if (sync_count(mine < c) < need) limit = c;
        }
    }
    const float thr_value = thr < kOrderedLowest ? -INFINITY : from_ordered(thr);    // below: no number
    if (key > thr || (key == thr && mine <= limit)) {
        const bool beside = tid < seg.head || tid < seg.tail;
        if (second >= thr_value || beside) t.wide[atomicAdd(&t.wides, 1)] = tid;
        else t.narrow[atomicAdd(&t.narrows, 1)] = tid;
        t.batch[tid] = batch;
    }
    sync_threads();
    auto offer = [&](float x, int j) {
        if (!(x >= thr_value)) return;
        const uint32_t o = ordered(x);
        if (o > thr || (o == thr && j <= limit)) {
            const int at = atomicAdd(&t.found, 1);
            if (at < kCandidates) t.cand[at] = (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~j);
        }
    };
    auto look = [&](int v) {
        const uint4 q[1] = {seg.load(v)};
        if (!(Ele<E>::template max_of<1>(q) >= thr_value)) return;
        float x[kPer];
        Ele<E>::unpack(q[0], x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) offer(x[e], seg.first + v * kPer + e);
    };
    for (int i = tid; i < t.narrows * kUnroll; i += kThreads) {
        const int bucket = t.narrow[i / kUnroll];
        const int v = (t.batch[bucket] * kUnroll + i % kUnroll) * kThreads + bucket;
        if (v < seg.n) look(v);
    }
    for (int b = warp; b < t.wides; b += kWarps) {
        const int bucket = t.wide[b];
        for (int v = bucket + lane * kThreads; v < seg.n; v += 32 * kThreads) look(v);
        if (lane == 0 && bucket < seg.head) offer(Ele<E>::load(seg.row + bucket), bucket);
        if (lane == 1 && bucket < seg.tail) offer(Ele<E>::load(seg.row + seg.after + bucket), seg.after + bucket);
    }
    sync_threads();
    const int found = t.found;
    if (found <= kCandidates) {
        // a key's place is the number of larger ones
        for (int i = tid; i < found; i += kThreads) {
            const uint64_t k = t.cand[i];
            int place = 0;
            for (int o = 0; o < found; ++o) place += t.cand[o] > k;
            if (place < n) list[place] = k;
        }
        if (tid == 0) t.count = found < n ? found : n;
        sync_threads();
        return;
    }
    // Large logits crowded into few buckets: the largest key below the last
    // one found, n times over the segment.
    uint64_t last = ~0ull;
    int count = 0;
    for (; count < n; ++count) {
        uint64_t best = 0;
        auto take = [&](float x, int j) {
            const uint64_t k = make_key(x, j);
            if (k < last && k > best) best = k;
        };
        for (int v = tid; v < seg.n; v += kThreads) {
            float x[kPer];
            Ele<E>::unpack(seg.load(v), x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) take(x[e], seg.first + v * kPer + e);
        }
        if (tid < seg.head) take(Ele<E>::load(seg.row + tid), tid);
        if (tid < seg.tail) take(Ele<E>::load(seg.row + seg.after + tid), seg.after + tid);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(~0u, best, o);
            if (k > best) best = k;
        }
        if (lane == 0) t.cand[warp] = best;
        sync_threads();
        for (int w = 0; w < kWarps; ++w)
            if (t.cand[w] > best) best = t.cand[w];
        sync_threads();
        if (!best) break;
        if (tid == 0) list[count] = best;
        last = best;
    }
    if (tid == 0) t.count = count;
    sync_threads();
}

// A cluster of a.cluster CTAs computes a row, a segment each, or one CTA a.rows
// rows one after another (a.rows is 1 in clusters).  A segment comes in chunks
// through a ring in shared memory: one warp starts asynchronous copies, into a slot as soon as all
// computing warps have given it back, and so runs ahead into the next row
// while this one's sums are joined, its alternatives selected or its gradient
// written.  The gradient takes the last chunks first, where the statistics left
// them in the ring, and the others are copied in again, from L2: the host
// splits rows only so far that those in flight fit there, as the CTAs of a row
// wait for one another (4096 x 131072 bf16 kept in the ring whole, in clusters of
// four: 454 us, in clusters of two 375; gradient stores are marked streaming to
// leave L2 to the logits).  The segments' statistics go from each CTA into
// every other one's shared memory, counted by an mbarrier.
// A thread whose copy has not arrived in time waits for none again: it reads
// its vectors of that chunk and all later ones from memory.  Its warp, if it is
// lane 0, gives no slot back any more, as it no longer knows that one was filled:
// what is in the ring then stays there for the threads that did see it arrive,
// and the warp that copies, which waits for every warp, starts no more copies.
// Statistics that have not arrived make the row NaN, and its alternatives none.
template <typename E, int OP, bool GRAD, bool TOP>
__global__ void __launch_bounds__(kBlock, ctas_of(GRAD)) rows_kernel(const Args a) {
    constexpr int kPer = Ele<E>::kPer;
    constexpr bool kEntropy = OP != kDistill;
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ Stats warp_stats[kWarps];
    __shared__ Exchange inbox[kMaxCluster], all;
    __shared__ PolicyLoss row_policy;
    __shared__ bool heard;                               // of every CTA of the row
    __shared__ volatile int gave_up;                     // on a copy
    __shared__ __align__(8) uint64_t full_bar[kSlotsMost], empty_bar[kSlotsMost], inbox_bar;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x % a.cluster);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / a.cluster) * a.rows;
    const int64_t row1 = min(a.T, row0 + a.rows);
    uint4* ring = reinterpret_cast<uint4*>(dyn);
    const uint32_t full = tcdt::smem_addr(full_bar), empty = tcdt::smem_addr(empty_bar);
    // the teacher's entries: tokens (-1: padding, or another CTA's; -2 up to a multiple of 4), P_k (before
    // that its logit), the student's logits there
    const int K4 = (a.K + 3) & ~3;
    int* tok = reinterpret_cast<int*>(ring + a.slots * kChunk);
    float* P = reinterpret_cast<float*>(tok + K4);
    float* zt = P + K4;
    TopState* top = reinterpret_cast<TopState*>(ring + a.slots * kChunk);

    // Rows of a policy or preference loss without a token are not read: all of theirs
    // is 0.  Those of weight 0 have a gradient of zeros, whatever they hold.
    auto unread = [&](int64_t r) {
        if constexpr (OP != kPolicy && OP != kScore) return false;
        const int64_t y = a.tokens[r];
        return y < 0 || y >= a.V;
    };
    auto weightless = [&](int64_t r) {
        if constexpr (OP != kPolicy) return false;
        return a.w[r] == 0.f;
    };

    if (tid == 0) {
        for (int i = 0; i < a.slots; ++i) {
            tcdt::mbar_init(full + 8 * i, 1);
            tcdt::mbar_init(empty + 8 * i, kWarps);
        }
        tcdt::mbar_init(tcdt::smem_addr(&inbox_bar), static_cast<uint32_t>(a.cluster));
        gave_up = 0;
        tcdt::fence_mbar_init();
    }
    if (OP == kDistill && tid < K4 - a.K) tok[a.K + tid] = -2;
    __syncthreads();
    if (a.cluster > 1) tcdt::cluster_sync_all();

    if (warp == kWarps) {
        // Chunk number q of this CTA goes to slot q % a.slots.
        if (lane == 0) {
            int slot = 0, started = 0;
            uint32_t parity = 1;            // an empty ring's slots count as given back
            bool ok = true;
            for (int64_t r = row0; ok && r < row1; ++r) {
                if (unread(r)) continue;
                const Segment<E> seg(a.z, r * a.ld, a.V, rank, a.cluster, a.per);
                const int chunks = seg.chunks(), again = GRAD && !weightless(r) ? chunks - min(chunks, a.slots) : 0;
                for (int i = 0; i < chunks + again; ++i) {
                    const int from = (i < chunks ? i : i - chunks) * kChunk;
                    ok = wait_slot(empty + 8 * slot, parity, 3 * a.limit_ns(), &gave_up);
                    if (!ok) break;
                    const uint32_t bytes = static_cast<uint32_t>(min(kChunk, seg.n - from)) * 16u;
                    tcdt::mbar_arrive_expect_tx(full + 8 * slot, bytes);
#ifdef TCDT_FAULT_INJECTION
                    if (!(started == a.fi_skip_copy && a.fi_here(rank)))
#endif
                        copy_bulk(tcdt::smem_addr(ring + slot * kChunk), seg.vec + from, bytes, full + 8 * slot);
                    ++started;
                    if (++slot == a.slots) slot = 0, parity ^= 1u;
                }
            }
            // a copy must not land in another CTA's memory
            for (int i = 0; i < a.slots && i < started; ++i)
                wait_limited(full + 8 * i, static_cast<uint32_t>((started - 1 - i) / a.slots) & 1u, a.limit_ns());
        }
        __syncwarp();
        if (a.cluster > 1) tcdt::cluster_sync_all();
        return;
    }

    int slot = 0;
    uint32_t parity = 0;
    bool late = false;
#ifdef TCDT_FAULT_INJECTION
    int64_t taken = 0;
#endif
    // the thread's vectors of a chunk, -inf beyond the segment's end; true if all are inside
    auto take = [&](const Segment<E>& seg, int chunk, bool give_back, uint4 (&q)[kUnroll]) {
#ifdef TCDT_FAULT_INJECTION
        if (taken++ == a.fi_late_chunk && a.fi_here(rank) && (a.fi_late_warps >> warp & 1u)) late = true;
#endif
        if (!late && !wait_limited(full + 8 * slot, parity, a.limit_ns())) late = true, gave_up = 1;
        const uint4* at = ring + slot * kChunk + tid;
        const bool inside = !late && (chunk + 1) * kChunk <= seg.n;
        if (inside) {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) q[k] = at[k * kThreads];
        } else {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int v = chunk * kChunk + k * kThreads + tid;
                if (v < seg.n) q[k] = late ? seg.load(v) : at[k * kThreads];
                else q[k] = make_uint4(Ele<E>::kNegInf, Ele<E>::kNegInf, Ele<E>::kNegInf, Ele<E>::kNegInf);
            }
        }
        if (give_back) {
            __syncwarp();
            if (lane == 0 && !late) tcdt::mbar_arrive(empty + 8 * slot);
        }
        if (++slot == a.slots) slot = 0, parity ^= 1u;
        return inside;
    };

    for (int64_t r = row0; r < row1; ++r) {
        const Segment<E> seg(a.z, r * a.ld, a.V, rank, a.cluster, a.per);
        const int chunks = seg.chunks(), kept = GRAD ? min(chunks, a.slots) : 0;    // kept in the ring
        // the segment's part of a gradient of zeros
        auto store_zeros = [&](E* out) {
            const bool whole = (reinterpret_cast<uintptr_t>(out + seg.first) & 15) == 0;
            const E zero = Ele<E>::round(0.f);
            if (whole)
                for (int v = tid; v < seg.n; v += kThreads)
                    __stcs(reinterpret_cast<uint4*>(out + seg.first) + v, make_uint4(0u, 0u, 0u, 0u));
            else
                for (int64_t i = tid; i < static_cast<int64_t>(seg.n) * kPer; i += kThreads) out[seg.first + i] = zero;
            if (tid < seg.head) out[tid] = zero;
            if (tid < seg.tail) out[seg.after + tid] = zero;
        };
        if constexpr (OP == kPolicy || OP == kScore) {
            if (unread(r)) {
                if (rank == 0 && tid == 0) {
                    if constexpr (OP == kPolicy) a.loss[r] = 0.f;
                    else if (a.state) a.state[r] = {0.f, INFINITY, 0.f, 0.f};
                    if (a.logprob) a.logprob[r] = 0.f;
                    if (a.entropy) a.entropy[r] = 0.f;
                    if (a.kl) a.kl[r] = 0.f;
                }
                if constexpr (GRAD) store_zeros(static_cast<E*>(a.dz) + r * a.ldd);
                continue;
            }
        }

        // The given token, or the teacher's entries, and the elements beside
        // the vectors: asked for here, used once the first chunk is there.
        constexpr int kEntries = LOGITS_MAX_TEACHER / kThreads;
        int64_t y[kEntries] = {};
        int token = -1;
        float z_token = 0.f;
        if constexpr (OP != kDistill) {
            y[0] = a.tokens ? a.tokens[r] : -1;
        } else {
#pragma unroll
            for (int i = 0; i < kEntries; ++i) {
                const int k = tid + i * kThreads;
                if (k < a.K) {
                    y[i] = a.tokens[r * a.ldt + k];
                    P[k] = teacher_value(a.teacher, a.teacher_type, r * a.ldt + k);
                }
            }
        }
        const float x_head = tid < seg.head ? Ele<E>::load(seg.row + tid) : -INFINITY;
        const float x_tail = tid < seg.tail ? Ele<E>::load(seg.row + seg.after + tid) : -INFINITY;
        auto given = [&] {
            if constexpr (OP != kDistill) {
                if (y[0] >= 0 && y[0] < a.V) {
                    token = static_cast<int>(y[0]);
                    z_token = Ele<E>::load(seg.row + token);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kEntries; ++i) {
                    const int k = tid + i * kThreads;
                    if (k >= a.K) break;
                    const bool real = y[i] >= 0 && y[i] < a.V;
                    const bool here = real && seg.holds(static_cast<int>(y[i]));
                    if (!real) P[k] = -INFINITY;
                    tok[k] = here ? static_cast<int>(y[i]) : -1;
                    zt[k] = here ? Ele<E>::load(seg.row + y[i]) : 0.f;
                }
            }
        };

        // statistics of the segment, and the buckets' maxima
        float bucket_max = -INFINITY, bucket_second = -INFINITY;     // of its chunks' maxima
        int bucket_batch = 0;
        Stats s = empty_stats();
        const uint64_t c2 = pair(a.c, a.c);
        {
            uint64_t m2 = pair(-s.m, -s.m), S2 = 0, U2 = 0;
            auto raise = [&](float m) {
                float x, y;
                unpair(S2, x, y);
                s.S = x + y;
                unpair(U2, x, y);
                s.U = x + y;
                raise_max(s, m, a.c);
                S2 = pair(s.S, 0.f), U2 = pair(s.U, 0.f);
                m2 = pair(-m, -m);
            };
            auto add = [&](uint64_t x2) {
                uint64_t u2 = mul2(add2(x2, m2), c2);
                if constexpr (kEntropy) u2 = max_nan2(u2, -200.f);
                const uint64_t e2 = ex2_2(u2);
                S2 = add2(S2, e2);
                if constexpr (kEntropy) U2 = fma2(e2, u2, U2);
            };
            if (chunks == 0) given();
            for (int b = 0; b < chunks; ++b) {
                uint4 q[kUnroll];
                take(seg, b, b < chunks - kept, q);
                if (b == 0) given();
                const float m = Ele<E>::template max_of<kUnroll>(q);
                if constexpr (TOP) {
                    bucket_second = fmaxf(bucket_second, fminf(bucket_max, m));
                    if (m > bucket_max) bucket_max = m, bucket_batch = b;
                }
                if (m > s.m) raise(m);
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    uint64_t x[kPer / 2];
                    Ele<E>::pairs(q[k], x);
#pragma unroll
                    for (int e = 0; e < kPer / 2; ++e) add(x[e]);
                }
            }
            if (tid < kPer) {
                const float m = fmaxf(x_head, x_tail);
                if (m > s.m) raise(m);
                add(pair(x_head, x_tail));
                if constexpr (TOP) {
                    if (x_head >= bucket_max) bucket_max = x_head, bucket_batch = kInHead;
                    if (x_tail > bucket_max) bucket_max = x_tail, bucket_batch = kInTail;
                }
            }
            float x, y;
            unpair(S2, x, y);
            s.S = x + y;
            unpair(U2, x, y);
            s.U = x + y;
        }

        // joined over the block by warp 0; the teacher's softmax and the
        // segment's part of a distillation loss are warp 1's
        // (of a thread's elements all but its maximum, 1 of S, went through ex2)
        s = warp_join<kEntropy>(s, 32, a.c, s.S > 1.f ? kEx2Lacks - __fdividef(kEx2Lacks, s.S) : 0.f);
        if (lane == 0) warp_stats[warp] = s;
        sync_threads();
        if (warp == 0) {
            s = lane < kWarps ? warp_stats[lane] : empty_stats();
            s = warp_join<kEntropy>(s, kWarps, a.c);
        }
        float A = 0.f, p = 0.f;
        if constexpr (OP == kDistill) {
            if (warp == 1) {
                const float sm = warp_max(lane < kWarps ? warp_stats[lane].m : -FLT_MAX);
                float m = -FLT_MAX, total = 0.f;
                for (int k = lane; k < a.K; k += 32) m = fmaxf(m, P[k]);
                m = warp_max(m);
                for (int k = lane; k < a.K; k += 32) total += ex2((P[k] - m) * a.c);
                total = warp_sum(total, 32);
                const float log2_total = lg2(total);
                for (int k = lane; k < a.K; k += 32) {
                    const float l = (P[k] - m) * a.c - log2_total, Pk = total != 0.f ? ex2(l) : 0.f;
                    P[k] = Pk;
                    if (tok[k] >= 0 && !(Pk <= 0.f)) {
                        A = fmaf(Pk, l * kLn2 - (zt[k] - sm) * a.inv_t, A);
                        p += Pk;
                    }
                }
                A = warp_sum(A, 32);
                p = warp_sum(p, 32);
                if (lane == 0) all.A = A, all.P = p;
            }
            sync_threads();
            if (warp == 0) A = all.A, p = all.P;
        }
        if constexpr (TOP)
            select_top<E>(*top, seg, ordered(bucket_max), bucket_batch, bucket_second, a.top);
        // The segments' statistics into every CTA's shared memory, lane i's
        // copy to CTA i, and the row's joined from them.
        if (warp == 0) {
            float advantage = 0.f, old_logprob = 0.f, ref_logprob = 0.f;      // asked for before the others' statistics
            if constexpr (OP == kPolicy) {
                advantage = a.advantage[r], old_logprob = a.old_logprob[r];
                if (a.ref_logprob) ref_logprob = a.ref_logprob[r];
            }
            Exchange x{s, A, p};
            bool arrived = true;
            if (a.cluster > 1) {
                const uint32_t bar = tcdt::smem_addr(&inbox_bar);
#ifdef TCDT_FAULT_INJECTION
                if (a.fi_silent && a.fi_here(rank)) {
                } else
#endif
                if (lane < a.cluster) {
                    const uint32_t to = tcdt::map_to_cta(tcdt::smem_addr(&inbox[rank]), static_cast<uint32_t>(lane));
                    st_cluster_f32(to, x.s.m), st_cluster_f32(to + 4, x.s.S), st_cluster_f32(to + 8, x.s.U);
                    st_cluster_f32(to + 12, x.A), st_cluster_f32(to + 16, x.P);
                    tcdt::mbar_arrive_cluster(tcdt::map_to_cta(bar, static_cast<uint32_t>(lane)));
                }
                // (a cluster's only row is phase 0; with the constant the compiler's arrangement of the whole
                // kernel took 2048 x 65537 with gradient from 98.1 us to 99.1)
                arrived = __all_sync(~0u, wait_cluster(bar, static_cast<uint32_t>(r - row0) & 1u, 2 * a.limit_ns()));
                x = lane < a.cluster ? inbox[lane] : Exchange{empty_stats(), 0.f, 0.f};
                s = warp_join<kEntropy>(x.s, kMaxCluster, a.c);
            }
            float l = 0.f, sum_P = 0.f;
            if constexpr (OP == kDistill) {
                // a part without teacher tokens has no maximum to shift by
                if (!(x.P <= 0.f)) l = s.S == 0.f ? x.A : fmaf(x.P, fmaf(s.m - x.s.m, a.inv_t, kLn2 * lg2(s.S)), x.A);
                sum_P = x.P;
                if (a.cluster > 1) l = warp_sum(l, kMaxCluster), sum_P = warp_sum(sum_P, kMaxCluster);
            }
            if (!arrived) s.S = NAN, l = NAN;
            __syncwarp();
            if (lane == 0) {
                all = {s, l, sum_P};
                // (computed by every thread, a policy loss took 3 % longer)
                if constexpr (OP == kPolicy) {
                    const float logprob =
                        s.S == 0.f ? -INFINITY : log_p(z_token, s.m, log_sum(s.S, s.U, a.c_rest), a.t, a.inv_t);
                    row_policy = policy_loss(a, logprob, advantage, old_logprob, ref_logprob);
                }
                if constexpr (TOP) heard = arrived;
            }
        }
        sync_threads();
        s = all.s;
        const float total_P = all.P;
        const bool nothing = s.S == 0.f;
        const float log2_S = lg2(s.S);
        const float entropy = nothing ? 0.f : kLn2 * (log2_S - s.U / s.S);
        if (rank == 0 && tid == 0) {
            if (a.lse) a.lse[r] = nothing ? -INFINITY : fmaf(s.m, a.inv_t, kLn2 * log2_S);
            if constexpr (OP != kDistill) {
                if (a.logprob)
                    a.logprob[r] = token < 0       ? 0.f
                                   : OP == kPolicy ? row_policy.logprob
                                   : nothing       ? -INFINITY
                                                   : log_p(z_token, s.m, log_sum(s.S, s.U, a.c_rest), a.t, a.inv_t);
                if (a.entropy) a.entropy[r] = entropy;
                if constexpr (OP == kPolicy) {
                    a.loss[r] = a.bonus != 0.f ? fmaf(-a.bonus, entropy, row_policy.loss) : row_policy.loss;
                    if (a.kl) a.kl[r] = row_policy.kl;
                }
                if constexpr (OP == kScore)
                    if (a.state) a.state[r] = {s.m, nothing ? INFINITY : log2_S, 0.f, 0.f};
            } else {
                a.loss[r] = a.t * (a.t * all.A);      // t^2 itself may be 0
            }
        }

        if constexpr (GRAD) {
            // p_j (ga + gb log2 p_j), and the given tokens' terms put in at the end
            float ga, gb = 0.f, g_token;
            if constexpr (OP != kDistill) {
                float g, h;
                if constexpr (OP == kPolicy) {
                    const float w = a.w[r];
                    g = w * row_policy.slope;
                    h = a.bonus != 0.f ? -a.bonus * w : 0.f;
                } else {
                    g = token >= 0 && a.g ? a.g[r] : 0.f;
                    h = a.h ? a.h[r] : 0.f;
                }
                ga = -a.inv_t * fmaf(h, entropy, g);
                gb = -a.inv_t * h * kLn2;
                g_token = a.inv_t * g;
            } else {
                g_token = a.w[r] * a.t;
                ga = g_token * total_P;
            }
            E* out = static_cast<E*>(a.dz) + r * a.ldd;
            const bool whole = (reinterpret_cast<uintptr_t>(out + seg.first) & 15) == 0;
            // (a row of nothing: every z - m is -inf, p and the factors are 0)
            const float shift = nothing ? 0.f : -log2_S;
            const uint64_t m2 = pair(-s.m, -s.m), shift2 = pair(shift, shift);
            const uint64_t ga2 = pair(nothing ? 0.f : ga, nothing ? 0.f : ga), gb2 = pair(gb, gb);
            // without a term of the entropy p_j's factor is the same for all of a row
            const bool plain = OP == kPolicy && a.bonus == 0.f;
            auto gradient = [&](uint64_t x2, bool plain) {
                uint64_t l2 = fma2(add2(x2, m2), c2, shift2);
                uint64_t g2 = ga2;
                if (OP != kDistill && !plain) {
                    l2 = max_nan2(l2, -200.f);
                    g2 = fma2(gb2, l2, ga2);
                }
                return mul2(ex2_2(l2), g2);
            };
            if ((slot -= kept) < 0) slot += a.slots, parity ^= 1u;
            const bool zeros = weightless(r);
            if (zeros) {
                for (int i = 0; i < kept; ++i) {
                    uint4 q[kUnroll];
                    take(seg, chunks - kept + i, true, q);
                }
                store_zeros(out);
            }
            for (int i = 0; i < chunks && !zeros; ++i) {
                const int b = i < kept ? chunks - kept + i : i - kept;
                uint4 q[kUnroll];
                const bool inside = take(seg, b, true, q);
                const int v0 = b * kChunk + tid;
                uint4* at = reinterpret_cast<uint4*>(out + seg.first) + v0;
                auto store_whole = [&](bool plain) {
#pragma unroll
                    for (int k = 0; k < kUnroll; ++k) {
                        uint64_t x[kPer / 2];
                        Ele<E>::pairs(q[k], x);
#pragma unroll
                        for (int e = 0; e < kPer / 2; ++e) x[e] = gradient(x[e], plain);
                        __stcs(at + k * kThreads, Ele<E>::pack_pairs(x));
                    }
                };
                if (inside && whole) {
                    if (OP == kPolicy && plain) store_whole(true);
                    else store_whole(false);
                } else {
#pragma unroll
                    for (int k = 0; k < kUnroll; ++k) {
                        const int v = v0 + k * kThreads;
                        if (v >= seg.n) continue;
                        uint64_t x[kPer / 2];
                        Ele<E>::pairs(q[k], x);
#pragma unroll
                        for (int e = 0; e < kPer / 2; ++e) x[e] = gradient(x[e], plain);
                        if (whole) {
                            at[k * kThreads] = Ele<E>::pack_pairs(x);
                        } else {
#pragma unroll
                            for (int e = 0; e < kPer / 2; ++e) {
                                float lo, hi;
                                unpair(x[e], lo, hi);
                                E* to = out + seg.first + static_cast<int64_t>(v) * kPer + 2 * e;
                                to[0] = Ele<E>::round(lo), to[1] = Ele<E>::round(hi);
                            }
                        }
                    }
                }
            }
            if (tid < kPer && !zeros) {
                float x0, x1;
                unpair(gradient(pair(x_head, x_tail), plain), x0, x1);
                if (tid < seg.head) out[tid] = Ele<E>::round(x0);
                if (tid < seg.tail) out[seg.after + tid] = Ele<E>::round(x1);
            }
            sync_threads();
            if constexpr (OP != kDistill) {
                if (tid == 0 && token >= 0 && !nothing && !zeros && seg.holds(token)) {
                    const float l = max_nan((z_token - s.m) * a.c - log2_S, -200.f);
                    out[token] = Ele<E>::round(fmaf(ex2(l), fmaf(gb, l, ga), g_token));
                }
            } else {
                for (int k = tid; k < a.K; k += kThreads) {
                    if (tok[k] < 0 || nothing) continue;
                    const int t = tok[k];
                    float p = 0.f;    // a token given twice: each of its entries writes the same sum
                    for (int i = 0; i < a.K; i += 4) {
                        const int4 o = *reinterpret_cast<const int4*>(tok + i);
                        if (o.x == t) p += P[i];
                        if (o.y == t) p += P[i + 1];
                        if (o.z == t) p += P[i + 2];
                        if (o.w == t) p += P[i + 3];
                    }
                    const float l = max_nan((zt[k] - s.m) * a.c - log2_S, -200.f);
                    out[tok[k]] = Ele<E>::round(fmaf(ga, ex2(l), -g_token * p));
                }
            }
        }

        if constexpr (TOP) {
            if (rank == 0 && !heard) {
                // no CTA's list is known to be whole: none is read
                for (int i = tid; i < a.top; i += kThreads) {
                    a.top_logprob[r * a.top + i] = NAN;
                    a.top_token[r * a.top + i] = -1;
                }
            } else if (rank == 0) {
                // the segments' lists side by side; a key's place is its place in its own list and the
                // number of larger keys in each of the others
                const int n = a.top, lists = a.cluster;
                const uint64_t* keys = top->list;
                const int* count = &top->count;
                int total = 0;
                for (int o = 0; o < lists; ++o)
                    total += lists == 1 ? *count
                                        : static_cast<int>(ld_cluster_u32(
                                              tcdt::map_to_cta(tcdt::smem_addr(count), static_cast<uint32_t>(o))));
                if (lists > 1) {
                    for (int i = tid; i < lists * n; i += kThreads) {
                        const uint32_t at = tcdt::map_to_cta(tcdt::smem_addr(keys + i % n), static_cast<uint32_t>(i / n));
                        top->cand[i] = static_cast<uint64_t>(ld_cluster_u32(at + 4)) << 32 | ld_cluster_u32(at);
                    }
                    sync_threads();
                    keys = top->cand;
                }
                const LogSum l = log_sum(s.S, s.U, a.c_rest);
                for (int i = tid; i < lists * n; i += kThreads) {
                    const uint64_t k = keys[i];
                    if (!k) continue;
                    int place = i % n;
                    for (int o = 0; o < lists; ++o) {
                        if (o == i / n) continue;
                        int lo = 0, hi = n;    // keys[o * n + 0 .. lo - 1] are larger, from hi on none is
                        while (lo < hi) {
                            const int mid = (lo + hi) / 2;
                            if (keys[o * n + mid] > k) lo = mid + 1;
                            else hi = mid;
                        }
                        place += lo;
                    }
                    if (place < n) {
                        const float z = from_ordered(static_cast<uint32_t>(k >> 32));
                        a.top_logprob[r * n + place] = log_p(z, s.m, l, a.t, a.inv_t);
                        a.top_token[r * n + place] = static_cast<int64_t>(~static_cast<uint32_t>(k));
                    }
                }
                for (int i = total + tid; i < n; i += kThreads) {
                    a.top_logprob[r * n + i] = -INFINITY;
                    a.top_token[r * n + i] = -1;
                }
            }
        }
        sync_threads();    // the row's entries, lists and `all` are done with
    }
    // nobody leaves while its shared memory may still be read
    __syncwarp();
    if (a.cluster > 1) tcdt::cluster_sync_all();
}

// ---- preference loss ---------------------------------------------------------
// The rows' log-probabilities and statistics (rows_kernel), then the pairs, then
// the gradient: a row's factor depends on all rows of its pair, so its logits are
// read a second time.  The gradient goes through the rows from the last one to
// the first: what the statistics read last is then still in L2.  4096 x 131072 bf16,
// eight pairs: 163 us (the time of the bytes), 8 and 301 (7.1 TB/s with what L2 held).
struct Pairs {
    const int64_t* offsets;           // [2 pairs + 1]
    const float* ref;                 // [T] or null
    const float* logprob;             // [T]
    const int64_t* tokens;            // [T]
    const float* w;                   // [pairs] or null
    int64_t T;
    int32_t V;
    float beta, smoothing;
    float* loss;                      // [pairs]
    float* reward;                    // [2 pairs]
    RowState* state;                  // [T]
};

constexpr int kPairThreads = 512;

// One CTA a pair.  Sums of a few thousand log-probabilities are kept in 64 bits:
// their difference is what counts.  The order of the additions is fixed.
__global__ void __launch_bounds__(kPairThreads) pairs_kernel(const Pairs a) {
    __shared__ double part[2][kPairThreads / 32];
    __shared__ float slope[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t pair = blockIdx.x;
    int64_t at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) at[i] = min(max(a.offsets[2 * pair + i], int64_t(0)), a.T);
    tcdt::griddep_wait();             // the rows' log-probabilities are there
    auto scored = [&](int64_t r) {
        const int64_t y = a.tokens[r];
        return y >= 0 && y < a.V;
    };
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        double sum = 0;
        for (int64_t r = at[side] + tid; r < at[side + 1]; r += kPairThreads)
            if (scored(r)) sum += static_cast<double>(a.logprob[r]) - (a.ref ? static_cast<double>(a.ref[r]) : 0.0);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) part[side][warp] = sum;
    }
    __syncthreads();
    if (tid == 0) {
        double reward[2] = {};
        for (int side = 0; side < 2; ++side) {
            for (int w = 0; w < kPairThreads / 32; ++w) reward[side] += part[side][w];
            reward[side] *= a.beta;
            a.reward[2 * pair + side] = static_cast<float>(reward[side]);
        }
        // -log sigma(m) = log1p(e^-|m|) + max(-m, 0), sigma from the same exponential.  |m| in two
        // fp32 parts, far + near: rounded to 32 bits it would be off by 2^-24 |m|, and so would
        // sigma, relatively.  (All of it in 64 bits took one thread 4 us.)
        const double margin = reward[0] - reward[1];
        const float m = static_cast<float>(margin), e = a.smoothing, far = fabsf(m);
        const float near = isfinite(m) ? static_cast<float>(fabs(margin) - static_cast<double>(far)) : 0.f;
        const float x0 = expf(-far), x = fmaf(-near, x0, x0), l = log1pf(x);
        const float less = x / (1.f + x), more = 1.f / (1.f + x);
        const float right = e == 1.f ? 0.f : (1.f - e) * (m < 0.f ? (l + near) + far : l);
        const float wrong = e == 0.f ? 0.f : e * (m > 0.f ? (l + near) + far : l);
        a.loss[pair] = m != m ? m : right + wrong;
        if (a.w) {
            const float d = e * (m < 0.f ? less : more) - (1.f - e) * (m < 0.f ? more : less);
            const float g = a.w[pair] == 0.f ? 0.f : d * a.beta * a.w[pair];
            slope[0] = g, slope[1] = -g;
        }
    }
    if (!a.w) return;
    __syncthreads();
    for (int side = 0; side < 2; ++side)
        for (int64_t r = at[side] + tid; r < at[side + 1]; r += kPairThreads) a.state[r].g = slope[side];
}

constexpr int kGradThreads = 256, kGradUnroll = 4;
constexpr int kGradVectors = kGradThreads * kGradUnroll * 4;     // of a CTA: 64 KB

// dlogits of a part of a row, g (1[j = y] - p_j) / temperature.
template <typename E>
__global__ void __launch_bounds__(kGradThreads) score_grad_kernel(const Args a, int parts) {
    constexpr int kPer = Ele<E>::kPer;
    const int tid = threadIdx.x;
    const int64_t r = a.T - 1 - static_cast<int64_t>(blockIdx.x) / parts;
    const int part = static_cast<int>(blockIdx.x % parts);
    const Segment<E> seg(a.z, r * a.ld, a.V, part, parts, kGradVectors);
    E* out = static_cast<E*>(a.dz) + r * a.ldd;
    const bool whole = (reinterpret_cast<uintptr_t>(out + seg.first) & 15) == 0;
    tcdt::griddep_wait();
    const RowState s = a.state[r];
    const bool zeros = s.g == 0.f || s.log2_S == INFINITY;
    const int64_t y = a.tokens[r];
    const float g = s.g * a.inv_t, shift = s.log2_S;
    auto p = [&](float z) { return ex2(fmaf(z - s.m, a.c, -shift)); };
    auto value = [&](float z, int j) { return zeros ? 0.f : j == y ? fmaf(-g, p(z), g) : -g * p(z); };
    const uint64_t c2 = pair(a.c, a.c), m2 = pair(-s.m, -s.m), shift2 = pair(-shift, -shift), g2 = pair(-g, -g);
    for (int v0 = tid; v0 < seg.n; v0 += kGradThreads * kGradUnroll) {
        uint4 q[kGradUnroll];
        if (!zeros) {
#pragma unroll
            for (int k = 0; k < kGradUnroll; ++k)
                if (v0 + k * kGradThreads < seg.n) q[k] = seg.load(v0 + k * kGradThreads);
        }
#pragma unroll
        for (int k = 0; k < kGradUnroll; ++k) {
            const int v = v0 + k * kGradThreads;
            if (v >= seg.n) continue;
            uint64_t x[kPer / 2];
            if (zeros) {
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) x[e] = 0;
            } else {
                Ele<E>::pairs(q[k], x);
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) x[e] = mul2(ex2_2(fma2(add2(x[e], m2), c2, shift2)), g2);
                const int64_t j = y - (seg.first + static_cast<int64_t>(v) * kPer);
                if (j >= 0 && j < kPer) {
#pragma unroll
                    for (int e = 0; e < kPer / 2; ++e) {
                        float lo, hi;
                        unpair(x[e], lo, hi);
                        x[e] = pair(j == 2 * e ? lo + g : lo, j == 2 * e + 1 ? hi + g : hi);
                    }
                }
            }
            if (whole) {
                __stcs(reinterpret_cast<uint4*>(out + seg.first) + v, Ele<E>::pack_pairs(x));
            } else {
#pragma unroll
                for (int e = 0; e < kPer / 2; ++e) {
                    float lo, hi;
                    unpair(x[e], lo, hi);
                    E* to = out + seg.first + static_cast<int64_t>(v) * kPer + 2 * e;
                    to[0] = Ele<E>::round(lo), to[1] = Ele<E>::round(hi);
                }
            }
        }
    }
    if (tid < seg.head) out[tid] = Ele<E>::round(value(zeros ? 0.f : Ele<E>::load(seg.row + tid), tid));
    if (tid < seg.tail) {
        const int j = seg.after + tid;
        out[j] = Ele<E>::round(value(zeros ? 0.f : Ele<E>::load(seg.row + j), j));
    }
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

#ifdef TCDT_FAULT_INJECTION
struct {
    uint64_t limit_ns = kWaitLimitNs;
    int64_t skip_copy = -1, late_chunk = -1;
    uint32_t late_warps = 0;
    int silent = 0, rank = -1;
} g_fi;
#endif

// What is asked once of a device: whether it is the kind the kernels are
// built for, and its number of SMs.
constexpr int kDevices = 64;
std::atomic<int> g_sms[kDevices];      // 0: not asked yet

gemm_status_t sms_of(int device, int* sms) {
    if (device < 0) return GEMM_ERR_INVALID_ARG;
    *sms = device < kDevices ? g_sms[device].load(std::memory_order_relaxed) : 0;
    if (*sms) return GEMM_OK;
    int count = 0, major = 0, minor = 0;
    gemm_status_t st = GEMM_OK;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count <= 0) st = GEMM_ERR_NO_DEVICE;
    else if (device >= count) st = GEMM_ERR_INVALID_ARG;
    else if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
             cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
             cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        st = GEMM_ERR_CUDA;
    else if (major != 10 || minor != 3) st = GEMM_ERR_NO_DEVICE;
    if (st != GEMM_OK) {
        cudaGetLastError();
        return st;
    }
    if (device < kDevices) g_sms[device].store(*sms, std::memory_order_relaxed);
    return GEMM_OK;
}

// Makes `device` current and restores the previous one.
struct OnDevice {
    int prev = -1;
    bool ok;
    explicit OnDevice(int device) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == device || cudaSetDevice(device) == cudaSuccess);
        if (!ok) cudaGetLastError();
        if (!ok || prev == device) prev = -1;
    }
    ~OnDevice() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

template <typename E, int OP, bool GRAD, bool TOP>
gemm_status_t launch(Args a, int64_t T, int device, int sms, cudaStream_t stream) {
    // The ring takes what shared memory kCtas CTAs an SM leave.
    constexpr int kCtas = ctas_of(GRAD);
    const int64_t chunks = (a.V / Ele<E>::kPer + kChunk - 1) / kChunk;
    const int64_t beside = TOP ? static_cast<int64_t>(sizeof(TopState)) : OP == kDistill ? (a.K + 3) / 4 * 48 : 0;
    int64_t slots = (kSharedOfSm / kCtas - 2048 - beside) / (kChunk * 16);
    const int64_t ctas_at_once = static_cast<int64_t>(kCtas) * sms;
    // CTAs of a row.  A gradient's rows in flight, which it reads twice, are to
    // fit L2 beside what it writes (4096 x 131072 bf16: 1 CTA a row 426 us, 2 375,
    // 3 478; 600 x 131072 fp32: 143, 131, 130 and 4 117; 300 x 131072 bf16, 79 MB
    // in all: 36 and 42).
    int64_t cluster = 1;
    if (GRAD)
        while (cluster < kMaxCluster && chunks > slots &&
               (T * cluster < ctas_at_once ? T : ctas_at_once / cluster) * a.V * static_cast<int64_t>(sizeof(E)) >
                   (cluster == 1 ? kInFlightWhole : kInFlight))
            ++cluster;
    // Few rows are split over up to two CTAs an SM (64 x 131072 bf16 with
    // gradient: 1 CTA a row 21 us, 2 15, 4 14, 8 19), in halves, as long as every
    // CTA has a chunk, or four where it selects alternatives of its own first
    // (1 x 131072 bf16: 1 CTA 16.4 us, 4 13.0, 8 13.6; 64 x 50001: 13.4, 14.0, 15.8).
    while (cluster * 2 <= kMaxCluster && T * cluster * 2 <= 2 * sms && chunks >= cluster * 2 * (TOP ? 4 : 1)) cluster *= 2;
    const int64_t each = chunks > 0 ? (chunks + cluster - 1) / cluster : 1;
    // Two rows one after another save a start where a row is short and the
    // CTAs are many (8192 x 8192 bf16 with gradient: 83 us with one, 74 with
    // two, 77 with four; 4096 x 131072 bf16, 64 alternatives: 217, 230, 241).
    const int64_t rows = cluster == 1 && each <= 2 && T >= 8 * ctas_at_once ? 2 : 1;
    if (slots > each * rows) slots = each * rows;
    if (slots > kSlotsMost) slots = kSlotsMost;
    a.T = T;
    a.cluster = static_cast<int>(cluster);
    a.per = static_cast<int>((a.V / Ele<E>::kPer + cluster - 1) / cluster);
    a.rows = static_cast<int>(rows);
    a.slots = static_cast<int>(slots);
#ifdef TCDT_FAULT_INJECTION
    a.fi_limit_ns = g_fi.limit_ns;
    a.fi_skip_copy = g_fi.skip_copy;
    a.fi_late_chunk = g_fi.late_chunk;
    a.fi_late_warps = g_fi.late_warps;
    a.fi_silent = g_fi.silent;
    a.fi_rank = g_fi.rank;
#endif
    const size_t dyn = static_cast<size_t>(slots) * kChunk * 16 + static_cast<size_t>(beside);
    const int64_t ctas = (T + rows - 1) / rows * cluster;
    auto kernel = rows_kernel<E, OP, GRAD, TOP>;
    if (ctas > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    // the kernel's shared-memory opt-in, once a device
    static std::atomic<uint64_t> prepared{0};
    const uint64_t bit = device < kDevices ? uint64_t(1) << device : 0;
    if (!(prepared.load(std::memory_order_relaxed) & bit) || !bit) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamicMost) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        prepared.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kBlock, 1, 1);
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
    int sms = 0;
    const gemm_status_t st = sms_of(device, &sms);
    if (st != GEMM_OK) return st;
    const OnDevice on(device);
    if (!on.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GEMM_F32) return launch<float, OP, GRAD, TOP>(a, T, device, sms, s);
    if (dtype == GEMM_F16) return launch<__half, OP, GRAD, TOP>(a, T, device, sms, s);
    return launch<__nv_bfloat16, OP, GRAD, TOP>(a, T, device, sms, s);
}

void fill_rows(Args& a, const void* logits, int64_t V, int64_t ld, float temperature) {
    a.z = logits;
    a.V = static_cast<int32_t>(V);
    a.ld = ld;
    a.t = temperature;
    a.inv_t = 1.0f / temperature;
    a.c = kLog2e / temperature;
    a.c_rest = static_cast<float>((1.4426950408889634 / temperature - a.c) / a.c);
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

gemm_status_t check_preference(gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                               const int64_t* tokens, float temperature, const logits_preference_t* preference,
                               const float* loss, const float* reward, const float* logprob) {
    const gemm_status_t st = check_rows(dtype, logits, T, V, ld, temperature);
    if (st != GEMM_OK) return st;
    if (!preference) return GEMM_ERR_INVALID_ARG;
    const logits_preference_t& q = *preference;
    if (q.pairs < 0 || !std::isfinite(q.beta) || !(q.smoothing >= 0.f && q.smoothing <= 1.f)) return GEMM_ERR_INVALID_ARG;
    if (q.pairs > kMaxExtent) return GEMM_ERR_UNSUPPORTED;
    if (q.pairs > 0 && (!q.offsets || !loss || !reward)) return GEMM_ERR_INVALID_ARG;
    if (T > 0 && (!tokens || !logprob)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(tokens, 8) || !aligned(q.offsets, 8) || !aligned(q.ref_logprob, 4) || !aligned(loss, 4) ||
        !aligned(reward, 4) || !aligned(logprob, 4))
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

// A kernel that may start while the one before it in the stream ends (it waits
// for it itself, see griddep_wait).
template <typename... P, typename... A>
gemm_status_t launch_dependent(void (*kernel)(P...), unsigned ctas, unsigned threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

template <typename E>
gemm_status_t launch_score_grad(const Args& a, cudaStream_t stream) {
    const int64_t vectors = a.V / Ele<E>::kPer;
    const int64_t parts = vectors > 0 ? (vectors + kGradVectors - 1) / kGradVectors : 1;
    if (parts * a.T > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    return launch_dependent(score_grad_kernel<E>, static_cast<unsigned>(parts * a.T), kGradThreads, stream, a,
                            static_cast<int>(parts));
}

// a.dz null: without the gradient.
gemm_status_t run_preference(int device, gemm_dtype_t dtype, Args a, int64_t T, const logits_preference_t& q,
                             const float* w, float* reward, void* stream) {
    if (T == 0 && q.pairs == 0) return GEMM_OK;
    int sms = 0;
    gemm_status_t st = sms_of(device, &sms);
    if (st != GEMM_OK) return st;
    const OnDevice on(device);
    if (!on.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.T = T;
    // refused before anything is launched
    if (a.dz && a.V > 0 && T * ((a.V / 4 + kGradVectors - 1) / kGradVectors + 1) > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    st = launch_type<kScore, false, false>(device, dtype, a, T, stream);
    if (st == GEMM_OK && q.pairs > 0) {
        Pairs p{q.offsets, q.ref_logprob, a.logprob, a.tokens, w, T, a.V, q.beta, q.smoothing, a.loss, reward, a.state};
        st = launch_dependent(pairs_kernel, static_cast<unsigned>(q.pairs), kPairThreads, s, p);
    }
    if (st != GEMM_OK || !a.dz || T == 0) return st;
    if (dtype == GEMM_F32) return launch_score_grad<float>(a, s);
    if (dtype == GEMM_F16) return launch_score_grad<__half>(a, s);
    return launch_score_grad<__nv_bfloat16>(a, s);
}

void fill_preference(Args& a, const int64_t* tokens, float* loss, float* logprob) {
    a.tokens = tokens;
    a.loss = loss;
    a.logprob = logprob;
}

gemm_status_t check_policy(gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                           const int64_t* tokens, float temperature, const logits_policy_t* policy,
                           const float* loss, const float* logprob, const float* kl, const float* entropy) {
    const gemm_status_t st = check_rows(dtype, logits, T, V, ld, temperature);
    if (st != GEMM_OK) return st;
    if (!policy) return GEMM_ERR_INVALID_ARG;
    const logits_policy_t& q = *policy;
    if (!(q.clip_low >= 0.f && q.clip_low <= 1.f) || !(q.clip_high >= 0.f) || !std::isfinite(q.clip_high) ||
        !std::isfinite(q.kl_coef) || !std::isfinite(q.entropy_bonus))
        return GEMM_ERR_INVALID_ARG;
    if (q.kl_coef != 0.f && !q.ref_logprob) return GEMM_ERR_INVALID_ARG;
    if (T > 0 && (!tokens || !q.old_logprob || !q.advantage || !loss)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(tokens, 8) || !aligned(q.old_logprob, 4) || !aligned(q.advantage, 4) || !aligned(q.ref_logprob, 4) ||
        !aligned(loss, 4) || !aligned(logprob, 4) || !aligned(kl, 4) || !aligned(entropy, 4))
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

void fill_policy(Args& a, const int64_t* tokens, const logits_policy_t& q, float* loss, float* logprob, float* kl,
                 float* entropy) {
    a.tokens = tokens;
    a.old_logprob = q.old_logprob;
    a.advantage = q.advantage;
    a.ref_logprob = q.ref_logprob;
    a.lo = 1.0f - q.clip_low;
    a.hi = 1.0f + q.clip_high;
    a.kl_coef = q.kl_coef;
    a.bonus = q.entropy_bonus;
    a.loss = loss;
    a.logprob = logprob;
    a.kl = kl;
    a.entropy = entropy;
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

gemm_status_t logits_policy(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                            const int64_t* tokens, float temperature, const logits_policy_t* policy, float* loss,
                            float* logprob, float* kl, float* entropy, void* stream) {
    const gemm_status_t st =
        check_policy(dtype, logits, T, V, ld, tokens, temperature, policy, loss, logprob, kl, entropy);
    if (st != GEMM_OK) return st;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_policy(a, tokens, *policy, loss, logprob, kl, entropy);
    return launch_type<kPolicy, false, false>(device, dtype, a, T, stream);
}

gemm_status_t logits_policy_grad(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                                 const int64_t* tokens, float temperature, const logits_policy_t* policy,
                                 const float* w, float* loss, float* logprob, float* kl, float* entropy, void* dlogits,
                                 int64_t ldd, void* stream) {
    gemm_status_t st = check_policy(dtype, logits, T, V, ld, tokens, temperature, policy, loss, logprob, kl, entropy);
    if (st == GEMM_OK) st = check_gradient(dtype, dlogits, T, V, ldd);
    if (st != GEMM_OK) return st;
    if (T > 0 && !w) return GEMM_ERR_INVALID_ARG;
    if (!aligned(w, 4)) return GEMM_ERR_MISALIGNED;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_policy(a, tokens, *policy, loss, logprob, kl, entropy);
    a.w = w;
    a.dz = dlogits;
    a.ldd = ldd;
    return launch_type<kPolicy, true, false>(device, dtype, a, T, stream);
}

gemm_status_t logits_preference(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V, int64_t ld,
                                const int64_t* tokens, float temperature, const logits_preference_t* preference,
                                float* loss, float* reward, float* logprob, void* stream) {
    const gemm_status_t st =
        check_preference(dtype, logits, T, V, ld, tokens, temperature, preference, loss, reward, logprob);
    if (st != GEMM_OK) return st;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_preference(a, tokens, loss, logprob);
    return run_preference(device, dtype, a, T, *preference, nullptr, reward, stream);
}

gemm_status_t logits_preference_grad(int device, gemm_dtype_t dtype, const void* logits, int64_t T, int64_t V,
                                     int64_t ld, const int64_t* tokens, float temperature,
                                     const logits_preference_t* preference, const float* w, float* loss, float* reward,
                                     float* logprob, void* dlogits, int64_t ldd, void* work, void* stream) {
    gemm_status_t st = check_preference(dtype, logits, T, V, ld, tokens, temperature, preference, loss, reward, logprob);
    if (st == GEMM_OK) st = check_gradient(dtype, dlogits, T, V, ldd);
    if (st != GEMM_OK) return st;
    if ((preference->pairs > 0 && !w) || (T > 0 && !work)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(w, 4) || !aligned(work, 16)) return GEMM_ERR_MISALIGNED;
    Args a{};
    fill_rows(a, logits, V, ld, temperature);
    fill_preference(a, tokens, loss, logprob);
    a.dz = V > 0 ? dlogits : nullptr;
    a.ldd = ldd;
    a.state = static_cast<RowState*>(work);
    return run_preference(device, dtype, a, T, *preference, w, reward, stream);
}

#ifdef TCDT_FAULT_INJECTION
// Test builds only (not part of the product library or of include/logits.h), for
// the calls that follow: see Args.
gemm_status_t logits_test_inject(uint64_t limit_ns, int64_t skip_copy, int64_t late_chunk, uint32_t late_warps,
                                 int silent, int rank) {
    g_fi = {limit_ns, skip_copy, late_chunk, late_warps, silent, rank};
    return GEMM_OK;
}
#endif

}  // extern "C"
