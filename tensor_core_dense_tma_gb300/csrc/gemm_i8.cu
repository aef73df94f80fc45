// gemm_i8.cu -- the product of 8-bit integers with a scale for each token
// (row of A) and channel (column of B), and the quantisation of rows
// (gemm_run_i8, gemm_run_i8_dynamic, gemm_quantize_rows_i8 of gemm.h).
//
//     D[i,j] = act(rs[i] cs[j] sum_k A[i,k] B[k,j] + bias[j])
//
// sm_103a has no 8-bit integer MMA on tcgen05.  An int8 value is exact in
// fp16 and the product of two is exact in fp32 (at most 2^14), so the codes
// are multiplied as fp16 with fp32 accumulation: partial sums within 2^24 are
// exact (any K up to 1024, or 1040 without the code -128; for larger K whenever
// the sums stay within it).  Larger ones lose what does not fit 24 bits, toward
// zero, at every step of 16 codes (all products of one sign, one range of K: the
// mean loss is 2^-20.1 of the sum at K = 2048, 2^-16 at 8192, 2^-14.3 at 16384).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gemm.h"
#include "gemm_i8_kernel.cuh"
#include "gemm_internal.cuh"

using namespace tcdt_host;

namespace {

constexpr int kThreads = 256;

// int8 rows (16-byte aligned, ld elements apart) as fp16 rows (ldh apart, a
// multiple of 8), zero in columns K..ldh-1; 16 codes a thread.  8192 x 8192
// codes: 67 MB read, 134 MB written.
__global__ void __launch_bounds__(kThreads) widen_kernel(const int8_t* q, int64_t ld, __half* h, int64_t ldh,
                                                         int64_t rows, int32_t K) {
    tcdt_i8::grid_release();
    const int32_t per_row = static_cast<int32_t>((K + 15) / 16);
    const int64_t total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / per_row;
        const int32_t k = static_cast<int32_t>(i - r * per_row) * 16;
        const int8_t* src = q + r * ld + k;
        uint4 c;
        if (k + 16 <= K) {
            c = *reinterpret_cast<const uint4*>(src);
        } else {    // nothing after the row's last code is read
            uint32_t w[4] = {};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k + e < K) w[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(src[e])) << (8 * (e % 4));
            c = make_uint4(w[0], w[1], w[2], w[3]);
        }
        uint4 lo, hi;
        tcdt_i8::widen4(c.x, lo.x, lo.y);
        tcdt_i8::widen4(c.y, lo.z, lo.w);
        tcdt_i8::widen4(c.z, hi.x, hi.y);
        tcdt_i8::widen4(c.w, hi.z, hi.w);
        uint4* dst = reinterpret_cast<uint4*>(h + r * ldh + k);
        dst[0] = lo;
        if (k + 8 < ldh) dst[1] = hi;
    }
}

template <typename E>
__device__ __forceinline__ float as_float(E x) { return static_cast<float>(x); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Both divisions are IEEE, so that the codes are those of the definition.  A
// quotient that is no number (a row with an infinity or a NaN) has code 0: the
// row's other codes are 0 as well, and 0 times its scale makes results NaN.
__device__ __forceinline__ int code_of(float x, float scale) {
    const float c = scale != 0.f ? __fdiv_rn(x, scale) : 0.f;
    return c == c ? __float2int_rn(fminf(fmaxf(c, -127.f), 127.f)) : 0;
}

__device__ __forceinline__ void store_code(int8_t* p, int q) { *p = static_cast<int8_t>(q); }
__device__ __forceinline__ void store_code(__half* p, int q) { *p = __int2half_rn(q); }

__device__ __forceinline__ void store_codes(int8_t* p, const int (&q)[8]) {
    uint2 v = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v.x |= static_cast<uint32_t>(q[e] & 255) << (8 * e);
        v.y |= static_cast<uint32_t>(q[4 + e] & 255) << (8 * e);
    }
    *reinterpret_cast<uint2*>(p) = v;
}
__device__ __forceinline__ void store_codes(__half* p, const int (&q)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2 h = __floats2half2_rn(static_cast<float>(q[2 * e]), static_cast<float>(q[2 * e + 1]));
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive elements, 16-byte aligned.
template <typename E>
struct Eight {
    uint4 v[sizeof(E) / 2];
    __device__ __forceinline__ void load(const E* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E)) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ float at(int e) const { return as_float(reinterpret_cast<const E*>(v)[e]); }
};

// One CTA a row: scale = max |x| / 127, code = round(x / scale).  A row of
// zeros has scale 0 and codes 0.  WHOLE: rows of X on 16-byte boundaries and
// rows of Q on those of eight codes are read and written eight elements at a
// time, the first kKeep of a thread staying in registers between the passes
// (rows of 8192 elements are read once).
template <typename E, typename Q, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const E* x, int64_t ldx, Q* q, int64_t ldq, float* scale,
                                                            int32_t K) {
    constexpr int kKeep = 4;
    __shared__ float part[kThreads / 32];
    tcdt_i8::grid_release();
    const int64_t r = blockIdx.x;
    const E* row = x + r * ldx;
    Q* out = q + r * ldq;
    const int32_t eights = WHOLE ? K / 8 : 0;
    Eight<E> keep[kKeep];
    float top = 0.f;
    if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int32_t c = threadIdx.x + i * kThreads;
            if (c < eights) keep[i].load(row + c * 8);
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (threadIdx.x + i * kThreads < eights) {
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(keep[i].at(e)));
            }
        for (int32_t c = threadIdx.x + kKeep * kThreads; c < eights; c += kThreads) {
            Eight<E> v;
            v.load(row + static_cast<int64_t>(c) * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v.at(e)));
        }
    }
    for (int32_t k = eights * 8 + threadIdx.x; k < K; k += kThreads) top = max_nan(top, fabsf(as_float(row[k])));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max_nan(top, part[w]);
    const float s = __fdiv_rn(top, 127.f);
    if (threadIdx.x == 0) scale[r] = s;
    if constexpr (WHOLE) {
        auto put = [&](const Eight<E>& v, int32_t c) {
            int code[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) code[e] = code_of(v.at(e), s);
            store_codes(out + static_cast<int64_t>(c) * 8, code);
        };
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (threadIdx.x + i * kThreads < eights) put(keep[i], threadIdx.x + i * kThreads);
        for (int32_t c = threadIdx.x + kKeep * kThreads; c < eights; c += kThreads) {
            Eight<E> v;
            v.load(row + static_cast<int64_t>(c) * 8);
            put(v, c);
        }
    }
    for (int32_t k = eights * 8 + threadIdx.x; k < K; k += kThreads) store_code(out + k, code_of(as_float(row[k]), s));
}

template <typename E, typename Q>
void launch_quantize_type(const void* x, int64_t R, int64_t K, int64_t ldx, Q* q, int64_t ldq, float* scale,
                          cudaStream_t s) {
    const bool whole = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ldx * sizeof(E)) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(q) % (8 * sizeof(Q)) == 0 && ldq % 8 == 0;
    const E* e = static_cast<const E*>(x);
    const unsigned grid = static_cast<unsigned>(R);
    if (whole) quantize_kernel<E, Q, true><<<grid, kThreads, 0, s>>>(e, ldx, q, ldq, scale, static_cast<int32_t>(K));
    else quantize_kernel<E, Q, false><<<grid, kThreads, 0, s>>>(e, ldx, q, ldq, scale, static_cast<int32_t>(K));
}

template <typename Q>
gemm_status_t launch_quantize(const void* x, gemm_dtype_t t, int64_t R, int64_t K, int64_t ldx, Q* q, int64_t ldq,
                              float* scale, cudaStream_t s) {
    if (t == GEMM_F32) launch_quantize_type<float>(x, R, K, ldx, q, ldq, scale, s);
    else if (t == GEMM_F16) launch_quantize_type<__half>(x, R, K, ldx, q, ldq, scale, s);
    else launch_quantize_type<__nv_bfloat16>(x, R, K, ldx, q, ldq, scale, s);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t launch_widen(gemm_plan* plan, const int8_t* q, int64_t ld, __half* h, int64_t ldh, int64_t rows,
                           int64_t K, cudaStream_t s) {
    const int64_t threads = rows * ((K + 15) / 16);
    int64_t grid = (threads + kThreads - 1) / kThreads;
    if (grid > 16LL * plan->sm_count) grid = 16LL * plan->sm_count;
    widen_kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(q, ld, h, ldh, rows, static_cast<int32_t>(K));
    if (cudaGetLastError() != cudaSuccess) return GEMM_ERR_CUDA;
    ++plan->launches;
    return GEMM_OK;
}

// The plan's buffer for codes and row scales, grown to `bytes`.  A buffer that
// was outgrown stays until the plan is destroyed: kernels in flight and
// captured graphs hold its address.  Each is at least twice the one before,
// so they are together smaller than the newest.
gemm_status_t reserve(gemm_plan* plan, size_t bytes) {
    if (bytes <= plan->i8_bytes) return GEMM_OK;
    size_t want = plan->i8_bytes ? 2 * plan->i8_bytes : size_t(1) << 20;
    if (want < bytes) want = bytes;
    if (plan->i8_buffers == kI8Buffers) return GEMM_ERR_CUDA;
    void* p = nullptr;
    if (cudaMalloc(&p, want) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    plan->d_i8[plan->i8_buffers++] = p;
    plan->i8_bytes = want;
    return GEMM_OK;
}

// Makes the plan's device current, and the previous one again at the end.
struct OnDevice {
    int prev = -1, device;
    bool ok;
    explicit OnDevice(int d) : device(d) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == d || cudaSetDevice(d) == cudaSuccess);
        if (!ok) cudaGetLastError();
    }
    ~OnDevice() {
        if (ok && prev != device) cudaSetDevice(prev);
    }
};

constexpr int64_t kMaxExtent = 0x7FFFF000;
bool float_type(gemm_dtype_t d) { return d == GEMM_F32 || d == GEMM_F16 || d == GEMM_BF16; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

gemm_status_t check_product(gemm_plan* plan, const void* B, const void* D, int64_t M, int64_t N, int64_t K,
                            int64_t ldb, int64_t ldd, gemm_dtype_t out, const gemm_epilogue_t* ep) {
    if (!plan || !float_type(out)) return GEMM_ERR_INVALID_ARG;
    if (ep && (static_cast<int>(ep->act) < 0 || static_cast<int>(ep->act) > 2)) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (plan->in_dtype != GEMM_F16 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!D || ldd < N) return GEMM_ERR_INVALID_ARG;
    if (ldd > (int64_t(1) << 40) || ldb > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (((M + 15) / 16) * ((N + 15) / 16) > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;    // gemm_run's limit
    if (!aligned(D, out == GEMM_F32 ? 4 : 2)) return GEMM_ERR_MISALIGNED;
    if (K == 0) return GEMM_OK;
    if (!B || ldb < K) return GEMM_ERR_INVALID_ARG;
    if (!aligned(B, 16) || ldb % 16) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

// Kernels of the product, by the number of tokens M.
enum Path { kDot, kTile, kPair, kWide };

Path path_of(int64_t M, int64_t N, int64_t K, int sms) {
    // Whole-number sums: K products of up to 2^14 stay within 31 bits.
    // Measured against the tile kernel (us, 1 / 4 / 8 tokens): 2048 x 2048
    // weights 3.4 / 3.4 / 4.6 to 6.1 / 6.2 / 6.4, 4096 x 4096 4.9 / 6.9 / 11.3 to
    // 9.2 / 9.2 / 9.3, 8192 x 8192 12.6 / 18.7 / 26.2 to 15.9 / 16.1 / 16.1, and
    // with 1 token quantised in the call 14.2 to 17.0.
    if (K < (1 << 17)) {
        const int64_t weights = N * K;
        if (M <= 2) return kDot;
        if (M <= 4 && weights <= (1 << 24)) return kDot;
        if (M <= 8 && weights <= (1 << 22)) return kDot;
    }
    // Few tokens or few tiles of 128 x 128: those, which then share K in clusters or
    // have an SM of their own (1024 x 8192 weights, 1024 tokens: 25 us, pairs 45,
    // widened first 74; 640 x 16000, 3500 tokens, 140 tiles: 91, 105, 109).
    const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128);
    if (M <= 256 || tiles <= sms) return kTile;
    // Otherwise the least of three estimates in us, fitted to 97 measured sizes from
    // 8192 x 300 to 640 x 16000 weights and 512 to 10000 tokens with bf16 results;
    // the choice cost 1.2 % over the best of the three on average, 15 % at most.
    // 128 x 128 tiles run two an SM, whose starts and epilogues fill each other's
    // gaps but whose MMAs do not overlap the last wave; 256 x 256 tiles on CTA pairs
    // run one an SM; the fp16 kernel divides its last wave, after both operands were
    // widened.  8192 x 8192 weights, 512 / 1024 / 1536 / 4097 tokens: 56 / 109 / 165 /
    // - us, 46 / 92 / 138 / 363 and 91 / 123 / 158 / 344; 4096 x 512, 4097 tokens: 31,
    // 38, 35; 1024 x 8192, 4097 tokens: 72, 62, 72.
    const double k = K / 1000.0, pairs = (M + 255) / 256 * ((N + 255) / 256), wave = sms / 2;
    const double round_tiles = std::ceil(tiles / (2.0 * sms));
    const double tile = 3.4 + 4.6 * std::max(1.0, tiles / (2.0 * sms)) + 6.3 * k * round_tiles;
    const double pair = 2.5 + std::ceil(pairs / wave) * (6.2 + 5.3 * k);
    const double wide = 12.5 + 0.75e-3 * (static_cast<double>(N) + M) * k + pairs / wave * (3.9 + 3.45 * k);
    return tile <= std::min(pair, wide) ? kTile : pair <= wide ? kPair : kWide;
}

// The kernel may start before the one that makes the tokens' codes has
// finished (it waits for it before it reads them, see grid_wait).
unsigned dependent(cudaLaunchAttribute& attr) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    return 1;
}

// Channels over x, tiles of tokens over y and z (token_tile).
dim3 tile_grid(int64_t x, int64_t token_tiles) {
    const int64_t z = (token_tiles + 65534) / 65535;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>((token_tiles + z - 1) / z), static_cast<unsigned>(z));
}

template <int MT, int R>
gemm_status_t launch_dot(gemm_plan* plan, const tcdt_i8::Params& p, bool after_tokens, gemm_dtype_t out,
                         cudaStream_t s) {
    // warps that share a channel's row: few channels otherwise leave SMs idle
    tcdt_i8::Params q = p;
    const int64_t groups = (p.N + R - 1) / R;
    q.splits = 1;
    while (q.splits < tcdt_i8::kDotWarps && groups * q.splits < 16LL * plan->sm_count && p.K / 16 >= 64 * q.splits)
        q.splits *= 2;
    const int64_t per_block = tcdt_i8::kDotWarps / q.splits;
    const unsigned grid = static_cast<unsigned>((groups + per_block - 1) / per_block);
    auto kernel = out == GEMM_F32   ? tcdt_i8::dot_kernel<MT, R, tcdt::kOutF32>
                  : out == GEMM_F16 ? tcdt_i8::dot_kernel<MT, R, tcdt::kOutF16>
                                    : tcdt_i8::dot_kernel<MT, R, tcdt::kOutBF16>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(tcdt_i8::kDotWarps * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = after_tokens ? dependent(attr[0]) : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, q) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    ++plan->launches;
    return GEMM_OK;
}

template <int BN, int OUT>
gemm_status_t launch_tile(gemm_plan* plan, tcdt_i8::Params p, const __half* x, int64_t ldx, cudaStream_t s) {
    using Cfg = tcdt_i8::TileConfig<BN>;
    CUtensorMap tmW, tmX;
    gemm_status_t st = encode_map(plan, &tmW, p.B, static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N),
                                  static_cast<uint64_t>(p.ldb), Cfg::KS, 128, GEMM_E4M3,
                                  Cfg::KS == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (st == GEMM_OK)
        st = encode_map(plan, &tmX, x, static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M),
                        static_cast<uint64_t>(ldx), 64, BN, GEMM_F16);
    if (st != GEMM_OK) return st;
    p.idesc = make_idesc(true, 0, false, false, 128, BN);
    p.status = plan->d_status;
    p.timeout_ns = plan->timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    p.fi_skip_load = plan->fi_skip_load;
#endif
    const int64_t tiles_n = (p.N + 127) / 128, tiles_m = (p.M + BN - 1) / BN;
    const int64_t blocks = (p.K + Cfg::KS - 1) / Cfg::KS;
    // CTAs that share a tile's K.  Four while all run at once (2048 x 2048
    // weights, 16 tokens: 10.3 us with 1, 8.0 with 2, 6.6 with 4, 6.8 with 8);
    // eight only where that leaves half of the SMs idle (1024 x 8192: 10.8 us
    // with 4, 8.4 with 8).
    const int64_t tiles = tiles_n * tiles_m;
    p.splits = 1;
    while (p.splits < 4 && tiles * p.splits * 2 <= 2 * static_cast<int64_t>(plan->sm_count) && blocks >= 2 * p.splits)
        p.splits *= 2;
    if (p.splits == 4 && tiles * 8 <= plan->sm_count / 2 && blocks >= 16) p.splits = 8;
    auto kernel = tcdt_i8::tile_kernel<BN, OUT>;
    bool& prepared = plan->i8_prepared[BN == 16 ? 0 : BN == 32 ? 1 : BN == 64 ? 2 : 3][OUT];
    if (!prepared && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    prepared = true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = tile_grid(tiles_n * p.splits, tiles_m);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    cfg.numAttrs = dependent(attr[0]);
    if (p.splits > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    ++plan->launches;
    return GEMM_OK;
}

template <int BN>
gemm_status_t launch_tile_out(gemm_plan* plan, const tcdt_i8::Params& p, const __half* x, int64_t ldx,
                              gemm_dtype_t out, cudaStream_t s) {
    if (out == GEMM_F32) return launch_tile<BN, tcdt::kOutF32>(plan, p, x, ldx, s);
    if (out == GEMM_F16) return launch_tile<BN, tcdt::kOutF16>(plan, p, x, ldx, s);
    return launch_tile<BN, tcdt::kOutBF16>(plan, p, x, ldx, s);
}

template <int OUT>
gemm_status_t launch_pair(gemm_plan* plan, tcdt_i8::Params p, const __half* x, int64_t ldx, cudaStream_t s) {
    using Cfg = tcdt_i8::PairConfig;
    CUtensorMap tmW, tmX;
    gemm_status_t st = encode_map(plan, &tmW, p.B, static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N),
                                  static_cast<uint64_t>(p.ldb), Cfg::KS, 128, GEMM_E4M3, CU_TENSOR_MAP_SWIZZLE_64B);
    if (st == GEMM_OK)
        st = encode_map(plan, &tmX, x, static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M),
                        static_cast<uint64_t>(ldx), 64, Cfg::BN / 2, GEMM_F16);
    if (st != GEMM_OK) return st;
    p.idesc = make_idesc(true, 0, false, false, 256, Cfg::BN);
    p.status = plan->d_status;
    p.timeout_ns = plan->timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    p.fi_skip_load = plan->fi_skip_load;
#endif
    auto kernel = tcdt_i8::pair_kernel<OUT>;
    bool& prepared = plan->i8_prepared[4][OUT];
    if (!prepared && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    prepared = true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = tile_grid((p.N + int64_t{255}) / 256 * 2, (p.M + int64_t{Cfg::BN - 1}) / Cfg::BN);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    cfg.numAttrs = 1 + dependent(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    ++plan->launches;
    return GEMM_OK;
}

// The product once arguments are checked: A's codes as given, or made from X
// in the plan's buffer, where the tokens (and on the wide path the weights)
// also become fp16.
gemm_status_t run_product(gemm_plan* plan, const int8_t* A, const void* X, gemm_dtype_t xt, const int8_t* B, void* D,
                          int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd, gemm_dtype_t out,
                          const gemm_epilogue_t* ep_in, cudaStream_t s) {
    gemm_epilogue_t ep{};
    if (ep_in) ep = *ep_in;
    if (K == 0) return run_keep_nan(plan, nullptr, nullptr, D, M, N, 0, 8, 8, ldd, out, &ep, s);
    const Path path = path_of(M, N, K, plan->sm_count);
    const int64_t ldh = round_up(K, path == kDot ? 16 : 8);
    const size_t a_bytes = static_cast<size_t>(round_up(M * ldh * (path == kDot ? 1 : 2), 256));
    const size_t b_bytes = path == kWide ? static_cast<size_t>(round_up(N * ldh * 2, 256)) : 0;
    gemm_status_t st = reserve(plan, a_bytes + b_bytes + static_cast<size_t>(M) * 4);
    if (st != GEMM_OK) return st;
    char* ws = static_cast<char*>(plan->d_i8[plan->i8_buffers - 1]);
    __half* a = reinterpret_cast<__half*>(ws);
    __half* b = reinterpret_cast<__half*>(ws + a_bytes);
    float* rs = reinterpret_cast<float*>(ws + a_bytes + b_bytes);
    if (X) {
        st = path == kDot ? launch_quantize(X, xt, M, K, lda, reinterpret_cast<int8_t*>(ws), ldh, rs, s)
                          : launch_quantize(X, xt, M, K, lda, a, ldh, rs, s);
        if (st == GEMM_OK) ++plan->launches;
        ep.row_scale = rs;
    } else if (path != kDot) {
        st = launch_widen(plan, A, lda, a, ldh, M, K, s);
    }
    if (st != GEMM_OK) return st;
    if (path == kWide) {
        st = launch_widen(plan, B, ldb, b, ldh, N, K, s);
        if (st != GEMM_OK) return st;
        return run_keep_nan(plan, a, b, D, M, N, K, ldh, ldh, ldd, out, &ep, s);
    }
    tcdt_i8::Params p{};
    p.M = static_cast<int32_t>(M), p.N = static_cast<int32_t>(N), p.K = static_cast<int32_t>(K);
    p.A = X ? reinterpret_cast<const int8_t*>(ws) : A;
    p.lda = X ? ldh : lda;
    p.B = B, p.ldb = ldb;
    p.D = D, p.ldd = ldd;
    p.rs = ep.row_scale, p.cs = ep.col_scale, p.bias = ep.bias;
    p.act = static_cast<uint32_t>(ep.act);
    if (path == kDot) {
        if (M == 1) return launch_dot<1, 2>(plan, p, X != nullptr, out, s);
        if (M == 2) return launch_dot<2, 2>(plan, p, X != nullptr, out, s);
        if (M <= 4) return launch_dot<4, 4>(plan, p, X != nullptr, out, s);
        return launch_dot<8, 4>(plan, p, X != nullptr, out, s);
    }
    if (path == kPair) {
        if (out == GEMM_F32) return launch_pair<tcdt::kOutF32>(plan, p, a, ldh, s);
        if (out == GEMM_F16) return launch_pair<tcdt::kOutF16>(plan, p, a, ldh, s);
        return launch_pair<tcdt::kOutBF16>(plan, p, a, ldh, s);
    }
    if (M <= 16) return launch_tile_out<16>(plan, p, a, ldh, out, s);
    if (M <= 32) return launch_tile_out<32>(plan, p, a, ldh, out, s);
    // 128 tokens a tile once such tiles are half as many as SMs (8192 x 8192
    // weights, 128 tokens: 23.4 us to 26.5 with 64 a tile; 4096 x 4096: 14.3 to 13.1)
    const int64_t tiles = (N + 127) / 128 * ((M + 127) / 128);
    if (M <= 64 || tiles < 64) return launch_tile_out<64>(plan, p, a, ldh, out, s);
    return launch_tile_out<128>(plan, p, a, ldh, out, s);
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_i8(gemm_plan_t plan, const int8_t* A, const int8_t* B, void* D, int64_t M, int64_t N,
                          int64_t K, int64_t lda, int64_t ldb, int64_t ldd, gemm_dtype_t out_dtype,
                          const gemm_epilogue_t* ep, void* stream) {
    const gemm_status_t st = check_product(plan, B, D, M, N, K, ldb, ldd, out_dtype, ep);
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    if (K > 0) {
        if (!A || lda < K) return GEMM_ERR_INVALID_ARG;
        if (lda > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
        if (!aligned(A, 16) || lda % 16) return GEMM_ERR_MISALIGNED;
    }
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    return run_product(plan, A, nullptr, GEMM_F32, B, D, M, N, K, lda, ldb, ldd, out_dtype, ep,
                       static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_i8_dynamic(gemm_plan_t plan, const void* X, gemm_dtype_t x_dtype, const int8_t* B, void* D,
                                  int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldb, int64_t ldd,
                                  gemm_dtype_t out_dtype, const gemm_epilogue_t* ep, void* stream) {
    if (!float_type(x_dtype) || (ep && ep->row_scale)) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_product(plan, B, D, M, N, K, ldb, ldd, out_dtype, ep);
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    if (K > 0) {
        if (!X || ldx < K) return GEMM_ERR_INVALID_ARG;
        if (ldx > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
        if (!aligned(X, x_dtype == GEMM_F32 ? 4 : 2)) return GEMM_ERR_MISALIGNED;
    }
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    return run_product(plan, nullptr, X, x_dtype, B, D, M, N, K, ldx, ldb, ldd, out_dtype, ep,
                       static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_quantize_rows_i8(int device, const void* X, gemm_dtype_t x_dtype, int64_t R, int64_t K,
                                    int64_t ldx, int8_t* Q, int64_t ldq, float* scale, void* stream) {
    if (!float_type(x_dtype) || R < 0 || K < 0 || ldx < K || ldq < K) return GEMM_ERR_INVALID_ARG;
    if (R > kMaxExtent || K > kMaxExtent || ldx > (int64_t(1) << 40) || ldq > (int64_t(1) << 40))
        return GEMM_ERR_UNSUPPORTED;
    if (R > 0 && (!scale || (K > 0 && (!X || !Q)))) return GEMM_ERR_INVALID_ARG;
    if (!aligned(X, x_dtype == GEMM_F32 ? 4 : 2) || !aligned(scale, 4)) return GEMM_ERR_MISALIGNED;
    int count = 0;
    if (device < 0) return GEMM_ERR_INVALID_ARG;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count <= 0) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (device >= count) return GEMM_ERR_INVALID_ARG;
    if (R == 0) return GEMM_OK;
    const OnDevice on(device);
    if (!on.ok) return GEMM_ERR_CUDA;
    return launch_quantize(X, x_dtype, R, K, ldx, Q, ldq, scale, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
