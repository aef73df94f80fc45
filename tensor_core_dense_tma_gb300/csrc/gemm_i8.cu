// gemm_i8.cu -- the product of 8-bit integers with a scale for each token
// (row of A) and channel (column of B), and the quantisation of rows
// (gemm_run_i8, gemm_run_i8_dynamic, gemm_quantize_rows_i8 of gemm.h).
//
//     D[i,j] = act(rs[i] cs[j] sum_k A[i,k] B[k,j] + bias[j])
//
// sm_103a has no 8-bit integer MMA on tcgen05.  An int8 value is exact in
// fp16 and the product of two is exact in fp32 (at most 2^14), so the codes
// are multiplied as fp16 with fp32 accumulation: every partial sum below
// 2^24 is exact (any K up to 1040; for larger K whenever the sums stay below
// it), larger ones round as fp32 sums do.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm.h"
#include "gemm_internal.cuh"

using namespace tcdt_host;

namespace {

constexpr int kThreads = 256;

// int8 rows (ld elements apart, 16-byte aligned) as fp16 rows (ldh apart),
// zero in columns K..ldh-1; 16 codes a thread.
__global__ void __launch_bounds__(kThreads) widen_kernel(const int8_t* q, int64_t ld, __half* h, int64_t ldh,
                                                         int64_t rows, int32_t K) {
    const int32_t per_row = static_cast<int32_t>((K + 15) / 16);
    const int64_t total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / per_row;
        const int32_t k = static_cast<int32_t>(i - r * per_row) * 16;
        const int8_t* src = q + r * ld + k;
        __half* dst = h + r * ldh + k;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (k + e < ldh) dst[e] = k + e < K ? __short2half_rn(src[e]) : __half(0.f);
    }
}

template <typename E>
__device__ __forceinline__ float as_float(E x) { return static_cast<float>(x); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ void store_code(int8_t* p, float q) { *p = static_cast<int8_t>(__float2int_rn(q)); }
__device__ __forceinline__ void store_code(__half* p, float q) { *p = __int2half_rn(__float2int_rn(q)); }

// One CTA a row: scale = max |x| / 127, code = round(x / scale), both
// divisions IEEE so that the codes are those of the definition.  A row of
// zeros has scale 0 and codes 0.
template <typename E, typename Q>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const E* x, int64_t ldx, Q* q, int64_t ldq, float* scale,
                                                            int32_t K) {
    __shared__ float part[kThreads / 32];
    const int64_t r = blockIdx.x;
    const E* row = x + r * ldx;
    float top = 0.f;
    for (int32_t k = threadIdx.x; k < K; k += kThreads) top = max_nan(top, fabsf(as_float(row[k])));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max_nan(top, part[w]);
    const float s = __fdiv_rn(top, 127.f);
    if (threadIdx.x == 0) scale[r] = s;
    for (int32_t k = threadIdx.x; k < K; k += kThreads) {
        const float c = s != 0.f ? __fdiv_rn(as_float(row[k]), s) : 0.f;
        store_code(q + r * ldq + k, fminf(fmaxf(c, -127.f), 127.f));
    }
}

template <typename Q>
gemm_status_t launch_quantize(const void* x, gemm_dtype_t t, int64_t R, int64_t K, int64_t ldx, Q* q, int64_t ldq,
                              float* scale, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(R);
    const int32_t k = static_cast<int32_t>(K);
    if (t == GEMM_F32)
        quantize_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float*>(x), ldx, q, ldq, scale, k);
    else if (t == GEMM_F16)
        quantize_kernel<<<grid, kThreads, 0, s>>>(static_cast<const __half*>(x), ldx, q, ldq, scale, k);
    else
        quantize_kernel<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx, q, ldq, scale, k);
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

// The plan's buffer for fp16 codes and row scales, grown to `bytes`.
gemm_status_t reserve(gemm_plan* plan, size_t bytes) {
    if (bytes <= plan->i8_bytes) return GEMM_OK;
    if (plan->d_i8) cudaFree(plan->d_i8);    // waits for kernels that still use it
    plan->d_i8 = nullptr;
    plan->i8_bytes = 0;
    if (cudaMalloc(&plan->d_i8, bytes) != cudaSuccess) {
        cudaGetLastError();
        plan->d_i8 = nullptr;
        return GEMM_ERR_CUDA;
    }
    plan->i8_bytes = bytes;
    return GEMM_OK;
}

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
    if (!aligned(D, out == GEMM_F32 ? 4 : 2)) return GEMM_ERR_MISALIGNED;
    if (K == 0) return GEMM_OK;
    if (!B || ldb < K) return GEMM_ERR_INVALID_ARG;
    if (!aligned(B, 16) || ldb % 16) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

// The product once A's codes are to be put into the plan's buffer as fp16
// rows: either widened from int8 (A) or quantised from X.
gemm_status_t run_product(gemm_plan* plan, const int8_t* A, const void* X, gemm_dtype_t xt, const int8_t* B, void* D,
                          int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd, gemm_dtype_t out,
                          const gemm_epilogue_t* ep_in, cudaStream_t s) {
    gemm_epilogue_t ep{};
    if (ep_in) ep = *ep_in;
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess || (prev != plan->device && cudaSetDevice(plan->device) != cudaSuccess)) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    const int64_t ldh = round_up(K, 8);
    const size_t a_bytes = static_cast<size_t>(round_up(M * ldh * 2, 256));
    const size_t b_bytes = static_cast<size_t>(round_up(N * ldh * 2, 256));
    gemm_status_t st = reserve(plan, a_bytes + b_bytes + static_cast<size_t>(M) * 4);
    if (st == GEMM_OK) {
        char* ws = static_cast<char*>(plan->d_i8);
        __half* a = reinterpret_cast<__half*>(ws);
        __half* b = reinterpret_cast<__half*>(ws + a_bytes);
        float* rs = reinterpret_cast<float*>(ws + a_bytes + b_bytes);
        if (X) {
            st = launch_quantize(X, xt, M, K, lda, a, ldh, rs, s);
            ++plan->launches;
            ep.row_scale = rs;
        } else {
            st = launch_widen(plan, A, lda, a, ldh, M, K, s);
        }
        if (st == GEMM_OK) st = launch_widen(plan, B, ldb, b, ldh, N, K, s);
        if (st == GEMM_OK)
            st = gemm_run_ep(plan, a, b, nullptr, D, M, N, K, ldh, ldh, ldd, GEMM_ROW_MAJOR, GEMM_COL_MAJOR, GEMM_F32,
                             out, 1.0f, 0.0f, &ep, s);
    }
    if (prev != plan->device) cudaSetDevice(prev);
    return st;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_i8(gemm_plan_t plan, const int8_t* A, const int8_t* B, void* D, int64_t M, int64_t N,
                          int64_t K, int64_t lda, int64_t ldb, int64_t ldd, gemm_dtype_t out_dtype,
                          const gemm_epilogue_t* ep, void* stream) {
    const gemm_status_t st = check_product(plan, B, D, M, N, K, ldb, ldd, out_dtype, ep);
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    if (K == 0)
        return gemm_run_ep(plan, nullptr, nullptr, nullptr, D, M, N, 0, 8, 8, ldd, GEMM_ROW_MAJOR, GEMM_COL_MAJOR,
                           GEMM_F32, out_dtype, 1.0f, 0.0f, ep, stream);
    if (!A || lda < K) return GEMM_ERR_INVALID_ARG;
    if (lda > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(A, 16) || lda % 16) return GEMM_ERR_MISALIGNED;
    return run_product(plan, A, nullptr, GEMM_F32, B, D, M, N, K, lda, ldb, ldd, out_dtype, ep,
                       static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_i8_dynamic(gemm_plan_t plan, const void* X, gemm_dtype_t x_dtype, const int8_t* B, void* D,
                                  int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldb, int64_t ldd,
                                  gemm_dtype_t out_dtype, const gemm_epilogue_t* ep, void* stream) {
    if (!float_type(x_dtype) || (ep && ep->row_scale)) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_product(plan, B, D, M, N, K, ldb, ldd, out_dtype, ep);
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    if (K == 0)
        return gemm_run_ep(plan, nullptr, nullptr, nullptr, D, M, N, 0, 8, 8, ldd, GEMM_ROW_MAJOR, GEMM_COL_MAJOR,
                           GEMM_F32, out_dtype, 1.0f, 0.0f, ep, stream);
    if (!X || ldx < K) return GEMM_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 40)) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(X, x_dtype == GEMM_F32 ? 4 : 2)) return GEMM_ERR_MISALIGNED;
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
    int count = 0, prev = -1;
    if (device < 0) return GEMM_ERR_INVALID_ARG;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count <= 0) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (device >= count) return GEMM_ERR_INVALID_ARG;
    if (R == 0) return GEMM_OK;
    if (cudaGetDevice(&prev) != cudaSuccess || (prev != device && cudaSetDevice(device) != cudaSuccess)) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    const gemm_status_t st = launch_quantize(X, x_dtype, R, K, ldx, Q, ldq, scale, static_cast<cudaStream_t>(stream));
    if (prev != device) cudaSetDevice(prev);
    return st;
}

}  // extern "C"
