// adapters.cu -- low-rank adapters of many requests beside a shared product, and
// the gradients of their factors (include/adapters.h).
//
//     h[i] = s A X[i],   D[i] = W^T X[i] + bias + U h[i]
//     d_down[g] = sum of p[i] X[i]^T,   d_up[g] = sum of dD[i] h[i]^T over the rows of g
//
// h and p are kept as a high and a low part of the plan's type, high = round(h) and
// low = round(h - high): products with both, added in fp32, lose 2^-17 (bf16) of h,
// where high alone would lose 2^-9, as much as the rounding of D.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "adapters.h"
#include "gemm_internal.cuh"

using namespace tcdt_host;

namespace {

constexpr int kThreads = 256;

// A stack of matrices, element (g, i, j) at p + g * stride + i * si + j * sj.
struct Stack {
    const void* p;
    int64_t stride, si, sj;
};

struct Rows {
    const int32_t* index;
    const float* scale;
    int32_t count, rank, part;      // part: columns of the high parts, and of the low ones
    int64_t M;
};

__device__ __forceinline__ float value(__half x) { return __half2float(x); }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(float x) { return x; }
template <typename E>
__device__ __forceinline__ E rounded(float x);
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }

// The adapter of a row, -1 for none.
__device__ __forceinline__ int adapter_of(const Rows& a, int64_t i) {
    const int g = a.index[i];
    return g >= 0 && g < a.count ? g : -1;
}

// h as its two parts; an infinity or a NaN is all in the high one.
template <typename E>
__device__ __forceinline__ void store_hidden(E* row, int r, int part, float h) {
    const E high = rounded<E>(h);
    const float rest = h - value(high);
    row[r] = high;
    row[part + r] = rounded<E>(isfinite(value(high)) ? rest : 0.f);
}

template <typename E>
__device__ __forceinline__ float load_hidden(const E* row, int r, int part) {
    return value(row[r]) + value(row[part + r]);
}

// h of a row, one CTA a row.
template <typename E>
__global__ void __launch_bounds__(kThreads) hidden_kernel(const Rows a, const E* X, int64_t ldx, int64_t K,
                                                          const Stack down, E* hidden, int64_t ldh) {
    const int64_t i = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = adapter_of(a, i);
    const E* x = X + i * ldx;
    E* row = hidden + i * ldh;
    const float s = g < 0 ? 0.f : a.scale ? a.scale[g] : 1.f;
    const E* A = static_cast<const E*>(down.p) + (g < 0 ? 0 : g) * down.stride;
    for (int r = a.rank + tid; r < a.part; r += kThreads) store_hidden<E>(row, r, a.part, 0.f);
    for (int r0 = 0; r0 < a.rank; r0 += kThreads / 32) {
        const int r = r0 + warp;
        float h = 0.f;
        if (g >= 0 && r < a.rank)
            for (int64_t k = lane; k < K; k += 32) h = fmaf(value(x[k]), value(A[r * down.si + k * down.sj]), h);
        for (int o = 16; o; o >>= 1) h += __shfl_xor_sync(~0u, h, o);
        if (lane == 0 && r < a.rank) store_hidden<E>(row, r, a.part, g < 0 ? 0.f : s * h);
    }
}

// D = work + bias + U h.
template <typename E, typename O>
__global__ void __launch_bounds__(kThreads) add_kernel(const Rows a, const float* work, const float* bias, int64_t N,
                                                       const Stack up, const E* hidden, int64_t ldh, O* D, int64_t ldd) {
    __shared__ float h[GEMM_ADAPTERS_MAX_RANK];
    const int64_t i = blockIdx.x;
    const int g = adapter_of(a, i);
    if (threadIdx.x < a.rank) h[threadIdx.x] = load_hidden<E>(hidden + i * ldh, threadIdx.x, a.part);
    __syncthreads();
    const int64_t n = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
    if (n >= N) return;
    const E* U = static_cast<const E*>(up.p) + (g < 0 ? 0 : g) * up.stride + n * up.si;
    float y = 0.f;
    if (g >= 0)
        for (int r = 0; r < a.rank; ++r) y = fmaf(value(U[r * up.sj]), h[r], y);
    y += work[i * N + n];
    D[i * ldd + n] = rounded<O>(bias ? y + bias[n] : y);
}

// sum over an adapter's rows of left[i] right[i]^T for 16 of the rank's values and
// 256 columns: out[g * stride + r * sr + c * sc].
template <typename E, typename O>
__global__ void __launch_bounds__(kThreads) factor_grad_kernel(const Rows a, const E* hidden, int64_t ldh, const E* X,
                                                               int64_t ldx, int64_t columns, O* out, int64_t stride,
                                                               int64_t sr, int64_t sc) {
    const int g = blockIdx.z, r0 = blockIdx.y * 16;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    float sum[16] = {};
    for (int64_t i = 0; i < a.M; ++i) {
        if (adapter_of(a, i) != g) continue;
        const float x = c < columns ? value(X[i * ldx + c]) : 0.f;
        for (int r = 0; r < 16; ++r)
            if (r0 + r < a.rank) sum[r] = fmaf(load_hidden<E>(hidden + i * ldh, r0 + r, a.part), x, sum[r]);
    }
    if (c >= columns) return;
    for (int r = 0; r < 16; ++r)
        if (r0 + r < a.rank) out[g * stride + (r0 + r) * sr + c * sc] = rounded<O>(sum[r]);
}

// ---- host ------------------------------------------------------------------
constexpr int64_t kMaxExtent = 0x7FFFF000;
constexpr int64_t kMaxStride = int64_t(1) << 40;
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool layout_ok(gemm_layout_t l) { return l == GEMM_ROW_MAJOR || l == GEMM_COL_MAJOR; }

int part_of(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

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

gemm_status_t check_adapters(const gemm_plan* plan, int64_t M, int64_t N, int64_t K, gemm_dtype_t out,
                             const gemm_adapters_t* a) {
    if (!plan || !a || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (a->count < 0 || a->rank < 1 || a->rank > GEMM_ADAPTERS_MAX_RANK) return GEMM_ERR_INVALID_ARG;
    if (out != GEMM_F32 && out != GEMM_F16 && out != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (plan->in_dtype != GEMM_F16 && plan->in_dtype != GEMM_BF16) return GEMM_ERR_UNSUPPORTED;
    if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent || a->count > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    if (M > 0 && !a->index) return GEMM_ERR_INVALID_ARG;
    if (!aligned(a->index, 4) || !aligned(a->scale, 4)) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

// A stack of count matrices of rows x cols, rows of ld elements that start on
// 16-byte boundaries.
gemm_status_t check_stack(int64_t count, const void* p, int64_t inner, int64_t ld, int64_t stride) {
    if (count == 0) return GEMM_OK;
    if (!p || ld < inner || stride < 0) return GEMM_ERR_INVALID_ARG;
    if (ld > kMaxStride || stride > kMaxStride) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || ld % 8 || (count > 1 && stride % 8)) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

gemm_status_t check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!p || ld < cols) return GEMM_ERR_INVALID_ARG;
    if (ld > kMaxStride) return GEMM_ERR_UNSUPPORTED;
    return aligned(p, 16) && ld % 8 == 0 ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

Rows rows_of(const gemm_adapters_t& a, int64_t M) {
    return {a.index, a.scale, static_cast<int32_t>(a.count), static_cast<int32_t>(a.rank), part_of(a.rank), M};
}

gemm_status_t launched(gemm_plan* plan) {
    if (cudaGetLastError() != cudaSuccess) return GEMM_ERR_CUDA;
    ++plan->launches;
    return GEMM_OK;
}

template <typename E>
gemm_status_t run_hidden(gemm_plan* plan, const Rows& r, const void* X, int64_t ldx, int64_t K, const Stack& down,
                         void* hidden, int64_t ldh, cudaStream_t s) {
    if (r.M == 0) return GEMM_OK;
    hidden_kernel<E><<<static_cast<unsigned>(r.M), kThreads, 0, s>>>(r, static_cast<const E*>(X), ldx, K, down,
                                                                     static_cast<E*>(hidden), ldh);
    return launched(plan);
}

template <typename E>
gemm_status_t run_add(gemm_plan* plan, const Rows& r, const void* work, const float* bias, int64_t N, const Stack& up,
                      const void* hidden, int64_t ldh, gemm_dtype_t out, void* D, int64_t ldd, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(r.M), static_cast<unsigned>((N + kThreads - 1) / kThreads), 1);
    const float* w = static_cast<const float*>(work);
    const E* h = static_cast<const E*>(hidden);
    if (out == GEMM_F32) add_kernel<E, float><<<grid, kThreads, 0, s>>>(r, w, bias, N, up, h, ldh, static_cast<float*>(D), ldd);
    else if (out == GEMM_F16) add_kernel<E, __half><<<grid, kThreads, 0, s>>>(r, w, bias, N, up, h, ldh, static_cast<__half*>(D), ldd);
    else add_kernel<E, __nv_bfloat16><<<grid, kThreads, 0, s>>>(r, w, bias, N, up, h, ldh, static_cast<__nv_bfloat16*>(D), ldd);
    return launched(plan);
}

template <typename E>
gemm_status_t run_factor_grad(gemm_plan* plan, const Rows& r, const void* hidden, int64_t ldh, const void* X, int64_t ldx,
                              int64_t columns, gemm_dtype_t out, void* d, int64_t stride, int64_t sr, int64_t sc,
                              cudaStream_t s) {
    if (!d || columns == 0 || r.count == 0) return GEMM_OK;
    const dim3 grid(static_cast<unsigned>((columns + kThreads - 1) / kThreads), static_cast<unsigned>((r.rank + 15) / 16),
                    static_cast<unsigned>(r.count));
    const E *h = static_cast<const E*>(hidden), *x = static_cast<const E*>(X);
    if (out == GEMM_F32) factor_grad_kernel<E, float><<<grid, kThreads, 0, s>>>(r, h, ldh, x, ldx, columns, static_cast<float*>(d), stride, sr, sc);
    else factor_grad_kernel<E, E><<<grid, kThreads, 0, s>>>(r, h, ldh, x, ldx, columns, static_cast<E*>(d), stride, sr, sc);
    return launched(plan);
}

}  // namespace

extern "C" {

int64_t gemm_adapters_hidden_width(int64_t rank) {
    return rank < 1 || rank > GEMM_ADAPTERS_MAX_RANK ? 0 : 2 * part_of(rank);
}

int64_t gemm_adapters_work_bytes(int64_t M, int64_t N) { return M > 0 && N > 0 ? M * N * 4 : 0; }

gemm_status_t gemm_run_adapters(gemm_plan_t plan, const void* X, const void* W, void* D, int64_t M, int64_t N,
                                int64_t K, int64_t ldx, int64_t ldw, int64_t ldd, gemm_layout_t layoutW,
                                gemm_dtype_t out_dtype, const float* bias, const gemm_adapters_t* adapters,
                                void* hidden, int64_t ldh, void* work, void* stream) {
    gemm_status_t st = check_adapters(plan, M, N, K, out_dtype, adapters);
    if (st != GEMM_OK) return st;
    const gemm_adapters_t& a = *adapters;
    if (!layout_ok(layoutW) || !layout_ok(a.down_layout) || !layout_ok(a.up_layout)) return GEMM_ERR_INVALID_ARG;
    st = gemm_validate(plan->in_dtype, X, W, nullptr, D, M, N, K, ldx, ldw, ldd, GEMM_ROW_MAJOR, layoutW, GEMM_F32,
                       out_dtype, 0.0f);
    if (st != GEMM_OK) return st;
    const bool down_row = a.down_layout == GEMM_ROW_MAJOR, up_row = a.up_layout == GEMM_ROW_MAJOR;
    if (K > 0) st = check_stack(a.count, a.down, down_row ? K : a.rank, a.down_ld, a.down_stride);
    if (st == GEMM_OK && N > 0) st = check_stack(a.count, a.up, up_row ? a.rank : N, a.up_ld, a.up_stride);
    if (st == GEMM_OK) st = check_matrix(X, M, K, ldx);
    if (st == GEMM_OK) st = check_matrix(hidden, M, 2 * part_of(a.rank), ldh);
    if (st != GEMM_OK) return st;
    if (gemm_adapters_work_bytes(M, N) > 0 && !work) return GEMM_ERR_INVALID_ARG;
    if (!aligned(bias, 4) || !aligned(work, 16)) return GEMM_ERR_MISALIGNED;
    if (M == 0) return GEMM_OK;
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Rows r = rows_of(a, M);
    const Stack down{a.down, a.down_stride, down_row ? a.down_ld : 1, down_row ? 1 : a.down_ld};
    const Stack up{a.up, a.up_stride, up_row ? a.up_ld : 1, up_row ? 1 : a.up_ld};
    const bool half = plan->in_dtype == GEMM_F16;
    st = half ? run_hidden<__half>(plan, r, X, ldx, K, down, hidden, ldh, s)
              : run_hidden<__nv_bfloat16>(plan, r, X, ldx, K, down, hidden, ldh, s);
    if (st != GEMM_OK || N == 0) return st;
    st = gemm_run(plan, X, W, nullptr, work, M, N, K, ldx, ldw, N, GEMM_ROW_MAJOR, layoutW, GEMM_F32, GEMM_F32, 1.0f,
                  0.0f, stream);
    if (st != GEMM_OK) return st;
    return half ? run_add<__half>(plan, r, work, bias, N, up, hidden, ldh, out_dtype, D, ldd, s)
                : run_add<__nv_bfloat16>(plan, r, work, bias, N, up, hidden, ldh, out_dtype, D, ldd, s);
}

gemm_status_t gemm_adapters_grad(gemm_plan_t plan, const void* X, const void* dD, int64_t M, int64_t N, int64_t K,
                                 int64_t ldx, int64_t lddd, const gemm_adapters_t* adapters, const void* h,
                                 const void* p, int64_t ldh, gemm_dtype_t out_dtype, void* d_down, int64_t down_ld,
                                 int64_t down_stride, void* d_up, int64_t up_ld, int64_t up_stride, void* stream) {
    gemm_status_t st = check_adapters(plan, M, N, K, out_dtype, adapters);
    if (st != GEMM_OK) return st;
    if (out_dtype != GEMM_F32 && out_dtype != plan->in_dtype) return GEMM_ERR_UNSUPPORTED;
    const gemm_adapters_t& a = *adapters;
    const int64_t width = 2 * part_of(a.rank);
    if (d_down) {
        st = check_matrix(X, M, K, ldx);
        if (st == GEMM_OK) st = check_matrix(p, M, width, ldh);
        if (st == GEMM_OK && (down_ld < K || down_stride < 0)) st = GEMM_ERR_INVALID_ARG;
        if (st == GEMM_OK && (down_ld > kMaxStride || down_stride > kMaxStride)) st = GEMM_ERR_UNSUPPORTED;
    }
    if (d_up && st == GEMM_OK) {
        st = check_matrix(dD, M, N, lddd);
        if (st == GEMM_OK) st = check_matrix(h, M, width, ldh);
        if (st == GEMM_OK && (up_ld < a.rank || up_stride < 0)) st = GEMM_ERR_INVALID_ARG;
        if (st == GEMM_OK && (up_ld > kMaxStride || up_stride > kMaxStride)) st = GEMM_ERR_UNSUPPORTED;
    }
    if (st != GEMM_OK) return st;
    const uintptr_t esz = out_dtype == GEMM_F32 ? 4 : 2;
    if (!aligned(d_down, esz) || !aligned(d_up, esz)) return GEMM_ERR_MISALIGNED;
    if (a.count == 0 || (!d_down && !d_up)) return GEMM_OK;
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Rows r = rows_of(a, M);
    if (plan->in_dtype == GEMM_F16) {
        st = run_factor_grad<__half>(plan, r, p, ldh, X, ldx, K, out_dtype, d_down, down_stride, down_ld, 1, s);
        if (st == GEMM_OK) st = run_factor_grad<__half>(plan, r, h, ldh, dD, lddd, N, out_dtype, d_up, up_stride, 1, up_ld, s);
    } else {
        st = run_factor_grad<__nv_bfloat16>(plan, r, p, ldh, X, ldx, K, out_dtype, d_down, down_stride, down_ld, 1, s);
        if (st == GEMM_OK) st = run_factor_grad<__nv_bfloat16>(plan, r, h, ldh, dD, lddd, N, out_dtype, d_up, up_stride, 1, up_ld, s);
    }
    return st;
}

}  // extern "C"
