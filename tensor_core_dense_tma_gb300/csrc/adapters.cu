// adapters.cu -- low-rank adapters of many requests beside a shared product, and
// the gradients of their factors (include/adapters.h).
//
//     h[i] = s A X[i],   D[i] = W^T X[i] + bias + U h[i]
//     d_down[g] = sum of p[i] X[i]^T,   d_up[g] = sum of dD[i] h[i]^T over the rows of g
//
// h and p are kept as a high and a low part of the plan's type, high = round(h) and
// low = round(h - high): products with both, added in fp32, lose 2^-17 (bf16) of h,
// where high alone would lose 2^-9, as much as the rounding of D.  fp16 has no low parts below
// 2^-24; the gradients of the factors, whose sums over high and low parts are apart until they
// are stored, can have them times 2^11 (a third part: the product adds both in one sum).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "adapters.h"
#include "adapters_kernel.cuh"
#include "gemm_internal.cuh"

using namespace tcdt_host;

namespace {

using tcdt::adapter_split;
using tcdt::adapter_value;
using tcdt::FactorGradArgs;
using tcdt::HiddenArgs;

// ---- h of a few rows ---------------------------------------------------------
// One CTA for a row and four of its values: X and four rows of A are read once,
// 16 bytes a load, all loads of a thread under way together (K = 8192: four
// of X and sixteen of A), so a call takes about as long as one trip to memory.  With
// more rows X and A come again from L2 each time: hidden_tile_kernel then.
constexpr int kRowThreads = 256, kRowValues = 4;

struct RowArgs {
    const uint16_t* X;
    int64_t ldx, K;
    const uint16_t* down;             // [adapter][rank][K]
    int64_t down_ld, down_stride;
    const int32_t* index;
    const float* scale;
    int32_t count, rank, part;
    uint32_t wide;                    // 1: low, high and low parts times 2^11, else high and low ones
    uint16_t* hidden;
    int64_t ldh;
    uint32_t bf16;
};

__device__ __forceinline__ void unpack8(const uint4& v, bool bf16, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = adapter_value(w[e] & 0xFFFFu, bf16);
        x[2 * e + 1] = adapter_value(w[e] >> 16, bf16);
    }
}

__global__ void __launch_bounds__(kRowThreads) hidden_rows_kernel(const RowArgs a) {
    __shared__ float part[kRowThreads / 32][kRowValues];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t i = blockIdx.y;
    const int r0 = blockIdx.x * kRowValues;
    const bool bf16 = a.bf16 != 0;
    tcdt::griddep_launch();
    const int g = a.index[i];
    float sum[kRowValues] = {};
    const bool mine = g >= 0 && g < a.count && r0 < a.rank;
    if (mine) {
        const uint16_t* x = a.X + i * a.ldx;
        const uint16_t* A[kRowValues];
#pragma unroll
        for (int r = 0; r < kRowValues; ++r) A[r] = a.down + g * a.down_stride + min(r0 + r, a.rank - 1) * a.down_ld;
        const int64_t vectors = a.K >> 3;
#pragma unroll 4
        for (int64_t v = tid; v < vectors; v += kRowThreads) {
            float xv[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(x) + v), bf16, xv);
#pragma unroll
            for (int r = 0; r < kRowValues; ++r) {
                float av[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(A[r]) + v), bf16, av);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[r] = fmaf(xv[e], av[e], sum[r]);
            }
        }
        const int64_t k = vectors * 8 + tid;
        if (k < a.K) {
            const float xv = adapter_value(x[k], bf16);
#pragma unroll
            for (int r = 0; r < kRowValues; ++r) sum[r] = fmaf(xv, adapter_value(A[r][k], bf16), sum[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRowValues; ++r) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sum[r] += __shfl_xor_sync(~0u, sum[r], o);
        if (lane == 0) part[warp][r] = sum[r];
    }
    __syncthreads();
    if (tid < kRowValues) {
        const int r = r0 + tid;
        float h = 0.f;
        for (int w = 0; w < kRowThreads / 32; ++w) h += part[w][tid];
        h = mine && r < a.rank ? (a.scale ? a.scale[g] * h : h) : 0.f;
        uint16_t hi, lo;
        adapter_split(h, bf16, hi, lo);
        uint16_t* out = a.hidden + i * a.ldh + r;
        out[a.wide ? a.part : 0] = hi;
        out[a.wide ? 0 : a.part] = lo;
        if (a.wide) out[2 * a.part] = tcdt::adapter_rest(h, hi);
    }
}

// ---- host ------------------------------------------------------------------
constexpr int64_t kMaxExtent = 0x7FFFF000;
constexpr int64_t kMaxStride = int64_t(1) << 39;      // elements: below 2^40 bytes, what a tensor map takes

// Whether hidden_rows_kernel makes h (down factors K-contiguous): it reads X and A from
// L2 again for every row, so its time goes with rows x rank x K, whatever the rows'
// adapters are, while hidden_tile_kernel takes 6 to 11 us where a tile has one adapter and
// many times that where it has many.  Measured (us), rows / tiles of one adapter / of 64 in
// turn: K = 8192, rank 16: 64 rows 3.4 / 9.5 / 146, 256 rows 8.5 / 9.7 / 146, 512 rows 14 /
// 9.8 / 147; rank 64: 64 rows 8.9 / 11 / 330, 128 rows 15 / 11 / 331, 256 rows 28 / 11 /
// 336; K = 4096, rank 16: 256 rows 6.4 / 7.8, 512 rows 10.8 / 7.8.  2^25 is 256 x 16 x 8192;
// up to 128 rows, most likely tokens of different requests, twice that.
bool by_rows(int64_t M, int part, int64_t K) {
    return M <= 65535 && M * part <= (int64_t(1) << (M <= 128 ? 26 : 25)) / K;
}
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool layout_ok(gemm_layout_t l) { return l == GEMM_ROW_MAJOR || l == GEMM_COL_MAJOR; }

int part_of(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
int64_t hidden_columns(const gemm_adapters_t& a, bool wide) { return (wide ? 3 : 2) * part_of(a.rank); }

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
    if ((a->wide || a->wide_h) && plan->in_dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// A stack of count matrices of rows x cols, rows of ld elements that start on
// 16-byte boundaries.
gemm_status_t check_stack(int64_t count, const void* p, int64_t inner, int64_t ld, int64_t stride) {
    if (count == 0) return GEMM_OK;
    if (!p || ld < inner || stride < 0) return GEMM_ERR_INVALID_ARG;
    if (count > 1 && stride == 0) return GEMM_ERR_INVALID_ARG;
    if (ld >= kMaxStride || stride >= kMaxStride) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || ld % 8 || (count > 1 && stride % 8)) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

gemm_status_t check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!p || ld < cols) return GEMM_ERR_INVALID_ARG;
    if (ld >= kMaxStride) return GEMM_ERR_UNSUPPORTED;
    return aligned(p, 16) && ld % 8 == 0 ? GEMM_OK : GEMM_ERR_MISALIGNED;
}

// A stack that is written: its matrices do not overlap, lying one after another or row by row in turn.
gemm_status_t check_gradient(int64_t count, int64_t rows, int64_t inner, int64_t ld, int64_t stride) {
    if (count == 0 || rows == 0 || inner == 0) return GEMM_OK;
    if (ld < inner || stride < 0) return GEMM_ERR_INVALID_ARG;
    if (ld >= kMaxStride || stride >= kMaxStride) return GEMM_ERR_UNSUPPORTED;
    // whether n rows of `inner` at distances of `step` end before `next`
    auto fits = [&](int64_t n, int64_t step, int64_t next) {
        return next >= inner && (n == 1 || (step > 0 && n - 1 <= (next - inner) / step));
    };
    return count == 1 || fits(rows, ld, stride) || (stride >= inner && fits(count, stride, ld)) ? GEMM_OK
                                                                                               : GEMM_ERR_INVALID_ARG;
}

gemm_status_t launched(gemm_plan* plan, cudaError_t e) {
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    ++plan->launches;
    return GEMM_OK;
}

// One of the two tile kernels, in clusters of `splits` CTAs.
template <typename Args>
gemm_status_t launch_tiles(gemm_plan* plan, void (*kernel)(Args), const Args& a, int64_t ctas, bool& prepared,
                           cudaStream_t s) {
    const int most = tcdt::kAdapterSharedBytes + 1024;
    if (ctas > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED;
    if (!prepared) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        prepared = true;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(tcdt::kAdapterThreads, 1, 1);
    cfg.dynamicSmemBytes = most;
    cfg.stream = s;
    // (they start while the kernel before them ends, and wait for it themselves)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    return launched(plan, cudaLaunchKernelEx(&cfg, kernel, a));
}

// CTAs of a cluster: as many (a power of two) as fill two CTAs an SM once, while each has `least`
// blocks of the long axis.
int splits_of(const gemm_plan* plan, int64_t tiles, int64_t blocks, int64_t least) {
    int s = 1;
    while (s < 8 && tiles * s * 2 <= 2 * plan->sm_count && blocks >= 2 * s * least) s *= 2;
    return s;
}

gemm_status_t run_hidden(gemm_plan* plan, const gemm_adapters_t& a, const void* X, int64_t ldx, int64_t M, int64_t K,
                         void* hidden, int64_t ldh, cudaStream_t s) {
    const bool row = a.down_layout == GEMM_ROW_MAJOR;
    const int part = part_of(a.rank);
    const uint32_t bf16 = plan->in_dtype == GEMM_BF16 ? 1u : 0u;
    if (row && by_rows(M, part, K)) {
        const RowArgs r{static_cast<const uint16_t*>(X), ldx, K, static_cast<const uint16_t*>(a.down), a.down_ld,
                        a.down_stride, a.index, a.scale, static_cast<int32_t>(a.count), static_cast<int32_t>(a.rank), part,
                        a.wide ? 1u : 0u, static_cast<uint16_t*>(hidden), ldh, bf16};
        hidden_rows_kernel<<<dim3(part / kRowValues, static_cast<unsigned>(M)), kRowThreads, 0, s>>>(r);
        return launched(plan, cudaGetLastError());
    }
    HiddenArgs h;
    std::memset(&h, 0, sizeof(h));
    h.index = a.index;
    h.scale = a.scale;
    h.count = static_cast<int32_t>(a.count);
    h.rank = static_cast<int32_t>(a.rank);
    h.part = part;
    h.wide = a.wide ? 1u : 0u;
    h.rr = (h.rank + 15) / 16 * 16;
    h.a_mn = row ? 0u : 1u;
    h.per_stage = row && h.rr <= 32 ? 64 / h.rr : 1;
    h.pitch = row ? h.rr : h.rr <= 64 ? 64 : 128;
    h.idesc = make_idesc(true, input_format(plan->in_dtype), false, !row, 128, h.per_stage * h.pitch);
    h.idesc_one = make_idesc(true, input_format(plan->in_dtype), false, !row, 128, h.rr);
    h.M = static_cast<int32_t>(M);
    const int64_t step = 64 * tcdt::hidden_blocks(h.rr);
    h.k_steps = static_cast<int32_t>((K + step - 1) / step);
    h.splits = splits_of(plan, (M + 127) / 128, h.k_steps, 2);
    const int64_t ctas = (M + 127) / 128 * h.splits;
    h.stages = tcdt::kAdapterSharedBytes / tcdt::hidden_stage_bytes(h.rr);
    h.hidden = static_cast<uint16_t*>(hidden);
    h.ldh = ldh;
    h.bf16 = bf16;
    h.status = plan->d_status;
    h.timeout_ns = plan->timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    h.fi_skip_load = plan->fi_skip_load;
#endif
    gemm_status_t st = encode_map(plan, &h.tmX, X, K, M, ldx, 64, 128, plan->in_dtype);
    if (st == GEMM_OK)
        st = row ? encode_stack(plan, &h.tmA, a.down, K, a.rank, a.count, a.down_ld, a.down_stride, h.rr)
                 : encode_stack(plan, &h.tmA, a.down, a.rank, K, a.count, a.down_ld, a.down_stride, 64);
    if (st != GEMM_OK) return st;
    return launch_tiles(plan, tcdt::hidden_tile_kernel, h, ctas, plan->adapters_prepared[0], s);
}

}  // namespace

extern "C" {

int64_t gemm_adapters_hidden_width(int64_t rank) {
    return rank < 1 || rank > GEMM_ADAPTERS_MAX_RANK ? 0 : 2 * part_of(rank);
}

gemm_status_t gemm_run_adapters(gemm_plan_t plan, const void* X, const void* W, void* D, int64_t M, int64_t N,
                                int64_t K, int64_t ldx, int64_t ldw, int64_t ldd, gemm_layout_t layoutW,
                                gemm_dtype_t out_dtype, const float* bias, const gemm_adapters_t* adapters,
                                void* hidden, int64_t ldh, void* stream) {
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
    if (st == GEMM_OK) st = check_matrix(hidden, M, hidden_columns(a, a.wide), ldh);
    if (st != GEMM_OK) return st;
    if (!aligned(bias, 4)) return GEMM_ERR_MISALIGNED;
    if (M == 0) return GEMM_OK;
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0 || a.count == 0) {
        // no adapter adds anything
        st = launched(plan, cudaMemset2DAsync(hidden, ldh * 2, 0, 2 * hidden_columns(a, a.wide), M, s));
        if (st != GEMM_OK || N == 0) return st;
        const gemm_epilogue_t ep{bias, nullptr, nullptr, GEMM_ACT_NONE};
        return gemm_run_ep(plan, X, W, nullptr, D, M, N, K, ldx, ldw, ldd, GEMM_ROW_MAJOR, layoutW, GEMM_F32, out_dtype,
                           1.0f, 0.0f, &ep, stream);
    }
    Choice ch;
    if (N > 0) {
        st = choose_adapters(plan, M, N, K, layoutW, out_dtype, s, &ch);
        if (st != GEMM_OK) return st;
    }
    st = run_hidden(plan, a, X, ldx, M, K, hidden, ldh, s);
    if (st != GEMM_OK || N == 0) return st;
    const AdapterProblem p{a.index, a.count, a.rank, part_of(a.rank), hidden, ldh, a.up, a.up_ld, a.up_stride, a.up_layout};
    return launch_adapters(plan, ch, X, W, D, M, N, K, ldx, ldw, ldd, layoutW, out_dtype, bias, p, s);
}

gemm_status_t gemm_adapters_grad(gemm_plan_t plan, const void* X, const void* dD, int64_t M, int64_t N, int64_t K,
                                 int64_t ldx, int64_t lddd, const gemm_adapters_t* adapters, const void* h,
                                 const void* p, int64_t ldh, gemm_dtype_t out_dtype, void* d_down, int64_t down_ld,
                                 int64_t down_stride, void* d_up, int64_t up_ld, int64_t up_stride, void* stream) {
    gemm_status_t st = check_adapters(plan, M, N, K, out_dtype, adapters);
    if (st != GEMM_OK) return st;
    if (out_dtype != GEMM_F32 && out_dtype != plan->in_dtype) return GEMM_ERR_UNSUPPORTED;
    const gemm_adapters_t& a = *adapters;
    const int part = part_of(a.rank);
    const int64_t ldp = a.ldp ? a.ldp : ldh;
    if (d_down) {
        st = check_matrix(X, M, K, ldx);
        if (st == GEMM_OK) st = check_matrix(p, M, hidden_columns(a, a.wide), ldp);
        if (st == GEMM_OK) st = check_gradient(a.count, a.rank, K, down_ld, down_stride);
    }
    if (d_up && st == GEMM_OK) {
        st = check_matrix(dD, M, N, lddd);
        if (st == GEMM_OK) st = check_matrix(h, M, hidden_columns(a, a.wide_h), ldh);
        if (st == GEMM_OK) st = check_gradient(a.count, N, a.rank, up_ld, up_stride);
    }
    if (st != GEMM_OK) return st;
    const uintptr_t esz = out_dtype == GEMM_F32 ? 4 : 2;
    if (!aligned(d_down, esz) || !aligned(d_up, esz)) return GEMM_ERR_MISALIGNED;
    FactorGradArgs f;
    std::memset(&f, 0, sizeof(f));
    if (d_down) f.f[0].blocks = static_cast<int32_t>((K + 127) / 128);
    if (d_up) f.f[1].blocks = static_cast<int32_t>((N + 127) / 128);
    const int64_t items = a.count * (f.f[0].blocks + static_cast<int64_t>(f.f[1].blocks));
    if (items == 0) return GEMM_OK;
    const OnDevice on(plan->device);
    if (!on.ok) return GEMM_ERR_CUDA;
    const void* left[2] = {X, dD};
    // (the high parts and those times 2^11 of wide rows)
    const bool wide[2] = {a.wide != 0, a.wide_h != 0};
    const uint16_t* right[2] = {static_cast<const uint16_t*>(p), static_cast<const uint16_t*>(h)};
    const int64_t columns[2] = {K, N}, ld[2] = {ldx, lddd}, ld_right[2] = {ldp, ldh};
    for (int i = 0; i < 2 && M > 0; ++i) {
        if (f.f[i].blocks == 0) continue;
        f.f[i].low = wide[i] ? tcdt::kRestScale : 1.0f;
        st = encode_map(plan, &f.f[i].tmX, left[i], columns[i], M, ld[i], 64, 64, plan->in_dtype);
        if (st == GEMM_OK) st = encode_map(plan, &f.f[i].tmH, right[i] + (wide[i] ? part : 0), 2 * part, M, ld_right[i], 64, 64, plan->in_dtype);
        if (st != GEMM_OK) return st;
    }
    f.f[0].out = d_down, f.f[0].stride = down_stride, f.f[0].sr = down_ld, f.f[0].sc = 1;
    f.f[1].out = d_up, f.f[1].stride = up_stride, f.f[1].sr = 1, f.f[1].sc = up_ld;
    f.f[0].columns = static_cast<int32_t>(K), f.f[1].columns = static_cast<int32_t>(N);
    f.index = a.index;
    f.rank = static_cast<int32_t>(a.rank);
    f.part = part;
    f.idesc = make_idesc(true, input_format(plan->in_dtype), true, true, 128, 2 * part);
    f.M = M;
    // (an adapter has about its share of the tiles: 1000 rows of three adapters, 75 items, 9 us
    // with one CTA each, 13 with four, 19 with eight; 4096 of one, 64 items: 27, 17, 27)
    f.splits = splits_of(plan, items, (M + 63) / 64 / a.count, 8);
    f.stages = tcdt::kAdapterSharedBytes / tcdt::factor_stage_bytes(part);
    if (f.stages > tcdt::kAdapterMaxStages) f.stages = tcdt::kAdapterMaxStages;
    f.out_kind = out_dtype == GEMM_F32 ? 0u : out_dtype == GEMM_F16 ? 1u : 2u;
    f.status = plan->d_status;
    f.timeout_ns = plan->timeout_ns;
#ifdef TCDT_FAULT_INJECTION
    f.fi_skip_load = plan->fi_skip_load;
#endif
    return launch_tiles(plan, tcdt::factor_grad_kernel, f, items * f.splits, plan->adapters_prepared[1],
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
