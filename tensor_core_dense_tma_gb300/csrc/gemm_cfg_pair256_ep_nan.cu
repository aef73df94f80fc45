// gemm_cfg_pair256_ep_nan.cu -- kernels of the pair256 tile configuration with the
// fused epilogue whose ReLU keeps a NaN (fp32 accumulation), in a translation
// unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
namespace {
template <int OUT>
gemm_status_t launch(gemm_plan* plan, int slot, const Choice& ch, const Problem& pr, void* D, int64_t ldd,
                     gemm_dtype_t out, cudaStream_t s) {
    using Cfg = CfgPair256<false, OUT, tcdt::kInF16>;
    const gemm_status_t st = prepare<Cfg, tcdt::kEpKeepNan>(plan, kCfgPair256, slot);
    return st == GEMM_OK ? launch_tc<Cfg, tcdt::kEpKeepNan>(plan, ch, pr, nullptr, D, ldd, 1.0f, 0.0f, out, s) : st;
}
}  // namespace

gemm_status_t launch_pair256_ep_nan(gemm_plan* plan, int slot, const Choice& ch, const Problem& pr, void* D,
                                    int64_t ldd, cudaStream_t s) {
    if (slot == 0) return launch<tcdt::kOutF32>(plan, slot, ch, pr, D, ldd, GEMM_F32, s);
    if (slot == 1) return launch<tcdt::kOutF16>(plan, slot, ch, pr, D, ldd, GEMM_F16, s);
    return launch<tcdt::kOutBF16>(plan, slot, ch, pr, D, ldd, GEMM_BF16, s);
}
}  // namespace tcdt_host
