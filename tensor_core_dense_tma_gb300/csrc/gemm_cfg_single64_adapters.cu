// gemm_cfg_single64_adapters.cu -- kernels of the single64 tile configuration that add
// the rows' low-rank adapters, in a translation unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
TCDT_DEFINE_ADAPTERS(single64, CfgSingle64)
}  // namespace tcdt_host
