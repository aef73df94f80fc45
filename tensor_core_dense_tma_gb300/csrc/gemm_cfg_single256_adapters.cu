// gemm_cfg_single256_adapters.cu -- kernels of the single256 tile configuration that add
// the rows' low-rank adapters, in a translation unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
TCDT_DEFINE_ADAPTERS(single256, CfgSingle256)
}  // namespace tcdt_host
