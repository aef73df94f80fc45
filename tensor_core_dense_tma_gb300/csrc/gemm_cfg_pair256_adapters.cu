// gemm_cfg_pair256_adapters.cu -- kernels of the pair256 tile configuration that add
// the rows' low-rank adapters, in a translation unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
TCDT_DEFINE_ADAPTERS(pair256, CfgPair256)
}  // namespace tcdt_host
