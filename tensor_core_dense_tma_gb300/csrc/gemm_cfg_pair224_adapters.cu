// gemm_cfg_pair224_adapters.cu -- kernels of the pair224 tile configuration that add
// the rows' low-rank adapters, in a translation unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
TCDT_DEFINE_ADAPTERS(pair224, CfgPair224)
}  // namespace tcdt_host
