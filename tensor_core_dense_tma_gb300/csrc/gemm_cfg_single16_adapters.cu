// gemm_cfg_single16_adapters.cu -- kernels of the single16 tile configuration that add
// the rows' low-rank adapters, in a translation unit of their own.
#include "gemm_internal.cuh"

namespace tcdt_host {
TCDT_DEFINE_ADAPTERS(single16, CfgSingle16)
}  // namespace tcdt_host
