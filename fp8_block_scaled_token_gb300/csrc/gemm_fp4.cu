// gemm_fp4.cu -- instantiation of the small-M GEMM for mode kModeFp4 (E2M1
// operands with block scales applied by the tensor core).
#include "gemm_launch.cuh"

namespace fp8bs {

fp8bs_status launch_gemm_fp4(const GemmLaunch &L, const DeviceInfo &dev)
{
    return launch_gemm_mode<kModeFp4>(L, dev);
}

} // namespace fp8bs
