// moe_up.cu -- the expert layer's gate/up product (moe_gemm.cuh).
#include "moe_gemm.cuh"

namespace fp8bs {

fp8bs_status launch_moe_up(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    return launch_moe_phase<kMoeUp>(L, w, dev);
}

} // namespace fp8bs
