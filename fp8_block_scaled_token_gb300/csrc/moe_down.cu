// moe_down.cu -- the expert layer's down product (moe_gemm.cuh).
#include "moe_gemm.cuh"

namespace fp8bs {

fp8bs_status launch_moe_down(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    return launch_moe_phase<kMoeDown>(L, w, dev);
}

} // namespace fp8bs
