// expert_ffn.hip -- the experts' gated feed-forward block on gfx950, over rows sorted by expert:
//   act = silu(x Wg^T) * (x Wu^T)      ep_expert_gate_up, ep_expert_gate_up_fp8
//   out = act Wd^T                     ep_expert_down, ep_expert_down_fp8
#include "expert_gemm.hpp"

namespace ep {

hipError_t launch_expert_gate_up(const GemmArgs& g, bool fp8, hipStream_t stream) {
    return fp8 ? launch_gemm<GemmOp::kGateUp, true>(g, stream)
               : launch_gemm<GemmOp::kGateUp, false>(g, stream);
}

hipError_t launch_expert_down(const GemmArgs& g, bool fp8, hipStream_t stream) {
    return fp8 ? launch_gemm<GemmOp::kDown, true>(g, stream)
               : launch_gemm<GemmOp::kDown, false>(g, stream);
}

}  // namespace ep
