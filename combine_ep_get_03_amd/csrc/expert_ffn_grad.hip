// expert_ffn_grad.hip -- the gradients of the experts' gated feed-forward block on gfx950, over
// rows sorted by expert. With s = sigmoid(gate) and da = grad_out Wd:
//   grad_gate = da up s (1 + gate (1 - s)), grad_up = da gate s      ep_expert_down_grad
//   grad_x    = grad_gate Wg + grad_up Wu                            ep_expert_gate_up_grad
//   grad_W[e] = grad_rows^T input_rows over expert e's rows          ep_expert_weight_grad
#include "expert_gemm.hpp"

#ifndef EP_WG_ROWS
#define EP_WG_ROWS 640
#endif
namespace ep {

hipError_t launch_expert_down_grad(const GemmArgs& g, hipStream_t stream) {
    return launch_gemm<GemmOp::kDownGrad, false>(g, stream);
}

hipError_t launch_expert_gate_up_grad(const GemmArgs& g, hipStream_t stream) {
    return launch_gemm<GemmOp::kInputGrad, false>(g, stream);
}

hipError_t launch_expert_weight_grad(const GemmArgs& g, hipStream_t stream) {
    // an expert's rows are the inner size here
    if (g.num_rows / g.E > EP_WG_ROWS)
        return launch_shape<GemmShape<GemmOp::kWeightGrad, false, 256>>(g, stream);
    return launch_shape<GemmShape<GemmOp::kWeightGrad, false, 128>>(g, stream);
}

}  // namespace ep
