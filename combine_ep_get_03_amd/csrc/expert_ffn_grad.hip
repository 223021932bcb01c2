// expert_ffn_grad.hip -- the gradients of the experts' gated feed-forward block on gfx950, over
// rows sorted by expert. With s = sigmoid(gate) and da = grad_out Wd:
//   grad_gate = da up s (1 + gate (1 - s)), grad_up = da gate s      ep_expert_down_grad
//   grad_x    = grad_gate Wg + grad_up Wu                            ep_expert_gate_up_grad
//   grad_W[e] = grad_rows^T input_rows over expert e's rows          ep_expert_weight_grad
#include "expert_gemm.hpp"

namespace ep {

hipError_t launch_expert_down_grad(const GemmArgs& g, hipStream_t stream) {
    return launch_gemm<GemmOp::kDownGrad, false>(g, stream);
}

hipError_t launch_expert_gate_up_grad(const GemmArgs& g, hipStream_t stream) {
    return launch_gemm<GemmOp::kInputGrad, false>(g, stream);
}

hipError_t launch_expert_weight_grad(const GemmArgs& g, hipStream_t stream) {
    // The rows per expert are the inner size here: with few the time is that of the stores, which
    // the lower tiles' waves do not wait for; with many it is the products' (of 4096 x 7168
    // weights of 32 experts, fp32, lower against higher: 256 rows 1048 / 1053 us, 384 rows
    // 1249 / 1209, 512 rows 1461 / 1379).
    if (g.num_rows / g.E > 256)
        return launch_shape<GemmShape<GemmOp::kWeightGrad, false, 256>>(g, stream);
    return launch_shape<GemmShape<GemmOp::kWeightGrad, false, 128>>(g, stream);
}

}  // namespace ep
