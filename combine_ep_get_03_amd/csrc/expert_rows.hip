// expert_rows.hip -- the expert-major rows on gfx950: e4m3 rows out to the experts, the
// experts' rows back to their tokens with the gate weights applied, and the gradients of
// both ways. With q = expert_slot[t][j] of token t's j-th pair (q < 0: not routed):
//   permute fp8    row q of the codes and of the scales = token t's
//   unpermute      out[t] = bf16(sum over j of w[t][j] y[q] (+ addend[t])), fp32, ascending j
//   its gradient   grad_y[q] = bf16(w[t][j] grad_out[t]), grad_w[t][j] = <grad_out[t], y[q]>
//   permute's      grad_x[t] = bf16(sum over j of grad_perm_x[q]), grad_w[t][j] = grad_perm_w[q]
// All are bound by the bytes of the expert-major rows, which move once.
#include "expert_ops.hpp"

namespace ep {
namespace {

constexpr int kT = 256;  // threads per block
constexpr int kWaves = kT / kWave;

// Wave (t, j) copies token t's codes and scales to row q.
__global__ __launch_bounds__(kT) void permute_fp8_kernel(
    const u32x4* __restrict__ codes, const float* __restrict__ scales,
    const float* __restrict__ topk_w, int64_t pairs, int V, int G, int k,
    const int32_t* __restrict__ expert_slot, u32x4* __restrict__ perm_codes,
    float* __restrict__ perm_scales, float* __restrict__ perm_w, int32_t* __restrict__ perm_src,
    int64_t cap, int32_t* __restrict__ error_flag) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / kWave;
    if (p >= pairs) return;
    const int lane = lane_id();
    const int64_t q = expert_slot[p];
    if (q < 0) return;
    if (q >= cap) {
        if (lane == 0) raise_error(error_flag, kErrRecvOverflow);
        return;
    }
    const int64_t t = p / k;
    for (int v = lane; v < V; v += kWave) store_stream(perm_codes + q * V + v, codes[t * V + v]);
    for (int g = lane; g < G; g += kWave) perm_scales[q * G + g] = scales[t * G + g];
    if (lane == 0) {
        if (perm_w) perm_w[q] = topk_w[p];
        if (perm_src) perm_src[q] = static_cast<int32_t>(t);
    }
}

// One block per token.
__global__ __launch_bounds__(kT) void unpermute_kernel(
    const u32x4* __restrict__ rows, int64_t num_rows, const float* __restrict__ topk_w,
    const int32_t* __restrict__ expert_slot, int V, int k, const u32x4* addend, u32x4* out,
    const float* __restrict__ grad_perm_w, float* __restrict__ grad_w,
    int32_t* __restrict__ error_flag) {
    const int64_t t = blockIdx.x;
    const int32_t* slot = expert_slot + t * k;
    for (int v = threadIdx.x; v < V; v += kT) {
        float acc[8] = {};
        for (int j = 0; j < k; ++j) {
            const int64_t q = slot[j];
            if (q < 0 || q >= num_rows) continue;
            const float w = topk_w ? topk_w[t * k + j] : 1.0f;
            float f[8];
            widen8(load_stream(rows + q * V + v), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += w * f[i];
        }
        if (addend) {
            float f[8];
            widen8(addend[t * V + v], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
        out[t * V + v] = narrow8(acc);
    }
    for (int j = threadIdx.x; j < k; j += kT) {
        const int64_t q = slot[j];
        if (q >= num_rows) raise_error(error_flag, kErrSlotRange);
        if (grad_w) grad_w[t * k + j] = q >= 0 && q < num_rows ? grad_perm_w[q] : 0.0f;
    }
}

// One block per token: its pairs in turn.
__global__ __launch_bounds__(kT) void unpermute_grad_kernel(
    const u32x4* __restrict__ grad_out, const u32x4* rows, int64_t num_rows,
    const float* __restrict__ topk_w, const int32_t* __restrict__ expert_slot, int V, int k,
    u32x4* grad_rows, float* __restrict__ grad_w, int32_t* __restrict__ error_flag) {
    __shared__ float red[kWaves];
    const int64_t t = blockIdx.x;
    for (int j = 0; j < k; ++j) {
        const int64_t q = expert_slot[t * k + j];
        const bool routed = q >= 0 && q < num_rows;
        if (q >= num_rows && threadIdx.x == 0) raise_error(error_flag, kErrSlotRange);
        float dot = 0.0f;
        if (routed) {
            const float w = topk_w ? topk_w[t * k + j] : 1.0f;
            for (int v = threadIdx.x; v < V; v += kT) {
                float g[8];
                widen8(grad_out[t * V + v], g);
                if (grad_w) {
                    float f[8];
                    widen8(load_stream(rows + q * V + v), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot += g[i] * f[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] *= w;
                store_stream(grad_rows + q * V + v, narrow8(g));
            }
        }
        if (grad_w) {
            dot = wave_sum(dot);
            if (lane_id() == 0) red[threadIdx.x / kWave] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                float s = 0.0f;
                for (int i = 0; i < kWaves; ++i) s += red[i];
                grad_w[t * k + j] = s;
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_dispatch_permute_fp8(const void* x_fp8, const float* x_scales,
                                       const float* topk_w, int64_t T, int H, int k,
                                       const int32_t* expert_slot, void* perm_x,
                                       float* perm_scales, float* perm_w, int32_t* perm_src,
                                       int64_t cap, int32_t* error_flag, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    const int64_t pairs = T * k;
    const int64_t grid = (pairs + kWaves - 1) / kWaves;
    if (!grid_fits(grid, kT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(permute_fp8_kernel, dim3(static_cast<unsigned>(grid)), dim3(kT), 0, stream,
                       static_cast<const u32x4*>(x_fp8), x_scales, topk_w, pairs, H / 16, H / 128,
                       k, expert_slot, static_cast<u32x4*>(perm_x), perm_scales, perm_w, perm_src,
                       cap, error_flag);
    return hipGetLastError();
}

hipError_t launch_combine_unpermute(const void* rows, int64_t num_rows, const float* topk_w,
                                    const int32_t* expert_slot, int64_t T, int H, int k,
                                    const void* addend, void* out, int32_t* error_flag,
                                    hipStream_t stream) {
    if (T == 0) return hipSuccess;
    if (!grid_fits(T, kT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(unpermute_kernel, dim3(static_cast<unsigned>(T)), dim3(kT), 0, stream,
                       static_cast<const u32x4*>(rows), num_rows, topk_w, expert_slot, H / 8, k,
                       static_cast<const u32x4*>(addend), static_cast<u32x4*>(out),
                       static_cast<const float*>(nullptr), static_cast<float*>(nullptr),
                       error_flag);
    return hipGetLastError();
}

hipError_t launch_combine_unpermute_grad(const void* grad_out, const void* rows,
                                         int64_t num_rows, const float* topk_w,
                                         const int32_t* expert_slot, int64_t T, int H, int k,
                                         void* grad_rows, float* grad_w, int32_t* error_flag,
                                         hipStream_t stream) {
    if (T == 0) return hipSuccess;
    if (!grid_fits(T, kT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(unpermute_grad_kernel, dim3(static_cast<unsigned>(T)), dim3(kT), 0, stream,
                       static_cast<const u32x4*>(grad_out), static_cast<const u32x4*>(rows),
                       num_rows, topk_w, expert_slot, H / 8, k, static_cast<u32x4*>(grad_rows),
                       grad_w, error_flag);
    return hipGetLastError();
}

hipError_t launch_dispatch_permute_grad(const void* grad_rows, const float* grad_perm_w,
                                        int64_t num_rows, const int32_t* expert_slot, int64_t T,
                                        int H, int k, void* grad_x, float* grad_w,
                                        int32_t* error_flag, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    if (!grid_fits(T, kT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(unpermute_kernel, dim3(static_cast<unsigned>(T)), dim3(kT), 0, stream,
                       static_cast<const u32x4*>(grad_rows), num_rows,
                       static_cast<const float*>(nullptr), expert_slot, H / 8, k,
                       static_cast<const u32x4*>(nullptr), static_cast<u32x4*>(grad_x),
                       grad_perm_w, grad_w, error_flag);
    return hipGetLastError();
}

}  // namespace ep
