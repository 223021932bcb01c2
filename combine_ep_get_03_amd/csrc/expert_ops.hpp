// expert_ops.hpp -- device helpers and kernel launchers of the operators around the
// expert-major rows (expert_rows.hip) and of the RMS norm in front of them (rmsnorm.hip).
// Not part of the public ABI.
#pragma once

#include "ep_internal.hpp"

namespace ep {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values rounded to nearest even into one word of two bf16 (one packed convert).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const uint16_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(a));
    const uint16_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(b));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The eight bf16 channels of a 128-bit word, widened.
__device__ __forceinline__ void widen8(u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[2 * q] = bf16_lo(w[q]);
        f[2 * q + 1] = bf16_hi(w[q]);
    }
}

__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = bf16_pair(f[2 * q], f[2 * q + 1]);
    return w;
}

// Cross-lane moves in the vector pipe (DPP): lanes whose source is outside the row of 16, or
// that the masks leave out, take 0.
template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ float dpp_or_zero(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRowMask, 0xf,
                                                      kRowMask == 0xf));
}

// Sum over the wave's 64 lanes (all of them active), the same value in every lane: prefix
// sums within rows of 16 (row_shr 1, 2, 4, 8), then each row's last lane into the rows
// above it (row_bcast 15 and 31); lane 63 ends with the total.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_or_zero<0x111>(v);
    v += dpp_or_zero<0x112>(v);
    v += dpp_or_zero<0x114>(v);
    v += dpp_or_zero<0x118>(v);
    v += dpp_or_zero<0x142, 0xa>(v);
    v += dpp_or_zero<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}

// Largest of 16 aligned lanes (a row), in each of them: rotations by 8, 4, 2, 1. v >= 0.
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp_or_zero<0x128>(v));
    v = fmaxf(v, dpp_or_zero<0x124>(v));
    v = fmaxf(v, dpp_or_zero<0x122>(v));
    return fmaxf(v, dpp_or_zero<0x121>(v));
}

// Word v (16 bytes) of a buffer; zeros past its end.
template <int kPolicy>
__device__ __forceinline__ u32x4 load_word(__amdgpu_buffer_rsrc_t b, int v) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, v * 16, 0, kPolicy));
}

// Stores word v; dropped past the buffer's end.
template <int kPolicy>
__device__ __forceinline__ void store_word(__amdgpu_buffer_rsrc_t b, int v, u32x4 w) {
    __builtin_amdgcn_raw_buffer_store_b128(w, b, v * 16, 0, kPolicy);
}

// Row t of an array of rows of V words as a buffer; of no bytes when the array is null, so
// that its loads are zeros and its stores dropped without a branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const u32x4* rows, int64_t t, int V) {
    return raw_buffer(rows ? rows + t * V : nullptr, rows ? static_cast<uint32_t>(V) * 16u : 0u);
}

// ---------------------------------------------------------------- launchers
// Each returns hipSuccess or the error reported at launch. Arguments have been validated
// by the C ABI layer.

// rmsnorm.hip
constexpr int kNormGroup = 128;  // channels per e4m3 scale
hipError_t launch_rmsnorm(const void* x, const void* residual, const void* weight,
                          bool weight_fp32, float eps, int64_t T, int H, void* residual_out,
                          void* y, uint8_t* y_fp8, float* y_scales, hipStream_t stream);
size_t rmsnorm_grad_workspace_bytes(int64_t T, int H);
hipError_t launch_rmsnorm_grad(const void* grad_y, const void* grad_residual_out, const void* h,
                               const void* weight, bool weight_fp32, float eps, int64_t T, int H,
                               void* grad_x, float* grad_weight, void* workspace,
                               hipStream_t stream);

// expert_rows.hip
hipError_t launch_dispatch_permute_fp8(const void* x_fp8, const float* x_scales,
                                       const float* topk_w, int64_t T, int H, int k,
                                       const int32_t* expert_slot, void* perm_x,
                                       float* perm_scales, float* perm_w, int32_t* perm_src,
                                       int64_t cap, int32_t* error_flag, hipStream_t stream);
hipError_t launch_combine_unpermute(const void* rows, int64_t num_rows, const float* topk_w,
                                    const int32_t* expert_slot, int64_t T, int H, int k,
                                    const void* addend, void* out, int32_t* error_flag,
                                    hipStream_t stream);
hipError_t launch_combine_unpermute_grad(const void* grad_out, const void* rows,
                                         int64_t num_rows, const float* topk_w,
                                         const int32_t* expert_slot, int64_t T, int H, int k,
                                         void* grad_rows, float* grad_w, int32_t* error_flag,
                                         hipStream_t stream);
hipError_t launch_dispatch_permute_grad(const void* grad_rows, const float* grad_perm_w,
                                        int64_t num_rows, const int32_t* expert_slot, int64_t T,
                                        int H, int k, void* grad_x, float* grad_w,
                                        int32_t* error_flag, hipStream_t stream);

}  // namespace ep
