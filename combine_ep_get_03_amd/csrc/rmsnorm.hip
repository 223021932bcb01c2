// rmsnorm.hip -- the RMS norm in front of a mixture-of-experts block, with the residual's
// addition and an e4m3 output, and its gradient, on gfx950.
//
// With s = x + residual (fp32, not rounded), r = 1 / sqrt(mean(s^2) + eps):
//   residual_out = bf16(s),  y = bf16(s r w),
//   per group of 128 channels: a = max |s r w|, scale = a / 448, code = e4m3(s r w 448 / a).
// Gradient, from h = the saved residual_out: n = h r, g = grad_y w,
//   grad_x = bf16(r (g - n mean(g n)) + grad_residual_out),  grad_w = sum over tokens of
//   grad_y n. The two row sums, of h^2 and of g h, come from one pass: mean(g n) n r =
//   h r^3 mean(g h).
// Everything between the inputs and the outputs is fp32; each output is rounded once.
#include "expert_ops.hpp"

namespace ep {
namespace {

constexpr int kNT = 256;                // threads per block
constexpr int kNWaves = kNT / kWave;
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyAmax = 0x1p-100f;  // floor of a group's amax: 448 / amax stays finite

// Sum over the block, in every thread; red holds kNWaves floats per call site.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0) red[wave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kNWaves; ++i) s += red[i];
    __syncthreads();
    return s;
}

template <bool kF32>
__device__ __forceinline__ void load_weight8(const void* w, int v, float (&f)[8]) {
    if constexpr (kF32) {
        const float* p = static_cast<const float*>(w) + 8 * static_cast<int64_t>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = p[i];
    } else {
        widen8(static_cast<const u32x4*>(w)[v], f);
    }
}

// s = x + residual of word v, in fp32.
__device__ __forceinline__ void load_sum8(const u32x4* x, const u32x4* res, int64_t v,
                                          float (&f)[8]) {
    widen8(x[v], f);
    if (res) {
        float r[8];
        widen8(res[v], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += r[i];
    }
}

__device__ __forceinline__ float inv_rms(float sum_sq, int H, float eps) {
    return 1.0f / sqrtf(sum_sq / static_cast<float>(H) + eps);
}

// One block per token, the row read twice (the second time from the L2).
template <bool kF32>
__global__ __launch_bounds__(kNT) void rmsnorm_kernel(const u32x4* x, const u32x4* residual,
                                                      const void* weight, float eps, int V,
                                                      u32x4* residual_out, u32x4* y,
                                                      u32x2* y_fp8, float* y_scales) {
    __shared__ float red[kNWaves];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * V;
    const u32x4* res = residual ? residual + base : nullptr;
    float ss = 0.0f;
    for (int v = threadIdx.x; v < V; v += kNT) {
        float f[8];
        load_sum8(x + base, res, v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
    }
    const float r = inv_rms(block_sum(ss, red), 8 * V, eps);
    for (int v = threadIdx.x; v < V; v += kNT) {
        float f[8], w[8];
        load_sum8(x + base, res, v, f);
        load_weight8<kF32>(weight, v, w);
        if (residual_out) residual_out[base + v] = narrow8(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
        if (y) y[base + v] = narrow8(f);
        if (y_fp8) {  // a group is 16 aligned lanes, all inside the row or all past it
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
#pragma unroll
            for (int m = 8; m >= 1; m >>= 1) a = fmaxf(a, __shfl_xor(a, m, kWave));
            a = a > 0.0f ? fmaxf(a, kTinyAmax) : kE4m3Max;
            const float inv = kE4m3Max / a;
            u32x2 c;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q] * inv, f[4 * q + 1] * inv,
                                                               0, false);
                c[q] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(
                    f[4 * q + 2] * inv, f[4 * q + 3] * inv, lo, true));
            }
            y_fp8[base + v] = c;
            if (v % 16 == 0) y_scales[(base + v) / 16] = a / kE4m3Max;
        }
    }
}

// ---- gradient

// r of every row of h.
__global__ __launch_bounds__(kNT) void rmsnorm_rstd_kernel(const u32x4* h, float eps, int V,
                                                           float* rstd) {
    __shared__ float red[kNWaves];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * V;
    float ss = 0.0f;
    for (int v = threadIdx.x; v < V; v += kNT) {
        float f[8];
        widen8(h[base + v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
    }
    const float r = inv_rms(block_sum(ss, red), 8 * V, eps);
    if (threadIdx.x == 0) rstd[blockIdx.x] = r;
}

// Partial sums of grad_w: block (b, c) sums the rows of chunk c over words [64 b, 64 b + 64),
// each wave every fourth row; the waves' sums join in LDS in wave order.
__global__ __launch_bounds__(kNT) void rmsnorm_dw_kernel(const u32x4* dy, const u32x4* h,
                                                         const float* rstd, int64_t T, int V,
                                                         int64_t rows, float* part) {
    __shared__ float acc_lds[kNWaves][kWave][8];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int v = static_cast<int>(blockIdx.x) * kWave + lane;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * rows;
    const int64_t t1 = min(t0 + rows, T);
    float acc[8] = {};
    if (v < V) {
        for (int64_t t = t0 + wave; t < t1; t += kNWaves) {
            float g[8], n[8];
            widen8(dy[t * V + v], g);
            widen8(h[t * V + v], n);
            const float r = rstd[t];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += g[i] * (n[i] * r);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc_lds[wave][lane][i] = acc[i];
    __syncthreads();
    if (wave == 0 && v < V) {
        float* p = part + (static_cast<int64_t>(blockIdx.y) * V + v) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = 0.0f;
            for (int w = 0; w < kNWaves; ++w) s += acc_lds[w][lane][i];
            p[i] = s;
        }
    }
}

// grad_w = the chunks' partial sums, added in chunk order.
__global__ __launch_bounds__(kNT) void rmsnorm_dw_join_kernel(const float* part, int H,
                                                              int chunks, float* dw) {
    const int c = static_cast<int>(blockIdx.x) * kNT + threadIdx.x;
    if (c >= H) return;
    float s = 0.0f;
    for (int p = 0; p < chunks; ++p) s += part[static_cast<int64_t>(p) * H + c];
    dw[c] = s;
}

template <bool kF32>
__global__ __launch_bounds__(kNT) void rmsnorm_dx_kernel(const u32x4* dy, const u32x4* dres,
                                                         const u32x4* h, const void* weight,
                                                         float eps, int V, u32x4* dx) {
    __shared__ float red[kNWaves];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * V;
    float hh = 0.0f, gh = 0.0f;
    for (int v = threadIdx.x; v < V; v += kNT) {
        float g[8], f[8], w[8];
        widen8(dy[base + v], g);
        widen8(h[base + v], f);
        load_weight8<kF32>(weight, v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            hh += f[i] * f[i];
            gh += g[i] * w[i] * f[i];
        }
    }
    const float r = inv_rms(block_sum(hh, red), 8 * V, eps);
    const float c = block_sum(gh, red) / static_cast<float>(8 * V) * r * r;
    for (int v = threadIdx.x; v < V; v += kNT) {
        float g[8], f[8], w[8], d[8] = {};
        widen8(dy[base + v], g);
        widen8(h[base + v], f);
        load_weight8<kF32>(weight, v, w);
        if (dres) widen8(dres[base + v], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += r * (g[i] * w[i] - f[i] * c);
        dx[base + v] = narrow8(d);
    }
}

constexpr int kDwChunks = 64;  // partial rows of grad_w

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

hipError_t launch_rmsnorm(const void* x, const void* residual, const void* weight,
                          bool weight_fp32, float eps, int64_t T, int H, void* residual_out,
                          void* y, uint8_t* y_fp8, float* y_scales, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    if (!grid_fits(T, kNT)) return hipErrorInvalidConfiguration;
    const auto kernel = weight_fp32 ? rmsnorm_kernel<true> : rmsnorm_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(T)), dim3(kNT), 0, stream,
                       static_cast<const u32x4*>(x), static_cast<const u32x4*>(residual), weight,
                       eps, H / 8, static_cast<u32x4*>(residual_out), static_cast<u32x4*>(y),
                       reinterpret_cast<u32x2*>(y_fp8), y_scales);
    return hipGetLastError();
}

size_t rmsnorm_grad_workspace_bytes(int64_t T, int H) {
    if (T == 0) return 0;
    return align256(sizeof(float) * static_cast<size_t>(T)) +
           sizeof(float) * static_cast<size_t>(kDwChunks) * static_cast<size_t>(H);
}

hipError_t launch_rmsnorm_grad(const void* grad_y, const void* grad_residual_out, const void* h,
                               const void* weight, bool weight_fp32, float eps, int64_t T, int H,
                               void* grad_x, float* grad_weight, void* workspace,
                               hipStream_t stream) {
    if (T == 0) {
        if (!grad_weight) return hipSuccess;
        return launch_zero_ints(ZeroInts{{reinterpret_cast<int32_t*>(grad_weight)}, {H}}, stream);
    }
    if (!grid_fits(T, kNT)) return hipErrorInvalidConfiguration;
    const int V = H / 8;
    const auto* dy = static_cast<const u32x4*>(grad_y);
    const auto* hp = static_cast<const u32x4*>(h);
    const unsigned grid = static_cast<unsigned>(T);
    if (grad_weight) {  // before grad_x, which may take the place of any of its inputs
        float* rstd = static_cast<float*>(workspace);
        float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                               align256(sizeof(float) * static_cast<size_t>(T)));
        const int64_t rows = (T + kDwChunks - 1) / kDwChunks;
        const int chunks = static_cast<int>((T + rows - 1) / rows);
        hipLaunchKernelGGL(rmsnorm_rstd_kernel, dim3(grid), dim3(kNT), 0, stream, hp, eps, V, rstd);
        EP_RETURN_IF_LAUNCH_FAILED();
        hipLaunchKernelGGL(rmsnorm_dw_kernel,
                           dim3((V + kWave - 1) / kWave, static_cast<unsigned>(chunks)), dim3(kNT),
                           0, stream, dy, hp, rstd, T, V, rows, part);
        EP_RETURN_IF_LAUNCH_FAILED();
        hipLaunchKernelGGL(rmsnorm_dw_join_kernel, dim3((H + kNT - 1) / kNT), dim3(kNT), 0, stream,
                           part, H, chunks, grad_weight);
        EP_RETURN_IF_LAUNCH_FAILED();
    }
    const auto kernel = weight_fp32 ? rmsnorm_dx_kernel<true> : rmsnorm_dx_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kNT), 0, stream, dy,
                       static_cast<const u32x4*>(grad_residual_out), hp, weight, eps, V,
                       static_cast<u32x4*>(grad_x));
    return hipGetLastError();
}

}  // namespace ep
