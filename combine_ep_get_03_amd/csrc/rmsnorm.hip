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
#include <type_traits>

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

// The e4m3 codes of a lane's 8 channels, and the magnitude that its group of 128 channels (16
// aligned lanes, all inside the row or all past it) is scaled to 448 by: the largest of the
// group's numbers (a NaN is none, and keeps its NaN code), at least 2^-100, or 448 for a group
// of zeros. No clamp: the largest product is 448 within 2 u, which rounds to 448.
__device__ __forceinline__ float quantize8(const float (&f)[8], u32x2& code) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
    a = row_max(a);
    a = a > 0.0f ? fmaxf(a, kTinyAmax) : kE4m3Max;
    const float inv = kE4m3Max / a;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q] * inv, f[4 * q + 1] * inv, 0, false);
        code[q] = static_cast<uint32_t>(
            __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q + 2] * inv, f[4 * q + 3] * inv, lo, true));
    }
    return a;
}

// Rows wider than the registers hold (past 32768 channels): one block per token, the row read
// twice, the second time from the L2. 113 us for 1024 rows of 40960 (3.3 TB/s).
template <bool kF32>
__global__ __launch_bounds__(kNT) void rmsnorm_kernel(const u32x4* x, const u32x4* residual,
                                                      const void* weight, float eps, int64_t t0,
                                                      int64_t /*t_end*/, int V,
                                                      u32x4* residual_out, u32x4* y,
                                                      u32x2* y_fp8, float* y_scales) {
    __shared__ float red[kNWaves];
    const int64_t base = (t0 + blockIdx.x) * V;
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
        if (y_fp8) {
            u32x2 c;
            const float a = quantize8(f, c);
            y_fp8[base + v] = c;
            if (v % 16 == 0) y_scales[(base + v) / 16] = a / kE4m3Max;
        }
    }
}

constexpr int kMaxWaves = 16;  // per block

// Sums of kN values over the W waves of a row, in every thread; red: one slot per wave.
// The caller alternates between two such arrays, so one barrier per call is enough.
template <int kN>
__device__ __forceinline__ void waves_sum(float (&s)[kN], float (*red)[kN], int first, int W) {
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] = wave_sum(s[n]);
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0) {
#pragma unroll
        for (int n = 0; n < kN; ++n) red[wave][n] = s[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) s[n] = 0.0f;
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int n = 0; n < kN; ++n) s[n] += red[first + i][n];
    }
}

// The weights of word v, zeros past the row.
template <bool kF32>
__device__ __forceinline__ void weight_word(__amdgpu_buffer_rsrc_t wb, int v, float (&f)[8]) {
    if constexpr (kF32) {
        const u32x4 a = load_word<0>(wb, 2 * v), b = load_word<0>(wb, 2 * v + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(a[i]);
            f[4 + i] = __uint_as_float(b[i]);
        }
    } else {
        widen8(load_word<0>(wb, v), f);
    }
}

// The row in registers: NV words per lane, one row per wave (kOneWave: four rows per block of
// 256) or one per block. Everything is read once and written once; bound by those bytes.
// A missing residual or output is a buffer of no bytes. kPolicy: the cache policy of the
// rows' loads and stores.
//
// Measured on MI355X at 7168 channels with residual, bf16 and e4m3 outputs: 46.7 us at 4096
// tokens, 178.5 us at 16384 (5.9 TB/s), 4.0 us for one token. Two words per lane and 448
// threads; one word 50.6 and 190 us, four 50.7 and 188 us (cached accesses, where two took
// 49.3 and 184). Two neighbouring words per lane, for 128-bit code stores, 58.0 and 213 us:
// their loads and stores of the bf16 rows leave every other 16 bytes to a second access.
template <int NV, bool kF32, bool kOneWave, int kPolicy>
__global__ __launch_bounds__(kOneWave ? kNT : kMaxWaves * kWave) void rmsnorm_row_kernel(
    const u32x4* x, const u32x4* residual, const void* weight, float eps, int64_t t0, int64_t t_end,
    int V, u32x4* residual_out, u32x4* y, u32x2* y_fp8, float* y_scales) {
    __shared__ float red[kMaxWaves][1];
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int64_t t =
        t0 + (kOneWave ? static_cast<int64_t>(blockIdx.x) * kNWaves + wave : blockIdx.x);
    if (kOneWave && t >= t_end) return;
    const int v = kOneWave ? lane_id() : threadIdx.x;
    const int step = kOneWave ? kWave : blockDim.x;
    const __amdgpu_buffer_rsrc_t xb = row_buffer(x, t, V), rb = row_buffer(residual, t, V);
    u32x4 xv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) xv[i] = load_word<kPolicy>(xb, v + i * step);
#pragma unroll
    for (int i = 0; i < NV; ++i) rv[i] = load_word<kPolicy>(rb, v + i * step);
    const __amdgpu_buffer_rsrc_t wb =
        raw_buffer(weight, static_cast<uint32_t>(V) * (kF32 ? 32u : 16u));
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) weight_word<kF32>(wb, v + i * step, w[i]);
    float f[NV][8], ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float r[8];
        widen8(xv[i], f[i]);
        widen8(rv[i], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[i][e] += r[e];
            ss[0] += f[i][e] * f[i][e];
        }
    }
    if constexpr (kOneWave) ss[0] = wave_sum(ss[0]);
    else waves_sum<1>(ss, red, 0, blockDim.x / kWave);
    const float r = inv_rms(ss[0], 8 * V, eps);
    const __amdgpu_buffer_rsrc_t sb = row_buffer(residual_out, t, V), yb = row_buffer(y, t, V);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (residual_out) store_word<kPolicy>(sb, v + i * step, narrow8(f[i]));
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * r * w[i][e];
        if (y) store_word<kPolicy>(yb, v + i * step, narrow8(f[i]));
    }
    if (!y_fp8) return;
    const int64_t G = V / 16;
    const __amdgpu_buffer_rsrc_t cb = raw_buffer(y_fp8 + t * V, static_cast<uint32_t>(V) * 8u);
    const __amdgpu_buffer_rsrc_t gb = raw_buffer(y_scales + t * G, static_cast<uint32_t>(G) * 4u);
#pragma unroll
    for (int i = 0; i < NV; ++i) {  // a group is a row of 16 lanes
        const int vi = v + i * step;
        u32x2 c;
        const float a = quantize8(f[i], c);
        __builtin_amdgcn_raw_buffer_store_b64(c, cb, vi * 8, 0, kPolicy);
        if (vi % 16 == 0)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(a / kE4m3Max), gb, vi / 16 * 4, 0, 0);
    }
}

// From this many bytes of x on, the rows' loads and stores are non-temporal. Measured at 7168
// channels with all outputs, cached against non-temporal: 11.1 against 12.9 us at 1024 tokens
// (15 MB), 28.1 against 25.4 us at 2048 (29 MB), 49.5 against 46.7 us at 4096 (59 MB).
constexpr int64_t kNormStreamBytes = int64_t{24} << 20;
constexpr int64_t kMaxRows = int64_t{1} << 21;  // per launch

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

// The same word, unknown to the compiler: what was computed from it before is computed again
// instead of being kept in registers. On grad_y's words after the reduction it frees the
// registers that two words per lane lack by one (46.3 against 46.7 us at 4096 tokens of 7168
// channels); on h's words as well 48.9 us.
__device__ __forceinline__ u32x4 anew(u32x4 w) {
    asm volatile("" : "+v"(w));
    return w;
}

// One row's words of a lane; zeros where there is no row.
template <int NV, int kPolicy>
struct GradRow {
    u32x4 dy[NV], h[NV], dr[NV];

    __device__ __forceinline__ void load(const u32x4* grad_y, const u32x4* hh, const u32x4* grad_res,
                                         int64_t t, bool live, int V, int v, int step) {
        const __amdgpu_buffer_rsrc_t a = row_buffer(live ? grad_y : nullptr, t, V);
        const __amdgpu_buffer_rsrc_t b = row_buffer(live ? hh : nullptr, t, V);
        const __amdgpu_buffer_rsrc_t c = row_buffer(live ? grad_res : nullptr, t, V);
#pragma unroll
        for (int i = 0; i < NV; ++i) dy[i] = load_word<kPolicy>(a, v + i * step);
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = load_word<kPolicy>(b, v + i * step);
#pragma unroll
        for (int i = 0; i < NV; ++i) dr[i] = load_word<kPolicy>(c, v + i * step);
    }
};

// The gradient with the rows in registers: a block holds G rows at a time, W waves and NV
// words per lane for each, and walks rows G apart; the next rows' loads are in flight
// while the present ones are reduced and written. Each lane keeps the sum of its words'
// grad_w over the block's rows in registers; at the end the G rows' sums join in LDS and the
// block writes one partial row of grad_w (part [gridDim.x][8 V]).
template <int NV, bool kF32, bool kDw, int kPolicy>
__global__ __launch_bounds__(kMaxWaves* kWave) void rmsnorm_grad_row_kernel(
    const u32x4* grad_y, const u32x4* grad_res, const u32x4* h, const void* weight, float eps,
    int64_t T, int V, int W, u32x4* grad_x, float* part) {
    __shared__ float red[2][kMaxWaves][2];
    __shared__ float join[kDw ? kMaxWaves * kWave * NV * 8 : 1];
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int G = static_cast<int>(blockDim.x) / (kWave * W);
    const int g = wave / W;
    const int v = (wave - g * W) * kWave + lane_id();
    const int step = W * kWave;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
    const __amdgpu_buffer_rsrc_t wb =
        raw_buffer(weight, static_cast<uint32_t>(V) * (kF32 ? 32u : 16u));
    float w[NV][8], dw[NV][8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) weight_word<kF32>(wb, v + i * step, w[i]);
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * G;
    GradRow<NV, kPolicy> cur;
    cur.load(grad_y, h, grad_res, t0 + g, t0 + g < T, V, v, step);
    for (int par = 0; t0 < T; t0 += stride, par ^= 1) {
        const int64_t t = t0 + g, tn = t + stride;
        GradRow<NV, kPolicy> next;
        next.load(grad_y, h, grad_res, tn, tn < T, V, v, step);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[8], y[8];
            widen8(cur.h[i], f);
            widen8(cur.dy[i], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] += f[e] * f[e];
                s[1] += y[e] * w[i][e] * f[e];
            }
        }
        waves_sum<2>(s, red[par], g * W, W);
        const float r = inv_rms(s[0], 8 * V, eps);
        const float c = s[1] / static_cast<float>(8 * V) * r * r;
        const __amdgpu_buffer_rsrc_t xb = row_buffer(t < T ? grad_x : nullptr, t, V);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float d[8], f[8], y[8];
            widen8(cur.dr[i], d);
            widen8(cur.h[i], f);
            widen8(anew(cur.dy[i]), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[e] += r * (y[e] * w[i][e] - f[e] * c);
                if (kDw && t < T) dw[i][e] += y[e] * (f[e] * r);
            }
            store_word<kPolicyNt>(xb, v + i * step, narrow8(d));
        }
        cur = next;
    }
    if constexpr (kDw) {
        float* out = part + static_cast<int64_t>(blockIdx.x) * V * 8;
        if (G == 1) {
            const __amdgpu_buffer_rsrc_t ob = raw_buffer(out, static_cast<uint32_t>(V) * 32u);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(dw[i][4 * q + e]);
                    store_word<0>(ob, 2 * (v + i * step) + q, o);
                }
            }
        } else {
            const int row = step * NV * 8;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) join[g * row + (v + i * step) * 8 + e] = dw[i][e];
            __syncthreads();
            for (int c = threadIdx.x; c < V * 8; c += blockDim.x) {
                float s = 0.0f;
                for (int i = 0; i < G; ++i) s += join[i * row + c];
                out[c] = s;
            }
        }
    }
}

// grad_w = the blocks' partial rows: block b takes 32 columns (a cache line of each row), its
// half waves every 32nd row each, joined in their order.
constexpr int kSumCols = 32;
constexpr int kSumRows = kMaxWaves * kWave / kSumCols;
constexpr int kSumLoads = 8;  // in flight per lane: every row of 256 blocks
__global__ __launch_bounds__(kMaxWaves* kWave) void rmsnorm_dw_sum_kernel(const float* part, int H,
                                                                          int rows, float* dw) {
    __shared__ float acc[kSumRows][kSumCols];
    const int x = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    const int c = static_cast<int>(blockIdx.x) * kSumCols + x;
    // loads past the last row are zeros: no load waits behind a branch or a loop's rest
    const __amdgpu_buffer_rsrc_t pb =
        raw_buffer(part, static_cast<uint32_t>(rows) * static_cast<uint32_t>(H) * 4u);
    float s = 0.0f;
    for (int p0 = r; p0 < rows; p0 += kSumRows * kSumLoads) {
        float v[kSumLoads];
#pragma unroll
        for (int i = 0; i < kSumLoads; ++i)
            v[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                pb, ((p0 + i * kSumRows) * H + min(c, H - 1)) * 4, 0, 0));
#pragma unroll
        for (int i = 0; i < kSumLoads; ++i) s += v[i];
    }
    acc[r][x] = s;
    __syncthreads();
    if (r == 0 && c < H) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kSumRows; ++i) s += acc[i][x];
        dw[c] = s;
    }
}

// Blocks with grad_w: one per CU, each with as many rows at a time as 16 waves hold, so that
// the partial rows stay few. Measured at 7168 channels, two words per lane: 256 blocks of two
// rows at a time 46.8 us at 4096 tokens and 138.4 us at 14000; 512 blocks of one row 47.2 and
// 146.9 us (one word per lane: 256 blocks 52.6 and 157.7 us, 1024 blocks 64.5 and 168.2 us).
// Batches of up to 256 rows take a row per block: 256 tokens 11.1 us against 12.4 us where the
// two were compared, 9.5 us in the latest run. What one block holds at once needs no second
// launch: 8 tokens of 1024 channels 5.9 us from the host and 4.9 in a graph, against 9.3 and
// 5.2; two rounds of one block 6.0 and 6.6 (16 tokens).
constexpr int64_t kGradBlocks = 256;
// From this many bytes of h on, the rows' loads are non-temporal. Cached against
// non-temporal: 17.6 against 18.2 us at 1024 tokens of 7168 channels (15 MB), 23.8 against
// 25.0 us at 14000 of 1024 (29 MB), 51.3 against 46.8 us at 4096 of 7168 (59 MB).
constexpr int64_t kGradStreamBytes = int64_t{40} << 20;

// Launch shape of the gradient with rows in registers; W == 0 for rows wider than that.
struct GradShape {
    int nv, W, G;
    int64_t blocks;  // with grad_w
};

GradShape grad_shape(int64_t T, int V) {
    GradShape s{};
    const int words = (V + kWave - 1) / kWave;
    if (words > 2 * kMaxWaves) return s;
    s.nv = words > kMaxWaves / 2 ? 2 : 1;
    s.W = (words + s.nv - 1) / s.nv;
    const int most = kMaxWaves / s.W;
    s.G = T <= most ? most
                    : static_cast<int>(std::min<int64_t>(most, (T + kGradBlocks - 1) / kGradBlocks));
    s.blocks = std::min<int64_t>(kGradBlocks, (T + s.G - 1) / s.G);
    return s;
}

constexpr int kDwChunks = 64;  // partial rows of grad_w

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

hipError_t launch_rmsnorm(const void* x, const void* residual, const void* weight,
                          bool weight_fp32, float eps, int64_t T, int H, void* residual_out,
                          void* y, uint8_t* y_fp8, float* y_scales, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    const int V = H / 8;
    // launches of at most kMaxRows rows: a dispatch packet counts threads in 32 bits
    const auto launch = [&](auto kernel, int rows_per_block, int threads) {
        for (int64_t t0 = 0; t0 < T; t0 += kMaxRows) {
            const int64_t t_end = std::min(T, t0 + kMaxRows);
            const int64_t grid = (t_end - t0 + rows_per_block - 1) / rows_per_block;
            hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, stream,
                               static_cast<const u32x4*>(x), static_cast<const u32x4*>(residual),
                               weight, eps, t0, t_end, V, static_cast<u32x4*>(residual_out),
                               static_cast<u32x4*>(y), reinterpret_cast<u32x2*>(y_fp8), y_scales);
            EP_RETURN_IF_LAUNCH_FAILED();
        }
        return hipSuccess;
    };
    using Nt = std::integral_constant<int, kPolicyNt>;
    using Cached = std::integral_constant<int, 0>;
    const auto row = [&](auto nv, auto one_wave) {
        constexpr int n = decltype(nv)::value;
        constexpr bool one = decltype(one_wave)::value;
        const int threads = one ? kNT : kWave * ((V + kWave * n - 1) / (kWave * n));
        const auto with = [&](auto policy) {
            constexpr int p = decltype(policy)::value;
            return launch(weight_fp32 ? rmsnorm_row_kernel<n, true, one, p>
                                      : rmsnorm_row_kernel<n, false, one, p>,
                          one ? kNWaves : 1, threads);
        };
        return T * V * 16 >= kNormStreamBytes ? with(Nt{}) : with(Cached{});
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    if (V <= kWave) return row(One{}, std::true_type{});
    if (V <= 2 * kWave) return row(Two{}, std::true_type{});
    if (V <= 4 * kWave) return row(Four{}, std::true_type{});
    if (V <= 2 * kMaxWaves * kWave) return row(Two{}, std::false_type{});
    if (V <= 4 * kMaxWaves * kWave) return row(Four{}, std::false_type{});
    return launch(weight_fp32 ? rmsnorm_kernel<true> : rmsnorm_kernel<false>, 1, kNT);
}

size_t rmsnorm_grad_workspace_bytes(int64_t T, int H) {
    if (T == 0) return 0;
    // as many partial rows as any batch of up to T rows takes, so that a workspace for a
    // larger batch serves a smaller one
    if (grad_shape(T, H / 8).W)
        return sizeof(float) * static_cast<size_t>(std::min(T, kGradBlocks)) *
               static_cast<size_t>(H);
    return align256(sizeof(float) * static_cast<size_t>(T)) +
           sizeof(float) * static_cast<size_t>(kDwChunks) * static_cast<size_t>(H);
}

// Rows wider than the registers hold (past 16384 channels): every row is read from memory as
// often as it is used. 138 us for 1024 rows of 40960 (2.4 TB/s).
static hipError_t launch_wide_grad(const u32x4* dy, const u32x4* dres, const u32x4* h,
                                   const void* weight, bool weight_fp32, float eps, int64_t T,
                                   int H, u32x4* grad_x, float* grad_weight, void* workspace,
                                   hipStream_t stream) {
    if (!grid_fits(T, kNT)) return hipErrorInvalidConfiguration;
    const int V = H / 8;
    const unsigned grid = static_cast<unsigned>(T);
    if (grad_weight) {  // before grad_x, which may take the place of any of its inputs
        float* rstd = static_cast<float*>(workspace);
        float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                               align256(sizeof(float) * static_cast<size_t>(T)));
        const int64_t rows = (T + kDwChunks - 1) / kDwChunks;
        const int chunks = static_cast<int>((T + rows - 1) / rows);
        hipLaunchKernelGGL(rmsnorm_rstd_kernel, dim3(grid), dim3(kNT), 0, stream, h, eps, V, rstd);
        EP_RETURN_IF_LAUNCH_FAILED();
        hipLaunchKernelGGL(rmsnorm_dw_kernel,
                           dim3((V + kWave - 1) / kWave, static_cast<unsigned>(chunks)), dim3(kNT),
                           0, stream, dy, h, rstd, T, V, rows, part);
        EP_RETURN_IF_LAUNCH_FAILED();
        hipLaunchKernelGGL(rmsnorm_dw_join_kernel, dim3((H + kNT - 1) / kNT), dim3(kNT), 0, stream,
                           part, H, chunks, grad_weight);
        EP_RETURN_IF_LAUNCH_FAILED();
    }
    const auto kernel = weight_fp32 ? rmsnorm_dx_kernel<true> : rmsnorm_dx_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kNT), 0, stream, dy, dres, h, weight, eps, V,
                       grad_x);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(const void* grad_y, const void* grad_residual_out, const void* h,
                               const void* weight, bool weight_fp32, float eps, int64_t T, int H,
                               void* grad_x, float* grad_weight, void* workspace,
                               hipStream_t stream) {
    if (T == 0) {
        if (!grad_weight) return hipSuccess;
        return launch_zero_ints(ZeroInts{{reinterpret_cast<int32_t*>(grad_weight)}, {H}}, stream);
    }
    const int V = H / 8;
    const auto* dy = static_cast<const u32x4*>(grad_y);
    const auto* dres = static_cast<const u32x4*>(grad_residual_out);
    const auto* hp = static_cast<const u32x4*>(h);
    auto* dx = static_cast<u32x4*>(grad_x);
    const GradShape s = grad_shape(T, V);
    if (!s.W)
        return launch_wide_grad(dy, dres, hp, weight, weight_fp32, eps, T, H, dx, grad_weight,
                                workspace, stream);
    // Without grad_w nothing ties a block to many rows. Measured at 7168 channels against the
    // form with grad_w: 5.4 against 9.5 us at 256 tokens, 12.2 against 17.5 at 1024, 22.8
    // against 26.0 at 2048; but 51.9 against 46.2 at 4096 and 171.7 against 136.6 at 14000,
    // where a block that holds a row once has no next row in flight while it reduces and writes.
    const int64_t grid =
        grad_weight ? s.blocks : std::min<int64_t>((T + s.G - 1) / s.G, int64_t{1} << 16);
    // a single block's partial row is the sum (it leaves in 128-bit words)
    const bool direct = s.blocks == 1 && reinterpret_cast<uintptr_t>(grad_weight) % 16 == 0;
    float* part = direct ? grad_weight : static_cast<float*>(workspace);
    const auto launch = [&](auto nv, auto policy) {
        constexpr int n = decltype(nv)::value, p = decltype(policy)::value;
        const auto kernel =
            weight_fp32 ? (grad_weight ? rmsnorm_grad_row_kernel<n, true, true, p>
                                       : rmsnorm_grad_row_kernel<n, true, false, p>)
                        : (grad_weight ? rmsnorm_grad_row_kernel<n, false, true, p>
                                       : rmsnorm_grad_row_kernel<n, false, false, p>);
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kWave * s.W * s.G), 0,
                           stream, dy, dres, hp, weight, eps, T, V, s.W, dx, part);
        return hipGetLastError();
    };
    const auto with = [&](auto policy) {
        return s.nv == 1 ? launch(std::integral_constant<int, 1>{}, policy)
                         : launch(std::integral_constant<int, 2>{}, policy);
    };
    const hipError_t e = T * V * 16 >= kGradStreamBytes
                             ? with(std::integral_constant<int, kPolicyNt>{})
                             : with(std::integral_constant<int, 0>{});
    if (e != hipSuccess || !grad_weight || direct) return e;
    hipLaunchKernelGGL(rmsnorm_dw_sum_kernel, dim3((H + kSumCols - 1) / kSumCols),
                       dim3(kMaxWaves * kWave), 0, stream, part, H, static_cast<int>(s.blocks),
                       grad_weight);
    return hipGetLastError();
}

}  // namespace ep
