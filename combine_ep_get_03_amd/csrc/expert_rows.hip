// expert_rows.hip -- the expert-major rows on gfx950: e4m3 rows out to the experts, the
// experts' rows back to their tokens with the gate weights applied, and the gradients of
// both ways. With q = expert_slot[t][j] of token t's j-th pair (q < 0: not routed):
//   permute fp8    row q of the codes and of the scales = token t's
//   unpermute      out[t] = bf16(sum over j of w[t][j] y[q] (+ addend[t])), fp32, ascending j
//   its gradient   grad_y[q] = bf16(w[t][j] grad_out[t]), grad_w[t][j] = <grad_out[t], y[q]>
//   permute's      grad_x[t] = bf16(sum over j of grad_perm_x[q]), grad_w[t][j] = grad_perm_w[q]
// All are bound by the bytes of the expert-major rows, which move once.
#include "dispatch_rows.hpp"
#include "expert_ops.hpp"

namespace ep {
namespace {

constexpr int kT = 256;  // threads per block: a few waves, each with its own piece of work
constexpr int kUnpermuteThreads = 128;
constexpr int64_t kMaxWaves = int64_t{1} << 24;  // per launch: a wave's index stays 32 bits

// f(t0, t_end, grid) launches over token ranges of at most kMaxWaves waves, kThreads / 64 of
// them per block, and returns its launch's status; the first failure ends the call.
template <int kThreads, typename F>
hipError_t by_token_range(int64_t T, int waves_per_token, F&& f) {
    constexpr int kWaves = kThreads / kWave;
    const int64_t step = std::max<int64_t>(1, kMaxWaves / waves_per_token);
    for (int64_t t0 = 0; t0 < T; t0 += step) {
        const int64_t t_end = std::min(T, t0 + step);
        const int64_t grid = ((t_end - t0) * waves_per_token + kWaves - 1) / kWaves;
        if (!grid_fits(grid, kThreads)) return hipErrorInvalidConfiguration;
        const hipError_t e = f(t0, t_end, static_cast<unsigned>(grid));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Wave (t, d) copies token t's codes and scales to the rows of its pairs d kPairs ..
// (d + 1) kPairs - 1, in the form of the bf16 permute: the row's loads are issued before the
// slots arrive, the codes leave as one burst of 128-bit stores (store_row_pass) and the
// token's other waves find the row in the L2. HBM-write bound: 8 rows written per row read at
// top-8. 4096 tokens of 7168 channels over 256 experts: 46.1-46.9 us, 5.9 TB/s; guarded stores in a loop 47.2 us.
//
// One pair per wave from 2176 channels on. Narrower rows would be bound by the rate at which
// waves start, about four per nanosecond, so a wave takes two pairs, and up to 1024 channels
// four. Measured at 12000 tokens, top-8, with one, two and four: 24.5, 18.1, 15.8 us at 256
// channels; 27.0, 21.8, 21.0 at 1024; 32.1, 28.6, 29.9 at 1536; 38.9, 38.4, 39.9 at 2048; 75.8,
// 76.4, 77.8 at 4096.
//
// A row's scales (224 bytes at 7168 channels) fill no whole cache line, so neighbouring rows,
// written by waves of different XCDs, share lines. Cached scale stores let each L2 gather
// its share of a line; past about half of the L2s' 32 MB they are evicted half-filled, and
// non-temporal stores take over. Measured, cached against non-temporal: 46.0 against
// 51.5 us at 4096 tokens (7 MB of scales), 93.3 against 103.4 us at 8192 (15 MB), 172.8
// against 152.1 us at 12000 (22 MB), 236.6 against 229.3 us at 16384 (29 MB). Blocks dealt so
// that each XCD writes an eighth of the rows, and its L2 gathers whole lines, took 59.9 us at
// 4096 tokens, since a token's row is then fetched by five XCDs instead of two.
constexpr int64_t kCachedScaleBytes = int64_t{16} << 20;

template <int WPL, bool kMulti, int kScalePolicy, int kPairs>
__global__ __launch_bounds__(kT) void permute_fp8_kernel(
    const u32x4* __restrict__ codes, const float* __restrict__ scales,
    const float* __restrict__ topk_w, int64_t t0, int64_t t_end, int V, int G, int k,
    const int32_t* __restrict__ expert_slot, FastDiv D, u32x4* __restrict__ perm_codes,
    float* __restrict__ perm_scales, float* __restrict__ perm_w, int32_t* __restrict__ perm_src,
    int64_t cap, int32_t* __restrict__ error_flag) {
    int64_t t;
    int d;
    if (!dest_wave<kT>(t0, t_end, D, t, d)) return;
    const int lane = lane_id();
    int32_t q[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int j = d * kPairs + i;
        q[i] = kPairs == 1 || j < k ? expert_slot[t * k + min(j, k - 1)] : -1;
    }
    const u32x4* xr = codes + t * V;
    const float* sr = scales + t * G;
    u32x4 v[WPL];
    load_row_cached(v, xr, 0, V);  // first pass, issued before the slots are known
    const float s0 = sr[min(lane, G - 1)];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        if (q[i] < 0) continue;
        if (q[i] >= cap) {
            if (lane == 0) raise_error(error_flag, kErrRecvOverflow);
            continue;
        }
        const int64_t qi = q[i];
        u32x4* row = perm_codes + qi * V;
        for (int v0 = 0; v0 < V; v0 += kWave * WPL) {
            if (v0 != 0) load_row_cached(v, xr, v0, V);
            store_row_pass(row, V, v0, v);
            if constexpr (!kMulti) break;
        }
        const __amdgpu_buffer_rsrc_t sb =
            raw_buffer(perm_scales + qi * G, static_cast<uint32_t>(G) * 4u);
        float s = s0;
        for (int g = lane; g - lane < G; g += kWave) {  // stores past G are dropped
            if (g != lane) s = sr[min(g, G - 1)];
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), sb, g * 4, 0, kScalePolicy);
        }
        if (lane == 0) {
            if (perm_w) perm_w[qi] = topk_w[t * k + d * kPairs + i];
            if (perm_src) perm_src[qi] = static_cast<int32_t>(t);
        }
    }
}

// kB of token t's pairs, j0 .. j0 + kB - 1, for every lane of a wave alike: their weights, and
// their rows' places as buffers of V words. A pair that is not routed, out of range or past
// k gets a buffer of no bytes and the weight -0.0, so that its load returns zeros and its
// store is dropped without a branch: behind a branch of its own, each load would first
// wait for every load before it. Its product -0.0 changes no sum, a sum of -0.0 included.
// t has to be the same in all lanes.
template <int kB>
struct Pairs {
    int32_t q[kB];
    float w[kB];

    __device__ __forceinline__ Pairs(const int32_t* __restrict__ slot,
                                     const float* __restrict__ topk_w, int64_t t, int j0, int k,
                                     int64_t num_rows, int32_t& errbits) {
        const int64_t at = t * k;
#pragma unroll
        for (int i = 0; i < kB; ++i) q[i] = slot[at + min(j0 + i, k - 1)];
#pragma unroll
        for (int i = 0; i < kB; ++i) w[i] = 1.0f;
        if (topk_w) {
#pragma unroll
            for (int i = 0; i < kB; ++i) w[i] = topk_w[at + min(j0 + i, k - 1)];
        }
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            if (q[i] >= num_rows) errbits |= kErrSlotRange;
            if (q[i] >= num_rows || j0 + i >= k) q[i] = -1;
            if (q[i] < 0) w[i] = -0.0f;
        }
    }

    __device__ __forceinline__ __amdgpu_buffer_rsrc_t place(const u32x4* rows, int i, int V) const {
        return raw_buffer(rows + static_cast<int64_t>(max(q[i], 0)) * V,
                          q[i] >= 0 ? static_cast<uint32_t>(V) * 16u : 0u);
    }
};

// Wave (t, c) sums words [64 c, 64 c + 64) of token t's rows, one word per lane, kB rows'
// loads in flight together. Bound by the rows' reads (8 per row written at top-8). Measured
// on MI355X at 7168 channels, top-8 of 256 experts: 88.9 us at 4096 tokens and 398.3 us at
// 16384 with an addend (5.9 TB/s); 64 tokens 4.3 us. Blocks of 256 threads took 90.1 and
// 410.7 us, of 448 90.2 and 416.8 us; two words per lane 90.9 and 419.7 us; cached row loads
// 97.2 and 434.9 us; a block per token walking its pairs one after the other 99.2, 456.2 and
// (64 tokens) 12.7 us.
template <int kB>
__global__ __launch_bounds__(kUnpermuteThreads) void unpermute_kernel(
    const u32x4* __restrict__ rows, int64_t num_rows, const float* __restrict__ topk_w,
    const int32_t* __restrict__ expert_slot, int64_t t0, int64_t t_end, int V, int k, FastDiv C,
    const u32x4* addend, u32x4* out, const float* __restrict__ grad_perm_w,
    float* __restrict__ grad_w, int32_t* __restrict__ error_flag) {
    int64_t t;
    int c;
    if (!dest_wave<kUnpermuteThreads>(t0, t_end, C, t, c)) return;
    const int lane = lane_id();
    const int v = c * kWave + lane;
    const u32x4 ad = load_word<kPolicyNt>(row_buffer(addend, t, V), v);
    // under an addend the sum starts at -0.0, so that a token with no pair gets the addend's
    // own bits; without one at +0.0, which is what such a token then gets
    const float start = addend ? -0.0f : 0.0f;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = start;
    int32_t errbits = 0;
    for (int j0 = 0; j0 < k; j0 += kB) {
        const Pairs<kB> pr(expert_slot, topk_w, t, j0, k, num_rows, errbits);
        u32x4 p[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) p[i] = load_word<kPolicyNt>(pr.place(rows, i, V), v);
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            float f[8];
            widen8(p[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += pr.w[i] * f[e];
        }
    }
    float f[8];
    widen8(ad, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += acc[e];
    store_word<kPolicyNt>(row_buffer(out, t, V), v, narrow8(f));
    if (c == 0) {
        if (errbits && lane == 0) raise_error(error_flag, errbits);
        if (grad_w) {
            for (int j = lane; j < k; j += kWave) {
                const int64_t s = expert_slot[t * k + j];
                grad_w[t * k + j] = s >= 0 && s < num_rows ? grad_perm_w[s] : 0.0f;
            }
        }
    }
}

// Wave (t, j) has the pair's row to itself: kDot adds up <grad_out[t], row q> in registers and
// one wave reduction, kRows writes row q = w grad_out[t]; with both, the row is read before
// it is written, word by word, so grad_rows may be rows. grad_out's row is read with
// cached loads, which a token's other waves hit, and its first pass is issued before the
// slot arrives. A short-lived wave per pair keeps the rows in flight close together in
// memory: a block per token, all its pairs at once (one read of grad_out, dots joined
// through LDS), took 191.5 against 187.5 us at 4096 tokens and 9.3 against 8.2 us at 64.
//
// kLoad: the cache policy of the rows' loads. kStore: of their stores.
template <int WPL, bool kDot, bool kRows, int kLoad, int kStore, int kThreads>
__global__ __launch_bounds__(kThreads) void unpermute_grad_kernel(
    const u32x4* __restrict__ grad_out, const u32x4* rows, int64_t num_rows,
    const float* __restrict__ topk_w, const int32_t* __restrict__ expert_slot, int64_t t0,
    int64_t t_end, int V, int k, FastDiv D, u32x4* grad_rows, float* __restrict__ grad_w,
    int32_t* __restrict__ error_flag) {
    int64_t t;
    int j;
    if (!dest_wave<kThreads>(t0, t_end, D, t, j)) return;
    const int lane = lane_id();
    const int64_t at = t * k + j;
    const int64_t q = expert_slot[at];
    const float w = topk_w ? topk_w[at] : 1.0f;
    const __amdgpu_buffer_rsrc_t gb = row_buffer(grad_out, t, V);
    u32x4 g[WPL];
#pragma unroll
    for (int i = 0; i < WPL; ++i) g[i] = load_word<0>(gb, i * kWave + lane);
    if (q < 0 || q >= num_rows) {
        if (lane == 0) {
            if (kDot) grad_w[at] = 0.0f;
            if (q >= num_rows) raise_error(error_flag, kErrSlotRange);
        }
        return;
    }
    const __amdgpu_buffer_rsrc_t yb = row_buffer(rows, q, V);
    const __amdgpu_buffer_rsrc_t ob = row_buffer(grad_rows, q, V);
    float dot = 0.0f;
    for (int v0 = 0; v0 < V; v0 += kWave * WPL) {
        u32x4 y[WPL];
        if constexpr (kDot) {
#pragma unroll
            for (int i = 0; i < WPL; ++i) y[i] = load_word<kLoad>(yb, v0 + i * kWave + lane);
        }
        if (v0 != 0) {
#pragma unroll
            for (int i = 0; i < WPL; ++i) g[i] = load_word<0>(gb, v0 + i * kWave + lane);
        }
#pragma unroll
        for (int i = 0; i < WPL; ++i) {
            float gf[8];
            widen8(g[i], gf);
            if constexpr (kDot) {  // words past the row are zeros on both sides
                float f[8];
                widen8(y[i], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot += gf[e] * f[e];
            }
            if constexpr (kRows) {
#pragma unroll
                for (int e = 0; e < 8; ++e) gf[e] *= w;
                store_word<kStore>(ob, v0 + i * kWave + lane, narrow8(gf));
            }
        }
    }
    if constexpr (kDot) {
        dot = wave_sum(dot);
        if (lane == 0) grad_w[at] = dot;
    }
}

// Above this many bytes of routed rows the dots and the rows are two launches, one that
// mostly reads and one that mostly writes: HBM moves a stream of reads and then a stream of
// writes faster than the two mixed over scattered rows. Measured on MI355X, one launch
// against two: 188.1 against 168.1 us at 4096 tokens (470 MB of rows; 5.9 TB/s, of which the
// dots 6.4 and the rows 5.7), 394 against 338 us at 8192, 48.5 against 44.7 us at 1024
// (117 MB). Below it one launch with cached row loads, since a set this small may still lie
// in the 256 MB Infinity Cache, where the experts left it: 22.7 us against 28.1 us with
// non-temporal loads at 512 tokens (59 MB), and the second launch would be a larger share.
constexpr int64_t kOneLaunchBytes = int64_t{64} << 20;
// The launches that read rows take blocks of 512 threads, so that a top-8 token's waves share
// an XCD and its L2 fetches grad_out's row once: 10.6 against 11.1 us at 256 tokens, 169.8
// against 172.9 us at 4096 (128 threads 198.4 us). Below this many pairs that would leave CUs
// without a block, and blocks of 256 take over: 5.1 against 6.4 us at 64 tokens.
constexpr int64_t kWideBlockPairs = 2048;

}  // namespace

hipError_t launch_dispatch_permute_fp8(const void* x_fp8, const float* x_scales,
                                       const float* topk_w, int64_t T, int H, int k,
                                       const int32_t* expert_slot, void* perm_x,
                                       float* perm_scales, float* perm_w, int32_t* perm_src,
                                       int64_t cap, int32_t* error_flag, hipStream_t stream) {
    const int V = H / 16, G = H / kNormGroup;
    const bool cached = T * k * G * static_cast<int64_t>(sizeof(float)) <= kCachedScaleBytes;
    const auto with = [&](auto pairs) {
        constexpr int n = decltype(pairs)::value;
        const int waves = (k + n - 1) / n;
        const FastDiv fd = FastDiv::make(waves);
        return by_token_range<kT>(T, waves, [&](int64_t t0, int64_t t_end, unsigned grid) {
            return with_row_width<14, false>(V, [&](auto wpl, auto multi) {
                constexpr int w = decltype(wpl)::value;
                constexpr bool m = decltype(multi)::value;
                // the widths that take n pairs per wave: one word per lane four, two words two
                if constexpr (n == (w == 1 ? 4 : w == 2 ? 2 : 1)) {
                    const auto kernel = cached ? permute_fp8_kernel<w, m, 0, n>
                                               : permute_fp8_kernel<w, m, kPolicyNt, n>;
                    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kT), 0, stream,
                                       static_cast<const u32x4*>(x_fp8), x_scales, topk_w, t0,
                                       t_end, V, G, k, expert_slot, fd,
                                       static_cast<u32x4*>(perm_x), perm_scales, perm_w, perm_src,
                                       cap, error_flag);
                }
            });
        });
    };
    if (V <= kWave) return with(std::integral_constant<int, 4>{});
    if (V <= 2 * kWave) return with(std::integral_constant<int, 2>{});
    return with(std::integral_constant<int, 1>{});
}

static hipError_t launch_unpermute(const void* rows, int64_t num_rows, const float* topk_w,
                                   const int32_t* expert_slot, int64_t T, int H, int k,
                                   const void* addend, void* out, const float* grad_perm_w,
                                   float* grad_w, int32_t* error_flag, hipStream_t stream) {
    const int V = H / 8;
    const int C = (V + kWave - 1) / kWave;
    const FastDiv fd = FastDiv::make(C);
    const auto kernel = k <= 2   ? unpermute_kernel<2>
                        : k <= 4 ? unpermute_kernel<4>
                                 : unpermute_kernel<8>;
    return by_token_range<kUnpermuteThreads>(T, C, [&](int64_t t0, int64_t t_end, unsigned grid) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(kUnpermuteThreads), 0, stream,
                           static_cast<const u32x4*>(rows), num_rows, topk_w, expert_slot, t0,
                           t_end, V, k, fd, static_cast<const u32x4*>(addend),
                           static_cast<u32x4*>(out), grad_perm_w, grad_w, error_flag);
        return hipGetLastError();
    });
}

hipError_t launch_combine_unpermute(const void* rows, int64_t num_rows, const float* topk_w,
                                    const int32_t* expert_slot, int64_t T, int H, int k,
                                    const void* addend, void* out, int32_t* error_flag,
                                    hipStream_t stream) {
    return launch_unpermute(rows, num_rows, topk_w, expert_slot, T, H, k, addend, out, nullptr,
                            nullptr, error_flag, stream);
}

hipError_t launch_dispatch_permute_grad(const void* grad_rows, const float* grad_perm_w,
                                        int64_t num_rows, const int32_t* expert_slot, int64_t T,
                                        int H, int k, void* grad_x, float* grad_w,
                                        int32_t* error_flag, hipStream_t stream) {
    return launch_unpermute(grad_rows, num_rows, nullptr, expert_slot, T, H, k, nullptr, grad_x,
                            grad_perm_w, grad_w, error_flag, stream);
}

hipError_t launch_combine_unpermute_grad(const void* grad_out, const void* rows,
                                         int64_t num_rows, const float* topk_w,
                                         const int32_t* expert_slot, int64_t T, int H, int k,
                                         void* grad_rows, float* grad_w, int32_t* error_flag,
                                         hipStream_t stream) {
    const int V = H / 8;
    const FastDiv fd = FastDiv::make(k);
    const auto pass = [&](auto dot, auto write, auto load, auto store, auto threads, auto width) {
        constexpr bool d = decltype(dot)::value, r = decltype(write)::value;
        constexpr int ld = decltype(load)::value, st = decltype(store)::value;
        constexpr int n = decltype(threads)::value;
        return by_token_range<n>(T, k, [&](int64_t t0, int64_t t_end, unsigned grid) {
            return with_row_width<decltype(width)::value, false>(V, [&](auto wpl, auto) {
                hipLaunchKernelGGL((unpermute_grad_kernel<decltype(wpl)::value, d, r, ld, st, n>),
                                   dim3(grid), dim3(n), 0, stream,
                                   static_cast<const u32x4*>(grad_out),
                                   static_cast<const u32x4*>(rows), num_rows, topk_w, expert_slot,
                                   t0, t_end, V, k, fd, static_cast<u32x4*>(grad_rows), grad_w,
                                   error_flag);
            });
        });
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    constexpr std::integral_constant<int, 0> cached{};
    constexpr std::integral_constant<int, kPolicyNt> nt{};
    constexpr std::integral_constant<int, kPolicyNt | kPolicySc1> nt_device{};
    constexpr std::integral_constant<int, 256> t256{};
    constexpr std::integral_constant<int, 512> t512{};
    constexpr std::integral_constant<int, 7> w7{};
    constexpr std::integral_constant<int, 14> w14{};
    if (grad_w && T * k * V * 16 <= kOneLaunchBytes)
        return T * k >= kWideBlockPairs ? pass(yes, yes, cached, nt, t512, w14)
                                        : pass(yes, yes, cached, nt, t256, w14);
    if (grad_w) {
        const hipError_t e = pass(yes, no, nt, nt, t512, w7);
        if (e != hipSuccess) return e;
    }
    return pass(no, yes, nt, nt_device, t256, w7);
}

}  // namespace ep
