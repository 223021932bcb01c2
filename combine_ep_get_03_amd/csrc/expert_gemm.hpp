// expert_gemm.hpp -- the grouped matrix product behind the experts' own operators
// (expert_ffn.hip, expert_ffn_grad.hip): tiles of 256 x 256 outputs fed from LDS to the matrix
// cores, over rows sorted by expert whose counts are known on the device alone. Not part of
// the public ABI.
//
// One product is out[m][n] = sum over k of A[m][k] B[n][k] within one expert. The m side is the
// expert's rows (or, for a weight's gradient, the gradient's channels), the n side the output
// channels. An operand lies in memory either with k contiguous ("by rows") or with m or n
// contiguous ("by columns"); the second is turned on the way from LDS to the registers.
#pragma once

#include "expert_ops.hpp"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kTileM = 256;         // rows (m side) of a tile
constexpr int kTileN = 256;         // channels (n side) of a tile
constexpr int kGemmThreads = 512;   // 8 waves, 2 along m and 4 along n
constexpr int kGemmWaves = kGemmThreads / kWave;
constexpr int kStepBytes = 128;     // bytes of k per row and step: 64 bf16 or 128 e4m3
constexpr int kOperandBytes = 256 * kStepBytes;  // one operand of one step in LDS
constexpr int kScaleBytes = 2048;   // one step's row scales in LDS (the second half unused)
constexpr int kAmaxBytes = kTileM * 2 * 4 * 4;  // [row][gate, up][wave along n] magnitudes
constexpr uint32_t kOutOfBuffer = 0x80000000u;  // an offset past every buffer made here

enum class GemmOp {
    kGateUp,      // two projections, silu(gate) * up; A by rows, B by rows
    kDown,        // plain; A by rows, B by rows
    kDownGrad,    // through the activation; A by rows, B by columns
    kInputGrad,   // plain; A by rows, B by columns
    kWeightGrad,  // over the rows; A by columns, B by columns
};

// ---------------------------------------------------------------- asynchronous loads to LDS
// A raw buffer of `bytes` bytes from `base` (both the same in every lane) in scalar registers,
// as the inline loads below take it.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 scalar_buffer(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4 d;
    d[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(a));
    d[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32) & 0xffff);
    d[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
    d[3] = kRawBufferWord3;
    return d;
}

// Each lane's 16 (4) bytes at base + voff + soff go to LDS at lds + 16 (4) * lane. Lanes past
// the buffer's end write zeros. Inline so that the compiler does not order its LDS reads after
// these writes: the kernel waits and synchronises itself, once per step. Nothing is returned in
// registers. m0 is set in the same block as it is used.
__device__ __forceinline__ void load_lds16(i32x4 buf, uint32_t lds,
                                           uint32_t voff, uint32_t soff) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    soff = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
}
__device__ __forceinline__ void load_lds4(i32x4 buf, uint32_t lds, uint32_t voff,
                                          uint32_t soff) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    soff = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
}

template <int kOutstanding>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kOutstanding) : "memory");
}

// Every wave's LDS accesses before are done, and none after has begun.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char*)p));
}

// ---------------------------------------------------------------- which tile is whose
// The tiles of all experts in one order: expert after expert, and within one in bands of four
// along m with n inside, so that the 32 blocks of one die share four parts of A and eight of
// B in its L2. An expert of c rows has ceil(c / kTileM) tiles along m of about equal heights.
// Every lane holds the number of such tiles before its chunk of experts; a tile is found by a
// ballot and a walk through one chunk. Offsets are taken as non-negative and ascending, and
// clamped to num_rows; where they are not, nothing is computed.
constexpr int kBandM = 4;

struct Tile {
    int expert;
    int m0, n0;    // first row (within the expert) or channel of the m side, and of the n side
    int64_t row0;  // the expert's first row
    int rows;      // the expert's rows
    int height;    // valid rows (channels) of the m side in this tile
};

struct TileMap {
    const int32_t* offset;
    int64_t num_rows;
    int chunk, E, nt, first;
    int64_t total;
    bool by_rows;  // m tiles cover an expert's rows; else M channels, mt of them per expert
    int M, mt;

    __device__ __forceinline__ int tiles(int c) const { return (c + kTileM - 1) / kTileM; }

    __device__ __forceinline__ void init(const GemmArgs& g, bool rows, int n_tile) {
        offset = g.offset;
        num_rows = g.num_rows;
        E = g.E;
        by_rows = rows;
        M = g.M;
        nt = (g.N + n_tile - 1) / n_tile;
        chunk = (E + kWave - 1) / kWave;
        const int lane = lane_id();
        const int e0 = min(lane * chunk, E), e1 = min(e0 + chunk, E);
        int count = 0;
        int64_t prev = offset[e0];
        bool bad = prev < 0, over = false;
        for (int e = e0; e < e1; ++e) {
            const int64_t next = offset[e + 1];
            bad |= next < prev;
            over |= next > num_rows;
            count += tiles(static_cast<int>(min(next, num_rows) - min(prev, num_rows)));
            prev = next;
        }
        int sum = count;
        for (int d = 1; d < kWave; d *= 2) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        first = sum - count;
        mt = rows ? __builtin_amdgcn_readlane(sum, kWave - 1) : tiles(M);
        total = static_cast<int64_t>(mt) * nt * (rows ? 1 : E);
        bad = wave_ballot(bad) != 0;
        over = wave_ballot(over) != 0;
        if (bad) total = 0;
        if ((bad || over) && blockIdx.x == 0 && threadIdx.x == 0)
            raise_error(g.error_flag, kErrSlotRange);
    }

    __device__ __forceinline__ void place(Tile& t, int in_expert, int mts, int n_tile) const {
        const int band = in_expert / (kBandM * nt);
        const int r = in_expert - band * kBandM * nt;
        const int high = min(kBandM, mts - band * kBandM);
        const int n = r / high;
        t.n0 = n * n_tile;
        t.m0 = band * kBandM + (r - n * high);  // the m tile's number, made a row by the caller
    }

    __device__ __forceinline__ Tile find(int64_t index, int n_tile) const {
        Tile t;
        int mts, in_expert;
        if (by_rows) {
            const uint64_t le =
                wave_ballot(static_cast<int64_t>(first) * nt <= index);
            const int lane = 63 - __builtin_clzll(le);
            int base = __builtin_amdgcn_readlane(first, lane);
            int e = lane * chunk;
            int64_t a = min<int64_t>(offset[e], num_rows);
            for (;;) {
                const int64_t b = min<int64_t>(offset[e + 1], num_rows);
                mts = tiles(static_cast<int>(b - a));
                if (index < static_cast<int64_t>(base + mts) * nt) {
                    t.rows = static_cast<int>(b - a);
                    break;
                }
                base += mts;
                a = b;
                ++e;
            }
            t.expert = e;
            t.row0 = a;
            in_expert = static_cast<int>(index - static_cast<int64_t>(base) * nt);
            place(t, in_expert, mts, n_tile);
            const int each = ((t.rows + mts - 1) / mts + 15) & ~15;
            t.m0 *= each;
            t.height = min(each, t.rows - t.m0);
        } else {
            const int per = mt * nt;
            t.expert = static_cast<int>(index / per);
            in_expert = static_cast<int>(index - static_cast<int64_t>(t.expert) * per);
            t.row0 = min<int64_t>(offset[t.expert], num_rows);
            t.rows = static_cast<int>(min<int64_t>(offset[t.expert + 1], num_rows) - t.row0);
            place(t, in_expert, mt, n_tile);
            t.m0 *= kTileM;
            t.height = min(kTileM, M - t.m0);
        }
        return t;
    }
};

// ---------------------------------------------------------------- one operand's loads
// By rows: a step is 128 bytes of each of 256 rows, row after row in LDS, with a row's 16-byte
// word c at place c ^ (row & 7): eight lanes of a fragment's read, on eight rows, then hit
// eight different places. Each wave load writes eight rows. By columns: a step is 64 rows of k
// of 256 channels (512 bytes), with the 32-byte pair of words p at place p ^ turn(k), so that
// a transposing read's four rows (of each of two groups of lanes) lie in different banks.
__device__ __forceinline__ int turn(int k) { return (k & 3) | ((k >> 1) & 4); }

template <bool kByRows>
struct OperandLoads {
    static constexpr int kLoads = 4;  // per wave and step
    uint32_t voff[kLoads];

    // rows: valid rows from the first; width: valid bytes of a row of `stride`
    __device__ __forceinline__ void init_rows(int wave, int lane, int rows, uint32_t stride) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            const int row = (t * kGemmWaves + wave) * 8 + lane / 8;
            voff[t] = row < rows ? row * stride + (((lane & 7) ^ (lane >> 3)) * 16) : kOutOfBuffer;
        }
    }
    // columns: valid columns from col0
    __device__ __forceinline__ void init_columns(int wave, int lane, int col0, int columns,
                                                 uint32_t stride) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            const int k = (t * kGemmWaves + wave) * 2 + lane / 32;
            const int word = (lane & 31) ^ (2 * turn(k));
            voff[t] = word * 8 < columns ? k * stride + (col0 + word * 8) * 2 : kOutOfBuffer;
        }
    }
    // by rows, last step: words past the row's end read zeros
    __device__ __forceinline__ void cut(int lane, int words) {
        if (((lane & 7) ^ (lane >> 3)) >= words) {
#pragma unroll
            for (int t = 0; t < kLoads; ++t) voff[t] = kOutOfBuffer;
        }
    }
};

// ---------------------------------------------------------------- the kernel
template <GemmOp kOp, bool kFp8>
struct GemmShape {
    static constexpr bool kGated = kOp == GemmOp::kGateUp;
    static constexpr bool kAByRows = kOp != GemmOp::kWeightGrad;
    static constexpr bool kBByRows = kOp == GemmOp::kGateUp || kOp == GemmOp::kDown;
    static constexpr bool kOverRows = kOp == GemmOp::kWeightGrad;  // k runs over the rows
    static constexpr int kNTile = kGated ? kTileN / 2 : kTileN;    // output channels of a tile
    static constexpr int kElem = kFp8 ? 1 : 2;
    static constexpr int kStepK = kStepBytes / kElem;
    static constexpr int kStages = 2;
    static constexpr int kStageBytes = 2 * kOperandBytes + (kFp8 ? kScaleBytes : 0);
    static constexpr int kLoads = 8 + (kFp8 ? 1 : 0);  // per wave and step
    static constexpr bool kAmax = kGated;
    static constexpr int kLdsBytes = kStages * kStageBytes + (kAmax ? kAmaxBytes : 0);
    static_assert(kLdsBytes <= 160 * 1024, "LDS of one CU");
};

// The stream of steps that a block loads: its tiles one after the other, the steps of each.
template <GemmOp kOp, bool kFp8>
struct Producer {
    using S = GemmShape<kOp, kFp8>;
    const GemmArgs& g;
    const TileMap& map;
    int wave, lane;
    int64_t index, stride;
    int step, steps;
    Tile t;
    OperandLoads<S::kAByRows> a;
    OperandLoads<S::kBByRows> b;
    uint32_t scale_voff;
    const char *a_base = nullptr, *b_base = nullptr, *b_up = nullptr;
    uint32_t a_row, b_row;  // bytes between rows in memory

    __device__ __forceinline__ Producer(const GemmArgs& g_, const TileMap& m, int64_t first,
                                        int64_t by)
        : g(g_), map(m), wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)),
          lane(lane_id()), index(first), stride(by), step(0), steps(0), t{} {
        a_row = static_cast<uint32_t>(S::kOverRows ? g.M : g.K) * S::kElem;
        b_row = static_cast<uint32_t>(S::kBByRows ? g.K : g.N) * S::kElem;
        if (index < map.total) start();
    }

    __device__ __forceinline__ void start() {
        t = map.find(index, S::kNTile);
        step = 0;
        const int k = S::kOverRows ? t.rows : g.K;
        steps = (k + S::kStepK - 1) / S::kStepK;
        const char* rows_a = static_cast<const char*>(g.a) + t.row0 * a_row;
        if constexpr (S::kAByRows) {
            a_base = rows_a + static_cast<int64_t>(t.m0) * a_row;
            a.init_rows(wave, lane, t.height, a_row);
        } else {
            a_base = rows_a;
            a.init_columns(wave, lane, t.m0, t.height, a_row);
        }
        const int nv = min(S::kNTile, g.N - t.n0);
        if constexpr (S::kOverRows) {
            b_base = static_cast<const char*>(g.b) + t.row0 * b_row;
            b.init_columns(wave, lane, t.n0, nv, b_row);
        } else {
            const int64_t weights = static_cast<int64_t>(S::kGated ? 2 : 1) * g.N * g.K * S::kElem;
            b_base = static_cast<const char*>(g.b) + t.expert * weights;
            if constexpr (S::kBByRows) {
                b_base += static_cast<int64_t>(t.n0) * b_row;
                b_up = b_base + static_cast<int64_t>(g.N) * b_row;
                b.init_rows(wave, lane, nv, b_row);
                if constexpr (S::kGated) {  // tile rows 128..255 are the up projection's
#pragma unroll
                    for (int i = 2; i < 4; ++i) b.voff[i] = b.voff[i - 2];
                }
            } else {
                b.init_columns(wave, lane, t.n0, nv, b_row);
            }
        }
        if constexpr (kFp8) {  // waves 0..3 take 64 rows' scales each
            const int row = wave * kWave + lane;
            scale_voff = row < t.height ? static_cast<uint32_t>(row) * (g.K / 128) * 4u
                                        : kOutOfBuffer;
        }
    }

    __device__ __forceinline__ void issue(uint32_t lds) {
        while (step == steps && index < map.total) {  // an expert without rows has no steps
            index += stride;
            if (index < map.total) start();
        }
        const bool live = index < map.total;
        const int k0 = step * S::kStepK;
        if constexpr (S::kAByRows || S::kBByRows) {
            if (live && k0 + S::kStepK > g.K) {  // only at a tile's last step
                const int words = (g.K - k0) * S::kElem / 16;
                if constexpr (S::kAByRows) a.cut(lane, words);
                if constexpr (S::kBByRows) b.cut(lane, words);
            }
        }
        const uint32_t along = live ? static_cast<uint32_t>(step) * kStepBytes : 0u;
        const uint32_t dst = lds + wave * 1024;
        if constexpr (S::kAByRows) {
            const auto buf = scalar_buffer(a_base, live ? static_cast<uint32_t>(t.height) * a_row : 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_lds16(buf, dst + i * kGemmWaves * 1024, a.voff[i], along);
        } else {
            const uint32_t n = live ? min(64, t.rows - k0) : 0;
            const auto buf = scalar_buffer(a_base + static_cast<int64_t>(k0) * a_row, n * a_row);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_lds16(buf, dst + i * kGemmWaves * 1024, a.voff[i], 0);
        }
        const uint32_t dst_b = dst + kOperandBytes;
        if constexpr (S::kBByRows) {
            const uint32_t n = live ? static_cast<uint32_t>(min(S::kNTile, g.N - t.n0)) * b_row : 0;
            const auto buf = scalar_buffer(b_base, n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (S::kGated) {
                    const auto half = scalar_buffer(i < 2 ? b_base : b_up, n);
                    load_lds16(half, dst_b + i * kGemmWaves * 1024, b.voff[i], along);
                } else {
                    load_lds16(buf, dst_b + i * kGemmWaves * 1024, b.voff[i], along);
                }
            }
        } else {
            const uint32_t n = live ? min(64, (S::kOverRows ? t.rows : g.K) - k0) : 0;
            const auto buf = scalar_buffer(b_base + static_cast<int64_t>(k0) * b_row, n * b_row);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_lds16(buf, dst_b + i * kGemmWaves * 1024, b.voff[i], 0);
        }
        if constexpr (kFp8) {
            const uint32_t row = static_cast<uint32_t>(g.K / 128) * 4u;
            const auto buf = scalar_buffer(g.a_scales + (t.row0 + t.m0) * (g.K / 128),
                                        live ? static_cast<uint32_t>(t.height) * row : 0);
            load_lds4(buf, lds + 2 * kOperandBytes + wave * 256, scale_voff, live ? step * 4u : 0u);
        }
        ++step;
        if (!live) step = steps;
    }
};

__device__ __forceinline__ float silu_sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

__device__ __forceinline__ u32x2 bf16_four(const float (&v)[4]) {
    u32x2 w;
    w[0] = bf16_pair(v[0], v[1]);
    w[1] = bf16_pair(v[2], v[3]);
    return w;
}

__device__ __forceinline__ uint32_t e4m3_four(const float (&v)[4], float inv) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    return static_cast<uint32_t>(
        __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true));
}

constexpr float kE4m3Largest = 448.0f;
constexpr float kSmallestAmax = 0x1p-100f;

// What a group whose largest magnitude is a is scaled to 448 by.
__device__ __forceinline__ float group_amax(float a) {
    return a > 0.0f ? fmaxf(a, kSmallestAmax) : kE4m3Largest;
}

// A lane holds row (column) l % 16 of a fragment and the words of k that belong to l / 16.
template <GemmOp kOp, bool kFp8, int kMT>
__device__ __forceinline__ void gemm_step(f32x4 (&acc)[8][4], const char* lds_a, const char* lds_b,
                                          const char* lds_s, int wm, int wn, int lane,
                                          const float (&bs)[2]) {
    using S = GemmShape<kOp, kFp8>;
    const int row = lane & 15, quad = lane >> 4;
    const int by_row = row * kStepBytes + ((quad ^ (row & 7)) * 16);
    // by columns: lane's row of k within a group of 4, its 8 bytes within the pair
    const int f = (row >> 2) | ((quad & 1) << 2);
    const int by_col = (8 * quad + (row >> 2)) * 512 + (row & 3) * 8;
    auto n_first = [&](int j) {
        return S::kGated ? (j >> 1) * 128 + wn * 32 + (j & 1) * 16 : wn * 64 + j * 16;
    };
    auto read16 = [&](const char* base, bool rows, int first, int s) -> bf16x8 {
        if (rows)
            return *reinterpret_cast<const bf16x8*>(base + first * kStepBytes + (by_row ^ (s * 64)));
        const char* p = base + by_col + s * 32 * 512 + (((first >> 4) ^ f) * 32);
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        union {
            s16x4 h[2];
            bf16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 512));
        return u.v;
    };
    if constexpr (!kFp8) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 b[4], a[kMT];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = read16(lds_b, S::kBByRows, n_first(j), s);
#pragma unroll
            for (int i = 0; i < kMT; ++i) a[i] = read16(lds_a, S::kAByRows, (2 * i + wm) * 16, s);
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
        }
    } else {
        auto read32 = [&](const char* base, int first) -> i32x8 {
            union {
                u32x4 h[2];
                i32x8 v;
            } u;
            u.h[0] = *reinterpret_cast<const u32x4*>(base + first * kStepBytes + by_row);
            u.h[1] = *reinterpret_cast<const u32x4*>(base + first * kStepBytes + (by_row ^ 64));
            return u.v;
        };
        i32x8 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = read32(lds_b, n_first(j));
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const i32x8 a = read32(lds_a, (2 * i + wm) * 16);
            const float as = *reinterpret_cast<const float*>(lds_s + ((2 * i + wm) * 16 + row) * 4);
            const float sc[2] = {as * bs[0], as * bs[1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    b[j], a, zero, 0, 0, 0, 0, 0, 0);
                const float c = sc[S::kGated ? j >> 1 : 0];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[r], c, acc[i][j][r]);
            }
        }
    }
}

// What a tile's sums become in memory. Lane: row (2 i + wm) 16 + l % 16 of the tile, channels
// 4 (l / 16) .. + 3 of each subtile j.
template <GemmOp kOp, bool kFp8>
__device__ __forceinline__ void gemm_store(const GemmArgs& g, const Tile& t, f32x4 (&acc)[8][4],
                                           char* lds_amax, int mt, int wm, int wn, int lane) {
    const int quad = lane >> 4;
    const int64_t first_row = t.row0 + t.m0;
    if constexpr (kOp == GemmOp::kGateUp) {
        const int I = g.N;
        float(*amax)[2][4] = reinterpret_cast<float(*)[2][4]>(lds_amax);
        const bool quantise = g.codes != nullptr;
        if (quantise) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= mt) continue;
                float top[2] = {0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (kFp8) {
                            const float gate = acc[i][j][r];
                            acc[i][j][r] = gate * silu_sigmoid(gate) * acc[i][j + 2][r];
                            top[0] = fmaxf(top[0], fabsf(acc[i][j][r]));
                        } else {
                            top[0] = fmaxf(top[0], fabsf(acc[i][j][r]));
                            top[1] = fmaxf(top[1], fabsf(acc[i][j + 2][r]));
                        }
                    }
#pragma unroll
                for (int h = 0; h < (kFp8 ? 1 : 2); ++h) {
                    top[h] = fmaxf(top[h], __shfl_xor(top[h], 16));
                    top[h] = fmaxf(top[h], __shfl_xor(top[h], 32));
                    if (quad == 0) amax[(2 * i + wm) * 16 + (lane & 15)][h][wn] = top[h];
                }
            }
            lds_barrier();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = (2 * i + wm) * 16 + (lane & 15);
            if (i >= mt || m >= t.height) continue;
            const int64_t row = first_row + m;
            float inv[2], top[2];
            if (quantise) {
#pragma unroll
                for (int h = 0; h < (kFp8 ? 1 : 2); ++h) {
                    const float* p = amax[m][h];
                    top[h] = group_amax(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])));
                    inv[h] = kE4m3Largest / top[h];
                }
                if (wn == 0 && quad == 0) {
                    if constexpr (kFp8) {
                        g.scales[row * (I / 128) + t.n0 / 128] = top[0] / kE4m3Largest;
                    } else {
                        float* s = g.scales + row * (I / 64) + t.n0 / 128;
                        s[0] = top[0] / kE4m3Largest;
                        s[I / 128] = top[1] / kE4m3Largest;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = t.n0 + wn * 32 + j * 16 + quad * 4;
                if (c >= I) continue;
                float gate[4], up[4], act[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    gate[r] = acc[i][j][r];
                    up[r] = acc[i][j + 2][r];
                }
                if constexpr (kFp8) {
                    *reinterpret_cast<uint32_t*>(g.codes + row * I + c) = e4m3_four(gate, inv[0]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) act[r] = gate[r] * silu_sigmoid(gate[r]) * up[r];
                    uint16_t* o = static_cast<uint16_t*>(g.out) + row * I + c;
                    *reinterpret_cast<u32x2*>(o) = bf16_four(act);
                    if (g.gate_up) {
                        uint16_t* s = static_cast<uint16_t*>(g.gate_up) + row * 2 * I + c;
                        *reinterpret_cast<u32x2*>(s) = bf16_four(gate);
                        *reinterpret_cast<u32x2*>(s + I) = bf16_four(up);
                    }
                    if (quantise) {
                        uint8_t* s = g.codes + row * 2 * I + c;
                        *reinterpret_cast<uint32_t*>(s) = e4m3_four(gate, inv[0]);
                        *reinterpret_cast<uint32_t*>(s + I) = e4m3_four(up, inv[1]);
                    }
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = (2 * i + wm) * 16 + (lane & 15);
            if (i >= mt || m >= t.height) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = t.n0 + wn * 64 + j * 16 + quad * 4;
                if (c >= g.N) continue;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r];
                if constexpr (kOp == GemmOp::kWeightGrad) {
                    const int64_t at =
                        (static_cast<int64_t>(t.expert) * g.M + t.m0 + m) * g.N + c;
                    if (g.out_fp32) {
                        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
                        f32x4 w = {v[0], v[1], v[2], v[3]};
                        if (g.accumulate) w += *o;
                        *o = w;
                    } else {
                        u32x2* o = reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at);
                        if (g.accumulate) {
                            const u32x2 w = *o;
                            v[0] += bf16_lo(w[0]);
                            v[1] += bf16_hi(w[0]);
                            v[2] += bf16_lo(w[1]);
                            v[3] += bf16_hi(w[1]);
                        }
                        *o = bf16_four(v);
                    }
                } else if constexpr (kOp == GemmOp::kDownGrad) {
                    const int I = g.N;
                    const int64_t row = first_row + m;
                    float gate[4], up[4];
                    if (g.gate_up) {
                        const uint16_t* s =
                            static_cast<const uint16_t*>(g.gate_up) + row * 2 * I + c;
                        const u32x2 a = *reinterpret_cast<const u32x2*>(s);
                        const u32x2 b = *reinterpret_cast<const u32x2*>(s + I);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            gate[2 * q] = bf16_lo(a[q]);
                            gate[2 * q + 1] = bf16_hi(a[q]);
                            up[2 * q] = bf16_lo(b[q]);
                            up[2 * q + 1] = bf16_hi(b[q]);
                        }
                    } else {
                        const uint8_t* s = g.codes + row * 2 * I + c;
                        const int a = *reinterpret_cast<const int*>(s);
                        const int b = *reinterpret_cast<const int*>(s + I);
                        const float* sc = g.scales + row * (I / 64) + c / 128;
                        const float sg = sc[0], su = sc[I / 128];
                        gate[0] = __builtin_amdgcn_cvt_f32_fp8(a, 0) * sg;
                        gate[1] = __builtin_amdgcn_cvt_f32_fp8(a, 1) * sg;
                        gate[2] = __builtin_amdgcn_cvt_f32_fp8(a, 2) * sg;
                        gate[3] = __builtin_amdgcn_cvt_f32_fp8(a, 3) * sg;
                        up[0] = __builtin_amdgcn_cvt_f32_fp8(b, 0) * su;
                        up[1] = __builtin_amdgcn_cvt_f32_fp8(b, 1) * su;
                        up[2] = __builtin_amdgcn_cvt_f32_fp8(b, 2) * su;
                        up[3] = __builtin_amdgcn_cvt_f32_fp8(b, 3) * su;
                    }
                    float dg[4], du[4], act[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float sig = silu_sigmoid(gate[r]);
                        const float silu = gate[r] * sig;
                        du[r] = v[r] * silu;
                        dg[r] = v[r] * up[r] * sig * (1.0f + gate[r] * (1.0f - sig));
                        act[r] = silu * up[r];
                    }
                    uint16_t* o = static_cast<uint16_t*>(g.out) + row * 2 * I + c;
                    *reinterpret_cast<u32x2*>(o) = bf16_four(dg);
                    *reinterpret_cast<u32x2*>(o + I) = bf16_four(du);
                    if (g.act)
                        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.act) + row * I + c) =
                            bf16_four(act);
                } else {
                    uint16_t* o = static_cast<uint16_t*>(g.out) + (first_row + m) * g.N + c;
                    *reinterpret_cast<u32x2*>(o) = bf16_four(v);
                }
            }
        }
    }
}

// One tile's steps with kMT subtiles of 16 rows per wave. On entry the first step's loads are
// on their way.
template <GemmOp kOp, bool kFp8, int kMT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, const Tile& t, int steps,
                                          Producer<kOp, kFp8>& p, f32x4 (&acc)[8][4], char* lds,
                                          int& slot, int wm, int wn, int lane) {
    using S = GemmShape<kOp, kFp8>;
    const float* bs_row = nullptr;
    if constexpr (kFp8) {
        const int KB = g.K / 128;
        const int nb = S::kGated ? t.n0 / 128 : min((t.n0 + wn * 64) / 128, g.N / 128 - 1);
        bs_row = g.b_scales +
                 (static_cast<int64_t>(t.expert) * (S::kGated ? 2 : 1) * (g.N / 128) + nb) * KB;
    }
    for (int step = 0; step < steps; ++step) {
        wait_loads<0>();
        lds_barrier();
        char* now = lds + slot * S::kStageBytes;
        slot ^= 1;
        p.issue(lds_address(lds + slot * S::kStageBytes));
        float bs[2] = {1.0f, 1.0f};
        if constexpr (kFp8) {
            bs[0] = bs_row[step];
            if constexpr (S::kGated)
                bs[1] = bs_row[static_cast<int64_t>(g.N / 128) * (g.K / 128) + step];
        }
        gemm_step<kOp, kFp8, kMT>(acc, now, now + kOperandBytes, now + 2 * kOperandBytes, wm, wn,
                                  lane, bs);
    }
}

template <GemmOp kOp, bool kFp8>
__global__ __launch_bounds__(kGemmThreads, 1) void gemm_kernel(const GemmArgs g) {
    using S = GemmShape<kOp, kFp8>;
    __shared__ __attribute__((aligned(1024))) char lds[S::kLdsBytes];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;
    TileMap map;
    map.init(g, !S::kOverRows, S::kNTile);
    // block b runs on die b % 8: its tiles are neighbours of that die's other blocks' tiles
    const int per_die = gridDim.x / 8;
    const int64_t first = gridDim.x % 8 == 0
                              ? static_cast<int64_t>(blockIdx.x % 8) * per_die + blockIdx.x / 8
                              : blockIdx.x;
    Producer<kOp, kFp8> p(g, map, first, gridDim.x);
    int slot = 0;
    p.issue(lds_address(lds));
    for (int64_t index = first; index < map.total; index += gridDim.x) {
        const Tile t = map.find(index, S::kNTile);
        const int steps = ((S::kOverRows ? t.rows : g.K) + S::kStepK - 1) / S::kStepK;
        f32x4 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int mt = (t.height + 31) / 32;
        switch (mt) {
#define EP_GEMM_CASE(n)                                                                    \
    case n:                                                                                \
        gemm_tile<kOp, kFp8, n>(g, t, steps, p, acc, lds, slot, wm, wn, lane);             \
        break;
            EP_GEMM_CASE(1)
            EP_GEMM_CASE(2)
            EP_GEMM_CASE(3)
            EP_GEMM_CASE(4)
            EP_GEMM_CASE(5)
            EP_GEMM_CASE(6)
            EP_GEMM_CASE(7)
            EP_GEMM_CASE(8)
#undef EP_GEMM_CASE
        }
        gemm_store<kOp, kFp8>(g, t, acc, lds + S::kStages * S::kStageBytes, mt, wm, wn, lane);
    }
    wait_loads<0>();  // no load of the last step's outlives the block
}

template <GemmOp kOp, bool kFp8>
hipError_t launch_gemm(const GemmArgs& g, hipStream_t stream) {
    using S = GemmShape<kOp, kFp8>;
    constexpr int64_t kBlocks = 256;  // one per CU
    const int64_t nt = (g.N + S::kNTile - 1) / S::kNTile;
    const int64_t mt = S::kOverRows ? static_cast<int64_t>(g.E) * ((g.M + kTileM - 1) / kTileM)
                                    : g.num_rows / kTileM + std::min<int64_t>(g.E, g.num_rows);
    const int64_t blocks = std::min(kBlocks, mt * nt);
    if (blocks == 0) return hipSuccess;
    gemm_kernel<kOp, kFp8><<<static_cast<unsigned>(blocks), kGemmThreads, 0, stream>>>(g);
    return hipGetLastError();
}

}  // namespace ep
