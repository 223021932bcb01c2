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
constexpr int kHalfBytes = kOperandBytes / 2;
constexpr int kScaleBytes = 2048;   // one step's row scales in LDS (the second half unused)
constexpr int kScaleSlots = 4;
constexpr int kTableExperts = 1024; // with at most so many experts, their offsets are kept in LDS
constexpr int kTableBytes = (kTableExperts + 32) * 4;
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
// The tiles of all experts in one order: expert after expert, and within one in bands of at most
// kBandM tiles along m (of about equal numbers) with n outside, so that the 32 blocks of one die
// take about six parts of A and five to eight of B between them and share both in its L2.
// An expert of c rows has ceil(c / kTileM) tiles along m of about equal heights. Every lane
// holds the number of such tiles before its chunk of experts; a tile is found by a ballot and a
// walk through one chunk. Offsets are taken as non-negative and ascending, and clamped to
// num_rows; where they are not, nothing is computed.
// The blocks take tiles in rounds. Where the last round's tiles are at most half as many as the
// blocks, each is cut along m in two (in four: a quarter), so that the round takes that much
// less: `whole` tiles are not cut, `cut` pieces make one of the others.
constexpr int kBandM = 8;

struct Tile {
    int expert;
    int m0, n0;  // first row (within the expert) or channel of the m side, and of the n side
    int row0;    // the expert's first row
    int rows;    // the expert's rows
    int height;  // valid rows (channels) of the m side in this tile
};

// A block's next four tiles, in the lanes of one register: the loads run up to two tiles ahead of
// the products, and looking a tile up takes more registers than the products leave.
struct TileRing {
    int lanes = 0;
    __device__ __forceinline__ void put(int n, const Tile& t) {
        const int at = (n & 3) * 8;
        const int field[6] = {t.expert, t.m0, t.n0, t.row0, t.rows, t.height};
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const int v = __builtin_amdgcn_readfirstlane(field[i]);
            if (lane_id() == at + i) lanes = v;
        }
    }
    __device__ __forceinline__ Tile get(int n) const {
        const int at = (n & 3) * 8;
        int field[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) field[i] = __builtin_amdgcn_readlane(lanes, at + i);
        return Tile{field[0], field[1], field[2], field[3], field[4], field[5]};
    }
};

struct TileMap {
    const int32_t* offset;
    int64_t num_rows;
    int chunk, E, nt, first;
    int64_t total, whole;  // of all pieces; of the tiles before the last round's
    int cut;
    bool by_rows;  // m tiles cover an expert's rows; else M channels, mt of them per expert
    int M, mt;
    const int* table;  // the clamped offsets in LDS

    __device__ __forceinline__ int tiles(int c) const { return (c + kTileM - 1) / kTileM; }

    __device__ __forceinline__ int start(int e) const {
        return E <= kTableExperts ? table[e]
                                  : static_cast<int>(min<int64_t>(offset[e], num_rows));
    }

    // Ends with a barrier.
    __device__ __forceinline__ void init(const GemmArgs& g, bool rows, int n_tile, int* lds_table) {
        if (g.E <= kTableExperts)
            for (int e = threadIdx.x; e <= g.E; e += kGemmThreads)
                lds_table[e] = static_cast<int>(min<int64_t>(g.offset[e], g.num_rows));
        table = lds_table;
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
        const int blocks = gridDim.x;
        const int rest = static_cast<int>(total % blocks);
        cut = rest * 4 <= blocks ? 4 : rest * 2 <= blocks ? 2 : 1;
        whole = total - rest;
        total = whole + static_cast<int64_t>(rest) * cut;
        if ((bad || over) && blockIdx.x == 0 && threadIdx.x == 0)
            raise_error(g.error_flag, kErrSlotRange);
        lds_barrier();
    }

    __device__ __forceinline__ void place(Tile& t, int in_expert, int mts, int n_tile) const {
        const int bands = (mts + kBandM - 1) / kBandM;
        const int high = (mts + bands - 1) / bands;
        const int band = in_expert / (high * nt);
        const int r = in_expert - band * high * nt;
        const int here = min(high, mts - band * high);
        const int n = r / here;
        t.n0 = n * n_tile;
        t.m0 = band * high + (r - n * here);  // the m tile's number, made a row by the caller
    }

    // The piece's rows (channels): of `height` from t.m0 on its share, in whole subtiles.
    __device__ __forceinline__ void take(Tile& t, int piece, int pieces) const {
        const int each = ((t.height + pieces - 1) / pieces + 15) & ~15;
        t.m0 += piece * each;
        t.height = max(0, min(each, t.height - piece * each));
    }

    __device__ __forceinline__ Tile find(int64_t index, int n_tile) const {
        Tile t;
        int mts, in_expert, piece = 0, pieces = 1;
        if (index >= whole) {
            const int r = static_cast<int>(index - whole);
            index = whole + r / cut;
            piece = r % cut;
            pieces = cut;
        }
        if (by_rows) {
            const uint64_t le =
                wave_ballot(static_cast<int64_t>(first) * nt <= index);
            const int lane = 63 - __builtin_clzll(le);
            int base = __builtin_amdgcn_readlane(first, lane);
            int e = lane * chunk;
            int a = start(e);
            for (;;) {
                const int b = start(e + 1);
                mts = tiles(b - a);
                if (index < static_cast<int64_t>(base + mts) * nt) {
                    t.rows = b - a;
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
            t.row0 = start(t.expert);
            t.rows = start(t.expert + 1) - t.row0;
            place(t, in_expert, mt, n_tile);
            t.m0 *= kTileM;
            t.height = min(kTileM, M - t.m0);
        }
        take(t, piece, pieces);
        return t;
    }
};

// ---------------------------------------------------------------- one operand's loads
// An operand's step is two halves of 16 KB. By rows: 128 bytes of each of 128 rows, row after row
// in LDS, with a row's 16-byte word c at place c ^ (row & 7): eight lanes of a fragment's read,
// on eight rows, then hit eight different places. By columns: 64 rows of k of 128 channels (256
// bytes each), with the 32-byte pair of words p at place p ^ turn(k), so that a transposing
// read's four rows (of each of two groups of lanes) lie in different banks. Of the m side the
// first half holds the subtiles that the first phase of a step reads (32 `split` rows of the
// tile), the second half the rest.
__device__ __forceinline__ int turn(int k) { return (k & 3) | ((k >> 1) & 4); }

template <bool kByRows>
struct OperandLoads {
    uint32_t voff[4];  // of a wave's two loads of the first half, and of the second

    // rows: valid rows of the tile; the second half's first is row `split`
    __device__ __forceinline__ void init_rows(int wave, int lane, int rows, int split,
                                              uint32_t stride) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int r = ((t & 1) * kGemmWaves + wave) * 8 + lane / 8;
            const int row = t < 2 ? r : r + split;
            const bool in = row < rows && (t >= 2 || r < split);
            voff[t] = in ? row * stride + (((lane & 7) ^ (lane >> 3)) * 16) : kOutOfBuffer;
        }
    }
    // columns: valid columns from col0
    __device__ __forceinline__ void init_columns(int wave, int lane, int col0, int columns,
                                                 int split, uint32_t stride) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = ((t & 1) * kGemmWaves + wave) * 4 + lane / 16;
            const int c = ((lane & 15) ^ (2 * turn(k))) * 8;
            const int col = t < 2 ? c : c + split;
            const bool in = col < columns && (t >= 2 || c < split);
            voff[t] = in ? k * stride + (col0 + col) * 2 : kOutOfBuffer;
        }
    }
    // by rows, last step: words past the row's end read zeros
    __device__ __forceinline__ void cut(int lane, int words) {
        if (((lane & 7) ^ (lane >> 3)) >= words) {
#pragma unroll
            for (int t = 0; t < 4; ++t) voff[t] = kOutOfBuffer;
        }
    }
};

// A tile of mt pairs of subtiles is computed in two phases of about equal length.
__device__ __forceinline__ constexpr int first_phase(int mt) { return (mt + 1) / 2; }

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
    static constexpr int kStageBytes = 2 * kOperandBytes;  // the m side, then the n side
    static constexpr int kLoads = 8 + (kFp8 ? 1 : 0);      // per wave and step
    static constexpr int kScalesAt = kStages * kStageBytes;
    static constexpr int kAmaxAt = kScalesAt + (kFp8 ? kScaleSlots * kScaleBytes : 0);
    static constexpr int kTableAt = kAmaxAt + (kGated ? kAmaxBytes : 0);
    static constexpr int kLdsBytes = kTableAt + kTableBytes;
    static_assert(kLdsBytes <= 160 * 1024, "LDS of one CU");
};

// A tile without rows to sum over (an expert's weight gradient) or to compute still takes one step,
// of zeros.
template <GemmOp kOp, bool kFp8>
__device__ __forceinline__ int tile_steps(const GemmArgs& g, const Tile& t) {
    using S = GemmShape<kOp, kFp8>;
    const int k = t.height > 0 ? (S::kOverRows ? t.rows : g.K) : 0;
    return max(1, (k + S::kStepK - 1) / S::kStepK);
}

// The stream of steps that a block loads: its tiles one after the other, the steps of each.
template <GemmOp kOp, bool kFp8>
struct Producer {
    using S = GemmShape<kOp, kFp8>;
    const GemmArgs& g;
    const uint32_t lds;
    int wave, lane;
    int tile, tiles;  // the block's present one, and how many it has
    int step, steps;  // of the tile
    int count;        // of all steps so far
    bool live;
    Tile t;
    OperandLoads<S::kAByRows> a;
    OperandLoads<S::kBByRows> b;
    uint32_t scale_voff;
    const char *a_base = nullptr, *b_base = nullptr, *b_up = nullptr;
    uint32_t a_row, b_row;  // bytes between rows in memory

    __device__ __forceinline__ Producer(const GemmArgs& g_, uint32_t lds_, int tiles_,
                                        const TileRing& ring)
        : g(g_), lds(lds_), wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)),
          lane(lane_id()), tile(0), tiles(tiles_), step(0), steps(0), count(0), live(false), t{} {
        a_row = static_cast<uint32_t>(S::kOverRows ? g.M : g.K) * S::kElem;
        b_row = static_cast<uint32_t>(S::kBByRows ? g.K : g.N) * S::kElem;
        if (tile < tiles) start(ring);
    }

    __device__ __forceinline__ void start(const TileRing& ring) {
        t = ring.get(tile);
        step = 0;
        steps = tile_steps<kOp, kFp8>(g, t);
        const int split = 32 * first_phase((t.height + 31) / 32);
        const char* rows_a = static_cast<const char*>(g.a) + static_cast<int64_t>(t.row0) * a_row;
        if constexpr (S::kAByRows) {
            a_base = rows_a + static_cast<int64_t>(t.m0) * a_row;
            a.init_rows(wave, lane, t.height, split, a_row);
        } else {
            a_base = rows_a;
            a.init_columns(wave, lane, t.m0, t.height, split, a_row);
        }
        const int nv = min(S::kNTile, g.N - t.n0);
        if constexpr (S::kOverRows) {
            b_base = static_cast<const char*>(g.b) + static_cast<int64_t>(t.row0) * b_row;
            b.init_columns(wave, lane, t.n0, nv, kTileN / 2, b_row);
        } else {
            const int64_t weights = static_cast<int64_t>(S::kGated ? 2 : 1) * g.N * g.K * S::kElem;
            b_base = static_cast<const char*>(g.b) + t.expert * weights;
            if constexpr (S::kBByRows) {
                b_base += static_cast<int64_t>(t.n0) * b_row;
                b_up = b_base + static_cast<int64_t>(g.N) * b_row;
                b.init_rows(wave, lane, nv, kTileN / 2, b_row);
                if constexpr (S::kGated) {  // the second half is the up projection's
#pragma unroll
                    for (int i = 2; i < 4; ++i) b.voff[i] = b.voff[i - 2];
                }
            } else {
                b.init_columns(wave, lane, t.n0, nv, kTileN / 2, b_row);
            }
        }
        if constexpr (kFp8) {  // waves 0..3 take 64 rows' scales each
            const int row = wave * kWave + lane;
            scale_voff = row < t.height ? static_cast<uint32_t>(row) * (g.K / 128) * 4u
                                        : kOutOfBuffer;
        }
    }

    // The loads of the m side's half h of the present step.
    __device__ __forceinline__ void issue_a(int h) {
        const uint32_t dst = lds + (count & 1) * S::kStageBytes + h * kHalfBytes + wave * 1024;
        const int k0 = step * S::kStepK;
        i32x4 buf;
        uint32_t along = 0;
        if constexpr (S::kAByRows) {
            buf = scalar_buffer(a_base, live ? static_cast<uint32_t>(t.height) * a_row : 0);
            along = static_cast<uint32_t>(step) * kStepBytes;
        } else {
            const uint32_t n = live ? min(64, t.rows - k0) : 0;
            buf = scalar_buffer(a_base + static_cast<int64_t>(k0) * a_row, n * a_row);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_lds16(buf, dst + i * kGemmWaves * 1024, a.voff[2 * h + i], along);
    }

    // The next step's n side, the first half of its m side and its scales. With no step left the
    // loads go on, of buffers of no bytes, so that the counts of loads in flight hold.
    __device__ __forceinline__ void issue_first(const TileRing& ring) {
        if (step == steps && tile < tiles) {
            ++tile;
            if (tile < tiles) start(ring);
        }
        live = tile < tiles;
        if (!live) step = 0;
        const int k0 = step * S::kStepK;
        if constexpr (S::kAByRows || S::kBByRows) {
            if (live && k0 + S::kStepK > g.K) {  // only at a tile's last step
                const int words = (g.K - k0) * S::kElem / 16;
                if constexpr (S::kAByRows) a.cut(lane, words);
                if constexpr (S::kBByRows) b.cut(lane, words);
            }
        }
        const uint32_t dst =
            lds + (count & 1) * S::kStageBytes + kOperandBytes + wave * 1024;
        if constexpr (S::kBByRows) {
            const uint32_t along = static_cast<uint32_t>(step) * kStepBytes;
            const uint32_t n = live ? static_cast<uint32_t>(min(S::kNTile, g.N - t.n0)) * b_row : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_lds16(scalar_buffer(S::kGated && i >= 2 ? b_up : b_base, n),
                           dst + i * kGemmWaves * 1024, b.voff[i], along);
        } else {
            const uint32_t n = live ? min(64, (S::kOverRows ? t.rows : g.K) - k0) : 0;
            const auto buf = scalar_buffer(b_base + static_cast<int64_t>(k0) * b_row, n * b_row);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_lds16(buf, dst + i * kGemmWaves * 1024, b.voff[i], 0);
        }
        issue_a(0);
        if constexpr (kFp8) {
            const uint32_t row = static_cast<uint32_t>(g.K / 128) * 4u;
            const auto buf = scalar_buffer(g.a_scales + (static_cast<int64_t>(t.row0) + t.m0) * (g.K / 128),
                                           live ? static_cast<uint32_t>(t.height) * row : 0);
            load_lds4(buf, lds + S::kScalesAt + (count & 3) * kScaleBytes + wave * 256, scale_voff,
                      static_cast<uint32_t>(step) * 4u);
        }
    }

    // The second half of the step's m side; on to the next step.
    __device__ __forceinline__ void issue_second() {
        issue_a(1);
        ++count;
        if (live) ++step;
    }
};

// Fragments of one wave: lane l holds row (column) l % 16 of a subtile and the words of k that
// belong to l / 16: words l / 16 and 4 + l / 16 of the step's eight (any order of k will do as
// long as both operands have it).
union Fragment {
    u32x4 word[2];
    bf16x8 bf16[2];
    i32x8 e4m3;
};

struct LanePlace {
    int by_row;  // of the first word in a row subtile
    int by_col;  // of the first 8 bytes in the column subtile of pair 0, turned

    __device__ __forceinline__ explicit LanePlace(int lane) {
        const int row = lane & 15, quad = lane >> 4;
        by_row = row * kStepBytes + ((quad ^ (row & 7)) * 16);
        const int f = (row >> 2) | ((quad & 1) << 2);  // turn(k) of the lane's rows of k
        by_col = (8 * quad + (row >> 2)) * 256 + f * 32 + (row & 3) * 8;
    }
};

// The subtile whose first row (column) within `half` is `first`.
template <bool kByRows>
__device__ __forceinline__ void read_fragment(Fragment& out, const char* half, int first,
                                              const LanePlace& at) {
    if constexpr (kByRows) {
        const char* p = half + first * kStepBytes;
        out.word[0] = *reinterpret_cast<const u32x4*>(p + at.by_row);
        out.word[1] = *reinterpret_cast<const u32x4*>(p + (at.by_row ^ 64));
    } else {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const char* p = half + (at.by_col ^ (first * 2));  // pair first / 16, of 32 bytes
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            union {
                s16x4 h[2];
                u32x4 w;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + s * 32 * 256));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + s * 32 * 256 + 4 * 256));
            out.word[s] = u.w;
        }
    }
}

template <GemmOp kOp, bool kFp8>
__device__ __forceinline__ void read_n_side(Fragment (&b)[4], const char* operand, int wn,
                                            const LanePlace& at) {
    using S = GemmShape<kOp, kFp8>;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (S::kGated)  // gate's channels from the first half, up's from the second
            read_fragment<S::kBByRows>(b[j], operand + (j >> 1) * kHalfBytes, wn * 32 + (j & 1) * 16,
                                       at);
        else
            read_fragment<S::kBByRows>(b[j], operand + (wn >> 1) * kHalfBytes,
                                       (wn & 1) * 64 + j * 16, at);
    }
}

template <bool kFp8, bool kGated>
__device__ __forceinline__ void multiply(f32x4 (&acc)[4], const Fragment (&b)[4], const Fragment& a,
                                         float as, const float (&bs)[2]) {
    if constexpr (!kFp8) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j].bf16[s], a.bf16[s], acc[j], 0,
                                                                 0, 0);
    } else {
        const float sc[2] = {as * bs[0], as * bs[1]};
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            d[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j].e4m3, a.e4m3, zero, 0, 0, 0,
                                                                    0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[j][r] = fmaf(d[j][r], sc[kGated ? j >> 1 : 0], acc[j][r]);
        // the sums are made here: moved behind the wait that follows, they keep every product
        // of the phase in registers, which then spill
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[j]));
    }
}

// Two subtiles' sums of one row as eight consecutive channels per lane: lanes 0..31 take the
// first subtile's 16 channels, lanes 32..63 the second's.
__device__ __forceinline__ void eight_channels(const f32x4& a, const f32x4& b, float (&v)[8]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        // rows of 16 lanes: a = {a0 a1 b0 b1}, b = {a2 a3 b2 b3}, then {a0 a2 b0 b2}, {a1 a3 b1 b3}
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[r]),
                                                        __float_as_uint(b[r]), false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
        v[r] = __uint_as_float(y[0]);
        v[4 + r] = __uint_as_float(y[1]);
    }
}

__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t buf, uint32_t at, u32x4 w) {
    __builtin_amdgcn_raw_buffer_store_b128(w, buf, at, 0, 0);
}

__device__ __forceinline__ u32x2 e4m3_eight(const float (&v)[8], float inv) {
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lo =
            __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
        w[h] = static_cast<uint32_t>(
            __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, lo, true));
    }
    return w;
}

__device__ __forceinline__ void values_eight(u32x2 w, float scale, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = static_cast<int>(w[h]);
        v[4 * h] = __builtin_amdgcn_cvt_f32_fp8(c, 0) * scale;
        v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(c, 1) * scale;
        v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(c, 2) * scale;
        v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(c, 3) * scale;
    }
}

__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

constexpr float kE4m3Largest = 448.0f;
constexpr float kSmallestAmax = 0x1p-100f;

// What a group whose largest magnitude is a is scaled to 448 by.
__device__ __forceinline__ float group_amax(float a) {
    return a > 0.0f ? fmaxf(a, kSmallestAmax) : kE4m3Largest;
}

// What a tile's sums become in memory. Lane: row (2 i + wm) 16 + l % 16 of the tile, eight
// channels of each pair of subtiles. The tile's rows of an array are a buffer, so that rows past
// its height are dropped (or read as zeros) without a branch, and every tile of mt pairs of
// subtiles makes the same number of stores.
template <GemmOp kOp, bool kFp8, int kMT>
__device__ __forceinline__ void gemm_store(const GemmArgs& g, const Tile& t, f32x4 (&acc)[8][4],
                                           char* lds_amax, int wm, int wn, int lane) {
    const int quad = lane >> 4;
    const int64_t first_row = static_cast<int64_t>(t.row0) + t.m0;
    const uint32_t height = t.height;
    // the tile's rows of an array of `bytes` per row; none of it where the array is missing
    auto rows_of = [&](const void* base, uint32_t bytes) {
        const char* p = static_cast<const char*>(base) + (base ? first_row * bytes : 0);
        return raw_buffer(p, base ? height * bytes : 0);
    };
    const int in_pair = (quad >> 1) * 16 + (quad & 1) * 8;
    if constexpr (kOp == GemmOp::kGateUp) {
        const int I = g.N;
        float(*amax)[2][4] = reinterpret_cast<float(*)[2][4]>(lds_amax);
        const bool quantise = g.codes != nullptr;
        if constexpr (kFp8) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float gate = acc[i][j][r];
                        acc[i][j][r] = gate * sigmoid(gate) * acc[i][j + 2][r];
                    }
        }
        if (quantise) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int h = 0; h < (kFp8 ? 1 : 2); ++h) {
                    float top = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        top = fmaxf(top, fmaxf(fabsf(acc[i][2 * h][r]), fabsf(acc[i][2 * h + 1][r])));
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    if (quad == 0) amax[(2 * i + wm) * 16 + (lane & 15)][h][wn] = top;
                }
            lds_barrier();
        }
        const int c = t.n0 + wn * 32 + in_pair;
        const bool in = c < I;
        const auto act_rows = rows_of(g.out, I * 2u);
        const auto kept_rows = rows_of(g.gate_up, I * 4u);
        const auto code_rows = rows_of(g.codes, I * (kFp8 ? 1u : 2u));
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
            float gate[8], up[8];
            eight_channels(acc[i][0], acc[i][1], gate);
            if constexpr (!kFp8) eight_channels(acc[i][2], acc[i][3], up);
            if (quantise) {
                float inv[2];
#pragma unroll
                for (int h = 0; h < (kFp8 ? 1 : 2); ++h) {
                    const float* p = amax[m][h];
                    const float top = group_amax(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])));
                    inv[h] = kE4m3Largest / top;
                    if (wn == 0 && quad == 0 && m < height)
                        g.scales[(first_row + m) * (I / (kFp8 ? 128 : 64)) + h * (I / 128) +
                                 t.n0 / 128] = top / kE4m3Largest;
                }
                const uint32_t at = in ? m * (I * (kFp8 ? 1u : 2u)) + c : kOutOfBuffer;
                __builtin_amdgcn_raw_buffer_store_b64(e4m3_eight(gate, inv[0]), code_rows, at, 0, 0);
                if constexpr (!kFp8)
                    __builtin_amdgcn_raw_buffer_store_b64(e4m3_eight(up, inv[1]), code_rows, at, I, 0);
            }
            if constexpr (!kFp8) {
                if (g.gate_up) {
                    const uint32_t at = in ? m * (I * 4u) + c * 2u : kOutOfBuffer;
                    store16(kept_rows, at, narrow8(gate));
                    store16(kept_rows, in ? at + I * 2u : at, narrow8(up));
                }
#pragma unroll
                for (int r = 0; r < 8; ++r) gate[r] = gate[r] * sigmoid(gate[r]) * up[r];
                store16(act_rows, in ? m * (I * 2u) + c * 2u : kOutOfBuffer, narrow8(gate));
            }
        }
    } else if constexpr (kOp == GemmOp::kWeightGrad) {
        const uint32_t row_bytes = g.N * (g.out_fp32 ? 4u : 2u);
        const int64_t first = static_cast<int64_t>(t.expert) * g.M + t.m0;
        const auto rows = raw_buffer(static_cast<char*>(g.out) + first * row_bytes, height * row_bytes);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t c = t.n0 + wn * 64 + p * 32 + in_pair;
                const bool in = c < static_cast<uint32_t>(g.N);
                float v[8];
                eight_channels(acc[i][2 * p], acc[i][2 * p + 1], v);
                if (g.out_fp32) {
                    const uint32_t at = in ? m * row_bytes + c * 4u : kOutOfBuffer;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x4 w = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
                        const uint32_t to = in ? at + 16 * h : at;
                        if (g.accumulate)
                            w += __builtin_bit_cast(
                                f32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, to, 0, 0));
                        store16(rows, to, __builtin_bit_cast(u32x4, w));
                    }
                } else {
                    const uint32_t at = in ? m * row_bytes + c * 2u : kOutOfBuffer;
                    if (g.accumulate) {
                        float w[8];
                        widen8(__builtin_bit_cast(
                                   u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, at, 0, 0)),
                               w);
#pragma unroll
                        for (int r = 0; r < 8; ++r) v[r] += w[r];
                    }
                    store16(rows, at, narrow8(v));
                }
            }
        }
    } else if constexpr (kOp == GemmOp::kDownGrad) {
        const int I = g.N;
        const auto kept = rows_of(g.gate_up, I * 4u);
        const auto codes = rows_of(g.codes, I * 2u);
        const auto scales = rows_of(g.scales, (I / 64) * 4u);
        const auto grad = rows_of(g.out, I * 4u);
        const auto act = rows_of(g.act, I * 2u);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t c = t.n0 + wn * 64 + p * 32 + in_pair;
                const bool in = c < static_cast<uint32_t>(I);
                const uint32_t at = in ? m * (I * 4u) + c * 2u : kOutOfBuffer;
                float da[8], gate[8], up[8];
                eight_channels(acc[i][2 * p], acc[i][2 * p + 1], da);
                if (g.gate_up) {
                    widen8(__builtin_bit_cast(
                               u32x4, __builtin_amdgcn_raw_buffer_load_b128(kept, at, 0, 0)),
                           gate);
                    widen8(__builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         kept, in ? at + I * 2u : at, 0, 0)),
                           up);
                } else {
                    const uint32_t from = in ? m * (I * 2u) + c : kOutOfBuffer;
                    const uint32_t sc = in ? m * ((I / 64) * 4u) + c / 128 * 4u : kOutOfBuffer;
                    const u32x2 a = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_raw_buffer_load_b64(codes, from, 0, 0));
                    const u32x2 b = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_raw_buffer_load_b64(codes, in ? from + I : from, 0, 0));
                    const float sg =
                        __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(scales, sc, 0, 0));
                    const float su = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                        scales, in ? sc + I / 128 * 4u : sc, 0, 0));
                    values_eight(a, sg, gate);
                    values_eight(b, su, up);
                }
                float dg[8], du[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float s = sigmoid(gate[r]);
                    const float silu = gate[r] * s;
                    du[r] = da[r] * silu;
                    dg[r] = da[r] * up[r] * s * (1.0f + gate[r] * (1.0f - s));
                    up[r] *= silu;
                }
                store16(grad, at, narrow8(dg));
                store16(grad, in ? at + I * 2u : at, narrow8(du));
                if (g.act) store16(act, in ? m * (I * 2u) + c * 2u : kOutOfBuffer, narrow8(up));
            }
        }
    } else {
        const auto rows = rows_of(g.out, g.N * 2u);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t c = t.n0 + wn * 64 + p * 32 + in_pair;
                float v[8];
                eight_channels(acc[i][2 * p], acc[i][2 * p + 1], v);
                store16(rows,
                        c < static_cast<uint32_t>(g.N) ? m * (g.N * 2u) + c * 2u : kOutOfBuffer,
                        narrow8(v));
            }
        }
    }
}

// How many stores gemm_store is sure to make after its last load.
template <GemmOp kOp, bool kFp8>
__device__ __forceinline__ int stores_after(const GemmArgs& g, int mt) {
    if constexpr (kOp == GemmOp::kGateUp)
        return mt * (kFp8 ? 1 : 1 + (g.gate_up ? 2 : 0) + (g.codes ? 2 : 0));
    else if constexpr (kOp == GemmOp::kWeightGrad)
        return g.accumulate ? 0 : mt * (g.out_fp32 ? 4 : 2);
    else if constexpr (kOp == GemmOp::kDownGrad)
        return 0;
    else
        return mt * 2;
}

// All but the last kOutstanding loads have arrived, where at least `stores` stores were made
// after the loads that are waited for.
template <int kOutstanding>
__device__ __forceinline__ void wait_loads_before(int stores) {
    if (stores >= 32)
        wait_loads<kOutstanding + 32>();
    else if (stores >= 16)
        wait_loads<kOutstanding + 16>();
    else if (stores >= 8)
        wait_loads<kOutstanding + 8>();
    else
        wait_loads<kOutstanding>();
}

// Ends a slot: this wave's LDS reads are in registers, and every wave gets here.
__device__ __forceinline__ void end_slot() {
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// One tile's steps with kMT subtiles of 16 rows per wave. The block's two halves (waves 0..3 and
// 4..7, one of each on every SIMD) take turns: while one multiplies, the other reads its next
// fragments from LDS and issues loads, and a barrier ends each such slot. A step is four slots:
//   waves 0..3   read 1   multiply 1   read 2       multiply 2
//   waves 4..7   -        read 1       multiply 1   read 2       multiply 2
// where reading 1 takes the n side and the first half of the m side and issues the second half
// of the next step's m side; reading 2 takes the second half and issues the rest of the step
// after the next into the places that reading 1 has left. Every load has six slots to arrive: of
// a wave's loads all but the last kLoads have to be there at the end of every odd slot.
template <GemmOp kOp, bool kFp8, int kMT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, const Tile& t, int steps,
                                          Producer<kOp, kFp8>& p, f32x4 (&acc)[8][4],
                                          char* lds, int& count, int& stores,
                                          const TileRing& ring, int wm, int wn,
                                          const LanePlace& at, int lane) {
    using S = GemmShape<kOp, kFp8>;
    constexpr int kP = first_phase(kMT);
    const float* bs_row = nullptr;
    int64_t up_scales = 0;
    float bs[2] = {1.0f, 1.0f};
    if constexpr (kFp8) {
        const int KB = g.K / 128;
        const int nb = S::kGated ? t.n0 / 128 : min((t.n0 + wn * 64) / 128, g.N / 128 - 1);
        bs_row = g.b_scales +
                 (static_cast<int64_t>(t.expert) * (S::kGated ? 2 : 1) * (g.N / 128) + nb) * KB;
        up_scales = static_cast<int64_t>(g.N / 128) * KB;
    }
    if (wm) end_slot();
    for (int step = 0; step < steps; ++step, ++count) {
        const char* stage = lds + (count & 1) * S::kStageBytes;
        const char* scales = lds + S::kScalesAt + (count & 3) * kScaleBytes;
        Fragment b[4], a[kP];
        float as[kP];
        read_n_side<kOp, kFp8>(b, stage + kOperandBytes, wn, at);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            read_fragment<S::kAByRows>(a[i], stage, (2 * i + wm) * 16, at);
            if constexpr (kFp8)
                as[i] = *reinterpret_cast<const float*>(scales + ((2 * i + wm) * 16 + (lane & 15)) * 4);
        }
        if constexpr (kFp8) {
            bs[0] = bs_row[step];
            if constexpr (S::kGated) bs[1] = bs_row[up_scales + step];
        }
        p.issue_second();
        if (wm) wait_loads_before<S::kLoads>(stores);
        end_slot();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < kP; ++i) multiply<kFp8, S::kGated>(acc[i], b, a[i], as[i], bs);
        __builtin_amdgcn_s_setprio(0);
        if (!wm) wait_loads_before<S::kLoads>(stores);
        end_slot();
#pragma unroll
        for (int i = kP; i < kMT; ++i) {
            read_fragment<S::kAByRows>(a[i - kP], stage + kHalfBytes, (2 * (i - kP) + wm) * 16, at);
            if constexpr (kFp8)
                as[i - kP] =
                    *reinterpret_cast<const float*>(scales + ((2 * i + wm) * 16 + (lane & 15)) * 4);
        }
        p.issue_first(ring);
        if (wm) wait_loads_before<S::kLoads>(stores);
        end_slot();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = kP; i < kMT; ++i)
            multiply<kFp8, S::kGated>(acc[i], b, a[i - kP], as[i - kP], bs);
        __builtin_amdgcn_s_setprio(0);
        if (!wm) wait_loads_before<S::kLoads>(stores);
        stores = 0;
        end_slot();
    }
    if (!wm) end_slot();
    gemm_store<kOp, kFp8, kMT>(g, t, acc, lds + S::kAmaxAt, wm, wn, lane);
    stores = stores_after<kOp, kFp8>(g, kMT);
}

template <GemmOp kOp, bool kFp8>
__global__ __launch_bounds__(kGemmThreads, 1) void gemm_kernel(const GemmArgs g) {
    using S = GemmShape<kOp, kFp8>;
    __shared__ __attribute__((aligned(1024))) char lds[S::kLdsBytes];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;
    const LanePlace at(lane);
    TileMap map;
    map.init(g, !S::kOverRows, S::kNTile, reinterpret_cast<int*>(lds + S::kTableAt));
    // block b runs on die b % 8: its tiles are neighbours of that die's other blocks' tiles
    const int per_die = gridDim.x / 8;
    const int64_t first = gridDim.x % 8 == 0
                              ? static_cast<int64_t>(blockIdx.x % 8) * per_die + blockIdx.x / 8
                              : blockIdx.x;
    const int tiles =
        first < map.total ? static_cast<int>((map.total - first + gridDim.x - 1) / gridDim.x) : 0;
    TileRing ring;
    auto look_up = [&](int n) {
        if (n < tiles) ring.put(n, map.find(first + static_cast<int64_t>(n) * gridDim.x, S::kNTile));
    };
    look_up(0);
    look_up(1);
    look_up(2);
    Producer<kOp, kFp8> p(g, lds_address(lds), tiles, ring);
    int count = 0, stores = 0;
    p.issue_first(ring);
    p.issue_second();
    p.issue_first(ring);
    wait_loads<S::kLoads>();
    end_slot();
    for (int n = 0; n < tiles; ++n) {
        look_up(n + 3);
        const Tile t = ring.get(n);
        const int steps = tile_steps<kOp, kFp8>(g, t);
        f32x4 acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int mt = (t.height + 31) / 32;
        switch (max(mt, 1)) {  // a piece of a low tile may have got no row
#define EP_GEMM_CASE(n)                                                                   \
    case n:                                                                               \
        gemm_tile<kOp, kFp8, n>(g, t, steps, p, acc, lds, count, stores, ring, wm, wn, at, lane); \
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
    }
    wait_loads<0>();  // no load outlives the block
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
