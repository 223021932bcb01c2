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
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlocks = 256;        // one per CU; a power of two
constexpr int kStepBytes = 128;     // bytes of k per row and step: 64 bf16 or 128 e4m3
constexpr int kScaleSlots = 4;      // steps whose row scales are in LDS
// With at most so many experts, their offsets are kept in LDS; with more, a tile is looked up in memory
// (128 rows of each of 1024 / 1032 experts of 1024 x 512 weights: gate_up 558 / 579 us, e4m3 down 195 /
// 219, weight's gradient 1172 / 1286).
constexpr int kTableExperts = 1024;
constexpr int kRingBytes = 8 * 32;   // the next eight tiles
constexpr int kTableBytes = (kTableExperts + 32) * 4 + kRingBytes;
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
// registers. m0 is set in the same block as it is used. The compiler does not see the load either:
// a scalar that the vector unit wrote (v_readfirstlane) may be read by it after five wait states,
// which the block's first two instructions are.
__device__ __forceinline__ void load_lds16(i32x4 buf, uint32_t lds,
                                           uint32_t voff, uint32_t soff) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    soff = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(i32x4 buf, uint32_t lds, uint32_t voff,
                                          uint32_t soff) {
    lds = __builtin_amdgcn_readfirstlane(lds);
    soff = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(buf), "s"(soff)
                 : "memory", "m0");
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
// An expert of c rows has ceil(c / tile_m) tiles along m of about equal heights. Every lane
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

// A block's next eight tiles, in the lanes of one register: the loads run up to kStages steps, of
// as many tiles, ahead of the products, and looking a tile up takes more registers than the
// products leave.
struct TileRing {
    int lanes = 0;
    __device__ __forceinline__ void put(int n, const Tile& t) {
        const int at = (n & 7) * 8;
        const int field[6] = {t.expert, t.m0, t.n0, t.row0, t.rows, t.height};
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const int v = __builtin_amdgcn_readfirstlane(field[i]);
            if (lane_id() == at + i) lanes = v;
        }
    }
    __device__ __forceinline__ Tile get(int n) const {
        const int at = (n & 7) * 8;
        int field[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) field[i] = __builtin_amdgcn_readlane(lanes, at + i);
        return Tile{field[0], field[1], field[2], field[3], field[4], field[5]};
    }
};

// The number of expert e's first piece where its rows begin at `offset`: at least as many
// numbers lie between two experts' as the first one's rows have pieces.
__device__ __forceinline__ int first_piece(int offset, int e, int piece_rows) {
    return offset / piece_rows + e;
}

struct TileMap {
    const int32_t* offset;
    int64_t num_rows;
    int chunk, E, nt, first;
    int64_t total, whole;  // of all pieces; of the tiles before the last round's
    int cut;
    bool by_rows;  // m tiles cover an expert's rows; else M channels, mt of them per expert
    int M, mt;
    const int* table;  // the clamped offsets in LDS

    int tile_m;

    // unsigned: c may be as large as INT32_MAX
    __device__ __forceinline__ int tiles(int c) const {
        return static_cast<int>((static_cast<uint32_t>(c) + tile_m - 1) / tile_m);
    }

    __device__ __forceinline__ int start(int e) const {
        return E <= kTableExperts ? table[e]
                                  : static_cast<int>(min<int64_t>(offset[e], num_rows));
    }

    // Pieces of experts in the experts' place: of expert e those from number first_piece() on,
    // its rows cut every piece_rows, and empty ones up to the next expert's first. The offsets
    // are sound: number `pieces` - 1 is the largest.
    __device__ __forceinline__ void piece_offsets(const GemmArgs& g, int* lds_table) const {
        for (int e = threadIdx.x; e <= g.E; e += static_cast<int>(blockDim.x)) {
            const int a = static_cast<int>(min<int64_t>(g.offset[e], g.num_rows));
            const int b = e < g.E ? static_cast<int>(min<int64_t>(g.offset[e + 1], g.num_rows)) : a;
            const int from = first_piece(a, e, g.piece_rows);
            const int to = e < g.E ? first_piece(b, e + 1, g.piece_rows) : g.pieces + 1;
            for (int s = e > 0 ? from : 0; s < to; ++s)
                lds_table[s] = s < from ? a
                                        : static_cast<int>(min<int64_t>(
                                              a + static_cast<int64_t>(s - from) * g.piece_rows, b));
        }
    }

    // Every wave has to come here.
    __device__ __forceinline__ void init(const GemmArgs& g, bool rows, int m_tile, int n_tile,
                                         int* lds_table) {
        tile_m = m_tile;
        // one read of the offsets per block: the lanes' chunks are summed from LDS
        int bad_pair = 0, past = 0;
        for (int e = threadIdx.x; e <= g.E; e += static_cast<int>(blockDim.x)) {
            const int here = g.offset[e];
            const int before = e > 0 ? g.offset[e - 1] : 0;
            bad_pair |= here < before;
            past |= here > g.num_rows;
            if (g.E <= kTableExperts)
                lds_table[e] = static_cast<int>(min<int64_t>(here, g.num_rows));
        }
        if (threadIdx.x < 2) lds_table[kTableExperts + 2 + threadIdx.x] = 0;
        lds_barrier();
        if (bad_pair) lds_table[kTableExperts + 2] = 1;
        if (past) lds_table[kTableExperts + 3] = 1;
        lds_barrier();
        const bool bad = lds_table[kTableExperts + 2] != 0, over = lds_table[kTableExperts + 3] != 0;
        table = lds_table;
        offset = g.offset;
        num_rows = g.num_rows;
        E = g.E;
        if (!rows && g.piece_rows > 0) {
            E = g.pieces;
            if (!bad) piece_offsets(g, lds_table);
            lds_barrier();
        }
        by_rows = rows;
        M = g.M;
        nt = (g.N + n_tile - 1) / n_tile;
        chunk = (E + kWave - 1) / kWave;
        const int lane = lane_id();
        const int e0 = min(lane * chunk, E), e1 = min(e0 + chunk, E);
        int count = 0;
        if (!bad)
            for (int e = e0, prev = start(e0); e < e1; ++e) {
                const int next = start(e + 1);
                count += tiles(next - prev);
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
        if (bad) total = 0;
        // a grid of fewer blocks than CUs has one for every tile
        const int blocks = gridDim.x;
        const int rest = static_cast<int>(blocks == kBlocks ? total & (kBlocks - 1)
                                          : total < blocks  ? total
                                                            : 0);
        cut = rest * 4 <= blocks ? 4 : rest * 2 <= blocks ? 2 : 1;
        whole = total - rest;
        total = whole + static_cast<int64_t>(rest) * cut;
        if ((bad || over) && blockIdx.x == 0 && threadIdx.x == 0)
            raise_error(g.error_flag, kErrSlotRange);
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
            const int each =
                static_cast<int>((static_cast<uint32_t>(t.rows) + mts - 1) / mts + 15) & ~15;
            t.m0 *= each;
            t.height = min(each, t.rows - t.m0);
        } else {
            const int per = mt * nt;
            t.expert = index <= INT32_MAX ? static_cast<int>(index) / per
                                          : static_cast<int>(index / per);
            in_expert = static_cast<int>(index - static_cast<int64_t>(t.expert) * per);
            t.row0 = start(t.expert);
            t.rows = start(t.expert + 1) - t.row0;
            place(t, in_expert, mt, n_tile);
            t.m0 *= tile_m;
            t.height = min(tile_m, M - t.m0);
        }
        take(t, piece, pieces);
        return t;
    }
};

// ---------------------------------------------------------------- the kernels' shapes
// Tiles of 256 x 256 for many rows per expert: the matrix cores are what is short, and two steps
// in LDS are what fits beside them (gemm_kernel). Lower ones for fewer rows, where the time is
// that of the weights' way from memory: as many steps as fit are in LDS, and waves of their own
// do nothing but load (stream_kernel). A wave multiplies 64 channels with every second subtile of
// 16 rows.
template <GemmOp kOp_, bool kFp8_, int kTileM_, int kTileN_ = 256>
struct GemmShape {
    static constexpr GemmOp kOp = kOp_;
    static constexpr bool kFp8 = kFp8_;
    static constexpr int kTileM = kTileM_, kTileN = kTileN_;
    static constexpr bool kGated = kOp == GemmOp::kGateUp;
    static constexpr bool kAByRows = kOp != GemmOp::kWeightGrad;
    static constexpr bool kBByRows = kOp == GemmOp::kGateUp || kOp == GemmOp::kDown;
    static constexpr bool kOverRows = kOp == GemmOp::kWeightGrad;  // k runs over the rows
    static constexpr bool kWidened = kFp8 && kGated;               // multiplied as bf16
    static constexpr int kNTile = kGated ? kTileN / 2 : kTileN;    // output channels of a tile
    static constexpr int kElem = kFp8 ? 1 : 2;
    static constexpr int kStepK = kStepBytes / kElem;
    static constexpr int kMT = kTileM / 32;  // pairs of subtiles along m
    static constexpr int kNWaves = kTileN / 64;
    static constexpr int kWaves = 2 * kNWaves;              // waves that multiply
    static constexpr int kLoaders = kTileM == 256 ? 0 : 4;  // waves that load
    static constexpr int kThreads = (kWaves + kLoaders) * kWave;
    static constexpr int kMBytes = kTileM * kStepBytes;
    static constexpr int kStageBytes = kMBytes + kTileN * kStepBytes;  // the m side, the n side
    static constexpr int kScaleBytes = (kTileM < 64 ? 64 : kTileM) * 4;
    static constexpr int kAmaxBytes = kTileM * 2 * 4 * 4;  // [row][gate, up][wave along n]
    static constexpr int kBesides = (kFp8 ? kScaleSlots * kScaleBytes : 0) +
                                    (kGated ? kAmaxBytes : 0) + kTableBytes;
    static constexpr int kFit = (160 * 1024 - kBesides) / kStageBytes;
    static constexpr int kMost = kFp8 ? kScaleSlots : 8;  // the scales' places, the tile ring's
    static constexpr int kStages = kFit < kMost ? kFit : kMost;
    static constexpr int kScalesAt = kStages * kStageBytes;
    static constexpr int kAmaxAt = kScalesAt + (kFp8 ? kScaleSlots * kScaleBytes : 0);
    static constexpr int kTableAt = kAmaxAt + (kGated ? kAmaxBytes : 0);
    static constexpr int kLdsBytes = kTableAt + kTableBytes;
    static_assert(kLdsBytes <= 160 * 1024, "LDS of one CU");
    static_assert(kStages >= 2, "one step arrives while another is multiplied");
    static_assert(kAByRows || kTileM >= 128, "an m side by columns has halves of 128");
    static_assert(kBByRows || kTileN >= 128, "an n side by columns has halves of 128");
    static_assert(kTileM < 256 || (kStages == 2 && kTileN == 256 && !kFp8), "gemm_kernel");
};

// ---------------------------------------------------------------- one operand's loads
// By rows: 128 bytes of each row of a step, row after row in LDS, with a row's 16-byte word c at
// place c ^ (row & 7): eight lanes of a fragment's read, on eight rows, then hit eight different
// places. By columns: halves of 64 rows of k of 128 channels (256 bytes each), with the 32-byte
// pair of words p at place p ^ turn(k), so that a transposing read's four rows (of each of two
// groups of lanes) lie in different banks. Of the m side the first half holds the subtiles that
// the first phase of a step reads (32 `split` rows of the tile), the second half the rest.
__device__ __forceinline__ int turn(int k) { return (k & 3) | ((k >> 1) & 4); }

// A load of a wave is one unit of 1 KB: eight rows, or four rows of k of 128 columns. kUnits of them
// are shared by kWaves waves.
template <bool kByRows, int kUnits, int kWaves>
struct OperandLoads {
    static constexpr int kLoads = kUnits / kWaves;  // per wave
    static_assert(kUnits % kWaves == 0, "the same number for every wave");
    uint32_t voff[kLoads];

    __device__ __forceinline__ static int unit(int t, int wave) { return t * kWaves + wave; }

    // rows: valid rows of the tile, of which the first `split` are in the first 128 rows of LDS
    // and the others behind them
    __device__ __forceinline__ void init_rows(int wave, int lane, int rows, int split,
                                              uint32_t stride) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            const int r = unit(t, wave) * 8 + lane / 8;
            const bool second = r >= 128;
            const int row = second ? r - 128 + split : r;
            const bool in = row < rows && (second || r < split);
            voff[t] = in ? row * stride + (((lane & 7) ^ (lane >> 3)) * 16) : kOutOfBuffer;
        }
    }
    // columns: valid columns from col0, split alike
    __device__ __forceinline__ void init_columns(int wave, int lane, int col0, int columns,
                                                 int split, uint32_t stride) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            const bool second = unit(t, wave) >= 16;
            const int k = (unit(t, wave) & 15) * 4 + lane / 16;
            const int c = ((lane & 15) ^ (2 * turn(k))) * 8;
            const int col = second ? c + split : c;
            const bool in = col < columns && (second || c < split);
            voff[t] = in ? k * stride + (col0 + col) * 2 : kOutOfBuffer;
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

// How many of a tile's mt pairs of subtiles the first phase of a step takes.
__device__ __forceinline__ constexpr int first_phase(int mt) { return (mt + 1) / 2; }

// A tile without rows to sum over (an expert's weight gradient) or to compute still takes one step,
// of zeros.
template <class S>
__device__ __forceinline__ int tile_steps(const GemmArgs& g, const Tile& t) {
    const uint32_t k = t.height > 0 ? (S::kOverRows ? t.rows : g.K) : 0;
    return max(1, static_cast<int>((k + S::kStepK - 1) / S::kStepK));
}

// The stream of steps that a block loads: its tiles one after the other, the steps of each, by
// kWaves waves.
template <class S, int kWaves>
struct Producer {
    using ALoads = OperandLoads<S::kAByRows, S::kTileM / 8, kWaves>;
    using BLoads = OperandLoads<S::kBByRows, S::kTileN / 8, kWaves>;
    static constexpr int kLoads = ALoads::kLoads + BLoads::kLoads + (S::kFp8 ? 1 : 0);
    static constexpr bool kTwoParts = S::kLoaders == 0;  // the m side is read in two halves

    const GemmArgs& g;
    const uint32_t lds;
    int wave, lane;
    int tile, tiles;  // the block's present one, and how many it has
    int step, steps;  // of the tile
    int slot;         // the step's place in LDS
    int scale_slot;   // its scales'
    bool live;
    Tile t;
    ALoads a;
    BLoads b;
    uint32_t scale_voff;
    const char *a_base = nullptr, *b_base = nullptr, *b_up = nullptr;
    uint32_t a_row, b_row;  // bytes between rows in memory

    __device__ __forceinline__ Producer(const GemmArgs& g_, uint32_t lds_, int wave_, int tiles_,
                                        const TileRing& ring)
        : g(g_), lds(lds_), wave(wave_), lane(lane_id()), tile(0), tiles(tiles_), step(0), steps(0),
          slot(0), scale_slot(0), live(false), t{} {
        a_row = static_cast<uint32_t>(S::kOverRows ? g.M : g.K) * S::kElem;
        b_row = static_cast<uint32_t>(S::kBByRows ? g.K : g.N) * S::kElem;
        if (tile < tiles) start(ring);
    }

    __device__ __forceinline__ void start(const TileRing& ring) {
        t = ring.get(tile);
        step = 0;
        steps = tile_steps<S>(g, t);
        const int split = kTwoParts ? 32 * first_phase((t.height + 31) / 32) : 128;
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
            b.init_columns(wave, lane, t.n0, nv, 128, b_row);
        } else {
            const int64_t weights = static_cast<int64_t>(S::kGated ? 2 : 1) * g.N * g.K * S::kElem;
            b_base = static_cast<const char*>(g.b) + t.expert * weights;
            if constexpr (S::kBByRows) {
                b_base += static_cast<int64_t>(t.n0) * b_row;
                b_up = b_base + static_cast<int64_t>(g.N) * b_row;
                b.init_rows(wave, lane, nv, 128, b_row);
                if constexpr (S::kGated) {  // the second half is the up projection's
                    constexpr int kHalf = BLoads::kLoads / 2;
#pragma unroll
                    for (int i = kHalf; i < 2 * kHalf; ++i) b.voff[i] = b.voff[i - kHalf];
                }
            } else {
                b.init_columns(wave, lane, t.n0, nv, 128, b_row);
            }
        }
        if constexpr (S::kFp8) {  // a wave takes 64 rows' scales, some waves the same ones
            const int row = wave % (S::kScaleBytes / 256) * kWave + lane;
            scale_voff = row < t.height ? static_cast<uint32_t>(row) * (g.K / 128) * 4u
                                        : kOutOfBuffer;
        }
    }

    // The m side's loads from..to - 1 of the present step.
    __device__ __forceinline__ void load_m(int from, int to) {
        const uint32_t dst = lds + slot * S::kStageBytes;
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
        for (int i = 0; i < ALoads::kLoads; ++i)
            if (i >= from && i < to)
                load_lds16(buf, dst + a.unit(i, wave) * 1024, a.voff[i], along);
    }

    // The next step's n side, the first half of its m side (all of it, where it is loaded in one
    // part) and its scales. With no step left the loads go on, of buffers of no bytes, so that
    // the counts of loads in flight hold.
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
        const uint32_t dst = lds + slot * S::kStageBytes + S::kMBytes;
        if constexpr (S::kBByRows) {
            const uint32_t along = static_cast<uint32_t>(step) * kStepBytes;
            const uint32_t n = live ? static_cast<uint32_t>(min(S::kNTile, g.N - t.n0)) * b_row : 0;
#pragma unroll
            for (int i = 0; i < BLoads::kLoads; ++i)
                load_lds16(scalar_buffer(S::kGated && i >= BLoads::kLoads / 2 ? b_up : b_base, n),
                           dst + b.unit(i, wave) * 1024, b.voff[i], along);
        } else {
            const uint32_t n = live ? min(64, (S::kOverRows ? t.rows : g.K) - k0) : 0;
            const auto buf = scalar_buffer(b_base + static_cast<int64_t>(k0) * b_row, n * b_row);
#pragma unroll
            for (int i = 0; i < BLoads::kLoads; ++i)
                load_lds16(buf, dst + b.unit(i, wave) * 1024, b.voff[i], 0);
        }
        load_m(0, kTwoParts ? ALoads::kLoads / 2 : ALoads::kLoads);
        if constexpr (S::kFp8) {
            const uint32_t row = static_cast<uint32_t>(g.K / 128) * 4u;
            const auto buf =
                scalar_buffer(g.a_scales + (static_cast<int64_t>(t.row0) + t.m0) * (g.K / 128),
                              live ? static_cast<uint32_t>(t.height) * row : 0);
            load_lds4(buf,
                      lds + S::kScalesAt + scale_slot * S::kScaleBytes +
                          wave % (S::kScaleBytes / 256) * 256,
                      scale_voff, static_cast<uint32_t>(step) * 4u);
        }
        if constexpr (!kTwoParts) next();
    }

    // The second half of the step's m side; on to the next step.
    __device__ __forceinline__ void issue_second() {
        load_m(ALoads::kLoads / 2, ALoads::kLoads);
        next();
    }

    __device__ __forceinline__ void next() {
        if constexpr (S::kStages == 2)
            slot ^= 1;
        else
            slot = slot + 1 == S::kStages ? 0 : slot + 1;
        scale_slot = (scale_slot + 1) & (kScaleSlots - 1);
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

// The first tile row of a wave's subtile j of the n side: with two projections the gate's
// channels come from the first half, the up projection's from the second.
template <class S>
__device__ __forceinline__ int n_first(int j, int wn) {
    return S::kGated ? (j >> 1) * (S::kTileN / 2) + wn * 32 + (j & 1) * 16 : wn * 64 + j * 16;
}

template <class S>
__device__ __forceinline__ void read_n_side(Fragment (&b)[4], const char* operand, int wn,
                                            const LanePlace& at) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (S::kBByRows)
            read_fragment<true>(b[j], operand, n_first<S>(j, wn), at);
        else  // halves of 128 columns
            read_fragment<false>(b[j], operand + (wn >> 1) * (128 * kStepBytes),
                                 (wn & 1) * 64 + j * 16, at);
    }
}

__device__ __forceinline__ void multiply(f32x4 (&acc)[4], const Fragment (&b)[4],
                                         const Fragment& a) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j].bf16[s], a.bf16[s], acc[j], 0, 0, 0);
}

// 128 channels of e4m3 under one scale. The instruction adds its products in groups of eight, each
// product cut 14 bits below the group's largest one, and the groups in fp32 (measured: beside one
// product of 1.53 * 2^17 seven of 127 others of 2^2 are lost, and none of 2^3). So a block's sum is off
// by less than 7 * 2^-14 of its products' magnitudes, which ep.h states as 2^-11; with normally
// distributed codes by 1.5e-5 of its size. That is a choice: the products of widened codes
// (widened_step) keep fp32's bits and take 4150 against 2270 us at 131072 rows of 2048 x 7168, and the
// output is rounded to bf16. The fp32 scales of act, which would show it, come from widened_step.
__device__ __forceinline__ void multiply_e4m3(f32x4 (&acc)[4], const Fragment (&b)[4],
                                              const Fragment& a, float scale) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        d[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j].e4m3, a.e4m3, zero, 0, 0, 0,
                                                                0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = fmaf(d[j][r], scale, acc[j][r]);
    // the sums are made here: moved behind the wait that follows, they keep every product of the
    // step in registers, which then spill
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[j]));
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

template <int kPolicy = 0>
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t buf, uint32_t at, u32x4 w) {
    __builtin_amdgcn_raw_buffer_store_b128(w, buf, at, 0, kPolicy);
}

// Lane l holds two 16-byte words of row l % 16 of a subtile: its quarter (l / 16) of the first and
// of the second half of a 128-byte line. Exchanged between lanes eight apart, so that each of
// two stores writes eight whole lines: a = the words of rows 0..7, b = those of rows 8..15, a
// lane's being of row l % 8 (+ 8) and of half (l / 8) % 2.
__device__ __forceinline__ void whole_lines(u32x4& a, u32x4& b, int lane) {
    const bool low = (lane & 8) == 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t give = low ? b[i] : a[i];
        const uint32_t got = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
            0, static_cast<int>(give), 0x128, 0xf, 0xf, true));  // rotated by 8 within 16 lanes
        a[i] = low ? a[i] : got;
        b[i] = low ? got : b[i];
    }
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
// subtiles makes the same number of stores. What moves an access within a row is in its vector
// offset: a scalar offset is taken off the buffer's size before the comparison, and a piece that
// got no row has a buffer of none.
template <class S, int kMT>
__device__ __forceinline__ void gemm_store(const GemmArgs& g, const Tile& t, f32x4 (&acc)[S::kMT][4],
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
    if constexpr (S::kOp == GemmOp::kGateUp) {
        const int I = g.N;
        float(*amax)[2][4] = reinterpret_cast<float(*)[2][4]>(lds_amax);
        const bool quantise = g.codes != nullptr;
        if constexpr (S::kFp8) {
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
                for (int h = 0; h < (S::kFp8 ? 1 : 2); ++h) {
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
        const auto code_rows = rows_of(g.codes, I * (S::kFp8 ? 1u : 2u));
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
            float gate[8], up[8];
            eight_channels(acc[i][0], acc[i][1], gate);
            if constexpr (!S::kFp8) eight_channels(acc[i][2], acc[i][3], up);
            if (quantise) {
                float inv[2];
#pragma unroll
                for (int h = 0; h < (S::kFp8 ? 1 : 2); ++h) {
                    const float* p = amax[m][h];
                    const float top = group_amax(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])));
                    inv[h] = kE4m3Largest / top;
                    if (wn == 0 && quad == 0 && m < height)
                        g.scales[(first_row + m) * (I / (S::kFp8 ? 128 : 64)) + h * (I / 128) +
                                 t.n0 / 128] = top / kE4m3Largest;
                }
                const uint32_t at = in ? m * (I * (S::kFp8 ? 1u : 2u)) + c : kOutOfBuffer;
                __builtin_amdgcn_raw_buffer_store_b64(e4m3_eight(gate, inv[0]), code_rows, at, 0, 0);
                if constexpr (!S::kFp8)
                    __builtin_amdgcn_raw_buffer_store_b64(e4m3_eight(up, inv[1]), code_rows,
                                                          in ? at + I : at, 0, 0);
            }
            if constexpr (!S::kFp8) {
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
    } else if constexpr (S::kOp == GemmOp::kWeightGrad) {
        const uint32_t row_bytes = g.N * (g.out_fp32 ? 4u : 2u);
        const int64_t first = static_cast<int64_t>(t.expert) * g.M + t.m0;
        const auto rows = raw_buffer(static_cast<char*>(g.out) + first * row_bytes, height * row_bytes);
        const int half = (lane >> 3) & 1;
        constexpr int kPolicy = S::kLoaders > 0 ? kPolicyNt : 0;
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 7);
            if (g.out_fp32) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t c = t.n0 + wn * 64 + p * 32 + half * 16 + quad * 4;
                    const bool in = c < static_cast<uint32_t>(g.N);
                    u32x4 w[2] = {__builtin_bit_cast(u32x4, acc[i][2 * p]),
                                  __builtin_bit_cast(u32x4, acc[i][2 * p + 1])};
                    whole_lines(w[0], w[1], lane);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = in ? (m + 8 * h) * row_bytes + c * 4u : kOutOfBuffer;
                        if (g.accumulate)
                            w[h] = __builtin_bit_cast(
                                u32x4, __builtin_bit_cast(f32x4, w[h]) +
                                           __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                         rows, at, 0, 0)));
                        store16<kPolicy>(rows, at, w[h]);
                    }
                }
            } else {
                const uint32_t c = t.n0 + wn * 64 + half * 32 + in_pair;
                const bool in = c < static_cast<uint32_t>(g.N);
                u32x4 w[2];
                if (g.accumulate) {
                    // added in fp32, before the rounding: each pair's words where its sums are
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint32_t cp = t.n0 + wn * 64 + p * 32 + in_pair;
                        const uint32_t at =
                            cp < static_cast<uint32_t>(g.N)
                                ? ((2 * i + wm) * 16 + (lane & 15)) * row_bytes + cp * 2u
                                : kOutOfBuffer;
                        float v[8], old[8];
                        eight_channels(acc[i][2 * p], acc[i][2 * p + 1], v);
                        widen8(__builtin_bit_cast(
                                   u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, at, 0, 0)),
                               old);
#pragma unroll
                        for (int r = 0; r < 8; ++r) v[r] += old[r];
                        w[p] = narrow8(v);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        float v[8];
                        eight_channels(acc[i][2 * p], acc[i][2 * p + 1], v);
                        w[p] = narrow8(v);
                    }
                }
                whole_lines(w[0], w[1], lane);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    store16<kPolicy>(rows, in ? (m + 8 * h) * row_bytes + c * 2u : kOutOfBuffer, w[h]);
            }
        }
    } else if constexpr (S::kOp == GemmOp::kDownGrad) {
        const int I = g.N;
        const auto kept = rows_of(g.gate_up, I * 4u);
        const auto codes = rows_of(g.codes, I * 2u);
        const auto scales = rows_of(g.scales, (I / 64) * 4u);
        const auto grad = rows_of(g.out, I * 4u);
        const auto act = rows_of(g.act, I * 2u);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const uint32_t m = (2 * i + wm) * 16 + (lane & 15);
            u32x4 dgate[2], dup[2], again[2];
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
                dgate[p] = narrow8(dg);
                dup[p] = narrow8(du);
                again[p] = narrow8(up);
            }
            whole_lines(dgate[0], dgate[1], lane);
            whole_lines(dup[0], dup[1], lane);
            whole_lines(again[0], again[1], lane);
            const uint32_t c = t.n0 + wn * 64 + ((lane >> 3) & 1) * 32 + in_pair;
            const bool in = c < static_cast<uint32_t>(I);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t row = (2 * i + wm) * 16 + (lane & 7) + 8 * h;
                const uint32_t at = in ? row * (I * 4u) + c * 2u : kOutOfBuffer;
                store16(grad, at, dgate[h]);
                store16(grad, in ? at + I * 2u : at, dup[h]);
                if (g.act) store16(act, in ? row * (I * 2u) + c * 2u : kOutOfBuffer, again[h]);
            }
        }
    } else {
        const auto rows = rows_of(g.out, g.N * 2u);
        const uint32_t c = t.n0 + wn * 64 + ((lane >> 3) & 1) * 32 + in_pair;
        const bool in = c < static_cast<uint32_t>(g.N);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            u32x4 w[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float v[8];
                eight_channels(acc[i][2 * p], acc[i][2 * p + 1], v);
                w[p] = narrow8(v);
            }
            whole_lines(w[0], w[1], lane);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t m = (2 * i + wm) * 16 + (lane & 7) + 8 * h;
                store16(rows, in ? m * (g.N * 2u) + c * 2u : kOutOfBuffer, w[h]);
            }
        }
    }
}

// How many stores gemm_store is sure to make after its last load.
template <class S>
__device__ __forceinline__ int stores_after(const GemmArgs& g, int mt) {
    if constexpr (S::kOp == GemmOp::kGateUp)
        return mt * (S::kFp8 ? 1 : 1 + (g.gate_up ? 2 : 0) + (g.codes ? 2 : 0));
    else if constexpr (S::kOp == GemmOp::kWeightGrad)
        return g.accumulate ? 0 : mt * (g.out_fp32 ? 4 : 2);
    else if constexpr (S::kOp == GemmOp::kDownGrad)
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

// The products' scales of an e4m3 tile: one per step for the gate's (all) channels, one for the up
// projection's.
template <class S>
struct WeightScales {
    const float* row;
    int64_t up;
    __device__ __forceinline__ WeightScales(const GemmArgs& g, const Tile& t, int wn) {
        if constexpr (S::kFp8) {
            const int KB = g.K / 128;
            const int nb = S::kGated ? t.n0 / 128 : min((t.n0 + wn * 64) / 128, g.N / 128 - 1);
            row = g.b_scales +
                  (static_cast<int64_t>(t.expert) * (S::kGated ? 2 : 1) * (g.N / 128) + nb) * KB;
            up = static_cast<int64_t>(g.N / 128) * KB;
        }
    }
    __device__ __forceinline__ void read(int step, float (&bs)[2]) const {
        if constexpr (S::kFp8) {
            bs[0] = row[step];
            if constexpr (S::kGated) bs[1] = row[up + step];
        }
    }
};

// One tile's steps with kMT subtiles of 16 rows per wave. The block's two halves (waves 0..3 and
// 4..7, one of each on every SIMD) take turns: while one multiplies, the other reads its next
// fragments from LDS and issues loads, and a barrier ends each such slot. A step is four slots:
//   waves 0..3   read 1   multiply 1   read 2       multiply 2
//   waves 4..7   -        read 1       multiply 1   read 2       multiply 2
// where reading 1 takes the n side and the first half of the m side and issues the second half
// of the next step's m side; reading 2 takes the second half and issues the rest of the step
// after the next into the places that reading 1 has left. Every load has six slots to arrive: of
// a wave's loads all but the last kLoads have to be there at the end of every odd slot. The
// stores of the tile before lie between those loads in a tile's first step, and need not have
// ended there.
template <class S, int kMT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, const Tile& t, int steps,
                                          Producer<S, S::kWaves>& p, f32x4 (&acc)[S::kMT][4],
                                          char* lds, int& count, int& stores,
                                          const TileRing& ring, int wm, int wn,
                                          const LanePlace& at, int lane) {
    constexpr int kP = first_phase(kMT);
    constexpr int kLoads = Producer<S, S::kWaves>::kLoads;
    if (wm) end_slot();
    for (int step = 0; step < steps; ++step, ++count) {
        const char* stage = lds + (count & 1) * S::kStageBytes;
        Fragment b[4], a[kP];
        read_n_side<S>(b, stage + S::kMBytes, wn, at);
#pragma unroll
        for (int i = 0; i < kP; ++i)
            read_fragment<S::kAByRows>(a[i], stage, (2 * i + wm) * 16, at);
        p.issue_second();
        if (wm) wait_loads_before<kLoads>(stores);
        end_slot();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < kP; ++i) multiply(acc[i], b, a[i]);
        __builtin_amdgcn_s_setprio(0);
        if (!wm) wait_loads_before<kLoads>(stores);
        end_slot();
#pragma unroll
        for (int i = kP; i < kMT; ++i)
            read_fragment<S::kAByRows>(a[i - kP], stage + S::kMBytes / 2, (2 * (i - kP) + wm) * 16,
                                       at);
        p.issue_first(ring);
        if (wm) wait_loads_before<kLoads>(stores);
        end_slot();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = kP; i < kMT; ++i) multiply(acc[i], b, a[i - kP]);
        __builtin_amdgcn_s_setprio(0);
        if (!wm) wait_loads_before<kLoads>(stores);
        stores = 0;
        end_slot();
    }
    if (!wm) end_slot();
    gemm_store<S, kMT>(g, t, acc, lds + S::kAmaxAt, wm, wn, lane);
    stores = stores_after<S>(g, kMT);
}

// A block's tiles: every gridDim.x-th from its first. Block b runs on die b % 8: its tiles are
// neighbours of that die's other blocks' tiles.
struct BlockTiles {
    TileMap map;
    int64_t first;
    int count;
    TileRing ring;

    template <class S>
    __device__ __forceinline__ void init(const GemmArgs& g, char* lds) {
        map.init(g, !S::kOverRows, S::kTileM, S::kNTile, reinterpret_cast<int*>(lds + S::kTableAt));
        const int per_die = gridDim.x / 8;
        first = gridDim.x % 8 == 0
                    ? static_cast<int64_t>(blockIdx.x % 8) * per_die + blockIdx.x / 8
                    : blockIdx.x;
        const int64_t left = map.total - first + gridDim.x - 1;
        count = first >= map.total    ? 0
                : gridDim.x == kBlocks ? static_cast<int>(left / kBlocks)
                                       : static_cast<int>(left) / static_cast<int>(gridDim.x);
    }
    template <class S>
    __device__ __forceinline__ void look_up(int n) {
        if (n < count)
            ring.put(n, map.find(first + static_cast<int64_t>(n) * gridDim.x, S::kNTile));
    }
    // Tile n for the waves that do not look up themselves: they read it after a barrier.
    template <class S>
    __device__ __forceinline__ void publish(int n, char* lds) const {
        const int at = (n & 7) * 8, lane = lane_id();
        if (n < count && lane >= at && lane < at + 6)
            reinterpret_cast<int*>(lds + S::kTableAt)[kTableExperts + 32 + lane] = ring.lanes;
    }
    template <class S>
    __device__ __forceinline__ static Tile published(int n, const char* lds) {
        const int* p = reinterpret_cast<const int*>(lds + S::kTableAt) + kTableExperts + 32 +
                       (n & 7) * 8;
        int field[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) field[i] = __builtin_amdgcn_readfirstlane(p[i]);
        return Tile{field[0], field[1], field[2], field[3], field[4], field[5]};
    }
};

template <class S>
__device__ __forceinline__ void clear(f32x4 (&acc)[S::kMT][4]) {
#pragma unroll
    for (int i = 0; i < S::kMT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// One block per CU, two steps of 64 KB in LDS: per step of k an output takes 1/128 of an element from
// the L2, where a tile of 128 x 256 takes 1/85 and comes to that way's limit (about 23 TB/s). 32768
// rows of 4096 x 7168 weights of 32 experts take 1500 to 1630 us (1180 to 1280 TFLOP/s) at the 1.55
// GHz that the clock falls to, the matrix cores busy for .65 of the cycles; a plain library product of
// that size 1278 us at 1.62 GHz, busy for .88. Between products the block waits for its epilogue:
// down's gradient, with six arrays in it, takes 940 to 970 us, 780 of them products at that rate;
// the weights' 2080 to 2250 us with 3.8 GB of fp32 stores, which take 606 us alone.
template <class S>
__global__ __launch_bounds__(S::kThreads, 1) void gemm_kernel(const GemmArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[S::kLdsBytes];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / S::kNWaves, wn = wave % S::kNWaves;
    const LanePlace at(lane);
    BlockTiles tiles;
    tiles.init<S>(g, lds);
    for (int n = 0; n < S::kStages; ++n) tiles.look_up<S>(n);
    Producer<S, S::kWaves> p(g, lds_address(lds), wave, tiles.count, tiles.ring);
    int count = 0, stores = 0;
    p.issue_first(tiles.ring);
    p.issue_second();
    p.issue_first(tiles.ring);
    wait_loads<Producer<S, S::kWaves>::kLoads>();
    end_slot();
    for (int n = 0; n < tiles.count; ++n) {
        tiles.look_up<S>(n + S::kStages);
        const Tile t = tiles.ring.get(n);
        const int steps = tile_steps<S>(g, t);
        f32x4 acc[S::kMT][4];
        clear<S>(acc);
        switch (max((t.height + 31) / 32, 1)) {  // a piece of a low tile may have got no row
#define EP_GEMM_CASE(n)                                                                            \
    case n:                                                                                        \
        gemm_tile<S, n>(g, t, steps, p, acc, lds, count, stores, tiles.ring, wm, wn, at, lane);    \
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

// Sixteen e4m3 codes as bf16, which holds every one of them.
__device__ __forceinline__ void widen_codes(const u32x4& w, bf16x8 (&v)[2]) {
    union {
        bf16x2 pair[8];
        bf16x8 eight[2];
    } u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u.pair[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
        u.pair[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
    }
    v[0] = u.eight[0];
    v[1] = u.eight[1];
}

// A step of e4m3 rows with the products summed in fp32 throughout: the codes are widened to bf16
// for the bf16 matrix instruction. With normally distributed codes the e4m3 one's sums of 128 are
// off by 1.5e-5 of their size, these by 1e-8, and the fp32 scales of act show it. It takes twice
// the matrix time and the conversions on top, each as long as three other vector operations
// (weights of 4096 x 7168: 16 rows of each of 32 experts 160 us against 158, 128 rows of each of
// 256 experts 2690 to 2890 against 1800). Every wave converts what it reads, in registers; fewer
// waves with more channels each, conversions between the products, and conversions through fp32
// and a byte permute gained nothing.
// A step is two sums of 64 products (the words w of a fragment), each scaled and added, whatever
// the tile's height: a row's result does not depend on how the other experts' rows cut its tile.
// Tiles of four pairs of subtiles read one word of every fragment at a time, to stay within the
// registers; lower ones, which have room, both. One sum of 128 in the lower ones took 1544 against
// 1587 to 1657 us at 64 rows of each of 256 experts, and gave other bits than the high ones.
template <class S, int kMT>
__device__ __forceinline__ void widened_step(f32x4 (&acc)[S::kMT][4], const char* stage,
                                             const float* as, const float (&bs)[2], int wm, int wn,
                                             const LanePlace& at) {
    constexpr int kParts = kMT > 3 ? 2 : 1, kWords = 2 / kParts;
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
        bf16x8 a[kWords][kMT][2];
        auto read = [&](const char* base, int first, int w, bf16x8 (&v)[2]) {
            const int place = at.by_row ^ ((part + w) * 64);
            widen_codes(*reinterpret_cast<const u32x4*>(base + first * kStepBytes + place), v);
        };
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int i = 0; i < kMT; ++i) read(stage, (2 * i + wm) * 16, w, a[w][i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 d[kWords][kMT];
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                bf16x8 b[2];
                read(stage + S::kMBytes, n_first<S>(j, wn), w, b);
#pragma unroll
                for (int i = 0; i < kMT; ++i) d[w][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < kMT; ++i)
                        d[w][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[s], a[w][i][s],
                                                                          d[w][i], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                const float scale = as[i] * bs[S::kGated ? j >> 1 : 0];
#pragma unroll
                for (int w = 0; w < kWords; ++w)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[w][i][r], scale, acc[i][j][r]);
            }
        }
    }
}

// One tile's steps in the waves that multiply.
template <class S, int kMT>
__device__ __forceinline__ void stream_tile(const GemmArgs& g, const Tile& t, int steps,
                                            f32x4 (&acc)[S::kMT][4], char* lds, int& slot,
                                            int& scale_slot, int wm, int wn, const LanePlace& at,
                                            int lane) {
    const WeightScales<S> weight_scales(g, t, wn);
    float bs[2] = {1.0f, 1.0f};
    for (int step = 0; step < steps; ++step) {
        weight_scales.read(step, bs);
        lds_barrier();
        const char* stage = lds + slot * S::kStageBytes;
        const char* scales = lds + S::kScalesAt + scale_slot * S::kScaleBytes;
        slot = slot + 1 == S::kStages ? 0 : slot + 1;
        scale_slot = (scale_slot + 1) & (kScaleSlots - 1);
        float as[kMT];
        if constexpr (S::kFp8) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
                as[i] = *reinterpret_cast<const float*>(scales + ((2 * i + wm) * 16 + (lane & 15)) * 4);
        }
        if constexpr (S::kWidened) {
            widened_step<S, kMT>(acc, stage, as, bs, wm, wn, at);
            continue;
        }
        Fragment b[4], a[kMT];
        read_n_side<S>(b, stage + S::kMBytes, wn, at);
#pragma unroll
        for (int i = 0; i < kMT; ++i)
            read_fragment<S::kAByRows>(a[i], stage, (2 * i + wm) * 16, at);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            if constexpr (S::kFp8)
                multiply_e4m3(acc[i], b, a[i], as[i] * bs[0]);
            else
                multiply(acc[i], b, a[i]);
        }
    }
    gemm_store<S, kMT>(g, t, acc, lds + S::kAmaxAt, wm, wn, lane);
}

// Most waves multiply and four load: a load that memory holds up stops none of the products, and
// the stores of a tile wait for no load. All meet once a step: then step k has arrived, step
// k - 1 has been read, and the loaders go on to step k + kStages - 1 in its place. What bounds it
// is the weights' way from memory: 5.3 to 6.2 of the 6.2 TB/s that a copy reaches from 512 rows of
// 256 experts down to one token of eight (1213, 435, 81 us); with more rows the e4m3 products
// (131072 rows of 2048 x 7168 2120 to 2270 us) and the widened ones (32768 rows of 4096 x 7168
// 2690 to 2890 us) are. A call of a few us waits for 16 to 112 steps of about .3 us.
template <class S>
__global__ __launch_bounds__(S::kThreads, 1) void stream_kernel(const GemmArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[S::kLdsBytes];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    BlockTiles tiles;
    tiles.init<S>(g, lds);
    if (wave >= S::kWaves) {
        using P = Producer<S, S::kLoaders>;
        for (int n = 0; n < S::kStages; ++n) {
            tiles.look_up<S>(n);
            tiles.publish<S>(n, lds);
        }
        lds_barrier();
        P p(g, lds_address(lds), wave - S::kWaves, tiles.count, tiles.ring);
        const bool meets_after = S::kGated && g.codes;  // for the magnitudes of the tile's groups
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) p.issue_first(tiles.ring);
        for (int n = 0; n < tiles.count; ++n) {
            const int steps = tile_steps<S>(g, tiles.ring.get(n));
            for (int step = 0; step < steps; ++step) {
                wait_loads<(S::kStages - 2) * P::kLoads>();
                lds_barrier();
                p.issue_first(tiles.ring);
                if (step == 0) {
                    tiles.look_up<S>(n + S::kStages);
                    tiles.publish<S>(n + S::kStages, lds);
                }
            }
            if (meets_after) lds_barrier();
        }
        wait_loads<0>();  // no load outlives the block
        return;
    }
    const int wm = wave / S::kNWaves, wn = wave % S::kNWaves;
    const LanePlace at(lane);
    int slot = 0, scale_slot = 0;
    lds_barrier();
    for (int n = 0; n < tiles.count; ++n) {
        const Tile t = BlockTiles::published<S>(n, lds);
        const int steps = tile_steps<S>(g, t);
        f32x4 acc[S::kMT][4];
        clear<S>(acc);
        switch (max((t.height + 31) / 32, 1)) {
#define EP_STREAM_CASE(n)                                                                        \
    case n:                                                                                      \
        if constexpr (n <= S::kMT)                                                               \
            stream_tile<S, n>(g, t, steps, acc, lds, slot, scale_slot, wm, wn, at, lane);        \
        break;
            EP_STREAM_CASE(1)
            EP_STREAM_CASE(2)
            EP_STREAM_CASE(3)
            EP_STREAM_CASE(4)
#undef EP_STREAM_CASE
        }
    }
}

// Tiles of a call at most, as the host knows it.
template <class S>
int64_t most_tiles(const GemmArgs& g) {
    const int64_t nt = (g.N + S::kNTile - 1) / S::kNTile;
    if constexpr (S::kOverRows)
        return static_cast<int64_t>(g.piece_rows > 0 ? g.pieces : g.E) *
               ((g.M + S::kTileM - 1) / S::kTileM) * nt;
    return (g.num_rows / S::kTileM + std::min<int64_t>(g.E, g.num_rows)) * nt;
}

template <class S>
hipError_t launch_shape(const GemmArgs& g, hipStream_t stream) {
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(kBlocks, most_tiles<S>(g)));
    if (blocks == 0) return hipSuccess;
    if constexpr (S::kLoaders > 0)
        stream_kernel<S><<<blocks, S::kThreads, 0, stream>>>(g);
    else
        gemm_kernel<S><<<blocks, S::kThreads, 0, stream>>>(g);
    return hipGetLastError();
}

// Which tile, by the rows per expert that the host knows of (us on MI355X):
//   32 against 128 rows (weights of 4096 x 7168, 7168 x 2048 and 4096 x 1408): 17 skewed rows of
//     each of 128 experts, down's gradient 284 / 305; 16 rows of 256, e4m3 down 641 / 622; up to
//     20 rows within 1% otherwise; 32 rows of 32 experts, e4m3 186 / 163, bf16 338 / 314
//   128 against 256 rows (bf16, 4096 x 7168 weights of 32 experts): 64 rows 314 / 324, 128 rows
//     395 / 346, 1024 rows 1720 / 1540
// e4m3 keeps the 128 rows: the e4m3 instruction's products take half the time and the loads are
// what is short at either height (131072 rows of 2048 x 7168 2164 against 2310); widened to bf16
// they leave no registers for more. A call with fewer tiles of 128 rows than CUs takes the low
// ones, and narrow ones where those are at most one per CU too (one token over eight experts 81
// against 96 narrow and wide; 257 tokens of 1024 over 16 experts 17.1 against 19.8 low and not).
constexpr int64_t kLowRows = 20, kMidRows = 96;

template <GemmOp kOp, bool kFp8>
hipError_t launch_gemm(const GemmArgs& g, hipStream_t stream) {
    using Low = GemmShape<kOp, kFp8, 32>;
    using Mid = GemmShape<kOp, kFp8, 128>;
    const int64_t rows = g.num_rows / g.E;
    if (rows <= kLowRows || most_tiles<Mid>(g) < kBlocks) {
        // a narrow tile has half a group of the gate's 128 channels, so it writes no codes
        if constexpr (!kFp8) {
            using Narrow = GemmShape<kOp, kFp8, 32, 128>;
            if (!(kOp == GemmOp::kGateUp && g.codes) && most_tiles<Narrow>(g) <= kBlocks)
                return launch_shape<Narrow>(g, stream);
        }
        return launch_shape<Low>(g, stream);
    }
    if constexpr (!kFp8)
        if (rows > kMidRows) return launch_shape<GemmShape<kOp, kFp8, 256>>(g, stream);
    return launch_shape<Mid>(g, stream);
}

}  // namespace ep
