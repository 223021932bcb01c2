// expert_ffn_grad.hip -- the gradients of the experts' gated feed-forward block on gfx950, over
// rows sorted by expert. With s = sigmoid(gate) and da = grad_out Wd:
//   grad_gate = da up s (1 + gate (1 - s)), grad_up = da gate s      ep_expert_down_grad
//   grad_x    = grad_gate Wg + grad_up Wu                            ep_expert_gate_up_grad
//   grad_W[e] = grad_rows^T input_rows over expert e's rows          ep_expert_weight_grad
#include "expert_gemm.hpp"

#include <algorithm>

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

// ---------------------------------------------------------------- long sums, few tiles
// A block sums an expert's rows for one tile of the weight, so a weight of few tiles leaves most
// CUs idle for as long as its rows take. There the rows are cut into pieces of equal length, so
// many that their tiles fill the chip once; every piece's sums go to the workspace in fp32 (at
// most 64 MB), and a second launch adds each expert's in order. It pays from 512 rows per expert on,
// and from ten times as many as there are tiles: they share the CUs, and their sums are written
// and read once more. Measured (us on MI355X, whole / in pieces of the lower tiles / of the higher):
//   1 of 112 x 112 (1 tile)       384 rows 12 / 13 / 14    512 rows 15 / 13 / 15    4096 rows 70 / 15 / 16
//   1 of 2048 x 1024 (64)         512 rows 24 / 25 / 30    640 rows 27 / 26 / 31    4096 rows 98 / 35 / 43
//   1 of 1536 x 1792 (84)         1024 rows 36 / 28 / 36   4096 rows 98 / 47 / 51   8192 rows 181 / 74 / 70
//   3 of 1032 x 1000 (108)        1408 rows 41 / 33 / 36   2048 rows 53 / 44 / 41   8192 rows 176 / 110 / 83
//   32 of 192 x 496 (128)         1024 rows 29 / 31 / 33   1280 rows 33 / 34 / 36   4096 rows 84 / 65 / 61
//   1 of 2048 x 2048 (128)        1024 rows 35 / 36 / 37   1280 rows 40 / 40 / 38   16384 rows 335 / 230 / 156
// The higher tiles, half as many, leave room for more pieces; that is worth their longer steps and
// larger sums where the lower ones nearly fill the chip, or rows are very many. A weight of no more
// than 128 channels along m has as few tiles of either height: there the whole rows are as quick in
// the higher ones, and pieces (of the lower) pay only for what they save, against their bytes:
//   96 of 128 x 256 (96)          1024 rows 26 / 32 / 33   2048 rows 42 / 44 / 45   4096 rows 82 / 78 / 80
//   101 of 24 x 40 (101)          1024 rows 18 / 14 / 18   4096 rows 55 / 25 / 43
namespace {

template <int kTileM>
using WeightShape = GemmShape<GemmOp::kWeightGrad, false, kTileM>;

constexpr int64_t kLeastPiece = 256;  // four steps; 128 rows are slower from 8192 rows on (18 against 16 us)
constexpr int64_t kRowsPerTile = 10;
constexpr int64_t kBytesPerRow = 12500;  // of pieces per row of an expert, at M <= 128
constexpr int kManyPieces = 32;

struct Pieces {
    int rows = 0, count = 0;
    bool high = false;
};

template <int kTileM>
int64_t weight_tiles(int E, int M, int N) {
    constexpr int kTileN = WeightShape<kTileM>::kNTile;
    return static_cast<int64_t>(E) * ((M + kTileM - 1) / kTileM) * ((N + kTileN - 1) / kTileN);
}

Pieces pieces_of(int E, int64_t rows, int M, int N) {
    Pieces p;
    int64_t tiles = weight_tiles<128>(E, M, N);
    if (tiles > kBlocks / 2 || rows / E < std::max<int64_t>(512, kRowsPerTile * tiles)) return p;
    p.high = M > 128 && tiles > 64 && rows / E >= (tiles > 96 ? 2048 : 8192);
    if (p.high) tiles = weight_tiles<256>(E, M, N);
    const int64_t left = kBlocks - tiles;  // every expert may have one piece begun
    const int64_t each = std::max(kLeastPiece, (rows * (tiles / E) + left - 1) / left);
    p.rows = static_cast<int>(std::min<int64_t>((each + 63) / 64 * 64, INT32_MAX / 64 * 64));
    p.count = static_cast<int>(rows / p.rows) + E;
    if (M <= 128 && rows / E < static_cast<int64_t>(p.count) * M * N * 4 / kBytesPerRow) return Pieces{};
    return p;
}

// Adds the pieces of a word of four channels per lane, eight loads in flight: all of them in one
// wave, or (kWaves = 4) every fourth in each of a block's four and then their sums, which many
// pieces are worth (64 of 112 x 112 19.5 against 26 us; 2 of 2048 x 2048 140 against 126).
template <int kWaves>
__global__ __launch_bounds__(256) void weight_pieces_kernel(const GemmArgs g,
                                                            const f32x4* __restrict__ partial) {
    constexpr int kWords = 256 / kWaves;
    __shared__ f32x4 sums[kWaves][kWords];
    bool bad = false;
    for (int e = threadIdx.x; e <= g.E; e += 256)
        bad |= g.offset[e] < (e > 0 ? g.offset[e - 1] : 0);
    if (__syncthreads_or(bad)) return;
    const int word = threadIdx.x % kWords, wave = threadIdx.x / kWords;
    const int64_t per = static_cast<int64_t>(g.M) * g.N / 4;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kWords + word;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at < per * g.E) {
        const int e = static_cast<int>(at / per);
        auto first = [&](int i) {
            return first_piece(static_cast<int>(min<int64_t>(g.offset[i], g.num_rows)), i,
                               g.piece_rows);
        };
        const int from = first(e) + wave, to = first(e + 1);
        const int64_t next = kWaves * per;
        const f32x4* p = partial + from * per + (at - e * per);
        int left = to > from ? (to - from + kWaves - 1) / kWaves : 0;
        for (; left >= 8; left -= 8, p += 8 * next) {
            f32x4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i * next];
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
        for (; left > 0; --left, p += next) sum += *p;
    }
    if constexpr (kWaves > 1) {
        sums[wave][word] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += sums[w][word];
    }
    if (wave > 0 || at >= per * g.E) return;
    if (g.out_fp32) {
        f32x4* out = static_cast<f32x4*>(g.out) + at;
        if (g.accumulate) sum += *out;
        *out = sum;
    } else {
        u32x2* out = static_cast<u32x2*>(g.out) + at;
        if (g.accumulate) {
            const u32x2 old = *out;
            sum += f32x4{bf16_lo(old[0]), bf16_hi(old[0]), bf16_lo(old[1]), bf16_hi(old[1])};
        }
        *out = u32x2{bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
    }
}

}  // namespace

size_t expert_weight_grad_workspace_bytes(int E, int64_t rows, int M, int N) {
    return static_cast<size_t>(pieces_of(E, rows, M, N).count) * M * N * sizeof(float);
}

hipError_t launch_expert_weight_grad_split(const GemmArgs& g, float* workspace,
                                           hipStream_t stream) {
    const Pieces p = pieces_of(g.E, g.num_rows, g.M, g.N);
    if (p.count == 0) return launch_expert_weight_grad(g, stream);
    GemmArgs part = g;
    part.piece_rows = p.rows;
    part.pieces = p.count;
    GemmArgs join = part;
    part.out = workspace;
    part.out_fp32 = 1;
    part.accumulate = 0;
    const hipError_t st = p.high ? launch_shape<WeightShape<256>>(part, stream)
                                 : launch_shape<WeightShape<128>>(part, stream);
    if (st != hipSuccess) return st;
    const int64_t words = static_cast<int64_t>(g.E) * g.M * g.N / 4;
    const f32x4* sums = reinterpret_cast<const f32x4*>(workspace);
    if (p.count / g.E >= kManyPieces)
        weight_pieces_kernel<4><<<static_cast<unsigned>((words + 63) / 64), 256, 0, stream>>>(join, sums);
    else
        weight_pieces_kernel<1><<<static_cast<unsigned>((words + 255) / 256), 256, 0, stream>>>(join, sums);
    return hipGetLastError();
}

}  // namespace ep
