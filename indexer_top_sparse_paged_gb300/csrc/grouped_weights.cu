// After the attention over the grouped-head cache, where they are wanted: the positions' weights, summed from the logits.
// They need the rows' final sums, so the attention leaves its logits in the workspace (4 bytes a row and position, mostly
// in L2 still when they are read here: 22 MB of 67 come from memory). Latency of those reads bounds it: 32 sequences of 8K,
// 8 heads, 8 rows take 14 us beside the attention's 75 (kernel times).
#include <type_traits>

#include "grouped.cuh"

namespace dsa {

constexpr int kWeightsThreads = 256;
constexpr int kWeightsRows = 8;        // rows that a warp sums at a time (no more than a row tile has)

// The sequences b0 .. b0 + 255 in shared memory, with the position tiles of key heads and the attention's tiles that stand
// before each.
struct GroupedChunk {
    GroupedSeq seq[kWeightsThreads];
    int64_t units[kWeightsThreads + 1], tiles[kWeightsThreads];
    int64_t warp_sums[kWeightsThreads / 32];
};

__device__ __forceinline__ int64_t chunk_load(const GroupedArgs& a, GroupedChunk& c, int b0, int64_t tiles_before) {
    const int tid = threadIdx.x, b = b0 + tid;
    GroupedSeq s{};
    if (b < a.B) s = grouped_seq(a, b, false);
    int64_t all_units, all_tiles;
    const int64_t u = block_prefix<kWeightsThreads>(static_cast<int64_t>(s.tiles) * a.H_kv, &all_units, c.warp_sums);
    const int64_t t = block_prefix<kWeightsThreads>(grouped_seq_tiles(a, s), &all_tiles, c.warp_sums);
    c.seq[tid] = s;
    c.units[tid] = u;
    c.tiles[tid] = tiles_before + t;
    if (tid == 0) c.units[kWeightsThreads] = all_units;
    __syncthreads();
    return all_tiles;
}

// weights_out = weights + the sum over the rows of 2^(z - lse): a warp for each position tile of a key head, four positions
// a lane, so that a row's 128 logits are four coalesced loads. Where there are no more tiles than CTAs, a CTA's warps share a
// tile's rows instead (attention and weights of 14 sequences of 2000, one key head, 640 rows: 460 us a warp a tile, 162
// shared; 4 of 2000, 8 key heads: 64 rows 73 and 53, 16 rows 35 and 36; with 4096 tiles of 128 rows 360 and 379, with 16,000
// of 8 rows 150 and 321).
__global__ void __launch_bounds__(kWeightsThreads) grouped_weights_kernel(GroupedArgs a) {
    constexpr int kWarps = kWeightsThreads / 32;
    __shared__ GroupedChunk c;
    __shared__ float part[kWarps][kGroupedTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t before = 0;
    bool waited = false;
    for (int b0 = 0; b0 < a.B; b0 += kWeightsThreads) {
        if (b0) __syncthreads();  // these sequences take the others' place
        before += chunk_load(a, c, b0, before);
        if (!waited) griddep_wait();
        waited = true;
        const int64_t n = c.units[kWeightsThreads];
        auto work = [&](auto sharing) {
            constexpr bool kShare = decltype(sharing)::value;
            constexpr int kStep = kShare ? kWarps * kWeightsRows : kWeightsRows;
            const int mine = kShare ? warp : 0;
            for (int64_t u = blockIdx.x + (kShare ? 0 : static_cast<int64_t>(warp) * gridDim.x); u < n; u += static_cast<int64_t>(kWarps) * gridDim.x) {
                int i = 0, hi = min(kWeightsThreads, a.B - b0) - 1;  // the last sequence whose first unit is at or before u
                while (i < hi) {
                    const int mid = (i + hi + 1) >> 1;
                    if (c.units[mid] <= u) i = mid;
                    else hi = mid - 1;
                }
                const GroupedSeq s = c.seq[i];
                const int place = static_cast<int>(u - c.units[i]), h = place / s.tiles, tile = place - h * s.tiles;
                const int pos = tile * kGroupedTile + lane, left = s.len - pos;  // positions pos, pos + 32, + 64, + 96 below len
                const int64_t at = (static_cast<int64_t>(b0 + i) * a.H_kv + h) * a.max_blocks * kBlock + pos;
                float w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = mine == 0 && a.weights && 32 * k < left ? a.weights[at + 32 * k] : 0.0f;
                const float* lse = a.row_lse + static_cast<int64_t>(s.q0) * a.H + h * a.G;
                const int all = s.n * a.G;
                for (int row0 = mine * kWeightsRows; row0 < all; row0 += kStep) {
                    const int it = row0 / a.row_tile;
                    const int64_t t = c.tiles[i] + (static_cast<int64_t>(h) * s.items + it) * s.tiles + tile;
                    if (t >= a.max_tiles) break;
                    const int n_rows = min(kWeightsRows, all - row0);
                    const float* z = a.z + (t * a.row_tile + row0 - it * a.row_tile) * kGroupedTile + lane;
                    // lane k: row row0 + k's sum, as a logarithm
                    const int row = row0 + lane, tok = row / a.G;
                    const float e = lane < n_rows ? lse[static_cast<int64_t>(tok) * a.H + row - tok * a.G] : 0.0f;
#pragma unroll 4
                    for (int r = 0; r < n_rows; ++r) {
                        const float er = __shfl_sync(0xFFFFFFFFu, e, r);
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = z[r * kGroupedTile + 32 * k];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (x[k] != -INFINITY) w[k] += exp2f(x[k] - er);
                    }
                }
                if constexpr (kShare) {  // the warps' sums, in order (one tile a CTA at most: every warp comes here, or none)
#pragma unroll
                    for (int k = 0; k < 4; ++k) part[warp][32 * k + lane] = w[k];
                    __syncthreads();
                    if (warp == 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            for (int j = 1; j < kWarps; ++j) w[k] += part[j][32 * k + lane];
                    }
                }
                if (mine == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (32 * k < left) a.weights_out[at + 32 * k] = w[k];
                }
            }
        };
        if (n <= gridDim.x) work(std::true_type{});
        else work(std::false_type{});
    }
}

// A row tile has 8 rows at least, so that a warp's rows at a time are of one.
bool launch_grouped_weights(const GroupedArgs& a, cudaStream_t s, int* launches) {
    if (!launch_kernel(true, grouped_weights_kernel, dim3(4 * a.ctas), dim3(kWeightsThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
