// After the attention over the grouped-head cache, where they are wanted: the positions' weights, summed from the logits.
// They need the rows' final sums, so the attention leaves its logits in the workspace (4 bytes a row and position, mostly
// in L2 still when they are read here: 22 MB of 67 come from memory). Latency of those reads bounds it: 32 sequences of 8K,
// 8 heads, 8 rows take 12 us beside the attention's 77.
#include "grouped.cuh"

namespace dsa {

constexpr int kWeightsThreads = 256;

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
// a lane, so that a row's 128 logits are four coalesced loads.
__global__ void __launch_bounds__(kWeightsThreads) grouped_weights_kernel(GroupedArgs a) {
    __shared__ GroupedChunk c;
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kWeightsThreads / 32);
    int64_t before = 0;
    bool waited = false;
    for (int b0 = 0; b0 < a.B; b0 += kWeightsThreads) {
        if (b0) __syncthreads();  // these sequences take the others' place
        before += chunk_load(a, c, b0, before);
        if (!waited) griddep_wait();
        waited = true;
        const int64_t n = c.units[kWeightsThreads];
        for (int64_t u = blockIdx.x + static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x; u < n; u += warps) {
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
            for (int k = 0; k < 4; ++k) w[k] = a.weights && 32 * k < left ? a.weights[at + 32 * k] : 0.0f;
            const float* lse = a.row_lse + static_cast<int64_t>(s.q0) * a.H + h * a.G;
            for (int it = 0; it < s.items; ++it) {
                const int64_t t = c.tiles[i] + (static_cast<int64_t>(h) * s.items + it) * s.tiles + tile;
                if (t >= a.max_tiles) break;
                const int row0 = it * a.row_tile, rows = min(a.row_tile, s.n * a.G - row0);
                const float* z = a.z + t * a.row_tile * kGroupedTile + lane;
                for (int r0 = 0; r0 < rows; r0 += 32) {
                    // lane k: row r0 + k's sum, as a logarithm
                    const int row = row0 + r0 + lane, tok = row / a.G;
                    const float e = r0 + lane < rows ? lse[static_cast<int64_t>(tok) * a.H + row - tok * a.G] : 0.0f;
                    const int n_rows = min(32, rows - r0);
#pragma unroll 4
                    for (int r = 0; r < n_rows; ++r) {
                        const float er = __shfl_sync(0xFFFFFFFFu, e, r);
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = z[(r0 + r) * kGroupedTile + 32 * k];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (x[k] != -INFINITY) w[k] += exp2f(x[k] - er);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (32 * k < left) a.weights_out[at + 32 * k] = w[k];
        }
    }
}

bool launch_grouped_weights(const GroupedArgs& a, cudaStream_t s, int* launches) {
    if (!launch_kernel(true, grouped_weights_kernel, dim3(4 * a.ctas), dim3(kWeightsThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
