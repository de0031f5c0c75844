// After the attention over the grouped-head cache: the rows of items that were cut are joined from their partials, rows
// without positions are written, and, where they are wanted, the positions' weights are summed from the logits.
#include "grouped.cuh"

namespace dsa {

constexpr int kGroupedJoinThreads = 256;

__device__ __forceinline__ void store_row(void* out, bool f32, int64_t at, float x) {
    if (f32) static_cast<float*>(out)[at] = x;
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

// The sequences b0 .. b0 + 255 in shared memory, with the items (weights: position tiles of a key head) and the tiles
// that stand before each.
struct GroupedChunk {
    GroupedSeq seq[kGroupedJoinThreads];
    int64_t units[kGroupedJoinThreads + 1], tiles[kGroupedJoinThreads + 1];
    int64_t warp_sums[kGroupedJoinThreads / 32];
};

__device__ __forceinline__ int chunk_find(const GroupedChunk& c, int n, int64_t u) {
    int lo = 0, hi = n - 1;  // the last sequence whose first unit is at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c.units[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <bool kWeights>
__device__ __forceinline__ int64_t chunk_load(const GroupedArgs& a, GroupedChunk& c, int b0, int64_t tiles_before) {
    const int tid = threadIdx.x, b = b0 + tid;
    GroupedSeq s{};
    if (b < a.B) s = grouped_seq(a, b, false);
    const int64_t units = kWeights ? static_cast<int64_t>(s.tiles) * a.H_kv : static_cast<int64_t>(s.items) * a.H_kv;
    const int64_t tiles = b < a.B ? grouped_seq_tiles(a, s) : 0;
    int64_t all_units, all_tiles;
    __syncthreads();
    c.seq[tid] = s;
    const int64_t u = block_prefix<kGroupedJoinThreads>(b < a.B ? units : 0, &all_units, c.warp_sums);
    const int64_t t = block_prefix<kGroupedJoinThreads>(tiles, &all_tiles, c.warp_sums);
    c.units[tid] = u;
    c.tiles[tid] = tiles_before + t;
    if (tid == 0) c.units[kGroupedJoinThreads] = all_units;
    __syncthreads();
    return all_tiles;
}

__global__ void __launch_bounds__(kGroupedJoinThreads) grouped_join_kernel(GroupedArgs a) {
    __shared__ GroupedChunk c;
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    // the lengths are inputs: only the partials wait for the attention
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += kGroupedJoinThreads) total += chunk_load<false>(a, c, b0, 0);
    const int64_t per = max(static_cast<int64_t>(1), (total + a.ctas - 1) / a.ctas);
    griddep_wait();
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kGroupedJoinThreads) {
        if (a.B > kGroupedJoinThreads) before += chunk_load<false>(a, c, b0, before);
        const int64_t n = c.units[kGroupedJoinThreads];
        for (int64_t u = blockIdx.x; u < n; u += gridDim.x) {
            const int i = chunk_find(c, min(kGroupedJoinThreads, a.B - b0), u);
            const GroupedSeq s = c.seq[i];
            const int item = static_cast<int>(u - c.units[i]), h = item / s.items, row0 = (item - h * s.items) * a.row_tile;
            const int rows = min(a.row_tile, s.n * a.G - row0);
            const int64_t u0 = c.tiles[i] + static_cast<int64_t>(item) * s.tiles, u1 = u0 + s.tiles;
            const int c0 = static_cast<int>(u0 / per), c1 = s.tiles ? static_cast<int>((u1 - 1) / per) : c0;
            if (s.tiles && c0 == c1) continue;  // the attention wrote the rows
            for (int e = tid; e < rows * a.d_v; e += kGroupedJoinThreads) {
                const int r = e / a.d_v, col = e - r * a.d_v, row = row0 + r;
                float top = -INFINITY, sum = 0.0f, o = 0.0f;
                for (int p = c0; s.tiles && p <= c1; ++p)
                    top = fmaxf(top, a.part_ml[grouped_slot(p * per, max(p * per, u0), p) * a.row_tile + r].x);
                const float ref = top == -INFINITY ? 0.0f : top;
                for (int p = c0; s.tiles && p <= c1; ++p) {
                    const int64_t slot = static_cast<int64_t>(grouped_slot(p * per, max(p * per, u0), p)) * a.row_tile + r;
                    const float2 ml = a.part_ml[slot];
                    const float f = exp2f(ml.x - ref);
                    sum = fmaf(f, ml.y, sum);
                    o = fmaf(f, a.part_o[slot * a.d_v + col], o);
                }
                const int64_t at = static_cast<int64_t>(s.q0 + row / a.G) * a.H + h * a.G + row % a.G;
                store_row(a.out, a.type == DSA_F32, at * a.d_v + col, sum == 0.0f ? 0.0f : o / sum);
                if (col == 0) {
                    const float lse2 = sum == 0.0f ? -INFINITY : top + log2f(sum);
                    if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
                    if (a.weights_out) a.row_lse[at] = lse2;
                }
            }
        }
        if (a.B > kGroupedJoinThreads) __syncthreads();  // the next sequences take their place
    }
}

// weights_out = weights + the sum over the rows of 2^(z - lse): two position tiles a CTA at a time.
__global__ void __launch_bounds__(kGroupedJoinThreads) grouped_weights_kernel(GroupedArgs a) {
    __shared__ GroupedChunk c;
    const int tid = threadIdx.x, part = tid >> 7, j = tid & 127;
    int64_t before = 0;
    bool waited = false;
    for (int b0 = 0; b0 < a.B; b0 += kGroupedJoinThreads) {
        before += chunk_load<true>(a, c, b0, before);
        if (!waited) griddep_wait();
        waited = true;
        const int64_t n = c.units[kGroupedJoinThreads];
        for (int64_t u = 2 * static_cast<int64_t>(blockIdx.x) + part; u < n; u += 2 * static_cast<int64_t>(gridDim.x)) {
            const int i = chunk_find(c, min(kGroupedJoinThreads, a.B - b0), u);
            const GroupedSeq s = c.seq[i];
            const int64_t place = u - c.units[i];
            const int h = static_cast<int>(place / s.tiles), tile = static_cast<int>(place - static_cast<int64_t>(h) * s.tiles);
            const int pos = tile * kGroupedTile + j;
            if (pos >= s.len) continue;
            float w = 0.0f;
            for (int it = 0; it < s.items; ++it) {
                const int64_t t = c.tiles[i] + (static_cast<int64_t>(h) * s.items + it) * s.tiles + tile;
                if (t >= a.max_tiles) break;
                const int row0 = it * a.row_tile, rows = min(a.row_tile, s.n * a.G - row0);
                const float* z = a.z + (t * kGroupedTile + j) * a.row_tile;
                for (int r = 0; r < rows; ++r) {
                    const int row = row0 + r;
                    const float x = z[r], e = a.row_lse[static_cast<int64_t>(s.q0 + row / a.G) * a.H + h * a.G + row % a.G];
                    if (x != -INFINITY) w += exp2f(x - e);
                }
            }
            const int64_t at = (static_cast<int64_t>(b0 + i) * a.H_kv + h) * a.max_blocks * kBlock + pos;
            a.weights_out[at] = a.weights ? a.weights[at] + w : w;
        }
        if (a.B > kGroupedJoinThreads) __syncthreads();
    }
}

bool launch_grouped_join(const GroupedArgs& a, cudaStream_t s, int* launches) {
    if (!launch_kernel(true, grouped_join_kernel, dim3(a.ctas), dim3(kGroupedJoinThreads), 0, s, a)) return false;
    ++*launches;
    if (!a.weights_out) return true;
    if (!launch_kernel(true, grouped_weights_kernel, dim3(4 * a.ctas), dim3(kGroupedJoinThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
