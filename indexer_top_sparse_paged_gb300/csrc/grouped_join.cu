// After the attention over the grouped-head cache: the rows of items that were cut are joined from their partials, rows
// of sequences without positions are written, and, where they are wanted, the positions' weights are summed from the
// logits.
#include "grouped.cuh"

namespace dsa {

constexpr int kGroupedJoinThreads = 256;
constexpr int kJoinBatch = 8;  // partials a thread has in flight

__device__ __forceinline__ void store_row4(void* out, bool f32, int64_t at, float4 x) {
    if (f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = x;
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
}

// CTA (c, y): the item that was first cut where share c begins, four columns of a row a thread; and every a.ctas-th
// sequence's rows, if it has no positions.
__global__ void __launch_bounds__(kGroupedJoinThreads) grouped_join_kernel(GroupedArgs a) {
    const int c = blockIdx.x, step = gridDim.y * kGroupedJoinThreads, first = blockIdx.y * kGroupedJoinThreads + threadIdx.x;
    const int quads = a.d_v / 4;
    const bool f32 = a.type == DSA_F32;
    griddep_launch_dependents();
    for (int b = c; b < a.B; b += a.ctas) {  // (lengths are inputs: no wait)
        const GroupedSeq s = grouped_seq(a, b, false);
        if (s.tiles) continue;
        for (int64_t i = first; i < static_cast<int64_t>(s.n) * a.H * quads; i += step) {
            const int64_t row = static_cast<int64_t>(s.q0) * a.H + i / quads;
            store_row4(a.out, f32, row * a.d_v + i % quads * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            if (i % quads == 0) {
                if (a.lse) a.lse[row] = -INFINITY;
                if (a.weights_out) a.row_lse[row] = -INFINITY;
            }
        }
    }
    griddep_wait();
    const GroupedCut cut = a.cuts[c];
    for (int i = first; i < cut.rows * quads; i += step) {
        const int r = i / quads, e = 4 * (i - r * quads);
        float top = -INFINITY, sum = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p0 = 0; p0 < cut.parts; p0 += kJoinBatch) {
            float2 ml[kJoinBatch];
            float4 x[kJoinBatch];
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const int p = p0 + k;
                if (p >= cut.parts) {
                    ml[k] = make_float2(-INFINITY, 0.0f);
                    x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    continue;
                }
                const int64_t slot = static_cast<int64_t>(p ? 2 * (cut.slot0 / 2 + p) : cut.slot0) * a.row_tile + r;
                ml[k] = __ldcg(a.part_ml + slot);
                x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot * a.d_v + e));
            }
            float most = top;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) most = fmaxf(most, ml[k].x);
            const float ref = most == -INFINITY ? 0.0f : most, old = exp2f(top - ref);
            sum *= old;
            o.x *= old, o.y *= old, o.z *= old, o.w *= old;
            top = most;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const float f = exp2f(ml[k].x - ref);
                sum = fmaf(f, ml[k].y, sum);
                o.x = fmaf(f, x[k].x, o.x), o.y = fmaf(f, x[k].y, o.y), o.z = fmaf(f, x[k].z, o.z), o.w = fmaf(f, x[k].w, o.w);
            }
        }
        const int row = cut.row0 + r;
        const int64_t at = static_cast<int64_t>(cut.q0 + row / a.G) * a.H + cut.h * a.G + row % a.G;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        store_row4(a.out, f32, at * a.d_v + e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (e == 0) {
            const float lse2 = sum == 0.0f ? -INFINITY : top + log2f(sum);
            if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
            if (a.weights_out) a.row_lse[at] = lse2;
        }
    }
}

// The sequences b0 .. b0 + 255 in shared memory, with the position tiles of key heads and the attention's tiles that stand
// before each.
struct GroupedChunk {
    GroupedSeq seq[kGroupedJoinThreads];
    int64_t units[kGroupedJoinThreads + 1], tiles[kGroupedJoinThreads];
    int64_t warp_sums[kGroupedJoinThreads / 32];
};

__device__ __forceinline__ int64_t chunk_load(const GroupedArgs& a, GroupedChunk& c, int b0, int64_t tiles_before) {
    const int tid = threadIdx.x, b = b0 + tid;
    GroupedSeq s{};
    if (b < a.B) s = grouped_seq(a, b, false);
    int64_t all_units, all_tiles;
    const int64_t u = block_prefix<kGroupedJoinThreads>(static_cast<int64_t>(s.tiles) * a.H_kv, &all_units, c.warp_sums);
    const int64_t t = block_prefix<kGroupedJoinThreads>(grouped_seq_tiles(a, s), &all_tiles, c.warp_sums);
    c.seq[tid] = s;
    c.units[tid] = u;
    c.tiles[tid] = tiles_before + t;
    if (tid == 0) c.units[kGroupedJoinThreads] = all_units;
    __syncthreads();
    return all_tiles;
}

// weights_out = weights + the sum over the rows of 2^(z - lse): a warp for each position tile of a key head, four positions
// a lane, so that a row's 128 logits are four coalesced loads.
__global__ void __launch_bounds__(kGroupedJoinThreads) grouped_weights_kernel(GroupedArgs a) {
    __shared__ GroupedChunk c;
    const int lane = threadIdx.x & 31, warps = gridDim.x * (kGroupedJoinThreads / 32);
    int64_t before = 0;
    bool waited = false;
    for (int b0 = 0; b0 < a.B; b0 += kGroupedJoinThreads) {
        if (b0) __syncthreads();  // these sequences take the others' place
        before += chunk_load(a, c, b0, before);
        if (!waited) griddep_wait();
        waited = true;
        const int64_t n = c.units[kGroupedJoinThreads];
        for (int64_t u = blockIdx.x + static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x; u < n; u += warps) {
            int i = 0, hi = min(kGroupedJoinThreads, a.B - b0) - 1;  // the last sequence whose first unit is at or before u
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

bool launch_grouped_join(const GroupedArgs& a, cudaStream_t s, int* launches) {
    const int runs = (a.row_tile * (a.d_v / 4) + kGroupedJoinThreads - 1) / kGroupedJoinThreads;
    if (!launch_kernel(true, grouped_join_kernel, dim3(a.ctas, runs), dim3(kGroupedJoinThreads), 0, s, a)) return false;
    ++*launches;
    if (!a.weights_out) return true;
    if (!launch_kernel(true, grouped_weights_kernel, dim3(4 * a.ctas), dim3(kGroupedJoinThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
