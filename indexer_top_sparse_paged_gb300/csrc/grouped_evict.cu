// Eviction from the grouped-head cache by accumulated attention weight: one kernel selects the positions that every
// sequence and key head keeps, a second one moves their rows into the new blocks.
//
// The selection finds the weight of the last kept position by its bits, eight at a time from the top (a histogram of the
// positions that agree so far), and then writes the kept positions in order: all above it, and of those equal to it the
// first ones.
#include "grouped.cuh"

namespace dsa {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 256;

// Order of the weights as unsigned integers; NaN is the lowest, together with -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) { return ordered_bits(w != w ? -INFINITY : w); }

__global__ void __launch_bounds__(kSelectThreads) grouped_select_kernel(GroupedEvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t chosen, left;
    __shared__ int64_t warp_sums[kSelectThreads / 32];
    const int tid = threadIdx.x, b = blockIdx.x / a.H_kv, h = blockIdx.x - b * a.H_kv;
    griddep_launch_dependents();
    int n = a.seq_lens[b];
    if (n < 0 || n > a.max_blocks * kBlock) {
        if (tid == 0) atomicOr(a.err, DSA_FAULT_INDEX);
        n = 0;
    }
    const int64_t bh = blockIdx.x;
    const float* w = a.weights + bh * a.max_blocks * kBlock;
    int32_t* kept = a.kept + bh * a.keep;
    float* out = a.weights_out + bh * a.new_max_blocks * kBlock;
    const int m = min(n, a.keep);
    if (h == 0 && tid == 0) a.new_lens[b] = m;
    for (int i = m + tid; i < a.keep; i += kSelectThreads) kept[i] = -1;
    for (int i = m + tid; i < a.new_max_blocks * kBlock; i += kSelectThreads) out[i] = 0.0f;
    if (n <= a.keep) {
        for (int i = tid; i < n; i += kSelectThreads) {
            kept[i] = i;
            out[i] = w[i];
        }
        return;
    }
    const int lo = a.sink, hi = n - a.recent, want = a.keep - a.sink - a.recent;  // `want` of the positions lo .. hi - 1
    uint32_t prefix = 0;
    if (tid == 0) left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kSelectThreads) {
            const uint32_t k = weight_key(w[i]);
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t need = left, bin = 255;
            while (bin > 0 && hist[bin] < need) need -= hist[bin--];
            left = need;
            chosen = bin;
        }
        __syncthreads();
        prefix = prefix << 8 | chosen;
    }
    const uint32_t ties = left;  // of the positions whose weight is the last kept one's
    int64_t before = 0;          // kept so far, and ties so far in the upper half
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + tid;
        bool keep = false, tie = false;
        float x = 0.0f;
        if (i < n) {
            x = w[i];
            const uint32_t k = weight_key(x);
            keep = i < lo || i >= hi || k > prefix;
            tie = !keep && k == prefix;
        }
        int64_t all;
        const int64_t at = before + block_prefix<kSelectThreads>(tie ? 1ll << 32 : keep ? 1 : 0, &all, warp_sums);
        const uint32_t ties_before = static_cast<uint32_t>(at >> 32);
        const int slot = static_cast<int>(at & 0xFFFFFFFF) + static_cast<int>(min(ties_before, ties));
        if (keep || (tie && ties_before < ties)) {
            kept[slot] = i;
            out[slot] = x;
        }
        before += all;
    }
}

// One CTA per (new block, sequence and head, keys or values).
__global__ void __launch_bounds__(kMoveThreads) grouped_move_kernel(GroupedEvictArgs a) {
    __shared__ int64_t src_row[kBlock];
    __shared__ float src_scale[kBlock];
    __shared__ float red[kMoveThreads / 32];
    const int tid = threadIdx.x, blocks = (a.keep + kBlock - 1) / kBlock;
    const int bh_in = blockIdx.x / blocks, j = blockIdx.x - bh_in * blocks, b = bh_in / a.H_kv, h = bh_in - b * a.H_kv;
    const bool value = blockIdx.y;
    const int d = value ? a.d_v : a.d_qk, groups = d / 16;
    uint8_t* cache = value ? a.v : a.k;
    float* scales = value ? a.v_scale : a.k_scale;
    int n = a.seq_lens[b];
    if (n < 0 || n > a.max_blocks * kBlock) n = 0;
    const int m = min(n, a.keep), rows = min(kBlock, m - j * kBlock);
    if (rows <= 0) return;
    const int to = a.new_table[static_cast<int64_t>(b) * a.new_max_blocks + j];
    const bool to_ok = to >= 0 && to < a.num_blocks;
    if (!to_ok && tid == 0) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
    griddep_wait();
    if (tid < rows) {
        const int i = a.kept[(static_cast<int64_t>(b) * a.H_kv + h) * a.keep + j * kBlock + tid];
        const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + i / kBlock];
        const bool ok = blk >= 0 && blk < a.num_blocks;
        if (!ok) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
        const int64_t bh = static_cast<int64_t>(blk) * a.H_kv + h;
        src_row[tid] = ok ? bh * kBlock + i % kBlock : -1;
        src_scale[tid] = ok ? scales[bh] : 0.0f;
    }
    __syncthreads();
    if (!to_ok) return;
    const int64_t to_bh = static_cast<int64_t>(to) * a.H_kv + h;
    uint4* dst = reinterpret_cast<uint4*>(cache + to_bh * kBlock * d);
    if (n <= a.keep) {  // whole: copied as it is
        if (src_row[0] == to_bh * kBlock) return;
        for (int i = tid; i < rows * groups; i += kMoveThreads) {
            const int r = i / groups;
            if (src_row[r] >= 0) dst[i] = reinterpret_cast<const uint4*>(cache + src_row[r] * d)[i - r * groups];
        }
        if (tid == 0 && src_row[0] >= 0) scales[to_bh] = src_scale[0];
        return;
    }
    float amax = 0.0f;
    for (int i = tid; i < rows * groups; i += kMoveThreads) {
        const int r = i / groups;
        if (src_row[r] < 0) continue;
        float x[16];
        e4m3x16_values(reinterpret_cast<const uint4*>(cache + src_row[r] * d)[i - r * groups], x);
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e] * src_scale[r]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
    for (int i = tid; i < rows * groups; i += kMoveThreads) {
        const int r = i / groups;
        if (src_row[r] < 0) continue;
        float x[16];
        e4m3x16_values(reinterpret_cast<const uint4*>(cache + src_row[r] * d)[i - r * groups], x);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) y[f] = x[4 * e + f] * src_scale[r] / scale;
            w[e] = e4m3x4_codes(y[0], y[1], y[2], y[3]);
        }
        dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tid == 0) scales[to_bh] = scale;
}

bool launch_grouped_evict(const GroupedEvictArgs& a, cudaStream_t s, int* launches) {
    const unsigned heads = static_cast<unsigned>(a.B) * a.H_kv;
    if (!launch_kernel(false, grouped_select_kernel, dim3(heads), dim3(kSelectThreads), 0, s, a)) return false;
    ++*launches;
    const dim3 grid(heads * ((a.keep + kBlock - 1) / kBlock), 2);
    if (!launch_kernel(true, grouped_move_kernel, grid, dim3(kMoveThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
