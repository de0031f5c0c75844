// Append to the grouped-head cache: new keys and values as e4m3 codes against one scale per 64-token block and head.
//
// One CTA per (block that gets new tokens, head, keys or values): the new rows' largest magnitude gives the block's
// scale (no smaller than the one its earlier tokens have), then the rows are written as codes; where the scale has
// grown, the earlier codes are rounded anew against it. So a scale only ever grows while a block fills, and codes whose
// scale stays are not touched.
#include "grouped.cuh"

namespace dsa {

constexpr int kGroupedAppendThreads = 256;

// 16 elements of a new row.
__device__ __forceinline__ void load16(const float* p, float2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        x[2 * i] = make_float2(v.x, v.y);
        x[2 * i + 1] = make_float2(v.z, v.w);
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
}

struct AppendSeq {
    int row0, n;       // the sequence's new rows
    int first;         // position of the first one that is written
    int skipped;       // rows before it, whose positions are negative
    int blocks;        // blocks they reach into
};

__device__ __forceinline__ AppendSeq append_seq(const GroupedAppendArgs& a, int b, bool report) {
    AppendSeq s{b, 1, 0, 0, 0};
    if (a.cu) {
        s.row0 = a.cu[b];
        s.n = a.cu[b + 1] - s.row0;
    }
    const int len = a.seq_lens[b];
    if (s.row0 < 0 || s.row0 > a.T || s.n < 0 || s.n > a.T - s.row0 || len < 0 || len > a.max_blocks * kBlock) {
        if (report) atomicOr(a.err, DSA_FAULT_INDEX);
        return AppendSeq{0, 0, 0, 0, 0};
    }
    if (s.n > len) {
        if (report) atomicOr(a.err, DSA_FAULT_INDEX);
        s.skipped = s.n - len;
    }
    s.first = len - s.n + s.skipped;
    const int written = s.n - s.skipped;
    s.blocks = written ? (s.first + written - 1) / kBlock - s.first / kBlock + 1 : 0;
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kGroupedAppendThreads) grouped_append_kernel(GroupedAppendArgs a) {
    __shared__ int64_t warp_sums[kGroupedAppendThreads / 32], found[2];
    __shared__ float red[kGroupedAppendThreads / 32];
    const int tid = threadIdx.x, h = blockIdx.y >> 1;
    const bool value = blockIdx.y & 1;
    int64_t total, base;
    int b;
    find_place<kGroupedAppendThreads>(
        a.B, [&](int i) { return static_cast<int64_t>(append_seq(a, i, blockIdx.x == 0 && blockIdx.y == 0).blocks); },
        [](int64_t) { return static_cast<int64_t>(blockIdx.x); }, &total, &b, &base, warp_sums, found);
    if (b < 0) return;
    const AppendSeq s = append_seq(a, b, false);
    const int lb = s.first / kBlock + static_cast<int>(blockIdx.x - base);
    const int p0 = max(s.first, lb * kBlock), p1 = min(s.first + s.n - s.skipped, (lb + 1) * kBlock);  // new positions here
    const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + lb];
    if (blk < 0 || blk >= a.num_blocks) {
        if (tid == 0) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
        return;
    }
    const int d = value ? a.d_v : a.d_qk, groups = d / 16, slot0 = p0 - lb * kBlock, n = (p1 - p0) * groups;
    const int64_t st = value ? a.v_stride_t : a.k_stride_t, sh = value ? a.v_stride_h : a.k_stride_h;
    const T* x = static_cast<const T*>(value ? a.v_new : a.k_new) + (s.row0 + s.skipped + p0 - s.first) * st + h * sh;
    const int64_t bh = static_cast<int64_t>(blk) * a.H_kv + h;
    uint4* codes = reinterpret_cast<uint4*>((value ? a.v : a.k) + bh * kBlock * d);
    float* scale_at = (value ? a.v_scale : a.k_scale) + bh;
    float amax = 0.0f;
    for (int i = tid; i < n; i += kGroupedAppendThreads) {
        float2 y[8];
        load16(x + (i / groups) * st + (i % groups) * 16, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(y[j].x), fabsf(y[j].y)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    const float old = slot0 ? *scale_at : 0.0f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kGroupedAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float scale = slot0 ? fmaxf(old, amax / 448.0f) : unit_scale(amax);
    for (int i = tid; i < n; i += kGroupedAppendThreads) {
        float2 y[8];
        load16(x + (i / groups) * st + (i % groups) * 16, y);
        codes[slot0 * groups + i] = codes16(y, scale);
    }
    if (slot0 && scale > old) {
        for (int i = tid; i < slot0 * groups; i += kGroupedAppendThreads) {
            codes[i] = requantise16(codes[i], old, scale, 1.0f / scale);
        }
    }
    if (tid == 0) *scale_at = scale;
}

bool launch_grouped_append(const GroupedAppendArgs& a, cudaStream_t s, int* launches) {
    if (a.T == 0) return true;
    // a sequence's rows reach into (n + 126) / 64 blocks at most, and into n
    const int64_t most = static_cast<int64_t>(a.T) / kBlock + 2ll * a.B;
    const dim3 grid(static_cast<unsigned>(most < a.T ? most : a.T), 2 * a.H_kv);
    auto* kernel = a.type == DSA_F32 ? grouped_append_kernel<float> : grouped_append_kernel<__nv_bfloat16>;
    if (!launch_kernel(false, kernel, grid, dim3(kGroupedAppendThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
