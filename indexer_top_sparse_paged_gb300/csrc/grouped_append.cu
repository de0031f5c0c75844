// Append to the grouped-head cache: new keys and values as e4m3 codes against one scale per 64-token block and head.
//
// One CTA per (block that gets new tokens, head, keys or values): the new rows' largest magnitude gives the block's
// scale (no smaller than the one its earlier tokens have), then the rows are written as codes; where the scale has
// grown, the earlier codes are rounded anew against it. So a scale only ever grows while a block fills (but for that of
// nothing but zeros), and codes whose scale stays are not touched.
//
// One row a sequence: latency bounds it (32 sequences, 8 heads of 128 and 128: 5.2 us of kernel time, 17 - 18 us a call in a
// stream), which is why a CTA reads its rows once, into registers, and keeps the next on their way. A prompt's many rows: the
// instructions of rounding (2 x 4096 tokens: 17 us; its 50 MB take 7.4; 65% of the issue slots busy; every code is converted
// twice, so that a value near the middle of two codes is noticed).
#include "grouped.cuh"

namespace dsa {

constexpr int kGroupedAppendThreads = 256;

// 16 elements of a new row, as they are loaded; top: the bits of their largest magnitude (NaN above all).
template <typename T>
struct Elements16;
template <>
struct Elements16<float> {
    float4 v[4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
    }
    __device__ __forceinline__ void values(float2 (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = make_float2(v[i].x, v[i].y);
            x[2 * i + 1] = make_float2(v[i].z, v[i].w);
        }
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = max(t, max(max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu),
                           max(__float_as_uint(v[i].z) & 0x7FFFFFFFu, __float_as_uint(v[i].w) & 0x7FFFFFFFu)));
        return t;
    }
};
template <>
struct Elements16<__nv_bfloat16> {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v[0] = reinterpret_cast<const uint4*>(p)[0];
        v[1] = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void values(float2 (&x)[8]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = 0x7FFF7FFFu;
        const uint32_t a = __vmaxu2(__vmaxu2(v[0].x & m, v[0].y & m), __vmaxu2(v[0].z & m, v[0].w & m));
        const uint32_t b = __vmaxu2(__vmaxu2(v[1].x & m, v[1].y & m), __vmaxu2(v[1].z & m, v[1].w & m));
        const uint32_t t = __vmaxu2(a, b);
        return max(t << 16, t & 0xFFFF0000u);
    }
};

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

// kPieces: pieces of 16 elements a thread holds, 64 rows of a head together. Two of bf16 fit 64 registers, so 4 CTAs an SM (32
// single tokens 5.2 us; with 66 registers 6.5).
template <typename T, int kPieces>
__global__ void __launch_bounds__(kGroupedAppendThreads, sizeof(T) * kPieces == 4 ? 4 : 1) grouped_append_kernel(GroupedAppendArgs a, uint32_t k_magic, uint32_t v_magic) {
    __shared__ int64_t warp_sums[kGroupedAppendThreads / 32], found[2];
    __shared__ float red[2][kGroupedAppendThreads / 32];
    const int tid = threadIdx.x;
    // the block: unit blockIdx.x of the line of blocks that the sequences' new rows reach into
    int64_t total, base;
    int b;
    const bool report = blockIdx.x == 0 && blockIdx.y == 0;
    if (!a.cu) {
        b = blockIdx.x, base = b;  // one row, one block for each
        if (append_seq(a, b, blockIdx.y == 0 && tid == 0).blocks == 0) return;
    } else if (a.B <= 32) {  // every warp finds it for itself
        const int lane = tid & 31, blocks = lane < a.B ? append_seq(a, lane, report && tid < 32).blocks : 0;
        int x = blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        const int at = blockIdx.x;
        b = __ffs(__ballot_sync(0xFFFFFFFFu, at >= x - blocks && at < x)) - 1;
        if (b < 0) return;
        base = __shfl_sync(0xFFFFFFFFu, x - blocks, b);
    } else {
        find_place<kGroupedAppendThreads>(a.B, [&](int i) { return static_cast<int64_t>(append_seq(a, i, report).blocks); },
                                          [](int64_t) { return static_cast<int64_t>(blockIdx.x); }, &total, &b, &base, warp_sums, found);
        if (b < 0) return;
    }
    const AppendSeq s = append_seq(a, b, false);
    const int lb = s.first / kBlock + static_cast<int>(blockIdx.x - base);
    const int p0 = max(s.first, lb * kBlock), p1 = min(s.first + s.n - s.skipped, (lb + 1) * kBlock);  // new positions here
    const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + lb];
    if (blk < 0 || blk >= a.num_blocks) {
        if (tid == 0) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
        return;
    }
    const int slot0 = p0 - lb * kBlock;
    // its heads, keys and values in turn, the next one's rows on their way while this one's are written
    Elements16<T> next[kPieces];
    float next_old = 0.0f;
    auto load = [&](int y) {
        if (y >= 2 * a.H_kv) return;
        const bool value = y & 1;
        const int groups = (value ? a.d_v : a.d_qk) / 16, n = (p1 - p0) * groups;
        const int64_t st = value ? a.v_stride_t : a.k_stride_t, sh = value ? a.v_stride_h : a.k_stride_h;
        const T* x = static_cast<const T*>(value ? a.v_new : a.k_new) + (s.row0 + s.skipped + p0 - s.first) * st + (y >> 1) * sh;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int i = tid + p * kGroupedAppendThreads;
            const int r = groups == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), value ? v_magic : k_magic));
            if (i < n) next[p].load(x + r * st + (i - r * groups) * 16);
        }
        next_old = slot0 ? (value ? a.v_scale : a.k_scale)[static_cast<int64_t>(blk) * a.H_kv + (y >> 1)] : 0.0f;
    };
    load(blockIdx.y);
    for (int y = blockIdx.y, turn = 0; y < 2 * a.H_kv; y += gridDim.y, turn ^= 1) {
        const bool value = y & 1;
        const int d = value ? a.d_v : a.d_qk, groups = d / 16, n = (p1 - p0) * groups;
        const int64_t bh = static_cast<int64_t>(blk) * a.H_kv + (y >> 1);
        uint4* codes = reinterpret_cast<uint4*>((value ? a.v : a.k) + bh * kBlock * d);
        Elements16<T> piece[kPieces];
        const float old = next_old;
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            piece[p] = next[p];
            if (tid + p * kGroupedAppendThreads < n) top = max(top, piece[p].top());
        }
        load(y + gridDim.y);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((tid & 31) == 0) red[turn][tid >> 5] = __uint_as_float(top);
        __syncthreads();
        float amax = 0.0f;  // (fmaxf passes NaN over)
#pragma unroll
        for (int w = 0; w < kGroupedAppendThreads / 32; ++w) amax = fmaxf(amax, red[turn][w]);
        float scale = slot0 ? fmaxf(old, amax / 448.0f) : unit_scale(amax);
        if (slot0 && old == 1.0f && amax < 448.0f) {  // (the same for all threads)
            // Tokens of zeros leave the scale 1, against which smaller values would lose their bits: they count as none.
            uint32_t held = 0;
#pragma unroll 1
            for (int i = tid; i < slot0 * groups; i += kGroupedAppendThreads) {
                const uint4 c = codes[i];
                held |= (c.x | c.y | c.z | c.w) & 0x7F7F7F7Fu;
            }
            if (!__syncthreads_or(held != 0)) scale = unit_scale(amax);
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int i = tid + p * kGroupedAppendThreads;
            if (i >= n) break;
            float2 v[8];
            piece[p].values(v);
            codes[slot0 * groups + i] = codes16(v, scale);
        }
        if (slot0 && scale > old) {
            for (int i = tid; i < slot0 * groups; i += kGroupedAppendThreads) codes[i] = requantise16(codes[i], old, scale);
        }
        if (tid == 0) (value ? a.v_scale : a.k_scale)[bh] = scale;
    }
}

template <typename T>
static bool launch_typed(const GroupedAppendArgs& a, cudaStream_t s) {
    // a sequence's rows reach into (n + 126) / 64 blocks at most, and into n
    const int64_t most = static_cast<int64_t>(a.T) / kBlock + 2ll * a.B, units = most < a.T ? most : a.T;
    // one turn of six CTAs an SM, each with the same number of heads' keys and values, or a CTA for every one
    const int64_t turns = (2ll * a.H_kv * units + 6 * device_sm_count() - 1) / (6 * device_sm_count());
    const int64_t heads = (2 * a.H_kv + turns - 1) / turns;
    const int most_groups = (a.d_qk > a.d_v ? a.d_qk : a.d_v) / 16;
    const uint32_t gk = a.d_qk / 16, gv = a.d_v / 16;
    // umulhi(i, ceil(2^32 / groups)) = i / groups for i < 2^32 / groups
    const uint32_t k_magic = static_cast<uint32_t>(((1ll << 32) + gk - 1) / gk), v_magic = static_cast<uint32_t>(((1ll << 32) + gv - 1) / gv);
    auto* kernel = most_groups <= 8 ? grouped_append_kernel<T, 2> : grouped_append_kernel<T, 4>;
    return launch_kernel(false, kernel, dim3(static_cast<unsigned>(units), static_cast<unsigned>(heads)), dim3(kGroupedAppendThreads), 0, s, a,
                         k_magic, v_magic);
}

bool launch_grouped_append(const GroupedAppendArgs& a, cudaStream_t s, int* launches) {
    if (a.T == 0) return true;
    if (!(a.type == DSA_F32 ? launch_typed<float>(a, s) : launch_typed<__nv_bfloat16>(a, s))) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
