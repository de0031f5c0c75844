// Eviction from the grouped-head cache by accumulated attention weight: one kernel selects the positions that every
// sequence and key head keeps, a second one moves their rows into the new blocks.
//
// Selection: a cluster of CTAs for each (sequence, head), each with a run of its positions. The weight of the last kept
// position is found by its bits, eleven at a time from the top: every CTA counts the positions that agree so far in a
// histogram of the next bits, reads the others' through distributed shared memory, and all find the same bin. Keys stay
// in shared memory from the first pass on, as far as they fit (else they are read again). Then every warp counts what it
// keeps of its run -- all above the last weight, and of those equal to it the first ones -- and writes it in order.
// Latency and shared-memory atomics bound it (five cluster barriers; the weights are 4 MB): 128K positions for each of 8
// heads take 26 us, 8 x 8 heads of 16K 17. Clusters of 8 CTAs at most: of 16, which may not be spread over as many SMs, the
// former took 116 us. Each CTA sums a slice of the bins for all (33 us when every CTA summed them all).
//
// Move: a CTA for each (new block, sequence and head), keys and values together since they share the chain kept position
// -> block -> row. A thread keeps its 16-byte pieces in registers between the largest magnitude (of the codes' 7 low
// bits, which order as the values do) and the rounding against the new scale. 8 sequences cut from 16K to 8K, 8 heads of 128 and
// 128: 81 us (237 MB; the bytes take 41). Half of what is above them is the rounding's instructions, 65% of the issue slots
// busy (with a division for each code it took 128), the other half the copy itself: without rounding it takes 61, with two
// barriers and a chain of dependent loads between a block's loads and its stores. Five CTAs an SM at 48 registers, of which
// some spill (56 bytes of stores, 84 of loads a thread in the form for multiples of 32; forms of more pieces: three CTAs, 80
// registers).
//
// The quotient is the formula's, in fp32. Rows from the source block that holds the new block's largest value have the ratio
// 448 / (its code): where that code is 256, 320 or 384, times a power of two, one mantissa in eight lies exactly on the middle
// of two codes, and the roundings of scale and product decide. 0.1 - 0.2% of all codes come out one step off what 64 bits
// would give.
#include "grouped.cuh"

namespace dsa {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
static_assert(kSelectWarps == 32, "a lane for every warp");
constexpr int kSelectBins = 2048;
constexpr int kSelectMaxCluster = 8;
constexpr int kSelectKeys = 40960;  // keys that shared memory holds, beside the histograms
constexpr int kSelectBatch = 8;     // of a thread's, in flight
constexpr int kSelectWords = 8;     // 32 positions each, that a warp marks at a time
constexpr int kMoveThreads = 256;

// Order of the weights as unsigned integers; NaN is the lowest, together with -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) { return ordered_bits(w != w ? -INFINITY : w); }

// The weight of a key that is not -infinity's (-0 comes back as 0).
__device__ __forceinline__ float key_weight(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kLowestKey = 0x007FFFFFu;  // that of -infinity and of NaN

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

struct SelectShared {
    uint32_t hist[3][kSelectBins];
    uint32_t slice[3][kSelectBins / 2];  // of every CTA's histogram, the bins that this CTA sums up
    uint32_t slice_total[3];
    uint32_t counts[2];  // of this CTA's run: kept above the last weight (or by place), equal to it
    uint32_t warp_counts[kSelectWarps][2];
    uint32_t warp_sums[kSelectWarps];
    uint32_t bin, need;
};

// Inclusive sums over the block's threads; `all` is their total.
__device__ __forceinline__ uint32_t block_sums(SelectShared& S, uint32_t v, uint32_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) S.warp_sums[warp] = x;
    __syncthreads();
    const uint32_t w = S.warp_sums[lane];
    *all = __reduce_add_sync(0xFFFFFFFFu, w);
    return x + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0);
}

// The bin (from the top) that holds the `need`-th position of the cluster's histograms, and the rank within it. CTA r sums
// up the r-th slice of the bins over all CTAs; then all read the slices' totals, and the bins of the one slice that matters.
__device__ __forceinline__ void find_bin(SelectShared& S, int pass, int ctas, int rank, uint32_t need) {
    const int tid = threadIdx.x, lane = tid & 31, width = kSelectBins / ctas;  // (256 at least)
    // slice r: the bins down from kSelectBins - 1 - r * width
    uint32_t mine = 0, all = 0;
    if (ctas > 1) {
        if (tid < width) {
            const uint32_t at = smem_u32(&S.hist[pass][kSelectBins - 1 - rank * width - tid]);
            uint32_t theirs[kSelectMaxCluster];  // (all on their way at once)
#pragma unroll
            for (int c = 0; c < kSelectMaxCluster; ++c) theirs[c] = c < ctas ? ld_cluster_u32(mapa_shared(at, c)) : 0;
#pragma unroll
            for (int c = 0; c < kSelectMaxCluster; ++c) mine += theirs[c];
            S.slice[pass][tid] = mine;
        }
        block_sums(S, mine, &all);
        if (tid == 0) S.slice_total[pass] = all;
        cluster_sync_all();
        uint32_t t = lane < ctas ? ld_cluster_u32(mapa_shared(smem_u32(&S.slice_total[pass]), lane)) : 0, x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, x >= need && x - t < need)) - 1;  // (there is one)
        need -= __shfl_sync(0xFFFFFFFFu, x - t, from);
        mine = tid < width ? ld_cluster_u32(mapa_shared(smem_u32(&S.slice[pass][tid]), from)) : 0;
        const uint32_t sum = block_sums(S, mine, &all);
        if (sum >= need && sum - mine < need) {
            S.bin = kSelectBins - 1 - from * width - tid;
            S.need = need - (sum - mine);
        }
    } else {  // two bins a thread
        const int top = kSelectBins - 1 - 2 * tid;
        const uint32_t n0 = S.hist[pass][top], n1 = S.hist[pass][top - 1];
        const uint32_t sum = block_sums(S, n0 + n1, &all), before = sum - n0 - n1;
        if (sum >= need && before < need) {
            const bool first = before + n0 >= need;
            S.bin = first ? top : top - 1;
            S.need = need - before - (first ? 0 : n0);
        }
    }
    __syncthreads();
}
static_assert(kSelectBins == 2 * kSelectThreads, "two bins a thread");

// One CTA's part of a row's selection. kCached: the keys of its run [r0, r1) fit shared memory.
template <bool kCached>
__device__ __forceinline__ void select_run(const GroupedEvictArgs& a, SelectShared& S, uint32_t* keys, const float* w, int32_t* kept, float* out,
                                           int n, int r0, int r1, int ctas, int rank) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lo = a.sink, hi = n - a.recent;  // the positions to choose from
    const uint32_t want = a.keep - a.sink - a.recent;
    auto key_at = [&](int i) { return kCached ? keys[i - r0] : weight_key(w[i]); };
    uint32_t prefix = 0xFFFFFFFFu, need = 0;  // above every key: with none wanted, positions are kept by their place alone
    if (want > 0) {
        for (int i = tid; i < 3 * kSelectBins; i += kSelectThreads) S.hist[0][i] = 0;
        __syncthreads();
        for (int i0 = r0 + tid; i0 < r1; i0 += kSelectBatch * kSelectThreads) {
            float x[kSelectBatch];
#pragma unroll
            for (int e = 0; e < kSelectBatch; ++e) x[e] = i0 + e * kSelectThreads < r1 ? w[i0 + e * kSelectThreads] : 0.0f;
#pragma unroll
            for (int e = 0; e < kSelectBatch; ++e) {
                const int i = i0 + e * kSelectThreads;
                const uint32_t k = weight_key(x[e]);
                if (kCached && i < r1) keys[i - r0] = k;
                if (i >= lo && i < min(hi, r1)) atomicAdd(&S.hist[0][k >> 21], 1u);
            }
        }
        if (ctas > 1) cluster_sync_all();
        else __syncthreads();
        find_bin(S, 0, ctas, rank, want);
        prefix = S.bin, need = S.need;
        // the next bits of the positions that agree so far
        const int from = max(r0, lo), to = min(r1, hi);
        auto next_pass = [&](int pass, int above, int shift, uint32_t mask) {
            for (int i0 = from + tid; i0 < to; i0 += kSelectBatch * kSelectThreads) {
                uint32_t k[kSelectBatch];
#pragma unroll
                for (int e = 0; e < kSelectBatch; ++e) k[e] = i0 + e * kSelectThreads < to ? key_at(i0 + e * kSelectThreads) : 0;
#pragma unroll
                for (int e = 0; e < kSelectBatch; ++e)
                    if (i0 + e * kSelectThreads < to && k[e] >> above == prefix) atomicAdd(&S.hist[pass][(k[e] >> shift) & mask], 1u);
            }
            if (ctas > 1) cluster_sync_all();
            else __syncthreads();
            find_bin(S, pass, ctas, rank, need);
        };
        next_pass(1, 21, 10, 2047);
        prefix = prefix << 11 | S.bin, need = S.need;
        next_pass(2, 10, 0, 1023);
        prefix = prefix << 10 | S.bin, need = S.need;  // the last kept weight's key; how many of its equals are kept
    }
    // every warp's part of the run: what it keeps, and what equals the last weight, as bits
    const int part = ((r1 - r0 + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int p0 = min(r1, r0 + warp * part), p1 = min(r1, p0 + part);
    uint32_t key[kSelectWords], keeps[kSelectWords], ties[kSelectWords];  // of kSelectWords times 32 positions
    auto mark = [&](int i0) {
        const bool inside = want > 0 && i0 >= lo && min(i0 + 32 * kSelectWords, p1) <= hi;  // (all by their weights)
#pragma unroll
        for (int e = 0; e < kSelectWords; ++e) {
            const int i = i0 + 32 * e + lane;
            key[e] = i < p1 && want > 0 ? key_at(i) : 0;
        }
#pragma unroll
        for (int e = 0; e < kSelectWords; ++e) {
            const int i = i0 + 32 * e + lane;
            const bool held = !inside && (i < lo || i >= hi);
            keeps[e] = __ballot_sync(0xFFFFFFFFu, i < p1 && (held || key[e] > prefix));
            ties[e] = __ballot_sync(0xFFFFFFFFu, i < p1 && !held && key[e] == prefix);
        }
    };
    uint32_t above = 0, equal = 0;
    for (int i0 = p0; i0 < p1; i0 += 32 * kSelectWords) {
        mark(i0);
#pragma unroll
        for (int e = 0; e < kSelectWords; ++e) above += __popc(keeps[e]), equal += __popc(ties[e]);
    }
    if (lane == 0) S.warp_counts[warp][0] = above, S.warp_counts[warp][1] = equal;
    __syncthreads();
    const uint32_t warp_above = S.warp_counts[lane][0], warp_equal = S.warp_counts[lane][1];
    if (warp == 0) {
        const uint32_t all_above = __reduce_add_sync(0xFFFFFFFFu, warp_above), all_equal = __reduce_add_sync(0xFFFFFFFFu, warp_equal);
        if (lane == 0) S.counts[0] = all_above, S.counts[1] = all_equal;
    }
    uint32_t cta_above = 0, cta_equal = 0;
    if (ctas > 1) {
        cluster_sync_all();
        const uint32_t at = mapa_shared(smem_u32(S.counts), lane < rank ? lane : 0);  // lane c: the counts of CTA c
        cta_above = lane < rank ? ld_cluster_u32(at) : 0, cta_equal = lane < rank ? ld_cluster_u32(at + 4) : 0;
    }
    uint32_t above_before = __reduce_add_sync(0xFFFFFFFFu, cta_above + (lane < warp ? warp_above : 0));
    uint32_t equal_before = __reduce_add_sync(0xFFFFFFFFu, cta_equal + (lane < warp ? warp_equal : 0));
    const uint32_t below = (1u << lane) - 1;
    for (int i0 = p0; i0 < p1; i0 += 32 * kSelectWords) {
        if (part > 32 * kSelectWords) mark(i0);
#pragma unroll
        for (int e = 0; e < kSelectWords; ++e) {
            const uint32_t t = equal_before + __popc(ties[e] & below);
            if ((keeps[e] >> lane & 1) || ((ties[e] >> lane & 1) && t < need)) {
                const uint32_t slot = above_before + __popc(keeps[e] & below) + min(t, need);
                const int i = i0 + 32 * e + lane;
                kept[slot] = i;
                out[slot] = want > 0 && key[e] != kLowestKey ? key_weight(key[e]) : w[i];
            }
            above_before += __popc(keeps[e]);
            equal_before += __popc(ties[e]);
        }
    }
    if (ctas > 1) cluster_sync_all();  // no CTA's shared memory goes while another may read it
}

__global__ void __launch_bounds__(kSelectThreads) grouped_select_kernel(GroupedEvictArgs a, int ctas, int cached) {
    extern __shared__ uint32_t keys[];  // [cached]
    __shared__ SelectShared S;
    const int tid = threadIdx.x;
    const int bh = blockIdx.x / ctas, rank = blockIdx.x - bh * ctas, b = bh / a.H_kv;
    griddep_launch_dependents();
    int n = a.seq_lens[b];
    if (n < 0 || n > a.max_blocks * kBlock) {
        if (tid == 0) atomicOr(a.err, DSA_FAULT_INDEX);
        n = 0;
    }
    const float* w = a.weights + static_cast<int64_t>(bh) * a.max_blocks * kBlock;
    int32_t* kept = a.kept + static_cast<int64_t>(bh) * a.keep;
    float* out = a.weights_out + static_cast<int64_t>(bh) * a.new_max_blocks * kBlock;
    const int m = min(n, a.keep), all = tid + rank * kSelectThreads, step = ctas * kSelectThreads;
    if (bh - b * a.H_kv == 0 && rank == 0 && tid == 0) a.new_lens[b] = m;
    for (int i = m + all; i < a.keep; i += step) kept[i] = -1;
    for (int64_t i = m + all; i < static_cast<int64_t>(a.new_max_blocks) * kBlock; i += step) out[i] = 0.0f;
    if (n <= a.keep) {  // (for all CTAs of the cluster)
        for (int i = all; i < n; i += step) {
            kept[i] = i;
            out[i] = w[i];
        }
        return;
    }
    // this CTA's run [r0, r1)
    const int run = ((n + ctas - 1) / ctas + kSelectThreads - 1) / kSelectThreads * kSelectThreads;
    const int r0 = static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(rank) * run)), r1 = min(n, r0 + run);
    if (run <= cached) select_run<true>(a, S, keys, w, kept, out, n, r0, r1, ctas, rank);
    else select_run<false>(a, S, keys, w, kept, out, n, r0, r1, ctas, rank);
}

// The largest of 16 codes' magnitudes: e4m3 values order as their 7 low bits.
__device__ __forceinline__ uint32_t top_code(const uint4& v) {
    const uint32_t m = 0x007F007Fu;
    const uint32_t lo = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    const uint32_t hi = __vmaxu2(__vmaxu2(v.x >> 8 & m, v.y >> 8 & m), __vmaxu2(v.z >> 8 & m, v.w >> 8 & m));
    const uint32_t t = __vmaxu2(lo, hi);
    return max(t & 0xFFFFu, t >> 16);
}

// How a row's codes change with its scale. Where a code and its rounded quotient are normal numbers, the quotient's 4-bit
// significand and its distance in powers of two depend on the code's 3 mantissa bits alone, and so does the difference of
// the two codes as integers (exponent above mantissa): eight differences, modulo 128, to be looked up by byte
// permutations, four codes at a time. Codes too small for that (`floor` turns their sum's bit 7 off) take the formula:
// with normally distributed values one piece in some hundreds.
struct alignas(16) CodeStep {
    uint2 diff;      // bytes: difference for mantissa 0 .. 7
    uint32_t floor;  // each byte: 128 - the least magnitude it holds for (0: for none)
};

// Half of a row's differences (mantissas 4 * half + 0 .. 3) for the ratio of its scale to the new one, and whether all are
// certain: with the ratio as f 2^k, 1 <= f < 2, code (8 + mantissa) 2^e becomes (8 + mantissa) f 2^(e + k), whose
// significand is rounded in steps of 1 below 16 and of 2 from there on. A value within 2^-14 of the middle of two steps
// leaves it to the formula (the ratio and the products are off by some 2^-22 relatively).
__device__ __forceinline__ bool step_differences(float ratio, int half, uint32_t* diff, int* least) {
    const int k = static_cast<int>(__float_as_uint(ratio) >> 23) - 127;
    const float f = __uint_as_float((__float_as_uint(ratio) & 0x7FFFFFu) | 0x3F800000u);
    bool sure = k >= -5 && k < 7;
    *diff = 0;
    *least = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int mant = 4 * half + i;
        const float y = static_cast<float>(8 + mant) * f, z = y < 16.0f ? y : 0.5f * y;
        const float up = z + 12582912.0f, whole = up - 12582912.0f;  // 1.5 * 2^23: the nearest whole number, and its bits
        sure = sure && fabsf(fabsf(z - whole) - 0.5f) > 0x1p-14f;
        const int d = static_cast<int>(__float_as_uint(up) & 31u) - (y < 16.0f ? 8 : 0) + 8 * k - mant;
        *diff |= static_cast<uint32_t>(d & 0x7F) << (8 * i);
        *least = min(*least, d);
    }
    return sure;
}

__device__ __forceinline__ bool step_codes(const uint4& in, const CodeStep& c, uint4* out) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t r[4], large = 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mag = w[i] & 0x7F7F7F7Fu;
        large &= mag + c.floor;
        uint32_t pick = w[i] & 0x07070707u;  // the mantissas, side by side as the permutation's four selectors
        pick = (pick | pick >> 4) & 0x00FF00FFu;
        pick |= pick >> 8;
        const uint32_t sum = mag + __byte_perm(c.diff.x, c.diff.y, pick & 0xFFFFu);  // (at most 254 in a byte)
        r[i] = (sum & 0x7F7F7F7Fu) | (w[i] & 0x80808080u);
    }
    if (large != 0x80808080u) return false;
    *out = make_uint4(r[0], r[1], r[2], r[3]);
    return true;
}

// kVec: 16-byte vectors of a piece (two where the widths allow it: half the addresses); kPieces: pieces of a thread, which
// hold 64 rows of d_qk + d_v bytes together.
template <int kVec, int kPieces>
__global__ void __launch_bounds__(kMoveThreads, kVec * kPieces <= 4 ? 5 : 3) grouped_move_kernel(GroupedEvictArgs a, uint32_t magic) {
    __shared__ int32_t src_row[kBlock];
    __shared__ float src_scale[2][kBlock];
    __shared__ CodeStep step[2][kBlock];
    __shared__ float2 red[kMoveThreads / 32];
    constexpr int kBytes = 16 * kVec;
    const int tid = threadIdx.x, bh_in = blockIdx.x, b = bh_in / a.H_kv, h = bh_in - b * a.H_kv;
    int n = a.seq_lens[b];
    if (n < 0 || n > a.max_blocks * kBlock) n = 0;
    const int m = min(n, a.keep);
    const bool whole = n <= a.keep;
    const int gk = a.d_qk / kBytes, groups = gk + a.d_v / kBytes;
    griddep_wait();
    for (int j = blockIdx.y; j * kBlock < m; j += gridDim.y) {
        const int rows = min(kBlock, m - j * kBlock), total = rows * groups;
        const int to = a.new_table[static_cast<int64_t>(b) * a.new_max_blocks + j];
        const bool to_ok = to >= 0 && to < a.num_blocks;
        if (!to_ok && tid == 0) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
        __syncthreads();  // the last block's rows have been read
        if (tid < rows) {
            const int i = a.kept[static_cast<int64_t>(bh_in) * a.keep + j * kBlock + tid];
            const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + i / kBlock];
            const bool ok = blk >= 0 && blk < a.num_blocks;
            if (!ok) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
            const int bh = blk * a.H_kv + h;  // (the caches' rows are counted in 32 bits)
            src_row[tid] = ok ? bh * kBlock + i % kBlock : -1;
            src_scale[0][tid] = ok ? a.k_scale[bh] : 0.0f;
            src_scale[1][tid] = ok ? a.v_scale[bh] : 0.0f;
        }
        __syncthreads();
        const int to_bh = to * a.H_kv + h;
        if (!to_ok || (whole && src_row[0] == to_bh * kBlock)) continue;
        auto piece_at = [&](int of_row, int u) {  // piece u of a cache row: of its keys, then of its values
            const bool value = u >= gk;
            return reinterpret_cast<uint4*>((value ? a.v : a.k) + static_cast<int64_t>(of_row) * (value ? a.d_v : a.d_qk) + (value ? u - gk : u) * kBytes);
        };
        uint4 x[kPieces][kVec];
        int row[kPieces], unit[kPieces];  // -1: nothing there; the piece of the row
        float top[2] = {0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int i = tid + p * kMoveThreads;
            const int r = groups == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), magic));
            unit[p] = i - r * groups;
            const int src = i < total ? src_row[r] : -1;
            row[p] = src >= 0 ? r : -1;
            if (src >= 0) {
                const uint4* from = piece_at(src, unit[p]);
#pragma unroll
                for (int v = 0; v < kVec; ++v) x[p][v] = from[v];
            }
        }
        float scale[2] = {src_scale[0][0], src_scale[1][0]};
        if (!whole) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (row[p] < 0) continue;
                const bool value = unit[p] >= gk;
                uint32_t code = top_code(x[p][0]);
                if (kVec == 2) code = max(code, top_code(x[p][kVec - 1]));
                const float y = e4m3_to_float(code) * src_scale[value][row[p]];
                top[0] = fmaxf(top[0], value ? 0.0f : y);
                top[1] = fmaxf(top[1], value ? y : 0.0f);
            }
            // (magnitudes order as their bits do)
            const float k_top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top[0])));
            const float v_top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top[1])));
            if ((tid & 31) == 0) red[tid >> 5] = make_float2(k_top, v_top);
            __syncthreads();
            float2 t = red[0];
#pragma unroll
            for (int w = 1; w < kMoveThreads / 32; ++w) t = make_float2(fmaxf(t.x, red[w].x), fmaxf(t.y, red[w].y));
            scale[0] = unit_scale(t.x);
            scale[1] = unit_scale(t.y);
            // the rows' steps: two threads a row (of keys or of values)
            const int v = tid >> 7, r = (tid >> 1) & 63, half = tid & 1;
            const float from = src_scale[v][r], to_scale = v ? scale[1] : scale[0];
            uint32_t diff;
            int least;
            bool sure = step_differences(__fdividef(from, to_scale), half, &diff, &least);
            sure = __shfl_xor_sync(0xFFFFFFFFu, sure, 1) && sure && plain_scale(from) && plain_scale(to_scale);
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, 1));
            (&step[v][r].diff.x)[half] = diff;
            if (half == 0) step[v][r].floor = sure ? (120 + least) * 0x01010101u : 0;
            __syncthreads();
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (row[p] < 0) continue;
            const bool value = unit[p] >= gk;
            if (!whole) {
                const CodeStep c = step[value][row[p]];
                bool stepped = step_codes(x[p][0], c, &x[p][0]);
                if (!stepped) x[p][0] = requantise16(x[p][0], src_scale[value][row[p]], value ? scale[1] : scale[0]);
                if (kVec == 2) {
                    stepped = step_codes(x[p][kVec - 1], c, &x[p][kVec - 1]);
                    if (!stepped) x[p][kVec - 1] = requantise16(x[p][kVec - 1], src_scale[value][row[p]], value ? scale[1] : scale[0]);
                }
            }
            uint4* out = piece_at(to_bh * kBlock + row[p], unit[p]);
#pragma unroll
            for (int v = 0; v < kVec; ++v) out[v] = x[p][v];
        }
        if (tid == 0 && (!whole || src_row[0] >= 0)) {
            a.k_scale[to_bh] = scale[0];
            a.v_scale[to_bh] = scale[1];
        }
    }
}

bool launch_grouped_evict(const GroupedEvictArgs& a, cudaStream_t s, int* launches) {
    const unsigned heads = static_cast<unsigned>(a.B) * a.H_kv;
    // CTAs of a cluster: one turn of the SMs, and no fewer than 2048 positions each
    const int most = a.max_blocks * kBlock;
    int ctas = 1;
    while (ctas < kSelectMaxCluster && static_cast<int64_t>(heads) * 2 * ctas <= device_sm_count() && most >= 2 * ctas * 2048) ctas *= 2;
    const int run = ((most + ctas - 1) / ctas + kSelectThreads - 1) / kSelectThreads * kSelectThreads;
    const int cached = run < kSelectKeys ? run : kSelectKeys;
    const size_t smem = sizeof(uint32_t) * static_cast<size_t>(cached);
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(grouped_select_kernel), sizeof(uint32_t) * kSelectKeys)) return false;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(heads * ctas);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, grouped_select_kernel, a, ctas, cached) != cudaSuccess) return false;
    ++*launches;
    const int blocks = (a.keep + kBlock - 1) / kBlock;
    const dim3 grid(heads, blocks < 65535 ? blocks : 65535);
    const int vec = a.d_qk % 32 == 0 && a.d_v % 32 == 0 ? 2 : 1;
    const uint32_t groups = (a.d_qk + a.d_v) / (16 * vec), pieces = (kBlock * groups + kMoveThreads - 1) / kMoveThreads;
    // umulhi(i, ceil(2^32 / groups)) = i / groups for i < 2^32 / groups
    const uint32_t magic = static_cast<uint32_t>(((1ll << 32) + groups - 1) / groups);
    auto* move = vec == 2 ? (pieces <= 2 ? grouped_move_kernel<2, 2> : grouped_move_kernel<2, 4>)
                          : (pieces <= 4 ? grouped_move_kernel<1, 4> : grouped_move_kernel<1, 8>);
    if (!launch_kernel(true, move, grid, dim3(kMoveThreads), 0, s, a, magic)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
