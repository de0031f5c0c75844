// Shared by the kernels of the grouped-head cache: the arguments, the sequences' places and the work of the
// attention, which every CTA finds in the lengths itself.
//
// The G = H / H_kv query heads of a key head share its keys, so a sequence's n queries give each key head one column of
// n * G rows, row r = token r / G, head r % G of the group. An item is (sequence, key head, row_tile of those rows); its
// positions are cut into tiles of 128. All tiles of all items, in this order, are one line, and CTA c of C takes the
// tiles [c * per, (c + 1) * per), per = ceil(total / C): an even share of the cached bytes whatever the lengths. An item
// cut by that leaves a partial (maximum, sum, unnormalised output) in its CTA's slot, and the CTA that leaves the last one
// joins them in order of positions, so that results do not depend on timing.
#pragma once

#include "internal.h"

namespace dsa {

constexpr int kGroupedTile = 128;  // positions per tile: two cache blocks

struct GroupedSeq {
    int q0, n;       // first row of q, number of them
    int len;         // cached positions
    int items;       // row tiles
    int tiles;       // position tiles
};

// Sequence b's place. What the host cannot see is checked here: a bad entry is reported (`report`), and the sequence is
// left with no rows (cu) or no positions (seq_lens).
__device__ __forceinline__ GroupedSeq grouped_seq(const GroupedArgs& a, int b, bool report) {
    GroupedSeq s;
    s.q0 = b;
    s.n = 1;
    if (a.cu) {
        s.q0 = a.cu[b];
        s.n = a.cu[b + 1] - s.q0;
        if (s.q0 < 0 || s.q0 > a.T || s.n < 0 || s.n > a.T - s.q0) {
            if (report) atomicOr(a.err, DSA_FAULT_INDEX);
            s.q0 = s.n = 0;
        }
    }
    s.len = a.seq_lens[b];
    if (s.len < 0 || s.len > a.max_blocks * kBlock) {
        if (report) atomicOr(a.err, DSA_FAULT_INDEX);
        s.len = 0;
    }
    s.items = static_cast<int>((static_cast<int64_t>(s.n) * a.G + a.row_tile - 1) / a.row_tile);
    s.tiles = (s.len + kGroupedTile - 1) / kGroupedTile;
    return s;
}

__device__ __forceinline__ int64_t grouped_seq_tiles(const GroupedArgs& a, const GroupedSeq& s) {
    return static_cast<int64_t>(s.items) * s.tiles * a.H_kv;
}

// Tiles of a CTA's share.
__device__ __forceinline__ int64_t grouped_share(const GroupedArgs& a, int64_t total) {
    return total < (1ll << 30) ? (static_cast<int>(total) + a.ctas - 1) / a.ctas : (total + a.ctas - 1) / a.ctas;
}

// Sum over the block's threads, and the sum of the threads before this one.
template <int kThreads>
__device__ __forceinline__ int64_t block_prefix(int64_t x, int64_t* total, int64_t* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) y += t;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + y - x;
}

// The total of count(b) over all sequences b, and, with at = where(total), the sequence whose units hold unit `at` of their
// line, and the first unit of that sequence (b -1: there is none). All threads of the block call it.
template <int kThreads, typename Count, typename Where>
__device__ __forceinline__ int64_t find_place(int B, Count count, Where where, int64_t* total, int* b_out, int64_t* base_out,
                                              int64_t* warp_sums, int64_t* found) {
    if (threadIdx.x == 0) found[0] = -1;
    int64_t sum = 0, n = 0, before = 0, at = 0;
    const bool once = B <= kThreads;  // a thread's sequence stays in registers
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        n = b < B ? count(b) : 0;
        int64_t all;
        before = block_prefix<kThreads>(n, &all, warp_sums);
        sum += all;
    }
    at = where(sum);
    int64_t done = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int64_t all = 0;
        if (!once) {
            n = b < B ? count(b) : 0;
            before = done + block_prefix<kThreads>(n, &all, warp_sums);
        }
        if (at >= before && at < before + n) {
            found[0] = b;
            found[1] = before;
        }
        done += all;
    }
    __syncthreads();
    *total = sum;
    *b_out = static_cast<int>(found[0]);
    *base_out = found[1];
    return at;
}

// Slot of the partial that CTA c leaves of an item: its share's first item, if that is cut, uses slot 2c, and the last
// one 2c + 1 (an item that fills the whole share is its first).
__device__ __forceinline__ int grouped_slot(int64_t share_begin, int64_t piece_begin, int c) {
    return 2 * c + (piece_begin > share_begin ? 1 : 0);
}

__device__ __forceinline__ void store_quad(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store_quad(__nv_bfloat16* p, float4 x) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Joins an item's partials: slot0, then the first ones of the next CTAs. A warp takes kRows rows at a time (warp, + warps,
// ...), four columns a lane, kBatch partials of each on their way at once. row_at: the rows' places in lse and out.
template <typename T, int kRows, int kBatch>
__device__ __noinline__ void grouped_join(const GroupedArgs& a, const int* row_at, int rows, int slot0, int parts, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    for (int r0 = warp; r0 < rows; r0 += kRows * warps) {
        for (int e = 4 * lane; e < a.d_v; e += 128) {
            float top[kRows], sum[kRows];
            float4 o[kRows];
#pragma unroll
            for (int q = 0; q < kRows; ++q) top[q] = -INFINITY, sum[q] = 0.0f, o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int p0 = 0; p0 < parts; p0 += kBatch) {
                float2 ml[kRows][kBatch];
                float4 x[kRows][kBatch];
#pragma unroll
                for (int q = 0; q < kRows; ++q)
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int p = min(p0 + k, parts - 1), r = min(r0 + q * warps, rows - 1);
                        const int slot = (p ? 2 * (slot0 / 2 + p) : slot0) * a.row_tile + r;
                        ml[q][k] = __ldcg(a.part_ml + slot);
                        x[q][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + static_cast<int64_t>(slot) * a.d_v + e));
                    }
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    float most = top[q];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        if (p0 + k >= parts) ml[q][k] = make_float2(-INFINITY, 0.0f), x[q][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        most = fmaxf(most, ml[q][k].x);
                    }
                    const float ref = most == -INFINITY ? 0.0f : most, old = exp2f(top[q] - ref);
                    sum[q] *= old;
                    o[q].x *= old, o[q].y *= old, o[q].z *= old, o[q].w *= old;
                    top[q] = most;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const float f = exp2f(ml[q][k].x - ref);
                        const float4 y = x[q][k];
                        sum[q] = fmaf(f, ml[q][k].y, sum[q]);
                        o[q].x = fmaf(f, y.x, o[q].x), o[q].y = fmaf(f, y.y, o[q].y), o[q].z = fmaf(f, y.z, o[q].z), o[q].w = fmaf(f, y.w, o[q].w);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                const int r = r0 + q * warps;
                if (r >= rows) break;
                const int at = row_at[r];
                const float inv = sum[q] == 0.0f ? 0.0f : 1.0f / sum[q];
                store_quad(static_cast<T*>(a.out) + static_cast<int64_t>(at) * a.d_v + e, make_float4(o[q].x * inv, o[q].y * inv, o[q].z * inv, o[q].w * inv));
                if (e == 0) {
                    const float lse2 = sum[q] == 0.0f ? -INFINITY : top[q] + log2f(sum[q]);
                    if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
                    if (a.weights_out) a.row_lse[at] = lse2;
                }
            }
        }
    }
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);  // exact
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

// The scale that takes amax to the largest code (1 where that is 0, as it also is for the smallest magnitudes).
__device__ __forceinline__ float unit_scale(float amax) {
    const float s = amax / 448.0f;
    return s > 0.0f ? s : 1.0f;
}

__device__ __forceinline__ uint32_t e4m3x4_codes(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// Rounded quotients without the division, checked: the formulas' results are off the exact quotient by two roundings of
// 2^-24 at most, relatively, and x times (1 / scale, drawn in or out by 2^-21) by four, so the two products enclose them.
// Where both round to the same code, so does the formula's result; where they do not (a value next to the middle of two
// codes, one in some 2^17), the formula is followed. (Underflowing products belong to the code 0 either way.)
constexpr float kBelow = 1.0f - 0x1p-21f, kAbove = 1.0f + 0x1p-21f;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {  // one instruction
    uint64_t x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(z));
    return a;
}

// Codes of 16 values times r; false: some lie too near the middle of two codes.
__device__ __forceinline__ bool near_codes(const float2 (&x)[8], float r, uint4* codes) {
    const float2 below = make_float2(r * kBelow, r * kBelow), above = make_float2(r * kAbove, r * kAbove);
    uint32_t w[4], differ = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a0 = mul2(x[2 * i], below), a1 = mul2(x[2 * i + 1], below);
        const float2 b0 = mul2(x[2 * i], above), b1 = mul2(x[2 * i + 1], above);
        w[i] = e4m3x4_codes(a0.x, a0.y, a1.x, a1.y);
        differ |= w[i] ^ e4m3x4_codes(b0.x, b0.y, b1.x, b1.y);
    }
    *codes = make_uint4(w[0], w[1], w[2], w[3]);
    return differ == 0;
}

static __device__ __noinline__ uint4 divided_codes(float2 x0, float2 x1, float2 x2, float2 x3, float2 x4, float2 x5, float2 x6, float2 x7, float s) {
    return make_uint4(e4m3x4_codes(x0.x / s, x0.y / s, x1.x / s, x1.y / s), e4m3x4_codes(x2.x / s, x2.y / s, x3.x / s, x3.y / s),
                      e4m3x4_codes(x4.x / s, x4.y / s, x5.x / s, x5.y / s), e4m3x4_codes(x6.x / s, x6.y / s, x7.x / s, x7.y / s));
}

// Scales whose reciprocal, and products with it, neither overflow nor lose bits: the others divide.
__device__ __forceinline__ bool plain_scale(float scale) { return scale >= 0x1p-80f && scale <= 0x1p80f; }

// RNE_e4m3(x / scale) of 16 values, saturating at +-448.
__device__ __forceinline__ uint4 codes16(const float2 (&x)[8], float scale) {
    uint4 codes;
    if (plain_scale(scale) && near_codes(x, 1.0f / scale, &codes)) return codes;
    return divided_codes(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale);
}

// RNE_e4m3(fl(code * from) / scale) of 16 codes, saturating.
static __device__ __noinline__ uint4 requantise16(uint4 in, float from, float scale) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    float2 x[8];
    uint4 codes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
        x[i] = __half22float2(*reinterpret_cast<const __half2*>(&h));
    }
    const float r = from * (1.0f / scale);
    if (plain_scale(scale) && plain_scale(from) && r <= 0x1p100f && near_codes(x, r, &codes)) return codes;  // (codes of 0 may have any scale)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].x *= from, x[i].y *= from;
    return divided_codes(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale);
}

}  // namespace dsa
