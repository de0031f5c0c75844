// What the prompt attention's kernels share: the keys a token sees and the join of a row's parts.
#pragma once

#include "internal.h"

namespace dsa {

// Pairs of fp32 in one 64-bit register: two products or sums an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(v));
    return y;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

// Keys that the sequence's query token t sees: its first ones, up to its own position when causal.
__device__ __forceinline__ int prompt_keys_seen(const PromptArgs& a, int t, int lq, int lk) {
    return a.causal ? min(lk, max(0, lk - lq + t + 1)) : lk;
}

// Small calls (at most 32 sequences and 7 key tiles, so that nothing is split) have no work list: a warp reads
// every sequence's bounds, and all its lanes return unit `index`; false past the last one. The sequences
// whose bounds are no ranges have no units (reported by the first).
__device__ __forceinline__ bool prompt_self_unit(const PromptArgs& a, int index, PromptUnit& u) {
    const int lane = threadIdx.x & 31, G = a.H / a.H_kv;
    int q0 = 0, lq = 0, k0 = 0, lk = 0, n = 0;
    if (lane < a.B) {
        const int q1 = a.cu_q[lane + 1], k1 = a.cu_k[lane + 1];
        q0 = a.cu_q[lane];
        k0 = a.cu_k[lane];
        if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) {
            if (index == 0) atomicOr(a.err, DSA_FAULT_INDEX);
        } else {
            lq = q1 - q0;
            lk = k1 - k0;
            n = (lq * G + a.tile_rows - 1) / a.tile_rows;
        }
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
    }
    const unsigned owner = __ballot_sync(0xFFFFFFFFu, index >= upto - n && index < upto);
    if (!owner) return false;
    const int src = __ffs(owner) - 1;
    u.q0 = __shfl_sync(0xFFFFFFFFu, q0, src);
    u.lq = __shfl_sync(0xFFFFFFFFu, lq, src);
    u.k0 = __shfl_sync(0xFFFFFFFFu, k0, src);
    u.lk = __shfl_sync(0xFFFFFFFFu, lk, src);
    u.row0 = (index - __shfl_sync(0xFFFFFFFFu, upto - n, src)) * a.tile_rows;
    u.kt0 = 0;
    u.kt1 = (u.lk + kPromptKeys - 1) / kPromptKeys;
    u.slot = 0;
    u.part = 0;
    u.parts = 1;
    return true;
}

// Column c of row r of partial `slot`: the rows of a column lie side by side, so that a warp whose lanes hold
// rows writes and reads whole lines.
__device__ __forceinline__ int64_t part_at(const PromptArgs& a, int64_t slot, int c, int r) {
    return (slot * a.d_v + c) * a.slot_rows + r;
}

__device__ __forceinline__ void store_cols(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Joins row r (row0 + r of the sequence) of the partials slot0 .. slot0 + parts - 1 in that order and writes its
// columns c .. c + 7 out: sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p, the loads of kAhead parts in flight (past the last
// it is loaded again: without a branch between them the loads go out together).
template <int kAhead, typename T>
__device__ __forceinline__ void prompt_join(const PromptArgs& a, int64_t slot0, int parts, int q0, int row0, int hk, int r,
                                            int c) {
    const int G = a.H / a.H_kv, t = (row0 + r) / G;
    const int64_t at = (static_cast<int64_t>(q0) + t) * a.H + hk * G + (row0 + r - t * G);  // (token, head)
    const float2* ml = a.part_ml + slot0 * a.slot_rows + r;
    T* out = static_cast<T*>(a.out) + at * a.d_v;
    const int m = min(8, a.d_v - c);  // 8, or 4 (fp32 rows of an odd number of pieces)
    float M = -INFINITY, l = 0.0f, o[8] = {};
    for (int p0 = 0; p0 < parts; p0 += kAhead) {
        float2 v[kAhead];
        float y[kAhead][8];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {  // every load of these parts before the first is used
            const int p = min(p0 + i, parts - 1);
            v[i] = __ldcg(ml + static_cast<int64_t>(p) * a.slot_rows);
            const float* po = a.part_o + part_at(a, slot0 + p, c, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = e < m ? __ldcg(po + static_cast<int64_t>(e) * a.slot_rows) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            // a part without keys has no sum and wrote no columns (a NaN sum beside a maximum of -inf is joined)
            if (p0 + i >= parts || v[i].y == 0.0f) continue;
            const float top = fmaxf(M, v[i].x), f = exp2f(v[i].x - top), keep = exp2f(M - top);
            l = l * keep + f * v[i].y;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = o[e] * keep + f * y[i][e];
            M = top;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    if (m == 8) {
        store_cols(out + c, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < m) out[c + e] = static_cast<T>(o[e]);
    }
    if (c == 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

}  // namespace dsa
