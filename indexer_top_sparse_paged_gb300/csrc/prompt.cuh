// What the prompt attention's kernels share: the keys a token sees and the join of a row's parts.
#pragma once

#include "internal.h"

namespace dsa {

// Keys that the sequence's query token t sees: its first ones, up to its own position when causal.
__device__ __forceinline__ int prompt_keys_seen(const PromptArgs& a, int t, int lq, int lk) {
    return a.causal ? min(lk, max(0, t + 1 + lk - lq)) : lk;
}

// Columns e .. e + 3 of row r of the partials slot0 .. slot0 + parts - 1, joined in that order:
// sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p, and the row's lse.
__device__ __forceinline__ float4 prompt_join4(const PromptArgs& a, int64_t slot0, int parts, int r, int e, float* lse) {
    float M = -INFINITY;
    for (int p = 0; p < parts; ++p) M = fmaxf(M, __ldcg(&a.part_ml[(slot0 + p) * a.slot_rows + r]).x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M == -INFINITY) {  // no part saw a key
        *lse = -INFINITY;
        return o;
    }
    float l = 0.0f;
    for (int p = 0; p < parts; ++p) {
        const int64_t at = (slot0 + p) * a.slot_rows + r;
        const float2 ml = __ldcg(&a.part_ml[at]);
        if (ml.x == -INFINITY) continue;
        const float f = exp2f(ml.x - M);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * a.d_v + e));
        l += f * ml.y;
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
    }
    const float inv = 1.0f / l;
    *lse = (M + log2f(l)) * 0.6931471805599453f;
    return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

}  // namespace dsa
