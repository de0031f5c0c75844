// Dense attention over packed prompts on the CUDA cores: fp32, and bf16 widths the tensor-core kernel
// does not take.
//
//   z = sm_scale q k^T over the keys j <= i + lk - lq (causal) or all of them, out = softmax(z) v,
//   lse = log sum exp z; a row without keys gives 0 and -inf.
//
// One CTA per tile of 64 rows (token, head of the group) and key head, one pass over the keys in tiles
// of 32 with the running maximum and sum of each row in fp32. A thread holds 4 rows x 2 keys of the
// logits and 4 rows x d_v / 16 columns of the output in registers.
#include "prompt.cuh"

namespace dsa {
namespace psimt {

constexpr int kThreads = 256;
constexpr int kRows = kPromptSimtRows, kKeys = 32;

__host__ __device__ constexpr int pitch(int d) { return d + 4; }

inline size_t smem_bytes(int d_qk, int d_v) {
    return sizeof(float) * ((kRows + kKeys) * pitch(d_qk) + kKeys * pitch(d_v) + kRows * (kKeys + 1));
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <typename T, int kCols>  // kCols: float4 columns of the output per thread, ceil(d_v / 64)
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(PromptArgs a) {
    extern __shared__ float smem[];
    const int pq = pitch(a.d_qk), pv = pitch(a.d_v);
    float* sq = smem;
    float* sk = sq + kRows * pq;
    float* sv = sk + kKeys * pq;
    float* sp = sv + kKeys * pv;
    griddep_launch_dependents();
    griddep_wait();
    if (static_cast<int>(blockIdx.x) >= a.head->n_units) return;
    const PromptUnit u = a.units[blockIdx.x];
    const int hk = blockIdx.y, G = a.H / a.H_kv;
    const int q0 = u.q0, lq = u.lq, k0 = u.k0, lk = u.lk, nrows = lq * G, row0 = u.row0;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    // queries, and for each of the thread's rows the number of keys it sees
    for (int i = tid; i < kRows * (a.d_qk / 4); i += kThreads) {
        const int r = i / (a.d_qk / 4), e = 4 * (i - r * (a.d_qk / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < nrows) {
            const int t = (row0 + r) / G, g = (row0 + r) % G;
            v = load4(static_cast<const T*>(a.q) + (q0 + t) * a.q_stride_t + (hk * G + g) * a.q_stride_h + e);
        }
        store4(sq + r * pq + e, v);
    }
    int seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + 4 * ty + i;
        seen[i] = r < nrows ? prompt_keys_seen(a, r / G, lq, lk) : 0;
    }
    // this part's keys, up to the last that the tile's last row sees
    const int n_keys = min(prompt_keys_seen(a, (min(nrows, row0 + kRows) - 1) / G, lq, lk), u.kt1 * kPromptKeys);
    const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
    float m[4], l[4];
    float4 o[4][kCols];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int s0 = u.kt0 * kPromptKeys; s0 < n_keys; s0 += kKeys) {
        __syncthreads();
        for (int i = tid; i < kKeys * (a.d_qk / 4); i += kThreads) {
            const int r = i / (a.d_qk / 4), e = 4 * (i - r * (a.d_qk / 4));
            store4(sk + r * pq + e, s0 + r < lk ? load4(static_cast<const T*>(a.k) + (static_cast<int64_t>(k0) + s0 + r) * a.k_stride_t +
                                                        hk * a.k_stride_h + e)
                                                : make_float4(0.f, 0.f, 0.f, 0.f));
        }
        for (int i = tid; i < kKeys * (a.d_v / 4); i += kThreads) {
            const int r = i / (a.d_v / 4), e = 4 * (i - r * (a.d_v / 4));
            store4(sv + r * pv + e, s0 + r < lk ? load4(static_cast<const T*>(a.v) + (static_cast<int64_t>(k0) + s0 + r) * a.v_stride_t +
                                                        hk * a.v_stride_h + e)
                                                : make_float4(0.f, 0.f, 0.f, 0.f));
        }
        __syncthreads();
        float z[4][2] = {};
        for (int e = 0; e < a.d_qk; e += 4) {
            float4 kv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * pq + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 qv = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * pq + e);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    z[i][j] = fmaf(qv.x, kv[j].x, z[i][j]);
                    z[i][j] = fmaf(qv.y, kv[j].y, z[i][j]);
                    z[i][j] = fmaf(qv.z, kv[j].z, z[i][j]);
                    z[i][j] = fmaf(qv.w, kv[j].w, z[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) z[i][j] = s0 + tx + 16 * j < seen[i] ? z[i][j] * c2 : -INFINITY;
            float mt = fmaxf(z[i][0], z[i][1]);
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, w));
            const float m_new = fmaxf(m[i], mt);
            const float ref = m_new == -INFINITY ? 0.0f : m_new;  // no key yet: every weight is 0
            const float alpha = exp2f(m[i] - ref);
            const float p0 = exp2f(z[i][0] - ref), p1 = exp2f(z[i][1] - ref);
            l[i] = l[i] * alpha + (p0 + p1);  // this thread's keys; joined at the end
            m[i] = m_new;
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                o[i][j].x *= alpha;
                o[i][j].y *= alpha;
                o[i][j].z *= alpha;
                o[i][j].w *= alpha;
            }
            sp[(4 * ty + i) * (kKeys + 1) + tx] = p0;
            sp[(4 * ty + i) * (kKeys + 1) + tx + 16] = p1;
        }
        __syncwarp();  // a row's 16 threads are half a warp
        for (int r = 0; r < kKeys; ++r) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = sp[(4 * ty + i) * (kKeys + 1) + r];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int e = 4 * tx + 64 * j;
                if (e >= a.d_v) continue;
                const float4 v = *reinterpret_cast<const float4*>(sv + r * pv + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i][j].x = fmaf(p[i], v.x, o[i][j].x);
                    o[i][j].y = fmaf(p[i], v.y, o[i][j].y);
                    o[i][j].z = fmaf(p[i], v.z, o[i][j].z);
                    o[i][j].w = fmaf(p[i], v.w, o[i][j].w);
                }
            }
        }
    }
    const int64_t slot0 = (static_cast<int64_t>(u.slot) * a.H_kv + static_cast<int64_t>(hk) * u.parts);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], w);
        const int r = 4 * ty + i;
        if (row0 + r >= nrows) continue;
        if (u.parts > 1) {
            if (tx == 0) a.part_ml[(slot0 + u.part) * a.slot_rows + r] = make_float2(m[i], l[i]);
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int e = 4 * tx + 64 * j;
                if (e >= a.d_v) continue;
                a.part_o[part_at(a, slot0 + u.part, e, r)] = o[i][j].x;
                a.part_o[part_at(a, slot0 + u.part, e + 1, r)] = o[i][j].y;
                a.part_o[part_at(a, slot0 + u.part, e + 2, r)] = o[i][j].z;
                a.part_o[part_at(a, slot0 + u.part, e + 3, r)] = o[i][j].w;
            }
            continue;
        }
        const int64_t at = (static_cast<int64_t>(q0) + (row0 + r) / G) * a.H + hk * G + (row0 + r) % G;  // (token, head)
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const int e = 4 * tx + 64 * j;
            if (e < a.d_v)
                store4(static_cast<T*>(a.out) + at * a.d_v + e,
                       make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv));
        }
        if (tx == 0 && a.lse) a.lse[at] = l[i] > 0.0f ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, int kCols>
static bool launch_typed(const PromptArgs& a, cudaStream_t s) {
    const size_t smem = smem_bytes(a.d_qk, a.d_v);
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(prompt_simt_kernel<T, kCols>), smem)) return false;
    return launch_kernel(true, prompt_simt_kernel<T, kCols>, dim3(a.max_units, a.H_kv), dim3(kThreads), smem, s, a);
}

template <typename T>
static bool launch_cols(const PromptArgs& a, cudaStream_t s) {
    switch ((a.d_v + 63) / 64) {
        case 1: return launch_typed<T, 1>(a, s);
        case 2: return launch_typed<T, 2>(a, s);
        case 3: return launch_typed<T, 3>(a, s);
        default: return launch_typed<T, 4>(a, s);
    }
}

}  // namespace psimt

bool launch_prompt_simt(const PromptArgs& a, cudaStream_t s, int* launches) {
    const bool ok = a.type == DSA_F32 ? psimt::launch_cols<float>(a, s) : psimt::launch_cols<__nv_bfloat16>(a, s);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
