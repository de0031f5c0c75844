// Dense attention over packed prompts on the CUDA cores: fp32, and bf16 widths the tensor-core kernel
// does not take.
//
//   z = sm_scale q k^T over the keys j <= i + lk - lq (causal) or all of them, out = softmax(z) v,
//   lse = log sum exp z; a row without keys gives 0 and -inf.
//
// One CTA per tile of 64 rows (token, head of the group), key head and range of keys; one pass over the keys
// in tiles of 64 with the running maximum and sum of each row in fp32. A thread holds 4 rows x 4 keys of the
// logits and 4 rows x d_v / 16 columns of the output; multiply-adds are issued in pairs (fma.rn.f32x2): 8 (12)
// loads of 16 bytes a lane feed 64 (128) of them. 20 TFLOP/s at 4096 tokens, 8 heads of 128 (1.7 ms); five prompts of
// up to 600 tokens, 8 / 2 heads, 121 us. Bound by latency: 206 registers a thread leave one CTA of 8 warps to an SM,
// which issue in 37% (33%) of its cycles, waiting for shared memory (its pipe half used) and for their own last
// instruction; keys and values are waited for before every tile, with nothing under way during the arithmetic; and
// SMs that are done early stand idle, 23% (18%) of the time. Tiles of 4 x 8 a thread, with half the warps, were
// slower (213 us, then 130, for the five prompts).
#include "prompt.cuh"

namespace dsa {
namespace psimt {

constexpr int kThreads = 256;
constexpr int kRows = kPromptSimtRows, kKeys = 64;
constexpr int kPitchP = kKeys + 4;
constexpr int kR = 4, kJ = 4;  // rows and keys per thread
static_assert(kRows == kThreads / 16 * kR && kKeys == 16 * kJ, "16 threads a row");

__host__ __device__ constexpr int pitch(int d) { return d + 4; }

inline size_t smem_bytes(int d_qk, int d_v) {
    const int keys = kKeys * pitch(d_qk), weights = kRows * kPitchP;
    return sizeof(float) * (kRows * pitch(d_qk) + (keys > weights ? keys : weights) + kKeys * pitch(d_v));
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

// Row r of a tile of keys: 4 columns a lane, from src + r * stride into dst + r * pitch as fp32; rows from n on
// are zeros. fp32 rows arrive by themselves (cp.async), bf16 rows are widened on the way.
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int pitch, const T* src, int64_t stride, int d, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int r = threadIdx.x >> 5; r < kKeys; r += kThreads / 32) {
        for (int e = 4 * lane; e < d; e += 128) {
            if constexpr (sizeof(T) == 4)
                cp_async16(smem_u32(dst + r * pitch + e), r < n ? src + r * stride + e : src, r < n ? 16 : 0);
            else
                store4(dst + r * pitch + e, r < n ? load4(src + r * stride + e) : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
}

template <typename T, int kCols>  // kCols: float4 columns of the output per thread, ceil(d_v / 64)
__global__ void __launch_bounds__(kThreads, 1) prompt_simt_kernel(PromptArgs a) {
    extern __shared__ float smem[];
    const int pq = pitch(a.d_qk), pv = pitch(a.d_v);
    float* sq = smem;
    float* sk = sq + kRows * pq;
    float* sp = sk;  // the weights, once the logits are made
    float* sv = sk + max(kKeys * pq, kRows * kPitchP);
    griddep_launch_dependents();
    griddep_wait();
    for (int index = blockIdx.x;; index += gridDim.x) {
        PromptUnit u;
        if (a.self_plan) {
            if (!prompt_self_unit(a, index, u)) return;  // (every warp for itself)
        } else {
            if (index >= a.head->n_units) return;
            u = a.units[index];
        }
        const int hk = blockIdx.y, G = a.H / a.H_kv;
        const int q0 = u.q0, lq = u.lq, k0 = u.k0, lk = u.lk, nrows = lq * G, row0 = u.row0;
        const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;  // the thread's rows: kR * ty ..
        // queries, and for each of the thread's rows the number of keys it sees
        {
            const int lane = tid & 31;
            for (int r = tid >> 5; r < kRows; r += kThreads / 32) {
                const bool in = row0 + r < nrows;
                const int t = in ? (row0 + r) / G : 0, g = in ? row0 + r - t * G : 0;
                const T* src = static_cast<const T*>(a.q) + (q0 + t) * a.q_stride_t + (hk * G + g) * a.q_stride_h;
                for (int e = 4 * lane; e < a.d_qk; e += 128)
                    store4(sq + r * pq + e, in ? load4(src + e) : make_float4(0.f, 0.f, 0.f, 0.f));
            }
        }
        int seen[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int r = row0 + kR * ty + i;
            seen[i] = r < nrows ? prompt_keys_seen(a, r / G, lq, lk) : 0;
        }
        const bool idle = row0 + tid / 32 * 2 * kR >= nrows;  // none of the warp's rows exist: it only loads (16 tokens on 1000 keys: 201 us, then 170)
        // this part's keys, up to the last that the tile's last row sees
        const int n_keys = min(prompt_keys_seen(a, (min(nrows, row0 + kRows) - 1) / G, lq, lk), u.kt1 * kPromptKeys);
        const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
        float m[kR], l[kR];
        uint64_t o[kR][kCols][2];  // pairs of columns
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < kCols; ++j) o[i][j][0] = o[i][j][1] = 0;
        }
        for (int s0 = u.kt0 * kPromptKeys; s0 < n_keys; s0 += kKeys) {
            const int64_t at = static_cast<int64_t>(k0) + s0;
            load_rows(sk, pq, static_cast<const T*>(a.k) + at * a.k_stride_t + hk * a.k_stride_h, a.k_stride_t, a.d_qk, lk - s0);
            load_rows(sv, pv, static_cast<const T*>(a.v) + at * a.v_stride_t + hk * a.v_stride_h, a.v_stride_t, a.d_v, lk - s0);
            cp_async_commit();
            cp_async_wait<0>();
            __syncthreads();
            uint64_t zz[kR][kJ];  // sums over the even and the odd columns
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int j = 0; j < kJ; ++j) zz[i][j] = 0;
            if (!idle) {
#pragma unroll 2
                for (int e = 0; e < a.d_qk; e += 4) {
                    ulonglong2 kv[kJ];
#pragma unroll
                    for (int j = 0; j < kJ; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * pq + e);
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(sq + (kR * ty + i) * pq + e);
#pragma unroll
                        for (int j = 0; j < kJ; ++j) zz[i][j] = fma2(qv.y, kv[j].y, fma2(qv.x, kv[j].x, zz[i][j]));
                    }
                }
            }
            __syncthreads();  // every warp has read the keys
            if (!idle) {
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    float z[kJ], mt = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const float2 h = unpack2(zz[i][j]);
                        z[j] = s0 + tx + 16 * j < seen[i] ? (h.x + h.y) * c2 : -INFINITY;
                        mt = fmaxf(mt, z[j]);
                    }
#pragma unroll
                    for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, w));
                    const float m_new = fmaxf(m[i], mt);
                    const float ref = m_new == -INFINITY ? 0.0f : m_new;  // no key yet: every weight is 0
                    const float alpha = exp2f(m[i] - ref);
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const float w = exp2f(z[j] - ref);
                        sum += w;
                        sp[(kR * ty + i) * kPitchP + tx + 16 * j] = w;
                    }
                    l[i] = l[i] * alpha + sum;  // this thread's keys; joined at the end
                    m[i] = m_new;
                    if (alpha != 1.0f) {
                        const uint64_t aa = pack2(alpha, alpha);
#pragma unroll
                        for (int j = 0; j < kCols; ++j) {
                            o[i][j][0] = fma2(o[i][j][0], aa, 0);
                            o[i][j][1] = fma2(o[i][j][1], aa, 0);
                        }
                    }
                }
                __syncwarp();  // a row's 16 threads are in one warp
                for (int r = 0; r < kKeys; r += 4) {
                    float4 p[kR];
#pragma unroll
                    for (int i = 0; i < kR; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (kR * ty + i) * kPitchP + r);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int j = 0; j < kCols; ++j) {
                            const int e = 4 * tx + 64 * j;
                            if (e >= a.d_v) continue;
                            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sv + (r + q) * pv + e);
#pragma unroll
                            for (int i = 0; i < kR; ++i) {
                                const float w = q == 0 ? p[i].x : q == 1 ? p[i].y : q == 2 ? p[i].z : p[i].w;
                                const uint64_t ww = pack2(w, w);
                                o[i][j][0] = fma2(ww, v.x, o[i][j][0]);
                                o[i][j][1] = fma2(ww, v.y, o[i][j][1]);
                            }
                        }
                    }
                }
            }
            __syncthreads();  // the tiles may be filled again
        }
        const int64_t slot0 = (static_cast<int64_t>(u.slot) * a.H_kv + static_cast<int64_t>(hk) * u.parts);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], w);
            const int r = kR * ty + i;
            if (row0 + r >= nrows) continue;
            if (u.parts > 1) {
                if (tx == 0) a.part_ml[(slot0 + u.part) * a.slot_rows + r] = make_float2(m[i], l[i]);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const int e = 4 * tx + 64 * j;
                    if (e >= a.d_v) continue;
                    const float2 lo = unpack2(o[i][j][0]), hi = unpack2(o[i][j][1]);
                    a.part_o[part_at(a, slot0 + u.part, e, r)] = lo.x;
                    a.part_o[part_at(a, slot0 + u.part, e + 1, r)] = lo.y;
                    a.part_o[part_at(a, slot0 + u.part, e + 2, r)] = hi.x;
                    a.part_o[part_at(a, slot0 + u.part, e + 3, r)] = hi.y;
                }
                continue;
            }
            const int64_t at = (static_cast<int64_t>(q0) + (row0 + r) / G) * a.H + hk * G + (row0 + r) % G;  // (token, head)
            const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int e = 4 * tx + 64 * j;
                const float2 lo = unpack2(o[i][j][0]), hi = unpack2(o[i][j][1]);
                if (e < a.d_v)
                    store4(static_cast<T*>(a.out) + at * a.d_v + e, make_float4(lo.x * inv, lo.y * inv, hi.x * inv, hi.y * inv));
            }
            if (tx == 0 && a.lse) a.lse[at] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
        }
    }
}

template <typename T, int kCols>
static bool launch_typed(const PromptArgs& a, cudaStream_t s) {
    const size_t smem = smem_bytes(a.d_qk, a.d_v);
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(prompt_simt_kernel<T, kCols>), smem)) return false;
    // A CTA for every whole item, and for as many parts as the plan aims at; should there be more, a CTA takes
    // several. (One for every part that there could be, most of them empty, took 2 us longer for 5 prompts of up to
    // 600 tokens, 120 us.)
    const int items = static_cast<int>(static_cast<int64_t>(a.Tq) * (a.H / a.H_kv) / a.tile_rows) + a.B;
    const int parts = 2 * a.shares / a.H_kv, most = items > parts ? items : parts;
    const int grid = most < a.max_units ? most : a.max_units;
    return launch_kernel(!a.self_plan, prompt_simt_kernel<T, kCols>, dim3(grid, a.H_kv), dim3(kThreads), smem, s, a);
}

template <typename T>
static bool launch_cols(const PromptArgs& a, cudaStream_t s) {
    if (a.d_v <= 64) return launch_typed<T, 1>(a, s);
    if (a.d_v <= 128) return launch_typed<T, 2>(a, s);
    return launch_typed<T, 4>(a, s);
}

}  // namespace psimt

bool launch_prompt_simt(const PromptArgs& a, cudaStream_t s, int* launches) {
    const bool ok = a.type == DSA_F32 ? psimt::launch_cols<float>(a, s) : psimt::launch_cols<__nv_bfloat16>(a, s);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
