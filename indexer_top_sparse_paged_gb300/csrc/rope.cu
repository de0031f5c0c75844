// Rotary positions: the pairs of a head's rotated columns turn by position * frequency.
//
//   angle_i = p f_i,   y_a = s (x_a cos - x_b sin),   y_b = s (x_a sin + x_b cos)
//
// with (a, b) = (2i, 2i + 1) (interleaved) or (i, i + rot / 2) (half). The transpose turns the other
// way: it is the backward pass (the Jacobian s R is linear in x). The angle is formed in fp64 as turns,
// p * (f / 2 pi), whose fraction is exact to 4e-11 at a million positions; fp32 would keep no more
// than two digits of it there. Sine and cosine are taken of the fraction in fp32.
//
// One CTA per token: its first rot / 2 threads form the token's table of cosines and sines once for
// all heads (of up to four tensors), then every thread turns pairs.
#include "internal.h"

namespace dsa {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    dsa_rope_tensor x[DSA_ROPE_MAX_TENSORS];
    int n;
    int rot;
    const double* freq;
    const int32_t* seq_lens;
    const int32_t* q_pos;
    float scale;
    int transpose;
};

template <typename T>
__device__ __forceinline__ float rope_load(const T* p);
template <>
__device__ __forceinline__ float rope_load<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float rope_load<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    __shared__ float2 table[DSA_ROPE_MAX_WIDTH / 2];
    const int t = blockIdx.x, half = a.rot / 2;
    const int pos = a.q_pos ? a.q_pos[t] : a.seq_lens[t] - 1;
    for (int i = threadIdx.x; i < half; i += kRopeThreads) table[i] = rope_cos_sin(pos, a.freq[i], a.scale, a.transpose);
    __syncthreads();
    for (int k = 0; k < a.n; ++k) {
        const dsa_rope_tensor& x = a.x[k];
        const T* src = static_cast<const T*>(x.x) + t * x.x_stride_t;
        T* dst = static_cast<T*>(x.out) + t * x.out_stride_t;
        if (pos < 0 && src == dst) continue;
        const int step = x.layout == DSA_ROPE_INTERLEAVED ? 1 : half;
        for (int j = threadIdx.x; j < x.heads * half; j += kRopeThreads) {
            const int h = j / half, i = j - h * half;
            const int e = x.layout == DSA_ROPE_INTERLEAVED ? 2 * i : i;
            const T* s = src + h * x.x_stride_h + e;
            T* d = dst + h * x.out_stride_h + e;
            const float u = rope_load(s), v = rope_load(s + step);
            const float2 y = pos < 0 ? make_float2(u, v) : rope_turn(u, v, table[i]);
            rope_store(d, y.x);
            rope_store(d + step, y.y);
        }
    }
}

bool launch_rope(int type, const dsa_rope_tensor* x, int n, int rot, const double* freq, const int32_t* seq_lens,
                 const int32_t* q_pos, int T, float scale, bool transpose, cudaStream_t s, int* launches) {
    RopeArgs a{};
    a.rot = rot;
    a.freq = freq;
    a.seq_lens = seq_lens;
    a.q_pos = q_pos;
    a.scale = scale;
    a.transpose = transpose ? 1 : 0;
    for (int i = 0; i < n; ++i)
        if (x[i].heads > 0) a.x[a.n++] = x[i];
    if (T == 0 || a.n == 0) return true;
    const bool ok = type == DSA_F32
                        ? launch_kernel(false, rope_kernel<float>, dim3(T), dim3(kRopeThreads), 0, s, a)
                        : launch_kernel(false, rope_kernel<__nv_bfloat16>, dim3(T), dim3(kRopeThreads), 0, s, a);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
