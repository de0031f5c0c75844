// Rotary positions: the pairs of a head's rotated columns turn by position * frequency.
//
//   angle_i = p f_i,   y_a = s (x_a cos - x_b sin),   y_b = s (x_a sin + x_b cos)
//
// with (a, b) = (2i, 2i + 1) (interleaved) or (i, i + rot / 2) (half). The transpose turns the other
// way: it is the backward pass (the Jacobian s R is linear in x). The angle is formed as turns, p * (f / 2 pi),
// in 64-bit fixed point: off by at most 2^-33 turns, from the cut of the frequency's turns, and 2^-52 of the whole
// angle, from their two roundings in fp64 (2^-21 radians at position 2^31 of the fastest pair; the fp64 product of
// the definition itself rounds by half that). fp32 would keep no more than two digits of the fraction at a million
// positions. Sine and cosine are taken of the fraction in fp32.
//
// Bound by memory: the rotated columns are read and written once. One CTA per token, so that its table of
// rot / 2 cosines and sines is formed once for all heads of up to four tensors (one fp64 product and one
// sincospi each); every thread asks for up to four pieces of 16 bytes (half layout: pairs of pieces)
// before it waits for the table. 8192 tokens of 128 + 64 heads with 64 bf16 columns: 74 us, 80% of the measured
// copy bandwidth. Views that are not aligned to 16 bytes go pair by pair, and so do heads whose columns (half
// layout: halves) are one piece or no whole number of them.
#include "internal.h"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // pieces a thread has in flight

struct RopeArgs {
    dsa_rope_tensor x[DSA_ROPE_MAX_TENSORS];
    int per[DSA_ROPE_MAX_TENSORS];         // pieces per head (0: pair by pair)
    uint32_t magic[DSA_ROPE_MAX_TENSORS];  // j / per = umulhi(j, magic) for every piece j
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

// Word w of a piece as one (fp32) or two (bf16) values, and back.
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf16_word(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// A piece of adjacent pairs, turned by the table entries from i on.
template <typename T>
__device__ __forceinline__ uint4 turn_interleaved(const uint4& v, const float2* table) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 x = bf16_pair(w[k]), y = rope_turn(x.x, x.y, table[k]);
            w[k] = bf16_word(y.x, y.y);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 y = rope_turn(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]), table[k]);
            w[2 * k] = __float_as_uint(y.x);
            w[2 * k + 1] = __float_as_uint(y.y);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A piece of first and one of second elements of the same pairs.
template <typename T>
__device__ __forceinline__ void turn_half(uint4& a, uint4& b, const float2* table) {
    uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
            const float2 x = bf16_pair(u[k]), y = bf16_pair(v[k]);
            const float2 p = rope_turn(x.x, y.x, table[2 * k]), q = rope_turn(x.y, y.y, table[2 * k + 1]);
            u[k] = bf16_word(p.x, q.x);
            v[k] = bf16_word(p.y, q.y);
        } else {
            const float2 p = rope_turn(__uint_as_float(u[k]), __uint_as_float(v[k]), table[k]);
            u[k] = __float_as_uint(p.x);
            v[k] = __float_as_uint(p.y);
        }
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(v[0], v[1], v[2], v[3]);
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    __shared__ float2 table[DSA_ROPE_MAX_WIDTH / 2];
    constexpr int kElems = 16 / sizeof(T);  // of a piece
    const int t = blockIdx.x, half = a.rot / 2, tid = threadIdx.x;
    const int pos = a.q_pos ? a.q_pos[t] : a.seq_lens[t] - 1;
    bool ready = false;
    auto need_table = [&] {  // reached by the whole CTA together
        if (ready) return;
        ready = true;
        // a negative position turns nothing: the table's identity leaves every value as it is
        for (int i = tid; i < half; i += kRopeThreads)
            table[i] = pos < 0 ? make_float2(1.0f, 0.0f) : rope_cos_sin(pos, a.freq[i], a.scale, a.transpose);
        __syncthreads();
    };
    for (int k = 0; k < a.n; ++k) {
        const dsa_rope_tensor& x = a.x[k];
        const T* src = static_cast<const T*>(x.x) + t * x.x_stride_t;
        T* dst = static_cast<T*>(x.out) + t * x.out_stride_t;
        if (pos < 0 && src == dst) continue;
        const int per = a.per[k];
        if (per > 0) {
            const bool il = x.layout == DSA_ROPE_INTERLEAVED;
            const uint32_t magic = a.magic[k];
            const int total = x.heads * per;
            for (int base = 0; base < total; base += kRopeBatch * kRopeThreads) {  // the same turns for every thread
                const int j0 = base + tid;
                uint4 u[kRopeBatch], v[kRopeBatch];
                int h[kRopeBatch], e[kRopeBatch];
#pragma unroll
                for (int b = 0; b < kRopeBatch; ++b) {
                    const int j = j0 + b * kRopeThreads;
                    h[b] = static_cast<int>(__umulhi(static_cast<uint32_t>(j), magic));
                    e[b] = (j - h[b] * per) * kElems;
                    if (j >= total) continue;
                    const T* s = src + h[b] * x.x_stride_h + e[b];
                    u[b] = *reinterpret_cast<const uint4*>(s);
                    if (!il) v[b] = *reinterpret_cast<const uint4*>(s + half);
                }
                need_table();
#pragma unroll
                for (int b = 0; b < kRopeBatch; ++b) {
                    if (j0 + b * kRopeThreads >= total) break;
                    T* d = dst + h[b] * x.out_stride_h + e[b];
                    if (pos >= 0) {
                        if (il) u[b] = turn_interleaved<T>(u[b], table + e[b] / 2);
                        else turn_half<T>(u[b], v[b], table + e[b]);
                    }
                    *reinterpret_cast<uint4*>(d) = u[b];
                    if (!il) *reinterpret_cast<uint4*>(d + half) = v[b];
                }
            }
            continue;
        }
        need_table();
        const int step = x.layout == DSA_ROPE_INTERLEAVED ? 1 : half;
        for (int j = tid; j < x.heads * half; j += kRopeThreads) {
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
    const int64_t elems = type == DSA_F32 ? 4 : 8;  // of 16 bytes
    for (int i = 0; i < n; ++i) {
        if (x[i].heads <= 0) continue;
        const dsa_rope_tensor& r = x[i];
        const int cols = r.layout == DSA_ROPE_INTERLEAVED ? rot : rot / 2;
        const int64_t per = cols / elems, pieces = per * r.heads;
        const bool aligned = ((reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.out)) & 15) == 0 &&
                             (r.x_stride_t | r.x_stride_h | r.out_stride_t | r.out_stride_h) % elems == 0;
        // umulhi(j, ceil(2^32 / per)) = j / per while j * per < 2^32 (batches may ask for a few j past the end)
        if (aligned && cols % elems == 0 && per > 1 && (pieces + kRopeBatch * kRopeThreads) * per < (1ll << 32)) {
            a.per[a.n] = static_cast<int>(per);
            a.magic[a.n] = static_cast<uint32_t>(((1ull << 32) + per - 1) / per);
        }
        a.x[a.n++] = r;
    }
    if (T == 0 || a.n == 0) return true;
    const bool ok = type == DSA_F32
                        ? launch_kernel(false, rope_kernel<float>, dim3(T), dim3(kRopeThreads), 0, s, a)
                        : launch_kernel(false, rope_kernel<__nv_bfloat16>, dim3(T), dim3(kRopeThreads), 0, s, a);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
