// Cache append: new tokens' latent rows and indexer keys into their paged slots, the step before
// the indexer and the sparse attention ("How the Ascend Computing Platform Achieves Same-Day
// Inference Adaptation ..." §2.2 table: the cache update is fused with the flow that produces the
// new entries; "Day0 Inference Support ... on Huawei Ascend CANN Architecture" §2.2/§3: the
// indexer's keys are quantised on the way in).
//
// One CTA per new token t (sequence b, position pos in the sequence's tail) copies its latent
// row, and in the fp32 / bf16 modes its indexer key, into physical row
// block_table[b][pos / 64] * 64 + pos % 64. With FP8 e4m3 keys (one fp32 scale per 64-token
// block) the first new token of every touched block requantises the whole block: with
// x = code * scale_old (fp32) for the block's earlier tokens and the new keys' values,
// scale = amax / 448 (1 when amax is 0) and every code becomes RNE_e4m3(x / scale), saturating
// at +-448. The new tokens of one block must be consecutive rows (ascending positions). MXFP8
// keys have no block state: each new key's groups of 32 get their own E8M0 scale and codes.
// An FP8 latent cache (DSA_KV_FP8) has no block state either: each new row becomes one record,
// every 128-element tile quantised on its own (one warp per tile), in fp32: scale = amax / 448
// (1 when amax is 0), code = RNE_e4m3(x / scale), saturating ("Day0 Inference Support ... on
// Huawei Ascend CANN Architecture" §3: FP8 block quantisation in the attention stage).
#include "internal.h"

namespace dsa {

constexpr int kAppendThreads = 256;

struct AppendArgs {
    int mode;
    int kv_fp8;  // latent rows stored as FP8 records
    int B, max_blocks, num_blocks;
    int d_I, d;
    int T;
    const void* k_new;
    const void* kv_new;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* q_seq;
    const int32_t* q_pos;
    void* k_cache;
    void* k_scale;
    void* kv_cache;
    int* err;
};

// Sequence, position and physical cache block of new token t (-1 when invalid).
__device__ __forceinline__ int append_block(const AppendArgs& a, int t, int& b, int& pos) {
    b = a.q_seq ? a.q_seq[t] : t;
    if (b < 0 || b >= a.B) return -1;
    const int L = a.seq_lens[b];
    pos = a.q_pos ? a.q_pos[t] : L - 1;
    if (pos < 0 || pos >= L || pos / kBlock >= a.max_blocks) return -1;
    const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + pos / kBlock];
    return (blk >= 0 && blk < a.num_blocks) ? blk : -1;
}

__device__ __forceinline__ void copy_row(void* dst, const void* src, int bytes) {
    const uint4* s = static_cast<const uint4*>(src);
    uint4* d = static_cast<uint4*>(dst);
    for (int i = threadIdx.x; i < bytes / 16; i += kAppendThreads) d[i] = s[i];
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);  // exact
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

// One FP8 latent record from a bf16 row of d elements (d % 16 == 0): warp w quantises tiles
// w, w + 8, ...; lane l holds elements 4l .. 4l + 3 of the tile. The padding after the scales is
// zeroed.
__device__ void store_kv_record(uint8_t* rec, const uint16_t* x, int d) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ntiles = (d + 127) / 128;
    for (int j = warp; j < ntiles; j += kAppendThreads / 32) {
        const int e = 128 * j + 4 * lane;
        const bool in = e < d;  // d % 16 == 0: a lane's 4 elements are all in or all out
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (in) {
            const uint2 u = *reinterpret_cast<const uint2*>(x + e);
            v[0] = __uint_as_float(u.x << 16);
            v[1] = __uint_as_float(u.x & 0xFFFF0000u);
            v[2] = __uint_as_float(u.y << 16);
            v[3] = __uint_as_float(u.y & 0xFFFF0000u);
        }
        float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
        if (in) {
            uint32_t c = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(v[k] / scale, __NV_SATFINITE, __NV_E4M3)) << (8 * k);
            *reinterpret_cast<uint32_t*>(rec + e) = c;
        }
        if (lane == 0) *reinterpret_cast<float*>(rec + d + 4 * j) = scale;
    }
    for (int i = d + 4 * ntiles + static_cast<int>(threadIdx.x); i < DSA_KV_FP8_RECORD_BYTES(d); i += kAppendThreads)
        rec[i] = 0;
}

// New token t's rows into the paged caches (the whole CTA).
__device__ void append_token(const AppendArgs& a, int t) {
    __shared__ float red[kAppendThreads / 32];
    __shared__ int run_end;
    int b, pos;
    const int blk = append_block(a, t, b, pos);
    if (blk < 0) {
        if (threadIdx.x == 0) atomicOr(a.err, (b < 0 || b >= a.B) ? DSA_FAULT_INDEX : DSA_FAULT_BLOCK_TABLE);
        return;
    }
    const int64_t row = static_cast<int64_t>(blk) * kBlock + pos % kBlock;
    const int act = a.mode == DSA_F32 ? 4 : 2;
    if (a.kv_fp8) {
        store_kv_record(static_cast<uint8_t*>(a.kv_cache) + row * DSA_KV_FP8_RECORD_BYTES(a.d),
                        static_cast<const uint16_t*>(a.kv_new) + static_cast<int64_t>(t) * a.d, a.d);
    } else {
        copy_row(static_cast<uint8_t*>(a.kv_cache) + row * a.d * act,
                 static_cast<const uint8_t*>(a.kv_new) + static_cast<int64_t>(t) * a.d * act, a.d * act);
    }
    if (a.mode == DSA_MXFP8) {  // every group of 32 of the new key is quantised on its own
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k_new) + static_cast<int64_t>(t) * a.d_I);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.k_cache) + row * a.d_I);
        for (int g = threadIdx.x; g < a.d_I / 32; g += kAppendThreads) {
            uint32_t w[16], codes[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = src[4 * g + i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
            const int X = mx_encode32(w, codes);
            dst[2 * g] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            dst[2 * g + 1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
            static_cast<uint8_t*>(a.k_scale)[row * (a.d_I / 32) + g] = static_cast<uint8_t>(X + 127);
        }
        return;
    }
    if (a.mode != DSA_BF16_KFP8) {
        copy_row(static_cast<uint8_t*>(a.k_cache) + row * a.d_I * act,
                 static_cast<const uint8_t*>(a.k_new) + static_cast<int64_t>(t) * a.d_I * act, a.d_I * act);
        return;
    }
    // FP8 keys: the first new token of the block requantises it
    const int lb = pos / kBlock;
    if (t > 0) {
        int b0, p0;
        const int prev = append_block(a, t - 1, b0, p0);
        if (prev >= 0 && b0 == b && p0 / kBlock == lb) return;
    }
    // the block's run of new tokens: rows t .. run_end - 1
    if (threadIdx.x == 0) run_end = min(a.T, t + kBlock);  // a block holds at most 64 new tokens
    __syncthreads();
    if (threadIdx.x < kBlock && threadIdx.x > 0) {
        const int u = t + static_cast<int>(threadIdx.x);
        int b2, p2;
        const bool same = u < a.T && append_block(a, u, b2, p2) >= 0 && b2 == b && p2 / kBlock == lb;
        if (!same) atomicMin(&run_end, u);
    }
    __syncthreads();
    const int m = run_end - t;
    const int n_old = pos - lb * kBlock;  // the block's earlier tokens: slots [0, n_old)
    const float old_scale = static_cast<const float*>(a.k_scale)[blk];
    uint8_t* codes = static_cast<uint8_t*>(a.k_cache) + static_cast<int64_t>(blk) * kBlock * a.d_I;
    const uint16_t* knew = static_cast<const uint16_t*>(a.k_new) + static_cast<int64_t>(t) * a.d_I;
    const int n_elem_old = n_old * a.d_I, n_elem_new = m * a.d_I;
    // amax over the earlier tokens (code * old scale) and the new keys
    float amax = 0.0f;
    for (int i = threadIdx.x; i < n_elem_old; i += kAppendThreads) amax = fmaxf(amax, fabsf(e4m3_value(codes[i]) * old_scale));
    for (int i = threadIdx.x; i < n_elem_new; i += kAppendThreads)
        amax = fmaxf(amax, fabsf(__uint_as_float(static_cast<uint32_t>(knew[i]) << 16)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
    // every code of the block's tokens, re-rounded against the new scale
    for (int i = threadIdx.x; i < n_elem_old; i += kAppendThreads) {
        const float x = e4m3_value(codes[i]) * old_scale;
        codes[i] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(x / scale, __NV_SATFINITE, __NV_E4M3));
    }
    for (int i = threadIdx.x; i < n_elem_new; i += kAppendThreads) {
        const int u = t + i / a.d_I;  // each new row into its own slot
        const int pu = a.q_pos ? a.q_pos[u] : pos;
        const float x = __uint_as_float(static_cast<uint32_t>(knew[i]) << 16);
        codes[(pu % kBlock) * a.d_I + i % a.d_I] =
            static_cast<uint8_t>(__nv_cvt_float_to_fp8(x / scale, __NV_SATFINITE, __NV_E4M3));
    }
    if (threadIdx.x == 0) static_cast<float*>(a.k_scale)[blk] = scale;
}

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendArgs a) { append_token(a, blockIdx.x); }

// Indexer prolog: the cache append of the step's new tokens (CTAs 0 .. T - 1) and, in the same
// launch, the MXFP8 quantisation of the indexer query (the other CTAs, one group of 32 elements per
// thread, written as its exact bf16 values to q_out) -- the two independent preparations the
// indexer needs ("Day0 Inference Support ... on Huawei Ascend CANN Architecture" §2.2, Indexer
// Prolog: Q quantisation runs beside the other preparations instead of after them).
__global__ void __launch_bounds__(kAppendThreads)
    indexer_prolog_kernel(AppendArgs a, const uint16_t* __restrict__ q, uint16_t* __restrict__ q_out, int64_t q_groups) {
    if (static_cast<int>(blockIdx.x) < a.T) {
        append_token(a, blockIdx.x);
        return;
    }
    const int64_t g = static_cast<int64_t>(blockIdx.x - a.T) * kAppendThreads + threadIdx.x;
    if (g < q_groups) mx_quantize_group32(q + g * 32, q_out + g * 32);
}

// ------------------------------------------------------------------------------------------------
// the rotated append: the same caches, the new rows' rotary columns turned on the way in
// ------------------------------------------------------------------------------------------------

struct RopeAppendArgs {
    AppendArgs a;
    dsa_rope_append r;
    const double* freq;
    int token_ctas;  // CTAs of warps that each write one row; the rest requantise FP8-key blocks
    int jobs_per_cta;
};

__device__ __forceinline__ float row_value(const void* x, bool f32, int e) {
    return f32 ? static_cast<const float*>(x)[e]
               : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(x)[e]) << 16);
}

// The pairs first, first + step, ... of one row's rotated columns, turned in fp32 into buf[0 .. rot).
__device__ __forceinline__ void rotate_row(const RopeAppendArgs& p, const void* x, int offset, int layout, int pos,
                                           float* buf, int first, int step) {
    const int half = p.r.rot / 2;
    for (int i = first; i < half; i += step) {
        const int e0 = layout == DSA_ROPE_INTERLEAVED ? 2 * i : i;
        const int e1 = layout == DSA_ROPE_INTERLEAVED ? 2 * i + 1 : i + half;
        const bool f32 = p.a.mode == DSA_F32;
        const float u = row_value(x, f32, offset + e0), v = row_value(x, f32, offset + e1);
        const float2 cs = rope_cos_sin(pos, p.freq[i], p.r.scale, false);
        const float2 y = rope_turn(u, v, cs);
        buf[e0] = y.x;
        buf[e1] = y.y;
    }
}

// Elements e .. e + 3 of a row whose columns offset .. offset + rot come from buf (offset < 0: none).
__device__ __forceinline__ float4 row_load4(const void* x, bool f32, int e, const float* buf, int offset, int rot) {
    float v[4];
    if (f32) {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + e);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + e);
        v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
    if (offset >= 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (static_cast<unsigned>(e + k - offset) < static_cast<unsigned>(rot)) v[k] = buf[e + k - offset];
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float amax4(const float4& v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

__device__ __forceinline__ uint32_t e4m3x4(const float4& v) {
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(v.x, __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float_to_fp8(v.y, __NV_SATFINITE, __NV_E4M3)) << 8 |
           static_cast<uint32_t>(__nv_cvt_float_to_fp8(v.z, __NV_SATFINITE, __NV_E4M3)) << 16 |
           static_cast<uint32_t>(__nv_cvt_float_to_fp8(v.w, __NV_SATFINITE, __NV_E4M3)) << 24;
}

// One row of n elements (fp32 or bf16) into dst in the same type.
__device__ __forceinline__ void store_plain_row(const void* x, bool f32, int n, void* dst, const float* buf, int offset,
                                                int rot, int lane) {
    for (int e = 4 * lane; e < n; e += 128) {
        const float4 v = row_load4(x, f32, e, buf, offset, rot);
        if (f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(dst) + e) = v;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dst) + e) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
    }
}

// FP8 keys: the block of new token t, requantised as a whole if t is its first new token (the CTA).
__device__ void requantise_block_rope(const RopeAppendArgs& p, int t, float* buf) {
    const AppendArgs& a = p.a;
    __shared__ float red[kAppendThreads / 32];
    __shared__ int run_end;
    int b, pos;
    const int blk = append_block(a, t, b, pos);
    if (blk < 0) return;  // reported by the token's own warps
    const int lb = pos / kBlock;
    if (t > 0) {
        int b0, p0;
        if (append_block(a, t - 1, b0, p0) >= 0 && b0 == b && p0 / kBlock == lb) return;
    }
    if (threadIdx.x == 0) run_end = min(a.T, t + kBlock);
    __syncthreads();
    if (threadIdx.x < kBlock && threadIdx.x > 0) {
        const int u = t + static_cast<int>(threadIdx.x);
        int b2, p2;
        const bool same = u < a.T && append_block(a, u, b2, p2) >= 0 && b2 == b && p2 / kBlock == lb;
        if (!same) atomicMin(&run_end, u);
    }
    __syncthreads();
    const int m = run_end - t, n_old = pos - lb * kBlock, d_I = a.d_I;
    const uint16_t* knew = static_cast<const uint16_t*>(a.k_new) + static_cast<int64_t>(t) * d_I;
    const bool turned = p.r.k_offset >= 0;
    if (turned) {
        for (int u = threadIdx.x >> 5; u < m; u += kAppendThreads / 32)
            rotate_row(p, knew + u * d_I, p.r.k_offset, p.r.k_layout, a.q_pos ? a.q_pos[t + u] : pos, buf + u * p.r.rot,
                       threadIdx.x & 31, 32);
        __syncthreads();
    }
    auto fresh = [&](int i) {  // element i of the run's new keys
        const int u = i / d_I, e = i - u * d_I - p.r.k_offset;
        return turned && static_cast<unsigned>(e) < static_cast<unsigned>(p.r.rot) ? buf[u * p.r.rot + e]
                                                                                    : row_value(knew, false, i);
    };
    const float old_scale = static_cast<const float*>(a.k_scale)[blk];
    uint8_t* codes = static_cast<uint8_t*>(a.k_cache) + static_cast<int64_t>(blk) * kBlock * d_I;
    float amax = 0.0f;
    for (int i = threadIdx.x; i < n_old * d_I; i += kAppendThreads) amax = fmaxf(amax, fabsf(e4m3_value(codes[i]) * old_scale));
    for (int i = threadIdx.x; i < m * d_I; i += kAppendThreads) amax = fmaxf(amax, fabsf(fresh(i)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float scale = amax > 0.0f ? amax / 448.0f : 1.0f;
    for (int i = threadIdx.x; i < n_old * d_I; i += kAppendThreads)
        codes[i] = static_cast<uint8_t>(
            __nv_cvt_float_to_fp8(e4m3_value(codes[i]) * old_scale / scale, __NV_SATFINITE, __NV_E4M3));
    for (int i = threadIdx.x; i < m * d_I; i += kAppendThreads) {
        const int u = t + i / d_I;
        const int pu = a.q_pos ? a.q_pos[u] : pos;
        codes[(pu % kBlock) * d_I + i % d_I] =
            static_cast<uint8_t>(__nv_cvt_float_to_fp8(fresh(i) / scale, __NV_SATFINITE, __NV_E4M3));
    }
    if (threadIdx.x == 0) static_cast<float*>(a.k_scale)[blk] = scale;
}

// Warp jobs 2t and 2t + 1 write token t's latent row and its key: the rotated columns go through a
// per-warp buffer in shared memory in fp32 and are rounded once, into the cache's type. Bound by the chain
// of loads that leads to a token's place and by the arithmetic of its rows (a token's two warps execute 1458
// instructions for an FP8 record and an MXFP8 key, the divisions by its scales among them; the schedulers issue in 53%
// of the cycles). (One warp for both rows of a token, its tiles in registers, took 30 us for 8192 fp8 tokens of
// 512 + 128 from a cold L2, two warps without the prefetch and one tile at a time 24, this form 20.)
__global__ void __launch_bounds__(kAppendThreads) cache_append_rope_kernel(RopeAppendArgs p) {
    extern __shared__ float rope_buf[];
    const AppendArgs& a = p.a;
    if (static_cast<int>(blockIdx.x) >= p.token_ctas) {
        requantise_block_rope(p, blockIdx.x - p.token_ctas, rope_buf);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * p.jobs_per_cta + warp;
    if (warp >= p.jobs_per_cta || job >= 2ll * a.T) return;
    const int t = static_cast<int>(job >> 1);
    const bool key = job & 1;
    const bool f32 = a.mode == DSA_F32;
    const int act = f32 ? 4 : 2, n = key ? a.d_I : a.d, rot = p.r.rot;
    const int offset = key ? p.r.k_offset : p.r.kv_offset;
    const void* x = static_cast<const uint8_t*>(key ? a.k_new : a.kv_new) + static_cast<int64_t>(t) * n * act;
    // the row is on its way while the token's place is found (three loads, each waiting for the last)
    for (int o = 128 * lane; o < n * act; o += 128 * 32)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const uint8_t*>(x) + o));
    int b, pos;
    const int blk = append_block(a, t, b, pos);
    if (blk < 0) {
        if (lane == 0) atomicOr(a.err, (b < 0 || b >= a.B) ? DSA_FAULT_INDEX : DSA_FAULT_BLOCK_TABLE);
        return;
    }
    if (key && a.mode == DSA_BF16_KFP8) return;
    const int64_t row = static_cast<int64_t>(blk) * kBlock + pos % kBlock;
    float* buf = rope_buf + warp * rot;
    if (offset >= 0) {
        rotate_row(p, x, offset, key ? p.r.k_layout : p.r.kv_layout, pos, buf, lane, 32);
        __syncwarp();
    }
    if (!key && a.kv_fp8) {
        uint8_t* rec = static_cast<uint8_t*>(a.kv_cache) + row * DSA_KV_FP8_RECORD_BYTES(n);
        const int ntiles = (n + 127) / 128;
        constexpr int kTiles = 3;  // side by side: their reductions and divisions overlap
        for (int j0 = 0; j0 < ntiles; j0 += kTiles) {
            float4 v[kTiles];
            float amax[kTiles], scale[kTiles];
#pragma unroll
            for (int k = 0; k < kTiles; ++k) {
                const int e = 128 * (j0 + k) + 4 * lane;
                v[k] = e < n ? row_load4(x, f32, e, buf, offset, rot) : make_float4(0.f, 0.f, 0.f, 0.f);
                amax[k] = amax4(v[k]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < kTiles; ++k) amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xFFFFFFFFu, amax[k], o));
#pragma unroll
            for (int k = 0; k < kTiles; ++k) {
                const int e = 128 * (j0 + k) + 4 * lane;
                scale[k] = amax[k] > 0.0f ? amax[k] / 448.0f : 1.0f;
                if (e < n)
                    *reinterpret_cast<uint32_t*>(rec + e) =
                        e4m3x4(make_float4(v[k].x / scale[k], v[k].y / scale[k], v[k].z / scale[k], v[k].w / scale[k]));
                if (lane == 0 && j0 + k < ntiles) *reinterpret_cast<float*>(rec + n + 4 * (j0 + k)) = scale[k];
            }
        }
        for (int i = n + 4 * ntiles + lane; i < DSA_KV_FP8_RECORD_BYTES(n); i += 32) rec[i] = 0;
    } else if (key && a.mode == DSA_MXFP8) {
        for (int e0 = 0; e0 < n; e0 += 128) {  // eight lanes hold one group of 32
            const int e = e0 + 4 * lane;
            const float4 v = e < n ? row_load4(x, f32, e, buf, offset, rot) : make_float4(0.f, 0.f, 0.f, 0.f);
            float amax = amax4(v);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            if (e >= n) continue;
            const int X = mx_exponent(amax);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.k_cache) + row * n + e) =
                e4m3x4(make_float4(v.x * down, v.y * down, v.z * down, v.w * down));
            if ((lane & 7) == 0) static_cast<uint8_t*>(a.k_scale)[row * (n / 32) + e / 32] = static_cast<uint8_t>(X + 127);
        }
    } else {
        store_plain_row(x, f32, n, static_cast<uint8_t*>(key ? a.k_cache : a.kv_cache) + row * n * act, buf, offset, rot, lane);
    }
}

bool launch_cache_append_rope(const dsa_dims& d, bool kv_fp8, const dsa_rope_append& r, const double* freq,
                              const void* k_new, const void* kv_new, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* q_seq, const int32_t* q_pos, int T, void* k_cache,
                              void* k_scale, void* kv_cache, int* err, cudaStream_t s, int* launches) {
    if (T == 0) return true;
    RopeAppendArgs p{};
    p.a = AppendArgs{d.mode, kv_fp8 ? 1 : 0, d.B, d.max_blocks, d.num_blocks, d.d_I, d.d, T, k_new, kv_new, block_table,
                     seq_lens, q_seq, q_pos, k_cache, k_scale, kv_cache, err};
    p.r = r;
    p.freq = freq;
    p.jobs_per_cta = kAppendThreads / 32;
    p.token_ctas = static_cast<int>((2ll * T + p.jobs_per_cta - 1) / p.jobs_per_cta);
    const bool blocks = d.mode == DSA_BF16_KFP8;
    const size_t smem = sizeof(float) * r.rot * (blocks ? kBlock : kAppendThreads / 32);
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(cache_append_rope_kernel), smem)) return false;
    if (!launch_kernel(false, cache_append_rope_kernel, dim3(p.token_ctas + (blocks ? T : 0)), dim3(kAppendThreads), smem,
                       s, p))
        return false;
    ++*launches;
    return true;
}

bool launch_cache_append(const dsa_dims& d, bool kv_fp8, const void* k_new, const void* kv_new,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                         const int32_t* q_pos, int T, void* k_cache, void* k_scale, void* kv_cache, int* err,
                         cudaStream_t s, int* launches) {
    if (T == 0) return true;
    AppendArgs a{d.mode, kv_fp8 ? 1 : 0, d.B, d.max_blocks, d.num_blocks, d.d_I, d.d, T, k_new, kv_new, block_table,
                 seq_lens, q_seq, q_pos, k_cache, k_scale, kv_cache, err};
    if (!launch_kernel(false, cache_append_kernel, dim3(T), dim3(kAppendThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

bool launch_indexer_prolog(const dsa_dims& d, bool kv_fp8, const void* k_new, const void* kv_new,
                           const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                           const int32_t* q_pos, int T, void* k_cache, void* k_scale, void* kv_cache, const void* q_I,
                           void* q_out, int64_t q_elements, int* err, cudaStream_t s, int* launches) {
    const int64_t q_groups = q_out ? q_elements / 32 : 0;
    const int64_t q_ctas = (q_groups + kAppendThreads - 1) / kAppendThreads;
    if (T == 0 && q_ctas == 0) return true;
    AppendArgs a{d.mode, kv_fp8 ? 1 : 0, d.B, d.max_blocks, d.num_blocks, d.d_I, d.d, T, k_new, kv_new, block_table,
                 seq_lens, q_seq, q_pos, k_cache, k_scale, kv_cache, err};
    if (!launch_kernel(false, indexer_prolog_kernel, dim3(static_cast<unsigned>(T + q_ctas)), dim3(kAppendThreads), 0, s,
                       a, static_cast<const uint16_t*>(q_I), static_cast<uint16_t*>(q_out), q_groups))
        return false;
    ++*launches;
    return true;
}

}  // namespace dsa
