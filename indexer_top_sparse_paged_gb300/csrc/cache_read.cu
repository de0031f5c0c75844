// Cache read-back: ranges of the paged caches as dense rows, the inverse of the cache append. A
// chunked prompt reads its cached prefix back before projecting it up for the prompt attention.
//
// Row r of the outputs belongs to the sequence b with cu_rows[b] <= r < cu_rows[b + 1] and holds its
// position start[b] + r - cu_rows[b]: FP8 latent records as code * tile scale, FP8 keys as
// code * block scale, MXFP8 keys as code * 2^X, in fp32, rounded once to bf16; the other modes copy.
// Bound by memory: every code is read once and written once as two bytes.
#include "internal.h"

namespace dsa {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // rows per CTA

struct ReadArgs {
    int mode, kv_fp8;
    int B, max_blocks, num_blocks;
    int d_I, d;
    int R;
    const void* k_cache;
    const void* k_scale;
    const void* kv_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* start;
    const int32_t* cu_rows;
    void* k_out;
    void* kv_out;
    int* err;
};

// 16 codes at src times f -> 32 bytes of bf16 at dst.
__device__ __forceinline__ void read_codes16(const uint8_t* src, float f, uint8_t* dst) {
    uint4 lo, hi;
    e4m3x16_to_bf16_scaled(*reinterpret_cast<const uint4*>(src), f, lo, hi);
    reinterpret_cast<uint4*>(dst)[0] = lo;
    reinterpret_cast<uint4*>(dst)[1] = hi;
}

__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(ReadArgs a) {
    __shared__ int64_t phys[kReadRows];  // physical cache row, -1: zeros, -2: not written
    const int r0 = blockIdx.x * kReadRows, n = min(kReadRows, a.R - r0);
    if (static_cast<int>(threadIdx.x) < n) {
        const int r = r0 + threadIdx.x;
        int lo = 0, hi = a.B;  // the last b with cu_rows[b] <= r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_rows[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        int64_t p = -2;
        if (lo < a.B && a.cu_rows[lo] <= r) {
            const int64_t pos = static_cast<int64_t>(a.start ? a.start[lo] : 0) + r - a.cu_rows[lo];
            p = -1;
            if (pos < 0 || pos >= a.seq_lens[lo] || pos / kBlock >= a.max_blocks) {
                atomicOr(a.err, DSA_FAULT_INDEX);
            } else {
                const int blk = a.block_table[static_cast<int64_t>(lo) * a.max_blocks + pos / kBlock];
                if (blk < 0 || blk >= a.num_blocks) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
                else p = static_cast<int64_t>(blk) * kBlock + pos % kBlock;
            }
        }
        phys[threadIdx.x] = p;
    }
    __syncthreads();
    const int act = a.mode == DSA_F32 ? 4 : 2;
    const bool k_codes = a.mode == DSA_BF16_KFP8 || a.mode == DSA_MXFP8;
    if (a.kv_out) {
        const int units = a.kv_fp8 ? a.d / 16 : a.d * act / 16;  // 16 codes, or 16 bytes
        const int rec = a.kv_fp8 ? DSA_KV_FP8_RECORD_BYTES(a.d) : a.d * act;
        for (int i = threadIdx.x; i < n * units; i += kReadThreads) {
            const int r = i / units, u = i - r * units;
            const int64_t p = phys[r];
            if (p == -2) continue;
            const uint8_t* src = static_cast<const uint8_t*>(a.kv_cache) + p * rec;
            uint8_t* dst = static_cast<uint8_t*>(a.kv_out) + static_cast<int64_t>(r0 + r) * a.d * act;
            if (a.kv_fp8) {
                if (p >= 0) {
                    read_codes16(src + 16 * u, *reinterpret_cast<const float*>(src + a.d + 4 * (u / 8)), dst + 32 * u);
                } else {
                    reinterpret_cast<uint4*>(dst)[2 * u] = make_uint4(0, 0, 0, 0);
                    reinterpret_cast<uint4*>(dst)[2 * u + 1] = make_uint4(0, 0, 0, 0);
                }
            } else {
                reinterpret_cast<uint4*>(dst)[u] = p >= 0 ? reinterpret_cast<const uint4*>(src)[u] : make_uint4(0, 0, 0, 0);
            }
        }
    }
    if (a.k_out) {
        const int units = k_codes ? a.d_I / 16 : a.d_I * act / 16;
        for (int i = threadIdx.x; i < n * units; i += kReadThreads) {
            const int r = i / units, u = i - r * units;
            const int64_t p = phys[r];
            if (p == -2) continue;
            uint8_t* dst = static_cast<uint8_t*>(a.k_out) + static_cast<int64_t>(r0 + r) * a.d_I * act;
            if (k_codes) {
                if (p >= 0) {
                    const float f = a.mode == DSA_MXFP8
                                        ? e8m0_value(static_cast<const uint8_t*>(a.k_scale)[p * (a.d_I / 32) + u / 2])
                                        : static_cast<const float*>(a.k_scale)[p / kBlock];
                    read_codes16(static_cast<const uint8_t*>(a.k_cache) + p * a.d_I + 16 * u, f, dst + 32 * u);
                } else {
                    reinterpret_cast<uint4*>(dst)[2 * u] = make_uint4(0, 0, 0, 0);
                    reinterpret_cast<uint4*>(dst)[2 * u + 1] = make_uint4(0, 0, 0, 0);
                }
            } else {
                const uint8_t* src = static_cast<const uint8_t*>(a.k_cache) + p * a.d_I * act;
                reinterpret_cast<uint4*>(dst)[u] = p >= 0 ? reinterpret_cast<const uint4*>(src)[u] : make_uint4(0, 0, 0, 0);
            }
        }
    }
}

bool launch_cache_read(const dsa_dims& d, bool kv_fp8, const void* k_cache, const void* k_scale, const void* kv_cache,
                       const int32_t* block_table, const int32_t* seq_lens, const int32_t* start, const int32_t* cu_rows,
                       int R, void* k_out, void* kv_out, int* err, cudaStream_t s, int* launches) {
    if (R == 0 || (!k_out && !kv_out)) return true;
    ReadArgs a{d.mode, kv_fp8 ? 1 : 0, d.B, d.max_blocks, d.num_blocks, d.d_I, d.d, R, k_cache, k_scale, kv_cache,
               block_table, seq_lens, start, cu_rows, k_out, kv_out, err};
    if (!launch_kernel(false, cache_read_kernel, dim3((R + kReadRows - 1) / kReadRows), dim3(kReadThreads), 0, s, a))
        return false;
    ++*launches;
    return true;
}

}  // namespace dsa
