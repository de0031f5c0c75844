// Cache read-back: ranges of the paged caches as dense rows, the inverse of the cache append. A
// chunked prompt reads its cached prefix back before projecting it up for the prompt attention.
//
// Row r of the outputs belongs to the sequence b with cu_rows[b] <= r < cu_rows[b + 1] and holds its
// position start[b] + r - cu_rows[b]: FP8 latent records as code * tile scale, FP8 keys as
// code * block scale, MXFP8 keys as code * 2^X, in fp32, rounded once to bf16; the other modes copy.
// Every code is read once and written once as two bytes: 64K rows of 608 + 132 bytes take 27.5 us (141 MB, 76% of
// the measured copy bandwidth). No unit is full: the schedulers issue in 61% of the cycles, the integer pipe works
// in 51% of them and a warp mostly waits for its loads. 173 instructions go to 16 codes of each lane, about 60 of
// them the widening, the rest indexes and 64-bit addresses. One even turn of CTAs, each with a run of rows: its
// threads find one row's place each (a chain of loads that all CTAs begin with together), and then keep two pieces
// in flight (four, with fewer CTAs, took 31 us).
#include "internal.h"

namespace dsa {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 256;   // rows per CTA at most: a thread finds the place of one
constexpr int kReadLeast = 8;    // ... and at least, where there are enough CTAs
constexpr int kReadCtas = 6;     // per SM
constexpr int kReadBatch = 2;    // pieces a thread has in flight
constexpr int kReadSeqs = 1024;  // sequences whose first rows fit shared memory

struct ReadArgs {
    int mode;
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
    int rows;        // per CTA
    uint32_t magic;  // i / (pieces of a row) = umulhi(i, magic) for every piece of a CTA
};

// A row's piece: 16 codes (32 bytes of bf16 out) or 16 bytes copied.
struct ReadPiece {
    uint4 x;
    float f;        // scale of the codes
    uint8_t* dst;   // nullptr: nothing to write
    bool zero;
};

__device__ __forceinline__ void write_piece(const ReadPiece& p, bool codes) {
    if (!p.dst) return;
    uint4 lo = p.zero ? make_uint4(0, 0, 0, 0) : p.x, hi = lo;
    if (codes && !p.zero) e4m3x16_to_bf16_scaled(p.x, p.f, lo, hi);
    if (codes && (reinterpret_cast<uintptr_t>(p.dst) & 31) == 0) {  // whole sectors
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store_32b(p.dst, w);
        return;
    }
    reinterpret_cast<uint4*>(p.dst)[0] = lo;
    if (codes) reinterpret_cast<uint4*>(p.dst)[1] = hi;
}

// First the rows' places (the sequences' first rows in shared memory, so that the search waits for memory
// once, then each row's block), then every thread's pieces of latent rows and keys, kReadBatch at a time.
template <bool kKvCodes, int kKeyMode>  // latent rows as FP8 records; keys: DSA_BF16 (copied), DSA_BF16_KFP8, DSA_MXFP8
__global__ void __launch_bounds__(kReadThreads, kReadCtas) cache_read_kernel(ReadArgs a) {
    __shared__ int64_t phys[kReadRows];  // physical cache row, -1: zeros, -2: not written
    __shared__ int32_t cu[kReadSeqs + 1];
    const int r0 = blockIdx.x * a.rows, n = min(a.rows, a.R - r0), tid = threadIdx.x;
    const bool shared = a.B <= kReadSeqs;
    if (shared) {
        for (int i = tid; i <= a.B; i += kReadThreads) cu[i] = a.cu_rows[i];
        __syncthreads();
    }
    if (tid < n) {
        const int32_t* first = shared ? cu : a.cu_rows;
        const int r = r0 + tid;
        int lo = 0, hi = a.B;  // the last b with first[b] <= r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        int64_t p = -2;
        if (lo < a.B && first[lo] <= r) {
            const int64_t pos = static_cast<int64_t>(a.start ? a.start[lo] : 0) + r - first[lo];
            const bool in_table = pos >= 0 && pos / kBlock < a.max_blocks;
            const int blk = in_table ? a.block_table[static_cast<int64_t>(lo) * a.max_blocks + pos / kBlock] : -1;
            p = -1;
            if (!in_table || pos >= a.seq_lens[lo]) atomicOr(a.err, DSA_FAULT_INDEX);
            else if (blk < 0 || blk >= a.num_blocks) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
            else p = static_cast<int64_t>(blk) * kBlock + pos % kBlock;
        }
        phys[tid] = p;
    }
    __syncthreads();
    constexpr bool kKeyCodes = kKeyMode != DSA_BF16;
    const int act = a.mode == DSA_F32 ? 4 : 2;
    const int kv_rec = kKvCodes ? DSA_KV_FP8_RECORD_BYTES(a.d) : a.d * act, k_rec = kKeyCodes ? a.d_I : a.d_I * act;
    const int kv_units = !a.kv_out ? 0 : kKvCodes ? a.d / 16 : a.d * act / 16;
    const int units = kv_units + (!a.k_out ? 0 : kKeyCodes ? a.d_I / 16 : a.d_I * act / 16), total = n * units;
    for (int i0 = tid; i0 < total; i0 += kReadBatch * kReadThreads) {
        ReadPiece p[kReadBatch];
        bool key[kReadBatch];
#pragma unroll
        for (int b = 0; b < kReadBatch; ++b) {
            const int i = i0 + b * kReadThreads;
            p[b].dst = nullptr;
            key[b] = false;
            if (i >= total) continue;
            const int r = units == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.magic)), u = i - r * units;
            const int64_t row = phys[r], out = r0 + r;
            if (row == -2) continue;
            p[b].zero = row == -1;
            key[b] = u >= kv_units;
            if (!key[b]) {
                p[b].dst = static_cast<uint8_t*>(a.kv_out) + out * a.d * act + u * (kKvCodes ? 32 : 16);
                if (p[b].zero) continue;
                const uint8_t* src = static_cast<const uint8_t*>(a.kv_cache) + row * kv_rec;
                p[b].x = reinterpret_cast<const uint4*>(src)[u];
                if (kKvCodes) p[b].f = *reinterpret_cast<const float*>(src + a.d + 4 * (u / 8));
            } else {
                const int w = u - kv_units;
                p[b].dst = static_cast<uint8_t*>(a.k_out) + out * a.d_I * act + w * (kKeyCodes ? 32 : 16);
                if (p[b].zero) continue;
                p[b].x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k_cache) + row * k_rec)[w];
                if (kKeyMode == DSA_MXFP8) p[b].f = e8m0_value(static_cast<const uint8_t*>(a.k_scale)[row * (a.d_I / 32) + w / 2]);
                if (kKeyMode == DSA_BF16_KFP8) p[b].f = static_cast<const float*>(a.k_scale)[row / kBlock];
            }
        }
#pragma unroll
        for (int b = 0; b < kReadBatch; ++b) write_piece(p[b], kKvCodes == kKeyCodes ? kKvCodes : key[b] ? kKeyCodes : kKvCodes);
    }
}

bool launch_cache_read(const dsa_dims& d, bool kv_fp8, const void* k_cache, const void* k_scale, const void* kv_cache,
                       const int32_t* block_table, const int32_t* seq_lens, const int32_t* start, const int32_t* cu_rows,
                       int R, void* k_out, void* kv_out, int* err, cudaStream_t s, int* launches) {
    if (R == 0 || (!k_out && !kv_out)) return true;
    const int ctas = kReadCtas * device_sm_count();
    int rows = static_cast<int>((static_cast<int64_t>(R) + ctas - 1) / ctas);  // one even turn of CTAs
    rows = rows < kReadLeast ? kReadLeast : rows > kReadRows ? kReadRows : rows;
    const int act = d.mode == DSA_F32 ? 4 : 2, key = d.mode == DSA_F32 ? DSA_BF16 : d.mode;
    const int64_t units = (kv_out ? (kv_fp8 ? d.d / 16 : d.d * act / 16) : 0) +
                          (k_out ? (key != DSA_BF16 ? d.d_I / 16 : d.d_I * act / 16) : 0);
    // umulhi(i, ceil(2^32 / units)) = i / units while i * units < 2^32 (units are below 2^16)
    const int64_t most = ((1ll << 32) - 1) / (units * units);
    if (rows > most) rows = static_cast<int>(most);
    const uint32_t magic = units > 1 ? static_cast<uint32_t>(((1ll << 32) + units - 1) / units) : 0;
    ReadArgs a{d.mode, d.B, d.max_blocks, d.num_blocks, d.d_I, d.d, R, k_cache, k_scale, kv_cache,
               block_table, seq_lens, start, cu_rows, k_out, kv_out, err, rows, magic};
    auto* kernel = kv_fp8 ? (key == DSA_BF16 ? cache_read_kernel<true, DSA_BF16>
                             : key == DSA_MXFP8 ? cache_read_kernel<true, DSA_MXFP8> : cache_read_kernel<true, DSA_BF16_KFP8>)
                          : (key == DSA_BF16 ? cache_read_kernel<false, DSA_BF16>
                             : key == DSA_MXFP8 ? cache_read_kernel<false, DSA_MXFP8> : cache_read_kernel<false, DSA_BF16_KFP8>);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(R) + rows - 1) / rows);
    if (!launch_kernel(false, kernel, dim3(grid), dim3(kReadThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
