// Host side of the C ABI (include/dsa.h): argument checks, workspace layout, kernel selection and
// launch order. Nothing here allocates, frees or synchronises (dsa_read_error excepted).
//
// Kernel selection follows the shape of the call ("Adapting GPU Software Stacks ..." §3.3:
// separate implementations per path, chosen at run time from batch size and sequence length):
// tensor-core kernels for the 64x128 indexer and the 128-head x 576 latent attention, CUDA-core
// kernels for small shapes (the fp32 workload).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <vector>

#include "grouped.cuh"
#include "internal.h"

namespace dsa {

static thread_local int g_last_launches = 0;

constexpr int kMaxDevices = 64;

int device_sm_count() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev >= 0 && dev < kMaxDevices && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (dev >= 0 && dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool set_max_dynamic_smem(const void* func, size_t bytes) {
    struct Entry {
        int dev;
        const void* func;
        size_t bytes;
    };
    static std::mutex mu;
    static std::vector<Entry> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : done)
        if (e.dev == dev && e.func == func && e.bytes >= bytes) return true;
    if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
        return false;
    done.push_back({dev, func, bytes});
    return true;
}

bool indexer_uses_tc(const dsa_dims& d) {
    return (d.mode == DSA_BF16 || d.mode == DSA_BF16_KFP8 || d.mode == DSA_MXFP8) && d.H_I == 64 && d.d_I == 128;
}

bool attn_uses_tc(const dsa_dims& d) {
    return (d.mode == DSA_BF16 || d.mode == DSA_BF16_KFP8 || d.mode == DSA_MXFP8) && d.H == 128 && d.d == 576 &&
           d.d_v == 512;
}

// Widths that two query tiles and their accumulators leave room for in shared and tensor memory; the
// keys' and values' rows are found through tensor maps, whose outer strides are not 0.
bool prompt_uses_tc(const dsa_prompt_dims& p) {
    return p.type == DSA_BF16 && p.d_qk <= 192 && p.d_v <= 128 && p.k_stride_t > 0 && p.v_stride_t > 0;
}

int indexer_ctas(const dsa_dims& d) {
    const int sms = device_sm_count();
    const int G = indexer_uses_tc(d) ? sms : 2 * sms;
    return G < kMaxIndexerCtas ? G : kMaxIndexerCtas;
}

int attn_splits(const dsa_dims& d, int T) {
    if (!attn_uses_tc(d) || T <= 0) return 1;
    const int sms = device_sm_count();
    int S = sms / (2 * T);
    int smax = d.K / 64;
    if (smax > kMaxSplits) smax = kMaxSplits;
    if (S > smax) S = smax;
    return S < 1 ? 1 : S;
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool prefill_path(const dsa_dims& d, int T) { return indexer_uses_tc(d) && T >= 4 && T > d.B; }

WsLayout ws_layout(const dsa_dims& d, int T, bool allow_prefill) {
    WsLayout w{};
    w.G = indexer_ctas(d);
    w.S = attn_splits(d, T);
    w.NG = (allow_prefill && prefill_path(d, T)) ? T / 4 : 0;
    size_t off = 0;
    w.err = off;
    off += 256;
    w.tile_prefix = off;
    off = align256(off + sizeof(int32_t) * (static_cast<size_t>(T) + 1));
    w.group_prefix = off;
    off = align256(off + sizeof(int32_t) * (static_cast<size_t>(T) + 1));
    w.merge_count = off;
    off = align256(off + sizeof(int32_t) * (kMergeLevels - 1) * static_cast<size_t>(merge_group_bound(T, w.G)));
    w.slot_count = off;
    off = align256(off + sizeof(int32_t) * (static_cast<size_t>(w.G) + T));
    w.slots = off;
    off = align256(off + sizeof(uint64_t) * (static_cast<size_t>(w.G) + T) * d.K);
    w.slot_est = off;
    off = align256(off + sizeof(uint64_t) * (static_cast<size_t>(w.G) + T));
    w.q_mx = off;
    if (d.mode == DSA_MXFP8) off = align256(off + sizeof(uint16_t) * static_cast<size_t>(T) * d.H_I * d.d_I);
    w.idx = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T) * d.K);
    w.part_o = off;
    if (w.S > 1) off = align256(off + sizeof(float) * static_cast<size_t>(T) * w.S * d.H * d.d_v);
    w.part_ml = off;
    if (w.S > 1) off = align256(off + sizeof(float) * static_cast<size_t>(T) * w.S * 2 * d.H * 2);
    w.gemm_flag = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(w.NG));
    w.gemm_tile_prefix = off;
    off = align256(off + sizeof(int32_t) * (static_cast<size_t>(w.NG) + 1));
    w.scores = off;
    if (w.NG > 0) off = align256(off + sizeof(float) * static_cast<size_t>(T) * d.max_blocks * kBlock);
    w.total = off;
    return w;
}

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

static EncodeTiled encode_fn() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}

bool make_tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t cols, uint64_t rows,
                  uint64_t pitch_bytes, uint32_t box_cols, uint32_t box_rows) {
    EncodeTiled fn = encode_fn();
    if (!fn || rows == 0) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {pitch_bytes};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_tmap_3d(CUtensorMap* map, const void* base, const uint64_t (&dims)[3], const uint64_t (&strides)[2],
                  const uint32_t (&box)[3]) {
    EncodeTiled fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
    const cuuint64_t s[2] = {strides[0], strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), d, s, b, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------------------------------------
// argument checks
// ------------------------------------------------------------------------------------------------

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The public mode may carry DSA_KV_FP8 (the latent cache's storage); every kernel below takes the
// indexer-key mode alone, and the attention and the cache append get the flag on its own.
static dsa_status split_mode(const dsa_dims* in, dsa_dims* out, bool* kv8) {
    if (!in) return DSA_ERR_INVALID_ARG;
    *out = *in;
    *kv8 = (in->mode & DSA_KV_FP8) != 0;
    out->mode = in->mode & ~(DSA_KV_FP8 | DSA_Q_MX_READY);
    if (*kv8 && (out->mode == DSA_F32 || in->d % 16)) return DSA_ERR_UNSUPPORTED;
    if ((in->mode & DSA_Q_MX_READY) && out->mode != DSA_MXFP8) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

// DSA_Q_MX_READY: q_I already holds the MXFP8 values (dsa_indexer_prolog wrote them).
static bool q_mx_ready(const dsa_dims* in) { return (in->mode & DSA_Q_MX_READY) != 0; }

static dsa_status check_common(const dsa_dims* d) {
    if (!d) return DSA_ERR_INVALID_ARG;
    if (d->mode < DSA_F32 || d->mode > DSA_MXFP8) return DSA_ERR_UNSUPPORTED;
    if (d->block_size != kBlock) return DSA_ERR_UNSUPPORTED;
    if (d->B <= 0 || d->max_blocks <= 0 || d->num_blocks <= 0) return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(d->num_blocks) * kBlock >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->max_blocks) * kBlock >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    if (d->K <= 0 || d->K > 2048) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

static dsa_status check_indexer_dims(const dsa_dims* d) {
    dsa_status st = check_common(d);
    if (st != DSA_OK) return st;
    if (d->H_I <= 0 || d->d_I <= 0) return DSA_ERR_INVALID_ARG;
    if (indexer_uses_tc(*d)) return DSA_OK;
    if (d->H_I > 64 || d->d_I > 256) return DSA_ERR_UNSUPPORTED;
    const int unit = d->mode == DSA_F32 ? 4 : (d->mode == DSA_BF16 ? 8 : (d->mode == DSA_MXFP8 ? 32 : 16));
    if (d->d_I % unit) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

// The key scales a mode needs: fp32 per block (FP8 keys) or E8M0 bytes, 16-byte aligned (MXFP8,
// fetched with bulk copies).
static bool scale_ok(const dsa_dims* d, const void* k_I_scale) {
    if (d->mode == DSA_BF16_KFP8) return k_I_scale != nullptr;
    if (d->mode == DSA_MXFP8) return k_I_scale != nullptr && aligned16(k_I_scale);
    return true;
}

static dsa_status check_attn_dims(const dsa_dims* d) {
    dsa_status st = check_common(d);
    if (st != DSA_OK) return st;
    if (d->H <= 0 || d->d <= 0 || d->d_v <= 0 || d->d_v > d->d) return DSA_ERR_INVALID_ARG;
    if (attn_uses_tc(*d)) return DSA_OK;
    if (d->H > 128 || d->d > 1024) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

static dsa_status check_ws(const dsa_dims* d, int T, void* ws, size_t ws_bytes) {
    if (!ws) return DSA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return DSA_ERR_WORKSPACE;
    if (ws_bytes < ws_layout(*d, T).total) return DSA_ERR_WORKSPACE;
    return DSA_OK;
}

static dsa_status run_indexer(const dsa_dims* d, const void* q_I, const float* w, const void* k_I_cache,
                              const void* k_I_scale, const int32_t* block_table, const int32_t* seq_lens,
                              const int32_t* q_seq, const int32_t* q_pos, int32_t T, int32_t* idx, void* ws,
                              cudaStream_t stream, int* launches, bool allow_prefill = true, bool q_ready = false) {
    const WsLayout L = ws_layout(*d, T, allow_prefill);
    uint8_t* base = static_cast<uint8_t*>(ws);
    IndexerArgs a{};
    a.mode = d->mode;
    a.B = d->B;
    a.max_blocks = d->max_blocks;
    a.num_blocks = d->num_blocks;
    a.H_I = d->H_I;
    a.d_I = d->d_I;
    a.K = d->K;
    a.T = T;
    a.q_I = q_I;
    a.w = w;
    a.k_I = k_I_cache;
    a.k_I_scale = k_I_scale;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.q_seq = q_seq;
    a.q_pos = q_pos;
    a.tile_prefix = reinterpret_cast<int32_t*>(base + L.tile_prefix);
    a.group_prefix = reinterpret_cast<int32_t*>(base + L.group_prefix);
    a.merge_count = reinterpret_cast<int32_t*>(base + L.merge_count);
    a.slot_count = reinterpret_cast<int32_t*>(base + L.slot_count);
    a.slots = reinterpret_cast<uint64_t*>(base + L.slots);
    a.slot_est = reinterpret_cast<uint64_t*>(base + L.slot_est);
    a.idx = idx;
    a.err = reinterpret_cast<int*>(base + L.err);
    a.G = L.G;
    a.NG = q_seq ? L.NG : 0;
    a.gemm_flag = reinterpret_cast<int32_t*>(base + L.gemm_flag);
    a.gemm_tile_prefix = reinterpret_cast<int32_t*>(base + L.gemm_tile_prefix);
    a.scores = reinterpret_cast<float*>(base + L.scores);
    a.G2 = device_sm_count();
    if (d->mode == DSA_MXFP8 && !q_ready) {  // the quantised query first; the indexer kernels read it as bf16
        void* q_mx = base + L.q_mx;
        if (!launch_mx_quantize_q(q_I, q_mx, static_cast<int64_t>(T) * d->H_I * d->d_I, stream, launches))
            return DSA_ERR_LAUNCH;
        a.q_I = q_mx;
        a.after_quant = 1;
    }
    // decode calls on the tensor-core indexer plan inside its kernel (no plan kernel, no gap)
    a.self_plan = (a.NG == 0 && indexer_uses_tc(*d) && T <= kSelfPlanRows) ? 1 : 0;
    if (!a.self_plan && !launch_plan(a, stream, launches)) return DSA_ERR_LAUNCH;
    if (a.NG > 0 && !launch_indexer_prefill(a, stream, launches)) return DSA_ERR_LAUNCH;
    const bool ok = indexer_uses_tc(*d) ? launch_indexer_tc(a, stream, launches) : launch_indexer_simt(a, stream, launches);
    if (!ok) return DSA_ERR_LAUNCH;
    if (!launch_merge(a, stream, launches)) return DSA_ERR_LAUNCH;
    if (a.NG > 0 && !launch_prefill_topk(a, stream, launches)) return DSA_ERR_LAUNCH;
    return DSA_OK;
}

static dsa_status run_attn(const dsa_dims* d, bool kv8, const void* q, const void* kv_cache,
                           const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                           const int32_t* idx, int32_t T, float sm_scale, void* out, float* lse, void* ws,
                           cudaStream_t stream, int* launches, bool after_own_kernel) {
    const WsLayout L = ws_layout(*d, T);
    uint8_t* base = static_cast<uint8_t*>(ws);
    AttnArgs a{};
    a.mode = d->mode;
    a.B = d->B;
    a.max_blocks = d->max_blocks;
    a.num_blocks = d->num_blocks;
    a.H = d->H;
    a.d = d->d;
    a.d_v = d->d_v;
    a.K = d->K;
    a.T = T;
    a.sm_scale = sm_scale;
    a.q = q;
    a.kv = kv_cache;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.q_seq = q_seq;
    a.idx = idx;
    a.out = out;
    a.lse = lse;
    a.part_o = reinterpret_cast<float*>(base + L.part_o);
    a.part_ml = reinterpret_cast<float*>(base + L.part_ml);
    a.S = L.S;
    a.err = reinterpret_cast<int*>(base + L.err);
    a.after_own_kernel = after_own_kernel ? 1 : 0;
    a.kv_fp8 = kv8 ? 1 : 0;
    a.kv_rec = kv8 ? DSA_KV_FP8_RECORD_BYTES(d->d) : d->d * (d->mode == DSA_F32 ? 4 : 2);
    const bool ok = attn_uses_tc(*d) ? launch_attn_tc(a, stream, launches) : launch_attn_simt(a, stream, launches);
    return ok ? DSA_OK : DSA_ERR_LAUNCH;
}

// ------------------------------------------------------------------------------------------------
// scratch of dsa_indexer_topk_noalloc: one static device buffer per device, resolved once
// ------------------------------------------------------------------------------------------------

constexpr size_t kNoAllocScratchBytes = DSA_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

static std::mutex g_noalloc_mu;
static void* g_noalloc_base[kMaxDevices];

// Device address of the static scratch on the current device; the first call per device looks it
// up (this may load the module on that device, so it belongs before any stream capture).
static void* noalloc_scratch() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    if (!g_noalloc_base[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) return nullptr;
        if (reinterpret_cast<uintptr_t>(p) & 255u) return nullptr;
        g_noalloc_base[dev] = p;
    }
    return g_noalloc_base[dev];
}

// ------------------------------------------------------------------------------------------------
// hierarchical selection: the coarse and fine problems and the workspace that holds both
// ------------------------------------------------------------------------------------------------

struct HierLayout {
    dsa_dims coarse, fine;
    int pages;            // summary pages per sequence: ceil(max_blocks / 64)
    size_t coarse_ws;     // at offset 0: its error word is the call's
    size_t coarse_table;  // int32 [B][pages]
    size_t coarse_lens;   // int32 [B]
    size_t coarse_pos;    // int32 [T]
    size_t bidx;          // int32 [T][n_sel] chosen blocks
    size_t vtable;        // int32 [T][n_sel] virtual block tables
    size_t vlen;          // int32 [T]
    size_t vidx;          // int32 [T][K] fine Top-K in virtual positions
    size_t fine_ws;
    size_t total;
};

static HierLayout hier_layout(const dsa_dims& d, int T, int n_sel) {
    HierLayout h{};
    h.pages = (d.max_blocks + kBlock - 1) / kBlock;
    h.coarse = d;
    h.coarse.mode = DSA_BF16;
    h.coarse.max_blocks = h.pages;
    h.coarse.num_blocks = d.B * h.pages;
    h.coarse.K = n_sel;
    h.fine = d;
    h.fine.B = T;
    h.fine.max_blocks = n_sel;
    size_t off = 0;
    h.coarse_ws = off;
    off = align256(off + ws_layout(h.coarse, T).total);
    h.coarse_table = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(d.B) * h.pages);
    h.coarse_lens = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(d.B));
    h.coarse_pos = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T));
    h.bidx = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T) * n_sel);
    h.vtable = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T) * n_sel);
    h.vlen = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T));
    h.vidx = off;
    off = align256(off + sizeof(int32_t) * static_cast<size_t>(T) * d.K);
    h.fine_ws = off;
    off = align256(off + (T > 0 ? ws_layout(h.fine, T).total : 256));
    h.total = off;
    return h;
}

// ------------------------------------------------------------------------------------------------
// prompt attention: checks and workspace
// ------------------------------------------------------------------------------------------------

// Rows (token, head of the group), keys and tiles are counted in 32 bits, with room to round up to tiles.
constexpr int64_t kPromptCount = (1ll << 31) - (1 << 16);

struct PromptLayout {
    size_t head;      // PromptHead
    size_t units;     // PromptUnit [max_units]
    size_t joins;     // PromptJoin [max_slots / 2]
    size_t part_ml;   // float2 [max_slots * H_kv][slot_rows]
    size_t part_o;    // fp32 [max_slots * H_kv][d_v][slot_rows]
    size_t total;
    int tile_rows, max_units, ctas, shares, max_slots, slot_rows;
};

static dsa_status check_prompt_dims(const dsa_prompt_dims* p, int32_t Tq) {
    if (!p) return DSA_ERR_INVALID_ARG;
    if (p->type != DSA_F32 && p->type != DSA_BF16) return DSA_ERR_UNSUPPORTED;
    if (p->B <= 0 || p->H <= 0 || p->H_kv <= 0 || p->d_qk <= 0 || p->d_v <= 0 || Tq < 0) return DSA_ERR_INVALID_ARG;
    if (p->H % p->H_kv) return DSA_ERR_INVALID_ARG;
    if (p->d_qk > 256 || p->d_v > 256 || p->H_kv > 65535) return DSA_ERR_UNSUPPORTED;
    const int unit = p->type == DSA_F32 ? 4 : 8;  // elements per 16 bytes
    if (p->d_qk % unit || p->d_v % unit) return DSA_ERR_UNSUPPORTED;
    const int64_t strides[6] = {p->q_stride_t, p->q_stride_h, p->k_stride_t, p->k_stride_h, p->v_stride_t, p->v_stride_h};
    for (int64_t s : strides)
        if (s < 0 || s % unit || s > (1ll << 36)) return DSA_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(Tq) * (p->H / p->H_kv), limit = kPromptCount;
    if (rows + p->B >= limit || (rows / kPromptSimtRows + p->B) * p->H_kv >= limit) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

static PromptLayout prompt_layout(const dsa_prompt_dims& p, int Tq) {
    PromptLayout w{};
    const int64_t rows = static_cast<int64_t>(Tq) * (p.H / p.H_kv);
    w.tile_rows = prompt_uses_tc(p) ? kPromptTcRows : kPromptSimtRows;
    w.ctas = device_sm_count();
    // The plan makes fewer than 2 x shares partials over all key heads (see there), so at most 2 x shares / H_kv
    // of one head. Every size here grows with Tq, so that a workspace serves smaller calls.
    w.shares = 2 * w.ctas;
    w.max_slots = 2 * w.shares / p.H_kv;
    w.slot_rows = rows <= w.tile_rows / 2 ? static_cast<int>((rows + 31) / 32 * 32) : w.tile_rows;
    // every sequence fills whole tiles but its last
    w.max_units = static_cast<int>(rows / w.tile_rows) + p.B + w.max_slots;
    const size_t slots = static_cast<size_t>(w.max_slots) * p.H_kv;
    size_t off = 256;  // the error word
    w.head = off;
    off += 256;
    w.units = off;
    off = align256(off + sizeof(PromptUnit) * static_cast<size_t>(w.max_units));
    w.joins = off;
    off = align256(off + sizeof(PromptJoin) * static_cast<size_t>(w.max_slots / 2));
    w.part_ml = off;
    off = align256(off + sizeof(float2) * slots * w.slot_rows);
    w.part_o = off;
    off = align256(off + sizeof(float) * slots * w.slot_rows * p.d_v);
    w.total = off;
    return w;
}

static bool rope_layout_ok(int layout) { return layout == DSA_ROPE_INTERLEAVED || layout == DSA_ROPE_HALF; }

// ------------------------------------------------------------------------------------------------
// grouped-head cache: checks and workspace
// ------------------------------------------------------------------------------------------------

// Positions are counted in 32 bits, with room to round up to tiles.
constexpr int64_t kGroupedPositions = (1ll << 31) - (1 << 16);

static dsa_status check_grouped_dims(const dsa_grouped_dims* d) {
    if (!d) return DSA_ERR_INVALID_ARG;
    if ((d->type != DSA_F32 && d->type != DSA_BF16) || d->block_size != kBlock) return DSA_ERR_UNSUPPORTED;
    if (d->B <= 0 || d->max_blocks <= 0 || d->num_blocks <= 0 || d->H <= 0 || d->H_kv <= 0 || d->d_qk <= 0 || d->d_v <= 0)
        return DSA_ERR_INVALID_ARG;
    if (d->H % d->H_kv) return DSA_ERR_INVALID_ARG;
    if (d->d_qk > 256 || d->d_v > 256 || d->d_qk % 16 || d->d_v % 16) return DSA_ERR_UNSUPPORTED;
    // rows of the caches (the tensor maps count them in 32 bits), positions, and the grids
    if (static_cast<int64_t>(d->num_blocks) * d->H_kv * kBlock >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->max_blocks) * kBlock > kGroupedPositions) return DSA_ERR_UNSUPPORTED;
    if (d->H_kv > 32767 || static_cast<int64_t>(d->B) * d->H_kv >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

static bool grouped_strides_ok(const dsa_grouped_dims* d, int64_t st, int64_t sh) {
    const int64_t unit = d->type == DSA_F32 ? 4 : 8;  // elements per 16 bytes
    return st >= 0 && sh >= 0 && st % unit == 0 && sh % unit == 0 && st <= (1ll << 36) && sh <= (1ll << 36);
}

static bool ws_ok(const void* ws, size_t ws_bytes, size_t need) {
    return ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) && ws_bytes >= need;
}

static bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + b_bytes && y < x + a_bytes;
}

// Bytes of the weights of `blocks` blocks a sequence.
static size_t weights_bytes(const dsa_grouped_dims& d, int blocks) {
    return sizeof(float) * static_cast<size_t>(d.B) * d.H_kv * blocks * kBlock;
}

// The arrivals stand behind the error word, in the 256 bytes that dsa_workspace_init clears and no other call writes.
constexpr size_t kGroupedArrived = 16;

struct GroupedLayout {
    size_t part_ml, part_o, row_lse, z, total;
    int row_tile, ctas;
    int64_t max_tiles;
};

// Rows of an item: as many as the average sequence of the call has for a key head, in powers of two.
static GroupedLayout grouped_layout(const dsa_grouped_dims& d, int T, bool weights) {
    GroupedLayout w{};
    const int64_t G = d.H / d.H_kv;
    w.row_tile = grouped_row_tile(d, T);
    w.ctas = grouped_ctas(d);
    // Items of a key head: every sequence with rows fills whole ones but its last, which may hold a single row; where a token's
    // heads fill whole items, all are full.
    const int64_t some = T < d.B ? T : d.B, last = G % w.row_tile ? some * (w.row_tile - 1) : 0;
    w.max_tiles = (T * G + last) / w.row_tile * d.H_kv * ((d.max_blocks + 1) / 2);
    size_t off = 256;  // the error word
    const size_t slot_rows = static_cast<size_t>(2) * w.ctas * w.row_tile;
    w.part_ml = off;
    off = align256(off + sizeof(float2) * slot_rows);
    w.part_o = off;
    off = align256(off + sizeof(float) * slot_rows * d.d_v);
    w.row_lse = off;
    if (weights) off = align256(off + sizeof(float) * static_cast<size_t>(T) * d.H);
    w.z = off;
    if (weights) off = align256(off + sizeof(float) * static_cast<size_t>(w.max_tiles) * kGroupedTile * w.row_tile);
    w.total = off;
    return w;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_workspace_size(const dsa_dims* dims_in, int32_t T) {
    dsa_dims D;
    bool kv8;
    if (!dims_in || split_mode(dims_in, &D, &kv8) != DSA_OK) return 0;
    const dsa_dims* dims = &D;
    if (T < 0 || check_common(dims) != DSA_OK) return 0;
    return ws_layout(*dims, T).total;
}

dsa_status dsa_workspace_init(void* ws, size_t ws_bytes, dsa_stream_t stream) {
    if (!ws || ws_bytes < 256 || (reinterpret_cast<uintptr_t>(ws) & 255u)) return DSA_ERR_WORKSPACE;
    return cudaMemsetAsync(ws, 0, 256, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK
                                                                                              : DSA_ERR_LAUNCH;
}

dsa_status dsa_indexer_topk(const dsa_dims* dims_in, const void* q_I, const float* w, const void* k_I_cache,
                            const void* k_I_scale, const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* q_seq, const int32_t* q_pos, int32_t T, int32_t* idx, void* ws,
                            size_t ws_bytes, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_indexer_dims(dims);
    if (st != DSA_OK) return st;
    if (T < 0) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!q_I || !w || !k_I_cache || !block_table || !seq_lens || !idx)) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_I) || !aligned16(w) || !aligned16(k_I_cache)) return DSA_ERR_INVALID_ARG;
    st = check_ws(dims, T, ws, ws_bytes);
    if (st != DSA_OK) return st;
    int launches = 0;
    if (T > 0)
        st = run_indexer(dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, q_seq, q_pos, T, idx, ws,
                         reinterpret_cast<cudaStream_t>(stream), &launches, true, q_mx_ready(dims_in));
    g_last_launches = launches;
    return st;
}

dsa_status dsa_sparse_attn(const dsa_dims* dims_in, const void* q, const void* kv_cache, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* q_seq, const int32_t* idx, int32_t T,
                           float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_attn_dims(dims);
    if (st != DSA_OK) return st;
    if (T < 0) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !kv_cache || !block_table || !seq_lens || !idx || !out)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
    st = check_ws(dims, T, ws, ws_bytes);
    if (st != DSA_OK) return st;
    int launches = 0;
    if (T > 0)
        st = run_attn(dims, kv8, q, kv_cache, block_table, seq_lens, q_seq, idx, T, sm_scale, out, lse, ws,
                      reinterpret_cast<cudaStream_t>(stream), &launches, false);
    g_last_launches = launches;
    return st;
}

dsa_status dsa_decode(const dsa_dims* dims_in, const void* q_I, const float* w, const void* k_I_cache,
                      const void* k_I_scale, const int32_t* block_table, const int32_t* seq_lens, const void* q,
                      const void* kv_cache, float sm_scale, int32_t* idx, void* out, float* lse, void* ws,
                      size_t ws_bytes, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_indexer_dims(dims);
    if (st != DSA_OK) return st;
    st = check_attn_dims(dims);
    if (st != DSA_OK) return st;
    const int T = dims->B;
    if (!q_I || !w || !k_I_cache || !block_table || !seq_lens || !q || !kv_cache || !out) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_I) || !aligned16(w) || !aligned16(k_I_cache) || !aligned16(q) || !aligned16(kv_cache) ||
        !aligned16(out))
        return DSA_ERR_INVALID_ARG;
    st = check_ws(dims, T, ws, ws_bytes);
    if (st != DSA_OK) return st;
    const WsLayout L = ws_layout(*dims, T);
    int32_t* idx_buf = idx ? idx : reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + L.idx);
    int launches = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = run_indexer(dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, nullptr, nullptr, T, idx_buf, ws, s,
                     &launches, true, q_mx_ready(dims_in));
    if (st == DSA_OK)
        st = run_attn(dims, kv8, q, kv_cache, block_table, seq_lens, nullptr, idx_buf, T, sm_scale, out, lse, ws, s,
                      &launches, true);
    g_last_launches = launches;
    return st;
}

dsa_status dsa_indexer_topk_noalloc(const dsa_dims* dims_in, const void* q_I, const float* w, const void* k_I_cache,
                                    const void* k_I_scale, const int32_t* block_table, const int32_t* seq_lens,
                                    const int32_t* q_seq, const int32_t* q_pos, int32_t T, int32_t* idx,
                                    int32_t* fault_word, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_indexer_dims(dims);
    if (st != DSA_OK) return st;
    if (T < 0) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    // the indexer uses the workspace regions up to the attention's (error word, plan, candidates);
    // checked before the pointers, so that a size query with null buffers never launches anything
    if (ws_layout(*dims, T, false).idx > kNoAllocScratchBytes) return DSA_ERR_TOO_LARGE;
    if (T > 0 && (!q_I || !w || !k_I_cache || !block_table || !seq_lens || !idx)) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_I) || !aligned16(w) || !aligned16(k_I_cache)) return DSA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(fault_word) & 3u) return DSA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {  // no rows: no kernel and no scratch; only the caller's fault word is cleared
        g_last_launches = 0;
        if (fault_word && cudaMemsetAsync(fault_word, 0, sizeof(int32_t), s) != cudaSuccess) return DSA_ERR_LAUNCH;
        return DSA_OK;
    }
    void* ws = noalloc_scratch();
    if (!ws) return DSA_ERR_LAUNCH;
    int launches = 0;
    // the error word is the only scratch that must start at zero (every other region is written
    // before it is read within the call)
    if (cudaMemsetAsync(ws, 0, 256, s) != cudaSuccess) return DSA_ERR_LAUNCH;
    st = run_indexer(dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, q_seq, q_pos, T, idx, ws, s,
                     &launches, /*allow_prefill=*/false);
    if (st == DSA_OK && fault_word &&
        cudaMemcpyAsync(fault_word, ws, sizeof(int32_t), cudaMemcpyDeviceToDevice, s) != cudaSuccess)
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_cache_append(const dsa_dims* dims_in, const void* k_I_new, const void* kv_new,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                            const int32_t* q_pos, int32_t T, void* k_I_cache, void* k_I_scale, void* kv_cache,
                            void* ws, size_t ws_bytes, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (T < 0 || dims->d_I <= 0 || dims->d <= 0) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!k_I_new || !kv_new || !block_table || !seq_lens || !k_I_cache || !kv_cache)) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    const int act = dims->mode == DSA_F32 ? 4 : 2;
    if ((dims->d * act) % 16 || (dims->d_I * act) % 16) return DSA_ERR_UNSUPPORTED;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (!aligned16(k_I_new) || !aligned16(kv_new) || !aligned16(k_I_cache) || !aligned16(kv_cache))
        return DSA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (!launch_cache_append(*dims, kv8, k_I_new, kv_new, block_table, seq_lens, q_seq, q_pos, T, k_I_cache,
                             k_I_scale, kv_cache, static_cast<int*>(ws), reinterpret_cast<cudaStream_t>(stream),
                             &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_indexer_prolog(const dsa_dims* dims_in, const void* k_I_new, const void* kv_new,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                              const int32_t* q_pos, int32_t T_new, void* k_I_cache, void* k_I_scale, void* kv_cache,
                              const void* q_I, int32_t T_q, void* q_I_mx, void* ws, size_t ws_bytes,
                              dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (T_new < 0 || T_q < 0 || dims->d_I <= 0 || dims->d <= 0) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T_new != dims->B) return DSA_ERR_INVALID_ARG;
    if (T_new > 0 && (!k_I_new || !kv_new || !block_table || !seq_lens || !k_I_cache || !kv_cache))
        return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    const int act = dims->mode == DSA_F32 ? 4 : 2;
    if ((dims->d * act) % 16 || (dims->d_I * act) % 16) return DSA_ERR_UNSUPPORTED;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (!aligned16(k_I_new) || !aligned16(kv_new) || !aligned16(k_I_cache) || !aligned16(kv_cache))
        return DSA_ERR_INVALID_ARG;
    if (q_I_mx) {  // the query quantisation: MXFP8 only, both buffers [T_q][H_I][d_I] bf16
        if (dims->mode != DSA_MXFP8) return DSA_ERR_UNSUPPORTED;
        if (T_q > 0 && (!q_I || !aligned16(q_I) || !aligned16(q_I_mx))) return DSA_ERR_INVALID_ARG;
    }
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    const int64_t q_elements = q_I_mx ? static_cast<int64_t>(T_q) * dims->H_I * dims->d_I : 0;
    if (!launch_indexer_prolog(*dims, kv8, k_I_new, kv_new, block_table, seq_lens, q_seq, q_pos, T_new, k_I_cache,
                               k_I_scale, kv_cache, q_I, q_I_mx, q_elements, static_cast<int*>(ws),
                               reinterpret_cast<cudaStream_t>(stream), &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original_length,
                                double beta_fast, double beta_slow, double* freq_host) {
    if (!freq_host || rot < 2 || rot % 2) return DSA_ERR_INVALID_ARG;
    if (rot > DSA_ROPE_MAX_WIDTH || scaling < DSA_ROPE_LINEAR || scaling > DSA_ROPE_YARN) return DSA_ERR_UNSUPPORTED;
    if (!(base > 0.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return DSA_ERR_INVALID_ARG;
    const int half = rot / 2;
    double low = 0.0, high = 0.0;
    if (scaling == DSA_ROPE_YARN) {
        if (!(base > 1.0) || !(original_length > 0.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
            !std::isfinite(original_length) || !std::isfinite(beta_fast))
            return DSA_ERR_INVALID_ARG;
        // the pair that makes `turns` turns over the trained length: original_length f = 2 pi turns
        auto pair_of = [&](double turns) {
            return rot * std::log(original_length / (turns * 2.0 * M_PI)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.0);
        if (high - low < 0.001) high = low + 0.001;
    }
    if (scaling == DSA_ROPE_BASE && factor > 1.0 && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
    if (!std::isfinite(base) || !std::isfinite(std::pow(base, -2.0 * (half - 1) / rot))) return DSA_ERR_INVALID_ARG;
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == DSA_ROPE_LINEAR) f /= factor;
        if (scaling == DSA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        freq_host[i] = f;
    }
    return DSA_OK;
}

dsa_status dsa_rope(int32_t type, const dsa_rope_tensor* x, int32_t n, int32_t rot, const double* freq,
                    const int32_t* seq_lens, const int32_t* q_pos, int32_t T, float scale, int32_t transpose,
                    dsa_stream_t stream) {
    if (type != DSA_F32 && type != DSA_BF16) return DSA_ERR_UNSUPPORTED;
    if (!x || n <= 0 || rot < 2 || rot % 2 || T < 0 || !std::isfinite(scale)) return DSA_ERR_INVALID_ARG;
    if (n > DSA_ROPE_MAX_TENSORS || rot > DSA_ROPE_MAX_WIDTH) return DSA_ERR_UNSUPPORTED;
    const uintptr_t elem = type == DSA_F32 ? 4 : 2;
    for (int i = 0; i < n; ++i) {
        if (x[i].heads < 0 || !rope_layout_ok(x[i].layout)) return DSA_ERR_INVALID_ARG;
        if (static_cast<int64_t>(x[i].heads) * rot >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
        if (T > 0 && x[i].heads > 0) {
            const uintptr_t src = reinterpret_cast<uintptr_t>(x[i].x), dst = reinterpret_cast<uintptr_t>(x[i].out);
            if (!src || !dst || src % elem || dst % elem) return DSA_ERR_INVALID_ARG;
            if (src == dst && (x[i].x_stride_t != x[i].out_stride_t || x[i].x_stride_h != x[i].out_stride_h))
                return DSA_ERR_INVALID_ARG;
        }
    }
    if (T > 0 && (!freq || (reinterpret_cast<uintptr_t>(freq) & 7u) || (!q_pos && !seq_lens))) return DSA_ERR_INVALID_ARG;
    int launches = 0;
    const bool ok = launch_rope(type, x, n, rot, freq, seq_lens, q_pos, T, scale, transpose != 0,
                                reinterpret_cast<cudaStream_t>(stream), &launches);
    g_last_launches = launches;
    return ok ? DSA_OK : DSA_ERR_LAUNCH;
}

dsa_status dsa_cache_append_rope(const dsa_dims* dims_in, const dsa_rope_append* rope, const double* freq,
                                 const void* k_I_new, const void* kv_new, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* q_seq, const int32_t* q_pos, int32_t T,
                                 void* k_I_cache, void* k_I_scale, void* kv_cache, void* ws, size_t ws_bytes,
                                 dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (T < 0 || dims->d_I <= 0 || dims->d <= 0) return DSA_ERR_INVALID_ARG;
    if (!rope || rope->rot < 2 || rope->rot % 2 || !std::isfinite(rope->scale)) return DSA_ERR_INVALID_ARG;
    if (rope->rot > 256) return DSA_ERR_UNSUPPORTED;
    if (!rope_layout_ok(rope->k_layout) || !rope_layout_ok(rope->kv_layout)) return DSA_ERR_INVALID_ARG;
    if (rope->k_offset < -1 || (rope->k_offset >= 0 && rope->k_offset > dims->d_I - rope->rot)) return DSA_ERR_INVALID_ARG;
    if (rope->kv_offset < -1 || (rope->kv_offset >= 0 && rope->kv_offset > dims->d - rope->rot)) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!freq || (reinterpret_cast<uintptr_t>(freq) & 7u))) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!k_I_new || !kv_new || !block_table || !seq_lens || !k_I_cache || !kv_cache)) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    const int act = dims->mode == DSA_F32 ? 4 : 2;
    if ((dims->d * act) % 16 || (dims->d_I * act) % 16) return DSA_ERR_UNSUPPORTED;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (!aligned16(k_I_new) || !aligned16(kv_new) || !aligned16(k_I_cache) || !aligned16(kv_cache))
        return DSA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (!launch_cache_append_rope(*dims, kv8, *rope, freq, k_I_new, kv_new, block_table, seq_lens, q_seq, q_pos, T,
                                  k_I_cache, k_I_scale, kv_cache, static_cast<int*>(ws),
                                  reinterpret_cast<cudaStream_t>(stream), &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_cache_read(const dsa_dims* dims_in, const void* k_I_cache, const void* k_I_scale, const void* kv_cache,
                          const int32_t* block_table, const int32_t* seq_lens, const int32_t* start,
                          const int32_t* cu_rows, int32_t R, void* k_out, void* kv_out, void* ws, size_t ws_bytes,
                          dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (R < 0 || dims->d_I <= 0 || dims->d <= 0) return DSA_ERR_INVALID_ARG;
    const int act = dims->mode == DSA_F32 ? 4 : 2;
    if ((dims->d * act) % 16 || (dims->d_I * act) % 16) return DSA_ERR_UNSUPPORTED;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (dims->mode == DSA_BF16_KFP8 && dims->d_I % 16) return DSA_ERR_UNSUPPORTED;
    if (dims->d > 65536 || dims->d_I > 65536) return DSA_ERR_UNSUPPORTED;  // pieces of a row are counted in 16 bits
    if (R > 0 && (!block_table || !seq_lens || !cu_rows || (!k_out && !kv_out))) return DSA_ERR_INVALID_ARG;
    if (k_out && (!k_I_cache || !scale_ok(dims, k_I_scale) || !aligned16(k_I_cache) || !aligned16(k_out)))
        return DSA_ERR_INVALID_ARG;
    if (kv_out && (!kv_cache || !aligned16(kv_cache) || !aligned16(kv_out))) return DSA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (!launch_cache_read(*dims, kv8, k_I_cache, k_I_scale, kv_cache, block_table, seq_lens, start, cu_rows, R, k_out,
                           kv_out, static_cast<int*>(ws), reinterpret_cast<cudaStream_t>(stream), &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

size_t dsa_prompt_workspace_size(const dsa_prompt_dims* dims, int32_t Tq) {
    return check_prompt_dims(dims, Tq) == DSA_OK ? prompt_layout(*dims, Tq).total : 0;
}

dsa_status dsa_prompt_attn(const dsa_prompt_dims* dims, const void* q, const void* k, const void* v,
                           const int32_t* cu_q, const int32_t* cu_k, int32_t Tq, int32_t Tk, float sm_scale, void* out,
                           float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream) {
    dsa_status st = check_prompt_dims(dims, Tq);
    if (st != DSA_OK) return st;
    if (Tk < 0 || !(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
    if (Tk >= kPromptCount) return DSA_ERR_UNSUPPORTED;
    if (Tq > 0 && (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v)))) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
    const PromptLayout L = prompt_layout(*dims, Tq);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.total) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (Tq > 0) {
        uint8_t* base = static_cast<uint8_t*>(ws);
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        PromptArgs a{};
        a.type = dims->type;
        a.B = dims->B;
        a.H = dims->H;
        a.H_kv = dims->H_kv;
        a.d_qk = dims->d_qk;
        a.d_v = dims->d_v;
        a.causal = dims->causal ? 1 : 0;
        a.Tq = Tq;
        a.Tk = Tk;
        a.sm_scale = sm_scale;
        a.q = q;
        a.k = k;
        a.v = v;
        a.q_stride_t = dims->q_stride_t;
        a.q_stride_h = dims->q_stride_h;
        a.k_stride_t = dims->k_stride_t;
        a.k_stride_h = dims->k_stride_h;
        a.v_stride_t = dims->v_stride_t;
        a.v_stride_h = dims->v_stride_h;
        a.cu_q = cu_q;
        a.cu_k = cu_k;
        a.out = out;
        a.lse = lse;
        a.err = reinterpret_cast<int*>(base);
        a.tile_rows = L.tile_rows;
        a.max_units = L.max_units;
        a.ctas = L.ctas;
        a.shares = L.shares;
        a.max_slots = L.max_slots;
        a.slot_rows = L.slot_rows;
        a.head = reinterpret_cast<PromptHead*>(base + L.head);
        a.units = reinterpret_cast<PromptUnit*>(base + L.units);
        a.joins = reinterpret_cast<PromptJoin*>(base + L.joins);
        a.part_o = reinterpret_cast<float*>(base + L.part_o);
        a.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
        const bool tc = prompt_uses_tc(*dims);
        // Keys are split into parts of at least min_tiles tiles; where that cannot be and there are CTAs for
        // all units at once, their order does not matter either, and one launch does (a prompt of 100 tokens:
        // 17 us a call against 28).
        const int64_t items = static_cast<int64_t>(Tq) * (dims->H / dims->H_kv) / L.tile_rows + dims->B;
        a.min_tiles = tc ? kPromptTcMinTiles : kPromptSimtMinTiles;
        const bool whole = Tk <= (2 * a.min_tiles - 1) * kPromptKeys;
        a.self_plan = whole && dims->B <= 32 && items * dims->H_kv <= (tc ? L.ctas : 2 * L.ctas) ? 1 : 0;
        if (a.self_plan) a.max_units = static_cast<int>(items);
        if ((!a.self_plan && !launch_prompt_plan(a, s, &launches)) ||
            !(tc ? launch_prompt_tc(a, s, &launches) : launch_prompt_simt(a, s, &launches)) ||
            (!whole && !launch_prompt_join(a, s, &launches)))
            st = DSA_ERR_LAUNCH;
    }
    g_last_launches = launches;
    return st;
}

dsa_status dsa_grouped_append(const dsa_grouped_dims* dims, const void* k_new, int64_t k_stride_t, int64_t k_stride_h,
                              const void* v_new, int64_t v_stride_t, int64_t v_stride_h, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* cu, int32_t T, void* k_cache, float* k_scale,
                              void* v_cache, float* v_scale, void* ws, size_t ws_bytes, dsa_stream_t stream) {
    dsa_status st = check_grouped_dims(dims);
    if (st != DSA_OK) return st;
    if (T < 0 || (!cu && T != dims->B)) return DSA_ERR_INVALID_ARG;
    if (!grouped_strides_ok(dims, k_stride_t, k_stride_h) || !grouped_strides_ok(dims, v_stride_t, v_stride_h))
        return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!k_new || !v_new || !block_table || !seq_lens || !k_cache || !k_scale || !v_cache || !v_scale))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache)) return DSA_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, 256)) return DSA_ERR_WORKSPACE;
    int launches = 0;
    const GroupedAppendArgs a{dims->type, dims->B, dims->max_blocks, dims->num_blocks, dims->H_kv, dims->d_qk, dims->d_v, T,
                              k_new, v_new, k_stride_t, k_stride_h, v_stride_t, v_stride_h, block_table, seq_lens, cu,
                              static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scale, v_scale,
                              static_cast<int*>(ws)};
    if (!launch_grouped_append(a, reinterpret_cast<cudaStream_t>(stream), &launches)) st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

size_t dsa_grouped_workspace_size(const dsa_grouped_dims* dims, int32_t T, int32_t weights) {
    if (check_grouped_dims(dims) != DSA_OK || T < 0 || static_cast<int64_t>(T) * dims->H >= (1ll << 31)) return 0;
    return grouped_layout(*dims, T, weights != 0).total;
}

dsa_status dsa_grouped_attn(const dsa_grouped_dims* dims, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                            const void* k_cache, const float* k_scale, const void* v_cache, const float* v_scale,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int32_t T,
                            float sm_scale, void* out, float* lse, const float* weights, float* weights_out, void* ws,
                            size_t ws_bytes, dsa_stream_t stream) {
    dsa_status st = check_grouped_dims(dims);
    if (st != DSA_OK) return st;
    if (T < 0 || (!cu && T != dims->B) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * dims->H >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;  // rows are counted in 32 bits
    if (!grouped_strides_ok(dims, q_stride_t, q_stride_h)) return DSA_ERR_INVALID_ARG;
    if (!block_table || !seq_lens || !k_cache || !k_scale || !v_cache || !v_scale || (T > 0 && (!q || !out)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return DSA_ERR_INVALID_ARG;
    if (weights && !weights_out) return DSA_ERR_INVALID_ARG;
    const size_t w_bytes = weights_bytes(*dims, dims->max_blocks);
    if (weights != weights_out && overlap(weights, w_bytes, weights_out, w_bytes)) return DSA_ERR_INVALID_ARG;
    const GroupedLayout L = grouped_layout(*dims, T, weights_out != nullptr);
    if (!ws_ok(ws, ws_bytes, L.total)) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (T > 0 || weights_out) {
        uint8_t* base = static_cast<uint8_t*>(ws);
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        GroupedArgs a{};
        a.type = dims->type;
        a.B = dims->B;
        a.max_blocks = dims->max_blocks;
        a.num_blocks = dims->num_blocks;
        a.H = dims->H;
        a.H_kv = dims->H_kv;
        a.G = dims->H / dims->H_kv;
        a.d_qk = dims->d_qk;
        a.d_v = dims->d_v;
        a.T = T;
        a.q = q;
        a.q_stride_t = q_stride_t;
        a.q_stride_h = q_stride_h;
        a.k = static_cast<const uint8_t*>(k_cache);
        a.v = static_cast<const uint8_t*>(v_cache);
        a.k_scale = k_scale;
        a.v_scale = v_scale;
        a.block_table = block_table;
        a.seq_lens = seq_lens;
        a.cu = cu;
        a.sm_scale = sm_scale;
        a.out = out;
        a.lse = lse;
        a.weights = weights;
        a.weights_out = weights_out;
        a.err = reinterpret_cast<int*>(base);
        a.row_tile = L.row_tile;
        a.ctas = L.ctas;
        a.arrived = reinterpret_cast<uint32_t*>(base + kGroupedArrived);
        a.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
        a.part_o = reinterpret_cast<float*>(base + L.part_o);
        a.row_lse = reinterpret_cast<float*>(base + L.row_lse);
        a.z = reinterpret_cast<float*>(base + L.z);
        a.max_tiles = L.max_tiles;
        if (!launch_grouped_attn(a, s, &launches) || (weights_out && !launch_grouped_weights(a, s, &launches))) st = DSA_ERR_LAUNCH;
    }
    g_last_launches = launches;
    return st;
}

dsa_status dsa_grouped_evict(const dsa_grouped_dims* dims, const float* weights, int32_t keep, int32_t sink, int32_t recent,
                             const int32_t* block_table, const int32_t* seq_lens, const int32_t* new_table,
                             int32_t new_max_blocks, void* k_cache, float* k_scale, void* v_cache, float* v_scale,
                             int32_t* kept, int32_t* new_lens, float* weights_out, void* ws, size_t ws_bytes,
                             dsa_stream_t stream) {
    dsa_status st = check_grouped_dims(dims);
    if (st != DSA_OK) return st;
    if (keep <= 0 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > keep || new_max_blocks <= 0)
        return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(new_max_blocks) * kBlock > kGroupedPositions) return DSA_ERR_UNSUPPORTED;
    if (keep > new_max_blocks * kBlock) return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(dims->B) * dims->H_kv * ((keep + kBlock - 1) / kBlock) >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
    if (!weights || !block_table || !seq_lens || !new_table || !k_cache || !k_scale || !v_cache || !v_scale || !kept ||
        !new_lens || !weights_out)
        return DSA_ERR_INVALID_ARG;
    const size_t lens_bytes = sizeof(int32_t) * dims->B;
    if (overlap(weights, weights_bytes(*dims, dims->max_blocks), weights_out, weights_bytes(*dims, new_max_blocks)) ||
        overlap(seq_lens, lens_bytes, new_lens, lens_bytes))
        return DSA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return DSA_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, 256)) return DSA_ERR_WORKSPACE;
    int launches = 0;
    const GroupedEvictArgs a{dims->B, dims->max_blocks, dims->num_blocks, dims->H_kv, dims->d_qk, dims->d_v, keep, sink, recent,
                             new_max_blocks, weights, block_table, seq_lens, new_table, static_cast<uint8_t*>(k_cache),
                             static_cast<uint8_t*>(v_cache), k_scale, v_scale, kept, new_lens, weights_out,
                             static_cast<int*>(ws)};
    if (!launch_grouped_evict(a, reinterpret_cast<cudaStream_t>(stream), &launches)) st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

size_t dsa_hier_workspace_size(const dsa_dims* dims_in, int32_t T, int32_t n_sel) {
    dsa_dims D;
    bool kv8;
    if (!dims_in || split_mode(dims_in, &D, &kv8) != DSA_OK) return 0;
    const dsa_dims* dims = &D;
    if (T <= 0 || n_sel <= 0 || n_sel > 2048 || check_common(dims) != DSA_OK) return 0;
    return hier_layout(*dims, T, n_sel).total;
}

dsa_status dsa_block_summaries(const dsa_dims* dims_in, const void* k_I_cache, const void* k_I_scale,
                               const int32_t* block_table, const int32_t* seq_lens, uint16_t* summaries, void* ws,
                               size_t ws_bytes, dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (dims->d_I <= 0) return DSA_ERR_INVALID_ARG;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (!k_I_cache || !block_table || !seq_lens || !summaries) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (!launch_block_summaries(*dims, k_I_cache, k_I_scale, block_table, seq_lens, summaries, static_cast<int*>(ws),
                                reinterpret_cast<cudaStream_t>(stream), &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_block_summaries_append(const dsa_dims* dims_in, const void* k_I_cache, const void* k_I_scale,
                                      const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_seq,
                                      const int32_t* q_pos, int32_t T, uint16_t* summaries, void* ws, size_t ws_bytes,
                                      dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_common(dims);
    if (st != DSA_OK) return st;
    if (T < 0 || dims->d_I <= 0) return DSA_ERR_INVALID_ARG;
    if (dims->mode == DSA_MXFP8 && dims->d_I % 32) return DSA_ERR_UNSUPPORTED;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T > 0 && (!k_I_cache || !block_table || !seq_lens || !summaries)) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    if (!launch_summaries_append(*dims, k_I_cache, k_I_scale, block_table, seq_lens, q_seq, q_pos, T, summaries,
                                 static_cast<int*>(ws), reinterpret_cast<cudaStream_t>(stream), &launches))
        st = DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return st;
}

dsa_status dsa_indexer_topk_hier(const dsa_dims* dims_in, const void* q_I, const float* w, const void* k_I_cache,
                                 const void* k_I_scale, const int32_t* block_table, const int32_t* seq_lens,
                                 const int32_t* q_seq, const int32_t* q_pos, int32_t T, const uint16_t* summaries,
                                 int32_t n_sel, int32_t* idx, int32_t* blocks_out, void* ws, size_t ws_bytes,
                                 dsa_stream_t stream) {
    dsa_dims D;
    bool kv8;
    {
        const dsa_status split = split_mode(dims_in, &D, &kv8);
        if (split != DSA_OK) return split;
    }
    const dsa_dims* dims = &D;
    dsa_status st = check_indexer_dims(dims);
    if (st != DSA_OK) return st;
    if (dims->mode == DSA_F32) return DSA_ERR_UNSUPPORTED;  // the coarse stage scores bf16 summaries with bf16 q_I
    if (T < 0 || n_sel <= 0 || n_sel > 2048) return DSA_ERR_INVALID_ARG;
    if (!q_seq && T != dims->B) return DSA_ERR_INVALID_ARG;
    if (T == 0) return DSA_OK;
    if (!q_I || !w || !k_I_cache || !block_table || !seq_lens || !summaries || !idx) return DSA_ERR_INVALID_ARG;
    if (!scale_ok(dims, k_I_scale)) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q_I) || !aligned16(w) || !aligned16(k_I_cache) || !aligned16(summaries)) return DSA_ERR_INVALID_ARG;
    const HierLayout H = hier_layout(*dims, T, n_sel);
    if (check_indexer_dims(&H.coarse) != DSA_OK) return DSA_ERR_UNSUPPORTED;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < H.total) return DSA_ERR_WORKSPACE;
    uint8_t* base = static_cast<uint8_t*>(ws);
    auto at = [&](size_t off) { return reinterpret_cast<int32_t*>(base + off); };
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int launches = 0;
    int* fine_err = reinterpret_cast<int*>(base + H.fine_ws);
    if (!launch_hier_setup(dims->B, H.pages, T, seq_lens, q_seq, q_pos, at(H.coarse_table), at(H.coarse_lens),
                           at(H.coarse_pos), fine_err, s, &launches))
        return DSA_ERR_LAUNCH;
    // coarse: the indexer over the summaries, Top-n_sel blocks per row
    st = run_indexer(&H.coarse, q_I, w, summaries, nullptr, at(H.coarse_table), at(H.coarse_lens), q_seq,
                     at(H.coarse_pos), T, at(H.bidx), base + H.coarse_ws, s, &launches);
    if (st != DSA_OK) return st;
    if (!launch_hier_virtualize(dims->B, dims->max_blocks, n_sel, T, block_table, seq_lens, q_seq, q_pos, at(H.bidx),
                                at(H.vtable), at(H.vlen), blocks_out, s, &launches))
        return DSA_ERR_LAUNCH;
    // fine: the indexer over the tokens of the chosen blocks (one virtual sequence per row)
    st = run_indexer(&H.fine, q_I, w, k_I_cache, k_I_scale, at(H.vtable), at(H.vlen), nullptr, nullptr, T, at(H.vidx),
                     base + H.fine_ws, s, &launches);
    if (st != DSA_OK) return st;
    if (!launch_hier_remap(T, n_sel, dims->K, at(H.bidx), at(H.vidx), idx, fine_err, reinterpret_cast<int*>(base), s,
                           &launches))
        return DSA_ERR_LAUNCH;
    g_last_launches = launches;
    return DSA_OK;
}

dsa_status dsa_read_error(void* ws, int32_t* fault_bits, dsa_stream_t stream) {
    if (!ws) return DSA_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t v = 0;
    if (cudaStreamSynchronize(s) != cudaSuccess) return DSA_ERR_LAUNCH;
    if (cudaMemcpy(&v, ws, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return DSA_ERR_LAUNCH;
    // a call that gave up may have left arrivals behind the error word
    if (cudaMemset(ws, 0, v & DSA_FAULT_TIMEOUT ? 256 : sizeof v) != cudaSuccess) return DSA_ERR_LAUNCH;
    if (fault_bits) *fault_bits = v;
    if (v & DSA_FAULT_TIMEOUT) return DSA_ERR_TIMEOUT;
    return v ? DSA_ERR_DEVICE : DSA_OK;
}

dsa_status dsa_selftest_wait_timeout(void* ws, size_t ws_bytes, dsa_stream_t stream) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    int launches = 0;
    const bool ok = launch_wait_timeout(static_cast<int*>(ws), reinterpret_cast<cudaStream_t>(stream), &launches);
    g_last_launches = launches;
    return ok ? DSA_OK : DSA_ERR_LAUNCH;
}

int32_t dsa_last_launch_count(void) { return g_last_launches; }

const char* dsa_status_string(dsa_status status) {
    switch (status) {
        case DSA_OK: return "ok";
        case DSA_ERR_INVALID_ARG: return "invalid argument";
        case DSA_ERR_UNSUPPORTED: return "unsupported shape or mode";
        case DSA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case DSA_ERR_LAUNCH: return "kernel launch failed";
        case DSA_ERR_DEVICE: return "device-side fault (bad block-table entry or index)";
        case DSA_ERR_TIMEOUT: return "a pipeline wait inside a kernel timed out";
        case DSA_ERR_TOO_LARGE: return "call needs more scratch than the static buffer of dsa_indexer_topk_noalloc";
    }
    return "unknown status";
}

int32_t dsa_version(void) { return 100; }

}  // extern "C"
