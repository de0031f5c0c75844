// Attention over the grouped-head cache on tcgen05 tensor cores, whose operands are the cached e4m3 codes themselves.
//
// A cached value is code * scale with one scale per block and head, so products with codes need no widening: the scale of
// a block is a factor of its logits, or of its weights. What keeps the other operand's precision is that the tensor
// core's cost here goes with the cached rows, not with the few query rows: a query row is split into e4m3 parts of 4
// significand bits,
//   t = q 2^-e,  t = t_0 + t_1 / 16 + t_2 / 256 + ...,  t_i = e4m3(16^i * what is left),
// and so are the weights. Two parts hold a bf16 query exactly (elements below 2^-13 of its largest keep an absolute error
// of 2^-21 of that), three parts 11 bits of a weight (rounded to fp16 first; an absolute error of 2^-26 of the largest),
// six parts hold fp32. With the cached rows as the M side of both products the parts are extra columns:
//   S^T [128 positions x (parts * rows)] = K tile [128 x d_qk] . Q^T,   K-major, from shared memory as TMA wrote it
//   O^T [d_v x (parts * rows)] += V tile^T [d_v x 128] . P^T,            MN-major: the same row layout read the other way
// (M = 128, N = 16 .. 192), 32 bytes of K a step. Position = TMEM lane: a softmax thread holds its position's logits of
// all rows, only the running maximum crosses lanes, and O's rescaling touches few columns.
//
// Bytes bound it: 2 x 128 of a head's position at d = 128, and 4 products of N = 16 or 32 columns take a tenth of the time
// those bytes take. One CTA an SM works through its even share of the tiles (see grouped.cuh): a warp of TMA loads runs
// ahead as far as the ring allows, whatever items it crosses, one warp issues the products, kGroups warpgroups the softmax
// of kRW rows each, two warps bring the next item's queries.
#include "grouped.cuh"

namespace dsa {
namespace gtc {

constexpr int kChunk = 64 * 128;  // bytes of one block's 128 columns of codes
constexpr int kMaxStages = 6;
constexpr size_t kSmemLimit = 232448;

__host__ __device__ constexpr int pad16(int n) { return (n + 15) / 16 * 16; }

// Compiled forms: rows of a softmax thread, warpgroups that share a tile's rows, parts of a query and of a weight.
template <int kRW_, int kGroups_, int kQP_, int kPP_>
struct Form {
    static constexpr int kRW = kRW_, kGroups = kGroups_, kQP = kQP_, kPP = kPP_;
    static constexpr int kRows = kRW * kGroups;
    static constexpr int kSN = kQP * kRows;         // columns of S^T; thread-group g's are kQP * kRW from g * kQP * kRW
    static constexpr int kPN = pad16(kPP * kRows);  // columns of O^T
    static constexpr int kSoftWarps = 4 * kGroups;
    static constexpr int kThreads = 128 * kGroups + 128;
    static constexpr int kVCMax = kRows > 32 ? 1 : 2;  // chunks of 128 value columns (O^T's share of tensor memory)
    static constexpr int kColO = 2 * kSN;
    static constexpr int kCols = kColO + kVCMax * kPN + 8;  // (reads of 32 columns go past the last 24)
    static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kQBytes = kSN * 128;   // one 128-column chunk of the split queries
    static constexpr int kPBytes = kPN * 128;   // the split weights of a tile
    static_assert(kSN % 16 == 0 && kSN <= 256 && kPN <= 256 && kCols <= 512, "shapes of the products");
};

template <typename F>
struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], mma_done, met[F::kGroups];
    float4 scales[kMaxStages];                // of a tile's two blocks: keys, keys, values, values
    int valid[kMaxStages];                    // bits 0, 1: the blocks are there
    alignas(16) float q_factor[2][F::kRows];  // 2^e * sm_scale * log2(e), NaN for a query that is not finite
    alignas(16) int seen[2][F::kRows];        // positions below this are seen (rows past the last: 0)
    alignas(16) float red[2][F::kGroups][F::kRW][4];
    uint32_t tmem_base;
    int abort_flag;
    int64_t warp_sums[F::kThreads / 32];
    int64_t found[2];
};

template <typename F>
struct Layout {  // byte offsets; kc, vc: chunks of 128 columns of keys and values
    int stages;
    size_t stage, ring, q, p, ctl, total;
    __host__ __device__ Layout(int kc, int vc) {
        stage = static_cast<size_t>(2) * (kc + vc) * kChunk;
        const size_t rest = 2 * (static_cast<size_t>(kc) * F::kQBytes + F::kPBytes) + sizeof(Ctl<F>) + 1024;
        stages = static_cast<int>((kSmemLimit - rest) / stage);
        if (stages > kMaxStages) stages = kMaxStages;
        ring = 0;
        q = ring + stages * stage;
        p = q + 2 * static_cast<size_t>(kc) * F::kQBytes;
        ctl = p + 2 * static_cast<size_t>(F::kPBytes);
        total = ctl + sizeof(Ctl<F>) + 1024;
    }
};

// ------------------------------------------------------------------------------------------------
// tensor-core operands
// ------------------------------------------------------------------------------------------------

// Descriptor of an MN-major operand without swizzle: 16-byte pieces along MN, kSbo bytes apart, each with its 8 K rows 16
// bytes apart, and groups of 8 K rows kLbo bytes apart.
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// One K step (32 codes) of D (+)= A * B^T, kind::f8f6f4 (e4m3 both), issued by one elected lane of a converged warp.
__device__ __forceinline__ void warp_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// e4m3 in both operands is type 0, so the descriptor is that of kind::f16 with type 0.
constexpr uint32_t idesc_f8(int N, uint32_t a_mn, uint32_t b_mn) { return idesc_f16(128, N, 0u, a_mn, b_mn); }

__device__ __forceinline__ uint32_t cvt_e4m3x2(__half2 x) {
    return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 half2_of(uint32_t codes) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3));
}

// Splits two values (magnitudes up to 448) into kParts pairs of codes. bf16 calls split fp16 values: exact differences.
template <int kParts>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&parts)[kParts]) {
    if constexpr (kParts <= 3) {
        __half2 t = __floats2half2_rn(a, b);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            parts[i] = cvt_e4m3x2(t);
            if (i + 1 < kParts) t = __hmul2(__hsub2(t, half2_of(parts[i])), __float2half2_rn(16.0f));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            parts[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
            const float2 f = __half22float2(half2_of(parts[i]));
            a = (a - f.x) * 16.0f;
            b = (b - f.y) * 16.0f;
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The warp's largest value, NaN left out.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Columns addr .. addr + N - 1 of this thread's lane (N = 16, 24, 32 or 48; 24: the eight behind them are read too).
template <int N>
__device__ __forceinline__ void load_columns(uint32_t addr, float (&x)[N]) {
    static_assert(N == 16 || N == 24 || N == 32 || N == 48, "column counts of the compiled forms");
    if constexpr (N == 16) {
        uint32_t u[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
              "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
            : "r"(addr)
            : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        uint32_t u[32];
        tmem_ld32(addr, u);
        tmem_ld_wait(u);
#pragma unroll
        for (int i = 0; i < 32 && i < N; ++i) x[i] = __uint_as_float(u[i]);
        if constexpr (N == 48) {
            float y[16];
            load_columns<16>(addr + 32, y);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[32 + i] = y[i];
        }
    }
}

template <int N>
__device__ __forceinline__ void store_columns(uint32_t addr, const float (&x)[N]) {
    static_assert(N == 24 || N == 48, "column counts of the compiled forms");
    if constexpr (N == 24) {
        uint32_t u[16], w[8];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(x[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[16 + i]);
        tmem_st16(addr, u);
        tmem_st8(addr + 16, w);
    } else {
        uint32_t u[32], w[16];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(x[i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[32 + i]);
        tmem_st32(addr, u);
        tmem_st16(addr + 32, w);
    }
}

// ------------------------------------------------------------------------------------------------
// the pieces of a CTA's share
// ------------------------------------------------------------------------------------------------

struct Piece {
    int b, h, row0, rows, tile0, tile1;
    GroupedSeq s;
    int64_t t;  // its first tile in the call's line
};

struct Walk {
    int64_t t, end, base;
    int b;
};

__device__ __forceinline__ bool next_piece(const GroupedArgs& a, Walk& w, Piece& p) {
    while (w.t < w.end) {
        p.s = grouped_seq(a, w.b, false);
        const int64_t here = grouped_seq_tiles(a, p.s), local = w.t - w.base;
        if (local >= here) {
            w.base += here;
            ++w.b;
            continue;
        }
        const int item = static_cast<int>(local / p.s.tiles);
        p.b = w.b;
        p.h = item / p.s.items;
        p.row0 = (item - p.h * p.s.items) * a.row_tile;
        p.rows = min(a.row_tile, p.s.n * a.G - p.row0);
        p.tile0 = static_cast<int>(local - static_cast<int64_t>(item) * p.s.tiles);
        p.tile1 = static_cast<int>(min(static_cast<int64_t>(p.s.tiles), p.tile0 + (w.end - w.t)));
        p.t = w.t;
        w.t += p.tile1 - p.tile0;
        return true;
    }
    return false;
}

// 8 elements of a query row.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store_act(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_act(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, typename F>
__global__ void __launch_bounds__(F::kThreads, 1)
    grouped_tc_kernel(GroupedArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    constexpr int kRW = F::kRW, kRows = F::kRows, kGroups = F::kGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int kc = (a.d_qk + 127) / 128, vc = (a.d_v + 127) / 128;
    const Layout<F> lay(kc, vc);
    const int stages = lay.stages;
    Ctl<F>& S = *reinterpret_cast<Ctl<F>*>(smem + lay.ctl);
    const uint32_t sRing = smem_u32(smem), sQ = smem_u32(smem + lay.q), sP = smem_u32(smem + lay.p);
    const uint32_t stage_bytes = static_cast<uint32_t>(lay.stage), v_off = 2 * kc * kChunk;
    volatile int* abort_flag = &S.abort_flag;
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.q_full[i]), 2);
            mbar_init(smem_u32(&S.q_empty[i]), 1 + F::kSoftWarps);  // the products that read it, and the softmax's factors
            mbar_init(smem_u32(&S.s_full[i]), 1);
            mbar_init(smem_u32(&S.p_full[i]), F::kSoftWarps);
            mbar_init(smem_u32(&S.pv_done[i]), 1);
        }
        mbar_init(smem_u32(&S.mma_done), 1);
        for (int g = 0; g < kGroups; ++g) mbar_init(smem_u32(&S.met[g]), 4);
        S.abort_flag = 0;
        fence_mbar_init();
    }
    constexpr int kWarpLoad = F::kSoftWarps, kWarpMma = kWarpLoad + 1, kWarpQ = kWarpLoad + 2;
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&S.tmem_base), F::kTmemCols);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    // this CTA's share
    int64_t total, base;
    int b0;
    const int64_t begin = find_place<F::kThreads>(
        a.B, [&](int b) { return grouped_seq_tiles(a, grouped_seq(a, b, blockIdx.x == 0)); },
        [&](int64_t all) { return (all + a.ctas - 1) / a.ctas * blockIdx.x; }, &total, &b0, &base, S.warp_sums, S.found);
    const int64_t per = (total + a.ctas - 1) / a.ctas, end = min(total, begin + per);
    tc_fence_before();
    block_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem_base, 0);
    Walk w{begin, end, base, b0};
    Piece p;

    if (begin >= end) {
        if (threadIdx.x == 0) a.cuts[blockIdx.x].rows = 0;
    } else if (warp == kWarpLoad) {
        // --------------------------------------------------------------------------- TMA: keys and values
        // Lane l holds the table entry and scales of every 32nd block of the piece, the next 32 fetched while these load.
        int st = 0, phase = 1, tiles = 0;
        bool ok = true;
        while (ok && next_piece(a, w, p)) {
            const int32_t* table = a.block_table + static_cast<int64_t>(p.b) * a.max_blocks;
            const int blocks = min(2 * p.tile1, (p.s.len + kBlock - 1) / kBlock);
            auto fetch = [&](int first, int& row, float& ks, float& vs) {
                const int i = first + lane;
                row = -1, ks = vs = 0.0f;
                if (i >= blocks) return;
                const int blk = table[i];
                if (blk < 0 || blk >= a.num_blocks) {
                    atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
                    return;
                }
                row = blk * a.H_kv + p.h;
                ks = a.k_scale[row];
                vs = a.v_scale[row];
            };
            int row, row_next;
            float ks, vs, ks_next, vs_next;
            fetch(2 * p.tile0, row_next, ks_next, vs_next);
            for (int tile = p.tile0; ok && tile < p.tile1; ++tile) {
                const int j = (tile - p.tile0) & 15;
                if (j == 0) {
                    row = row_next, ks = ks_next, vs = vs_next;
                    fetch(2 * tile + 32, row_next, ks_next, vs_next);
                }
                const int r0 = __shfl_sync(0xFFFFFFFFu, row, 2 * j), r1 = __shfl_sync(0xFFFFFFFFu, row, 2 * j + 1);
                float4 sc;
                sc.x = __shfl_sync(0xFFFFFFFFu, ks, 2 * j), sc.y = __shfl_sync(0xFFFFFFFFu, ks, 2 * j + 1);
                sc.z = __shfl_sync(0xFFFFFFFFu, vs, 2 * j), sc.w = __shfl_sync(0xFFFFFFFFu, vs, 2 * j + 1);
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.empty[st]), phase, abort_flag, a.err));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&S.full[st]), dst = sRing + st * stage_bytes;
                    S.scales[st] = sc;
                    S.valid[st] = (r0 >= 0 ? 1 : 0) | (r1 >= 0 ? 2 : 0);
                    const uint32_t n = (r0 >= 0 ? 1 : 0) + (r1 >= 0 ? 1 : 0);
                    if (n) mbar_arrive_expect_tx(bar, n * (kc + vc) * kChunk);
                    else mbar_arrive(bar);
                    for (int c = 0; c < kc; ++c) {
                        if (r0 >= 0) tma_load_2d(dst + 2 * c * kChunk, &map_k, c * 128, r0 * kBlock, bar);
                        if (r1 >= 0) tma_load_2d(dst + (2 * c + 1) * kChunk, &map_k, c * 128, r1 * kBlock, bar);
                    }
                    for (int c = 0; c < vc; ++c) {
                        if (r0 >= 0) tma_load_2d(dst + v_off + 2 * c * kChunk, &map_v, c * 128, r0 * kBlock, bar);
                        if (r1 >= 0) tma_load_2d(dst + v_off + (2 * c + 1) * kChunk, &map_v, c * 128, r1 * kBlock, bar);
                    }
                }
                __syncwarp();
                ++tiles;
                if (++st == stages) st = 0, phase ^= 1;
            }
        }
        // nothing may still be landing when the CTA exits: each used stage's last load
        if (lane == 0) {
            for (int i = 0; i < stages && i < tiles; ++i) {
                if (--st < 0) st = stages - 1, phase ^= 1;
                mbar_wait_drain(smem_u32(&S.full[st]), phase ^ 1, a.err);
            }
        }
    } else if (warp == kWarpMma) {
        // --------------------------------------------------------------------------------- products
        // K Q^T of a tile runs one tile ahead of V^T P^T.
        int st = 0, phase = 0, st_v = 0, n = 0, item = 0;  // n: tiles whose logits were issued
        bool ok = true, open = false, first = false, first_v = false;  // open: the last tile's V^T P^T is still to come
        const int ksteps = (a.d_qk + 31) / 32;
        auto values = [&](int j) {  // V^T P^T of tile j
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.p_full[j & 1]), (j >> 1) & 1, abort_flag, a.err));
            if (!ok) return;
            tc_fence_after();
            for (int c = 0; c < vc; ++c) {
                const uint64_t da = sw128_desc(sRing + st_v * stage_bytes + v_off + 2 * c * kChunk, 0, 1024);
                const uint64_t db = plain_desc(sP + (j & 1) * F::kPBytes, 128, 2048);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    warp_mma_f8(tmem + F::kColO + c * F::kPN, da + k * (4096 >> 4), db + k * (512 >> 4), idesc_f8(F::kPN, 1u, 1u),
                                (first_v && k == 0) ? 0u : 1u);
            }
            warp_tc_commit(smem_u32(&S.empty[st_v]));
            warp_tc_commit(smem_u32(&S.pv_done[j & 1]));
            if (++st_v == stages) st_v = 0;
        };
        while (ok && next_piece(a, w, p)) {
            const int qb = item & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.q_full[qb]), (item >> 1) & 1, abort_flag, a.err));
            for (int tile = p.tile0; ok && tile < p.tile1; ++tile) {
                first = tile == p.tile0;
                // S[n & 1] is free: V^T P^T of tile n - 2 was issued after its weights came
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.full[st]), phase, abort_flag, a.err));
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < ksteps; ++k) {
                    const uint64_t da = sw128_desc(sRing + st * stage_bytes + (k >> 2) * 2 * kChunk, 0, 1024) + (k & 3) * 2;
                    const uint64_t db = sw128_desc(sQ + (qb * kc + (k >> 2)) * F::kQBytes, 0, 1024) + (k & 3) * 2;
                    warp_mma_f8(tmem + (n & 1) * F::kSN, da, db, idesc_f8(F::kSN, 0u, 0u), k ? 1u : 0u);
                }
                warp_tc_commit(smem_u32(&S.s_full[n & 1]));
                if (tile + 1 == p.tile1) warp_tc_commit(smem_u32(&S.q_empty[qb]));
                if (open) values(n - 1);
                open = true;
                first_v = first;
                ++n;
                if (++st == stages) st = 0, phase ^= 1;
            }
            ++item;
        }
        if (ok && open) values(n - 1);
        warp_tc_commit(smem_u32(&S.mma_done));  // every product issued so far
        if (lane == 0) mbar_wait_drain(smem_u32(&S.mma_done), 0, a.err);
    } else if (warp >= kWarpQ) {
        // --------------------------------------------------------------------------------- queries
        // Two warps split the rows of the next item's queries into parts; lane l holds columns 8l .. 8l + 7. First one
        // of them leaves word of the item that the share's begin cuts, for the join.
        if (threadIdx.x == kWarpQ * 32) {
            Walk w1 = w;
            next_piece(a, w1, p);
            const int64_t u0 = p.t - p.tile0, u1 = u0 + p.s.tiles;
            GroupedCut cut{};
            if (p.tile0 > 0 && begin - per <= u0) {
                const int c0 = blockIdx.x - 1;
                cut = GroupedCut{p.s.q0, p.h, p.row0, p.rows, grouped_slot(begin - per, u0, c0),
                                 static_cast<int>((u1 - 1) / per) - c0 + 1, {0, 0}};
            }
            a.cuts[blockIdx.x] = cut;
        }
        int item = 0;
        bool ok = true;
        const T* q = static_cast<const T*>(a.q);
        while (ok && next_piece(a, w, p)) {
            const int qb = item & 1;
            // (this wait lasts as long as an item; what stalls in it gives up by itself)
            const long long t0 = clock64();
            while (ok && !mbar_try_wait(smem_u32(&S.q_empty[qb]), ((item >> 1) & 1) ^ 1)) {
                if (clock64() - t0 > 64 * kWaitCycles) {
                    *abort_flag = 1;
                    atomicOr(a.err, DSA_FAULT_TIMEOUT);
                }
                ok = !*abort_flag;
                __nanosleep(64);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const int col = lane * 8;
#pragma unroll 4
            for (int r = warp - kWarpQ; r < kRows; r += 2) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.0f;
                const int row = p.row0 + r, i_tok = row / a.G;
                if (r < p.rows && col < a.d_qk)
                    load8(q + static_cast<int64_t>(p.s.q0 + i_tok) * a.q_stride_t + static_cast<int64_t>(p.h * a.G + row - i_tok * a.G) * a.q_stride_h + col, x);
                float top = 0.0f;
                bool fine = true;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    top = fmaxf(top, fabsf(x[i]));
                    fine = fine && isfinite(x[i]);
                }
                top = warp_max(top);
                fine = __all_sync(0xFFFFFFFFu, fine);
                // 2^-e takes the largest element into (224, 448]
                int e = 0;
                if (fine && top > 0.0f) {
                    e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 8, -120);
                    if (top * exp2f(static_cast<float>(-e)) > 448.0f) ++e;
                }
                const float down = exp2f(static_cast<float>(-e));
                uint32_t parts[4][F::kQP];
#pragma unroll
                for (int i = 0; i < 4; ++i) split_pair<F::kQP>(fine ? x[2 * i] * down : 0.0f, fine ? x[2 * i + 1] * down : 0.0f, parts[i]);
                if (col < kc * 128) {
                    const uint32_t chunk = sQ + (qb * kc + (col >> 7)) * F::kQBytes;
#pragma unroll
                    for (int i = 0; i < F::kQP; ++i) {
                        const int nrow = (r / kRW) * (F::kQP * kRW) + i * kRW + r % kRW, c16 = (col & 127) >> 4;
                        const uint32_t at = chunk + nrow * 128 + ((c16 ^ (nrow & 7)) << 4) + (col & 8);
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(parts[0][i] | parts[1][i] << 16),
                                     "r"(parts[2][i] | parts[3][i] << 16)
                                     : "memory");
                    }
                }
                if (lane == 0) {
                    S.q_factor[qb][r] = fine ? exp2f(static_cast<float>(e)) * (a.sm_scale * 1.4426950408889634f) : NAN;
                    S.seen[qb][r] = r < p.rows ? p.s.len - p.s.n + i_tok + 1 : 0;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.q_full[qb]));
            ++item;
        }
    } else {
        // --------------------------------------------------------------------------------- softmax
        const int group = warp >> 2, quarter = warp & 3, j = quarter * 32 + lane;  // j: position of the tile, TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t o_col = lane_base + F::kColO + group * F::kPP * kRW;
        int n = 0, st = 0, sphase = 0, item = 0, met = 0;
        bool ok = true;
        // The group's four warps meet (a barrier whose wait gives up, as every other).
        auto group_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.met[group]));
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.met[group]), met, abort_flag, a.err));
            met ^= 1;
        };
        while (ok && next_piece(a, w, p)) {
            const int qb = item & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.q_full[qb]), (item >> 1) & 1, abort_flag, a.err));
            float m[kRW], l[kRW], v_ref = 7.8886090522101181e-31f;  // 2^-100
#pragma unroll
            for (int r = 0; r < kRW; ++r) m[r] = -INFINITY, l[r] = 0.0f;
            const float* factor = S.q_factor[qb] + group * kRW;
            const int* seen = S.seen[qb] + group * kRW;
            // every row sees the positions below this
            const int all_see = p.s.len - p.s.n + p.row0 / a.G + 1;
            for (int tile = p.tile0; ok && tile < p.tile1; ++tile, ++n) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.full[st]), sphase, abort_flag, a.err) &&
                                                 mbar_wait(smem_u32(&S.s_full[n & 1]), (n >> 1) & 1, abort_flag, a.err));
                if (!ok) break;
                tc_fence_after();
                const float4 sc = S.scales[st];
                const int valid = S.valid[st], pos = tile * kGroupedTile + j;
                const float ks = quarter < 2 ? sc.x : sc.y, vs = quarter < 2 ? sc.z : sc.w;
                const bool here = (valid >> (quarter >> 1)) & 1 && pos < p.s.len;
                float z[kRW];
                {
                    float x[F::kQP * kRW];
                    load_columns<F::kQP * kRW>(lane_base + (n & 1) * F::kSN + group * F::kQP * kRW, x);
#pragma unroll
                    for (int r = 0; r < kRW; ++r) {
                        float y = x[(F::kQP - 1) * kRW + r];
#pragma unroll
                        for (int i = F::kQP - 2; i >= 0; --i) y = fmaf(y, 0.0625f, x[i * kRW + r]);
                        z[r] = y * (factor[r] * ks);
                    }
                }
                const bool whole = valid == 3 && (tile + 1) * kGroupedTile <= min(all_see, p.s.len);
                if (!whole) {
#pragma unroll
                    for (int r = 0; r < kRW; ++r) z[r] = here && pos < seen[r] ? z[r] : -INFINITY;
                    if (group == 0 && !here) {  // what the slot holds must not reach the products: 0 * NaN is NaN
                        for (int c = 0; c < vc; ++c) {
                            const uint32_t at = sRing + st * stage_bytes + v_off + 2 * c * kChunk + j * 128;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16 * i), "r"(0) : "memory");
                        }
                    }
                }
                if (a.weights_out && p.t + tile - p.tile0 < a.max_tiles) {
                    float* to = a.z + ((p.t + tile - p.tile0) * kRows + group * kRW) * kGroupedTile + j;
#pragma unroll
                    for (int r = 0; r < kRW; ++r)
                        if (group * kRW + r < p.rows) to[r * kGroupedTile] = z[r];
                }
                // the rows' maxima over the tile
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float top = warp_max(z[r]);
                    if (lane == (r & 31)) S.red[n & 1][group][r][quarter] = top;
                }
                group_sync();
                if (!ok) break;
                bool grown = false;
                float fac[kRW];
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const float4 t = *reinterpret_cast<const float4*>(S.red[n & 1][group][r]);
                    const float top = fmaxf(fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)), m[r]);
                    grown = grown || top > m[r];
                    fac[r] = top == -INFINITY ? 1.0f : ex2(m[r] - top);
                    m[r] = top;
                }
                // The weights carry their block's value scale, against a power of two no smaller than any so far.
                const float v_top = fmaxf(valid & 1 ? fabsf(sc.z) : 0.0f, valid & 2 ? fabsf(sc.w) : 0.0f);
                float v_fac = 1.0f;
                if (v_top > v_ref) {
                    const float ref = __uint_as_float((__float_as_uint(v_top) + 0x7FFFFFu) & 0x7F800000u);
                    v_fac = v_ref / ref;
                    grown = true;
                    v_ref = ref;
                }
                if (grown) {  // the same for all of the group's threads
#pragma unroll
                    for (int r = 0; r < kRW; ++r) l[r] *= fac[r];
                    if (tile > p.tile0) {
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.pv_done[(n - 1) & 1]), ((n - 1) >> 1) & 1, abort_flag, a.err));
                        if (!ok) break;
                        tc_fence_after();
                        for (int c = 0; c < vc; ++c) {
                            float o[F::kPP * kRW];
                            load_columns<F::kPP * kRW>(o_col + c * F::kPN, o);
#pragma unroll
                            for (int i = 0; i < F::kPP; ++i)
#pragma unroll
                                for (int r = 0; r < kRW; ++r) o[i * kRW + r] *= fac[r] * v_fac;
                            store_columns<F::kPP * kRW>(o_col + c * F::kPN, o);
                        }
                        tmem_st_wait();
                    }
                }
                if (n >= 2) {  // the products that read this buffer of weights are done
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.pv_done[n & 1]), ((n - 2) >> 1) & 1, abort_flag, a.err));
                    if (!ok) break;
                }
                const float tv = here ? vs * (256.0f / v_ref) : 0.0f;
                const uint32_t p_buf = sP + (n & 1) * F::kPBytes + j * 16;
#pragma unroll
                for (int r8 = 0; r8 < kRW; r8 += 8) {
                    uint32_t parts[4][F::kPP];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r8 + 2 * i;
                        const float p0 = ex2(z[r] - (m[r] == -INFINITY ? 0.0f : m[r]));
                        const float p1 = ex2(z[r + 1] - (m[r + 1] == -INFINITY ? 0.0f : m[r + 1]));
                        l[r] += p0;
                        l[r + 1] += p1;
                        split_pair<F::kPP>(p0 * tv, p1 * tv, parts[i]);
                    }
#pragma unroll
                    for (int i = 0; i < F::kPP; ++i) {
                        const int col = group * F::kPP * kRW + i * kRW + r8;
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(p_buf + (col >> 4) * 2048 + (col & 8)),
                                     "r"(parts[0][i] | parts[1][i] << 16), "r"(parts[2][i] | parts[3][i] << 16)
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.p_full[n & 1]));
                if (++st == stages) st = 0, sphase ^= 1;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.q_empty[qb]));
            ++item;
            // the item's end: sums over the positions, then the rows, or their partial
#pragma unroll
            for (int r = 0; r < kRW; ++r) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], o);
            }
            // (the maxima of the last tile have been read by all; those of the one before, long since)
#pragma unroll
            for (int r = 0; r < kRW; ++r)
                if (lane == (r & 31)) S.red[n & 1][group][r][quarter] = l[r];
            group_sync();
            ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.pv_done[(n - 1) & 1]), ((n - 1) >> 1) & 1, abort_flag, a.err));
            if (!ok) break;
            tc_fence_after();
            const bool complete = p.tile0 == 0 && p.tile1 == p.s.tiles;
            const int slot = grouped_slot(begin, p.t, blockIdx.x);
            const float unit = v_ref * (1.0f / 256.0f);
            for (int c = 0; c < vc; ++c) {
                float o[F::kPP * kRW];
                load_columns<F::kPP * kRW>(o_col + c * F::kPN, o);
                const int e = c * 128 + j;
#pragma unroll
                for (int r = 0; r < kRW; ++r) {
                    const int rr = group * kRW + r;
                    if (rr >= p.rows) break;
                    float y = o[(F::kPP - 1) * kRW + r];
#pragma unroll
                    for (int i = F::kPP - 2; i >= 0; --i) y = fmaf(y, 0.0625f, o[i * kRW + r]);
                    y *= unit;
                    const float4 t = *reinterpret_cast<const float4*>(S.red[n & 1][group][r]);
                    const float sum = (t.x + t.y) + (t.z + t.w);
                    const int row = p.row0 + rr, i_tok = row / a.G;
                    const int64_t at = static_cast<int64_t>(p.s.q0 + i_tok) * a.H + p.h * a.G + row - i_tok * a.G;
                    if (e < a.d_v) {
                        if (complete) store_act(static_cast<T*>(a.out) + at * a.d_v + e, sum == 0.0f ? 0.0f : y / sum);
                        else a.part_o[(static_cast<int64_t>(slot) * kRows + rr) * a.d_v + e] = sum == 0.0f ? 0.0f : y;
                    }
                    if (c == 0 && j == 0) {
                        const float lse2 = sum == 0.0f ? -INFINITY : m[r] + log2f(sum);
                        if (!complete) a.part_ml[slot * kRows + rr] = make_float2(m[r], sum);
                        if (complete && a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
                        if (complete && a.weights_out) a.row_lse[at] = lse2;
                    }
                }
            }
            tc_fence_before();  // O has been read before the next item's first product may overwrite it
            group_sync();       // and so have the sums, before the next item's maxima
        }
    }
    tc_fence_before();
    block_sync();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, F::kTmemCols);
    }
}

template <typename T, typename F>
static bool launch_form(const GroupedArgs& a, cudaStream_t s) {
    const int kc = (a.d_qk + 127) / 128, vc = (a.d_v + 127) / 128;
    const Layout<F> lay(kc, vc);
    if (vc > F::kVCMax || lay.stages < 2) return false;
    auto* kernel = grouped_tc_kernel<T, F>;
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), lay.total)) return false;
    CUtensorMap map_k, map_v;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.H_kv * kBlock;
    if (!make_tmap_2d(&map_k, a.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.d_qk, rows, a.d_qk, 128, kBlock) ||
        !make_tmap_2d(&map_v, a.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.d_v, rows, a.d_v, 128, kBlock))
        return false;
    return launch_kernel(false, kernel, dim3(a.ctas), dim3(F::kThreads), lay.total, s, a, map_k, map_v);
}

}  // namespace gtc

// Rows of an item: as many as the average sequence of the call has for a key head, in powers of two. Of fp32 queries and
// of wide values fewer: their parts fill tensor memory.
int grouped_row_tile(const dsa_grouped_dims& d, int T) {
    const int64_t rows = (static_cast<int64_t>(T) + d.B - 1) / d.B * (d.H / d.H_kv);
    const int most = d.type == DSA_F32 ? 16 : d.d_v > 128 ? 32 : 64;
    int tile = 8;
    while (tile < rows && tile < most) tile *= 2;
    return tile;
}

int grouped_ctas(const dsa_grouped_dims&) { return device_sm_count(); }

bool launch_grouped_attn(const GroupedArgs& a, cudaStream_t s, int* launches) {
    using namespace gtc;
    bool ok = false;
    if (a.type == DSA_F32) {
        ok = a.row_tile == 8 ? launch_form<float, Form<8, 1, 6, 6>>(a, s) : launch_form<float, Form<8, 2, 6, 6>>(a, s);
    } else {
        switch (a.row_tile) {
            case 8: ok = launch_form<__nv_bfloat16, Form<8, 1, 2, 3>>(a, s); break;
            case 16: ok = launch_form<__nv_bfloat16, Form<8, 2, 2, 3>>(a, s); break;
            case 32: ok = launch_form<__nv_bfloat16, Form<16, 2, 2, 3>>(a, s); break;
            default: ok = launch_form<__nv_bfloat16, Form<16, 4, 2, 3>>(a, s); break;
        }
    }
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
