// Attention over the grouped-head cache on tcgen05 tensor cores, whose operands are the cached e4m3 codes themselves.
//
// A cached value is code * scale with one scale per block and head, so products with codes need no widening: the scale of
// a block is a factor of its logits, or of its weights. What keeps the other operand's precision is that the tensor
// core's cost here goes with the cached rows, not with the few query rows: a query row is split into e4m3 parts of 4
// significand bits,
//   t = q 2^-e,  t = t_0 + t_1 / 16 + t_2 / 256 + ...,  t_i = e4m3(16^i * what is left),
// and so are the weights, in steps of 32 (what rounding leaves is half a step at most and has a sign, so a part is worth 5
// bits; queries go up to 448, where 32 times that half step would leave the codes' range). Two parts hold a bf16 query exactly
// (elements below 2^-13 of its largest keep an absolute error of 2^-21 of that), four parts every fp16 number up to 256, to
// which a weight is rounded (in steps of 16 small ones would be off by 2^-22, fp16's rounding is by 2^-25), six parts fp32 (small
// weights with an absolute error of 2^-35). With the cached rows as the M side of both products the parts are extra columns:
//   S^T [128 positions x (parts * rows)] = K tile [128 x d_qk] . Q^T,   K-major, from shared memory as TMA wrote it
//   O^T [d_v x (parts * rows)] += V tile^T [d_v x 128] . P^T,            MN-major: the same row layout read the other way
// (M = 128, N = 16 .. 256), 32 bytes of K a step: 46 cycles each up to N = 64, 128 at N = 256. Position = TMEM lane: a
// softmax thread holds its position's logits of all rows, so only maxima cross lanes, and O's rescaling touches few columns.
//
// Softmax: weights are formed against a row's reference m, its maximum when that was last looked at. As long as no logit of
// a tile passes m by more than 4 (in powers of two) the weights stay below 2^4 and are kept as they are; else m moves to the
// maximum, O^T and the sums are multiplied by 2^(m_old - m), and the tile's weights are formed again. So most tiles need no
// maxima across lanes, and no tile's weights wait for them: the warps exchange one flag at a barrier after the weights are
// written (drafts of 16 x 4 147 us with maxima in every tile, 121 without). The block's value scale is a factor of the
// weights, 1/4 .. 16 times: it stands against a power of two that the loads' warp chooses by the scales of 32 blocks at a time,
// 64^-i of it for smaller ones. Where that power changes, O^T is multiplied by the old one over the new (exactly); where it
// changes within a tile, the blocks take turns: weights of the first, its products, O^T moved, weights of the second. So a
// block with a large scale, be it of zeros, takes no bits from the light weights of others.
//
// What bounds it. One row a token and 8 heads a key head (N = 16 and 32): bytes; 32 sequences of 16K - 32K 254 us, 1.55 GB
// at 6.1 TB/s, 90% of a copy's rate; one of 1M 341 us, 93%. More rows: the softmax's instructions and their latencies, a
// row at a time (2 rows a token 82 us, 4 107, 8 184 where the bytes take 37). Few bytes: the launch and the items' chains.
// Scales that vary by two powers of two from block to block (standard deviation), where every other tile's blocks take turns:
// the decode batch 388 us; by one power 260.
// A tile's chain logits -> weights (about 1500 cycles) is longer than its bytes take (1400), so two sets of warps take
// tiles in turn, each with a maximum, a sum and an O^T of its own, and the set with an item's last tile puts the two
// together; where rows fill the warps of both, one set of kGroups warpgroups shares a tile's rows (see the forms below).
// One CTA an SM works through its even share of the tiles (see grouped.cuh): a warp of TMA loads runs ahead as far as the
// ring allows, whatever items it crosses; one warp issues the products, the values' as soon as their weights are there
// (d = 256, where the ring has 3 stages: 134 us when they stood behind the next keys', 102 so); two warps bring the next
// item's queries. 12 warps leave 168 registers a thread; more, of fewer rows or with spills, were slower but for 64 rows.
// The roles' loops drive each other out of the instruction cache, so what runs once or twice a tile is not unrolled (loops
// over the chunks of 128 columns, left to the compiler, made the code half again as long: 2 rows a token 82 us, so 102; the
// keys' products are, as their issue is what the decode batch waits for: 254 us, rolled 267).
// An item's end costs the products' and the softmax's latencies, which two sets overlap in part: 128 sequences of 1024 take 80
// us where the bytes take 40, of 16K and more a tenth above them.
#include <cfloat>
#include <cstddef>

#include "grouped.cuh"

namespace dsa {
namespace gtc {

constexpr int kChunk = 64 * 128;  // bytes of one block's 128 columns of codes
constexpr int kMaxStages = 6;
constexpr float kSlack = 4.0f;  // a weight is 2^kSlack at most,
constexpr float kTop = 16.0f;   // and kTop * 2^kSlack = 256 as it is split into codes (which end at 448)
constexpr int kQStep = 16, kPStep = 32;  // a part of a query, and of a weight, against the next
constexpr int kLeastRef = 27;   // exponents (127: of 1) of what value scales refer to: the least,
constexpr int kRefRange = 60;   // and how far they fall below an item's largest
constexpr size_t kSmemLimit = 232448;

__host__ __device__ constexpr int pad16(int n) { return (n + 15) / 16 * 16; }

// Where a CTA stands in its share; next_piece takes the next item, or what the share holds of it.
struct Walk {
    GroupedSeq s;
    int b, item, tile;  // the next piece's sequence, item of it (key head and row tile) and first tile
    int64_t left, t;    // tiles of the share from there on; place of that tile in the call's line
};

struct Piece {
    int h, row0, rows, tile0, tile1;
    int64_t t;
};

__device__ __forceinline__ bool next_piece(const GroupedArgs& a, Walk& w, Piece& p) {
    if (w.left <= 0) return false;
    while (!w.s.tiles || w.item >= w.s.items * a.H_kv) {  // (left > 0: there is a next one)
        w.s = grouped_seq(a, ++w.b, false);
        w.item = 0;
    }
    p.h = w.s.items == 1 ? w.item : w.item / w.s.items;
    p.row0 = (w.item - p.h * w.s.items) * a.row_tile;
    p.rows = min(a.row_tile, w.s.n * a.G - p.row0);
    p.tile0 = w.tile;
    p.tile1 = static_cast<int>(min(static_cast<int64_t>(w.s.tiles), w.tile + w.left));
    p.t = w.t;
    const int n = p.tile1 - p.tile0;
    w.t += n;
    w.left -= n;
    w.tile = 0;
    ++w.item;
    return true;
}

// What the products and the softmax need to know of a piece, beside its queries. tiles 0: there are no more.
struct Item {
    int tile0, tiles, len;
    int all_see;         // every row sees the positions below this
    int rows;
    int complete;        // the piece is a whole item; otherwise:
    int slot;            // its partial
    int c0, join_slot, parts;  // the CTA and slot of the item's first partial, and their number
    int64_t t;           // its first tile in the call's line
};

// Compiled forms: rows of a softmax thread, warpgroups that share a tile's rows, sets that take tiles in turn, parts of a
// query and of a weight, buffers of logits. (32 rows, drafts of 16 x 4, when they were tried: two warpgroups of 16 rows a thread
// 115 us, 106 now; one of 32 rows in each of two sets, four of 8 rows, or two of 16 rows in each of two sets 152 - 182.)
template <int kRW_, int kGroups_, int kSets_, int kQP_, int kPP_, int kSB_>
struct Form {
    static constexpr int kRW = kRW_, kGroups = kGroups_, kSets = kSets_, kQP = kQP_, kPP = kPP_, kSB = kSB_;
    static constexpr int kRows = kRW * kGroups;
    static constexpr int kSN = kQP * kRows;         // columns of S^T; group g's are kQP * kRW from g * kQP * kRW
    static constexpr int kPN = pad16(kPP * kRows);  // columns of O^T
    static constexpr int kSetWarps = 4 * kGroups, kSoftWarps = kSets * kSetWarps;
    static constexpr int kQWarps = 2;  // (12 warps in all leave 168 registers a thread)
    static constexpr int kThreads = 32 * (kSoftWarps + 2 + kQWarps);
    static constexpr int kVCMax = kRows > 16 ? 1 : 2;  // chunks of 128 value columns (O^T's share of tensor memory)
    static constexpr int kColO = kSB * kSN;
    static constexpr int kCols = kColO + kSets * kVCMax * kPN;
    static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kQBytes = kSN * 128;   // one 128-column chunk of the split queries
    static constexpr int kPBytes = kPN * 128;   // the split weights of a tile
    // Buffers of weights, and barriers for their coming and for the end of the products that read them. Before the keys'
    // products of tile n the values' are issued of all before n - kSB / 2 (tile n - 3 and before of two sets, n - 2 of one),
    // so that whoever has the logits of n knows that the phase before n's, tile n - kPB's, has ended on each of these
    // barriers. With two barriers for two sets, n - 2 might not have: the wait for n could take the phase before for its own.
    // (A tile whose blocks take turns has two phases of each; the first has been waited for when the second's weights come.)
    static constexpr int kPB = kSets == 2 ? 4 : 2;
    static_assert(kSN % 16 == 0 && kSN <= 256 && kPN <= 256 && kCols <= 512, "shapes of the products");
};

template <typename F>
struct Ctl {
    // barriers, with their arrivals in barrier_count
    uint64_t full[kMaxStages], empty[kMaxStages], s_full[F::kSB], pv_done[F::kPB], mma_done;
    uint64_t q_full[2], p_full[F::kPB], o_free, left[2], q_first, fin, q_empty[2];
    alignas(16) float2 scales[kMaxStages][2];  // of a tile's blocks: the keys' scale, the values' times kTop / what it refers to
    uint32_t refs[kMaxStages];                // bits 0, 1: the blocks are there; 2: they refer to different powers of two and
                                              // take turns; from 8 and 16: the exponents of these
    alignas(16) float q_factor[2][F::kRows];  // 2^e * sm_scale * log2(e)
    alignas(16) int seen[2][F::kRows];        // positions below this are seen (rows past the last: 0)
    alignas(16) int row_at[2][F::kRows];      // token * H + head
    alignas(16) float red[F::kSets * F::kGroups][F::kRW][4];  // maxima of a tile's rows, by warp
    alignas(16) uint32_t flag[2][F::kSets * F::kGroups][4];   // a warp's word on whether they must move
    int go[2][F::kSets * F::kGroups];         // whether the waits of a group's first warp ended well
    alignas(16) float2 fm[F::kSoftWarps][F::kRW];  // each warp's own: a row's factor, minus what its weights refer to
    alignas(16) float fac[F::kSoftWarps][F::kRW];  // and what its sums are to be multiplied by
    alignas(16) float fin_l[2][F::kSets][F::kRows][4], fin_m[2][F::kSets][F::kRows];  // a set's share of an item
    float fin_unit[2][F::kSets];  // of its O^T; 0: it had no tile
    Item item[2];
    uint32_t tmem_base;
    int abort_flag;
    int last_part;  // whether the CTA left the last partial of an item
    int64_t warp_sums[F::kThreads / 32];
    int64_t found[2];
};

template <typename F>
__device__ __forceinline__ int barrier_count(int i) {
    constexpr int kOnes = 2 * kMaxStages + F::kSB + F::kPB + 1, kSet = kOnes + 2, kSoft = kSet + F::kPB + 3, kLast = kSoft + 2;
    static_assert(offsetof(Ctl<F>, q_empty) == kLast * 8, "barriers in order");
    if (i < kOnes) return 1;
    if (i < kSet) return F::kQWarps;
    if (i < kSoft) return F::kSetWarps;     // p_full, o_free, left
    return i < kLast ? F::kSoftWarps : 1 + F::kSoftWarps;  // q_empty: the products that read it, too
}

template <typename F>
struct Layout {  // byte offsets; kc, vc: chunks of 128 columns of keys and values
    int stages;
    size_t stage, ring, q, p, ctl, total;
    __host__ __device__ Layout(int kc, int vc) {
        stage = static_cast<size_t>(2) * (kc + vc) * kChunk;
        const size_t rest = 2 * static_cast<size_t>(kc) * F::kQBytes + F::kPB * F::kPBytes + sizeof(Ctl<F>) + 1024;
        stages = static_cast<int>((kSmemLimit - rest) / stage);
        if (stages > kMaxStages) stages = kMaxStages;
        ring = 0;
        q = ring + stages * stage;
        p = q + 2 * static_cast<size_t>(kc) * F::kQBytes;
        ctl = p + F::kPB * static_cast<size_t>(F::kPBytes);
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
template <int kStep, int kParts>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&parts)[kParts]) {
    if constexpr (kParts <= 4) {
        __half2 t = __floats2half2_rn(a, b);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            parts[i] = cvt_e4m3x2(t);
            if (i + 1 < kParts) t = __hmul2(__hsub2(t, half2_of(parts[i])), __float2half2_rn(kStep));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            parts[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
            const float2 f = __half22float2(half2_of(parts[i]));
            a = (a - f.x) * kStep;
            b = (b - f.y) * kStep;
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

// Columns addr .. addr + N - 1 of this thread's lane.
template <int N>
__device__ __forceinline__ void load_columns(uint32_t addr, float (&x)[N]) {
    static_assert(N == 8 || N == 16 || N == 32 || N == 48, "column counts of the compiled forms");
    if constexpr (N == 8) {
        uint32_t u[8];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
            : "r"(addr)
            : "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else if constexpr (N == 16) {
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
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(u[i]);
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
    static_assert(N == 8 || N == 16 || N == 32, "column counts of the compiled forms");
    uint32_t u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = __float_as_uint(x[i]);
    if constexpr (N == 8) tmem_st8(addr, u);
    else if constexpr (N == 16) tmem_st16(addr, u);
    else tmem_st32(addr, u);
}

// This thread's products with the keys (times their block's scale), from the sums with each part of the queries (part i's rows side by side).
template <int kQP, int kRW>
__device__ __forceinline__ void load_logits(uint32_t addr, float scale, float (&s)[kRW]) {
    float x[kQP * kRW];
    load_columns<kQP * kRW>(addr, x);
#pragma unroll
    for (int r = 0; r < kRW; ++r) {
        s[r] = x[(kQP - 1) * kRW + r];
#pragma unroll
        for (int i = kQP - 2; i >= 0; --i) s[r] = fmaf(s[r], 1.0f / kQStep, x[i * kRW + r]);
        s[r] *= scale;
    }
}

// Eight rows' columns of O^T, put together from their parts, kStep columns apart.
template <int kPP, int kStep>
__device__ __forceinline__ void join_parts(uint32_t addr, float (&y)[8]) {
    load_columns<8>(addr + (kPP - 1) * kStep, y);
#pragma unroll
    for (int i = kPP - 2; i >= 0; --i) {
        float o[8];
        load_columns<8>(addr + i * kStep, o);
#pragma unroll
        for (int r = 0; r < 8; ++r) y[r] = fmaf(y[r], 1.0f / kPStep, o[r]);
    }
}

// Sums of kRW values over the warp's lanes; lane r's result is that of row r (kRW < 32: of row r % kRW, in every lane).
template <int kRW>
__device__ __forceinline__ float sum_rows(float (&x)[kRW], int lane) {
    // halve the rows a lane holds and double the lanes each sum covers: lane bit kRW / 2, then kRW / 4, ... chooses the half
#pragma unroll
    for (int w = kRW / 2; w > 0; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = up ? x[i] : x[i + w], own = up ? x[i + w] : x[i];
            x[i] = own + __shfl_xor_sync(0xFFFFFFFFu, give, w);
        }
    }
#pragma unroll
    for (int o = kRW; o < 32; o <<= 1) x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], o);
    return x[0];
}

// ------------------------------------------------------------------------------------------------
// queries and outputs
// ------------------------------------------------------------------------------------------------

// 8 elements of a query row, as they are loaded.
template <typename T>
struct Elements;
template <>
struct Elements<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Elements<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// Splits rows first, first + step, ... of an item's queries into parts, in shared memory as the products read them; lane l
// holds columns 8l .. 8l + 7.
template <typename T, typename F>
__device__ __forceinline__ void split_queries(const GroupedArgs& a, const GroupedSeq& seq, const Piece& p, Ctl<F>& S, int qb, uint32_t dst,
                                              int kc, int first, int step) {
    // (a rolled loop, the next row's elements on their way: its instructions are fetched once)
    const int lane = threadIdx.x & 31, col = lane * 8;
    // lane k looks after row first + k * step: its token and head
    const int mine = first + lane * step, row = p.row0 + mine, tok = row / a.G, head = p.h * a.G + row - tok * a.G;
    const bool live = mine < p.rows;
    const int64_t at = static_cast<int64_t>(seq.q0 + tok) * a.q_stride_t + static_cast<int64_t>(head) * a.q_stride_h;
    if (mine < F::kRows) {
        S.seen[qb][mine] = live ? seq.len - seq.n + tok + 1 : 0;
        S.row_at[qb][mine] = live ? (seq.q0 + tok) * a.H + head : 0;
    }
    Elements<T> next;
    auto load = [&](int k) {
        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, k);
        next = Elements<T>{};
        if (first + k * step < p.rows && col < a.d_qk) next.load(static_cast<const T*>(a.q) + from + col);
    };
    load(0);
#pragma unroll 1
    for (int k = 0, r = first; r < F::kRows; ++k, r += step) {
        float x[8];
        next.values(x);
        load((k + 1) & 31);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        // 2^-e takes the largest element into (224, 448]; a query that is not finite becomes codes of NaN
        const bool fine = top < 0x7F800000u;
        const int e = !fine ? 0 : max(static_cast<int>(top >> 23) - 127 - 8, -120) + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        // (finite and not 0: a position that is not seen has the logit -inf, and 0 times it were NaN)
        const float factor = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (a.sm_scale * 1.4426950408889634f);
        if (lane == 0) S.q_factor[qb][r] = fminf(fmaxf(factor, 0x1p-126f), FLT_MAX);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        uint32_t parts[4][F::kQP];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_pair<kQStep>(x[2 * i] * down, x[2 * i + 1] * down, parts[i]);
        if (col >= kc * 128) continue;
        const int nrow = (r / F::kRW) * (F::kQP * F::kRW) + r % F::kRW, c16 = (col & 127) >> 4;
        const uint32_t to = dst + (col >> 7) * F::kQBytes + nrow * 128 + ((c16 ^ (nrow & 7)) << 4) + (col & 8);
#pragma unroll
        for (int i = 0; i < F::kQP; ++i)  // (kRW is a multiple of 8: the parts' rows swizzle alike)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + i * F::kRW * 128),
                         "r"(fine ? parts[0][i] | parts[1][i] << 16 : 0x7F7F7F7Fu),
                         "r"(fine ? parts[2][i] | parts[3][i] << 16 : 0x7F7F7F7Fu));
    }
    fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ void store_act(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_act(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, typename F>
__global__ void __launch_bounds__(F::kThreads, 1)
    grouped_tc_kernel(GroupedArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    constexpr int kRW = F::kRW, kRows = F::kRows, kGroups = F::kGroups, kSets = F::kSets;
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

    constexpr int kWarpLoad = F::kSoftWarps, kWarpMma = kWarpLoad + 1, kWarpQ = kWarpLoad + 2;
    if (warp == 0) {
        for (int i = lane; i * 8 < static_cast<int>(offsetof(Ctl<F>, q_empty)) + 16; i += 32)
            mbar_init(smem_u32(&S) + i * 8, barrier_count<F>(i));
        if (lane == 0) S.abort_flag = 0;
        fence_mbar_init();
    } else if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&S.tmem_base), F::kTmemCols);
        tmem_relinquish();
    } else if (warp == kWarpLoad && lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    griddep_launch_dependents();
    // This CTA's share. Few sequences: every warp finds it for itself.
    Walk w{};
    int64_t per, begin;
    if (a.B <= 32) {
        if (lane < a.B) w.s = grouped_seq(a, lane, blockIdx.x == 0 && warp == 0);
        const int64_t n = grouped_seq_tiles(a, w.s);
        int64_t x = n;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        const int64_t total = __shfl_sync(0xFFFFFFFFu, x, 31);
        per = grouped_share(a, total);
        begin = per * blockIdx.x;
        w.left = min(total, begin + per) - begin;
        // the last sequence that begins at or before the share does and has tiles there
        w.b = __ffs(__ballot_sync(0xFFFFFFFFu, begin >= x - n && begin < x)) - 1;
        const int from = max(w.b, 0);
        const int64_t local = begin - __shfl_sync(0xFFFFFFFFu, x - n, from);
        w.s.q0 = __shfl_sync(0xFFFFFFFFu, w.s.q0, from);
        w.s.n = __shfl_sync(0xFFFFFFFFu, w.s.n, from);
        w.s.len = __shfl_sync(0xFFFFFFFFu, w.s.len, from);
        w.s.items = __shfl_sync(0xFFFFFFFFu, w.s.items, from);
        w.s.tiles = __shfl_sync(0xFFFFFFFFu, w.s.tiles, from);
        w.t = local;
        tc_fence_before();
        block_sync();
    } else {
        int64_t total, base;
        begin = find_place<F::kThreads>(
            a.B, [&](int b) { return grouped_seq_tiles(a, grouped_seq(a, b, blockIdx.x == 0)); },
            [&](int64_t all) { return grouped_share(a, all) * blockIdx.x; }, &total, &w.b, &base, S.warp_sums, S.found);
        per = grouped_share(a, total);
        w.left = min(total, begin + per) - begin;
        if (w.left > 0) w.s = grouped_seq(a, w.b, false);
        w.t = begin - base;
        tc_fence_before();
        block_sync();
    }
    tc_fence_after();
    if (w.left > 0) {  // (w.t: the share's begin in its sequence's tiles)
        w.item = w.t < (1ll << 31) ? static_cast<int>(w.t) / w.s.tiles : static_cast<int>(w.t / w.s.tiles);
        w.tile = static_cast<int>(w.t - static_cast<int64_t>(w.item) * w.s.tiles);
    }
    w.t = begin;
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem_base, 0);
    Piece p;

    if (warp == kWarpLoad) {
        // --------------------------------------------------------------------------- TMA: keys and values
        // Lane l holds the table entry and scales of every 32nd block of the piece, the next 32 fetched while these load.
        int st = 0, phase = 1, tiles = 0;
        bool ok = true;
        while (ok && next_piece(a, w, p)) {
            const int32_t* table = a.block_table + static_cast<int64_t>(w.b) * a.max_blocks;
            const int blocks = min(2 * p.tile1, (w.s.len + kBlock - 1) / kBlock);
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
            // What the weights of 32 blocks refer their value scales to: a power of two no smaller than any of them, kept from
            // before unless it is 4 times too large, or 64^-i of it for a scale that is 64^i times smaller or more. So a block's
            // weights keep their bits whatever the scales of others are, and O^T is seldom moved to another power (which loses
            // nothing, as long as they stay within 2^kRefRange of an item's largest).
            int unit = 0, most = 0;
            uint32_t refs;
            auto refer = [&]() {
                const bool there = row >= 0;
                const uint32_t bits = there ? __float_as_uint(vs) & 0x7FFFFFFFu : 0u;
                const int e = min(max(static_cast<int>((bits + 0x7FFFFFu) >> 23), kLeastRef), 254);  // 2^(e - 127) >= the scale
                const int top = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(e)));
                if (top > unit || top + 2 <= unit) unit = top;
                most = max(most, unit);
                const int mine = max(max(unit - (unit - e) / 6 * 6, most - kRefRange), kLeastRef);
                vs = __uint_as_float(bits) * __uint_as_float(static_cast<uint32_t>(258 - mine) << 23);  // kTop / 2^(mine - 127)
                const int next = __shfl_down_sync(0xFFFFFFFFu, mine, 1);
                const bool next_there = __shfl_down_sync(0xFFFFFFFFu, there, 1);
                const int first = there ? mine : next_there ? next : unit, second = next_there ? next : first;  // (even lanes: of their tile)
                refs = (there ? 1u : 0u) | (next_there ? 2u : 0u) | (first != second ? 4u : 0u) | first << 8 | second << 16;
            };
            fetch(2 * p.tile0, row_next, ks_next, vs_next);
            for (int tile = p.tile0; ok && tile < p.tile1; ++tile) {
                const int j = (tile - p.tile0) & 15;
                if (j == 0) {
                    row = row_next, ks = ks_next, vs = vs_next;
                    fetch(2 * tile + 32, row_next, ks_next, vs_next);
                }
                const int r0 = __shfl_sync(0xFFFFFFFFu, row, 2 * j), r1 = __shfl_sync(0xFFFFFFFFu, row, 2 * j + 1);
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.empty[st]), phase, abort_flag, a.err));
                if (!ok) break;
                const uint32_t bar = smem_u32(&S.full[st]), dst = sRing + st * stage_bytes;
                if (lane == 0) {
                    const uint32_t n = (r0 >= 0 ? 1 : 0) + (r1 >= 0 ? 1 : 0);
                    if (n) mbar_expect_tx(bar, n * (kc + vc) * kChunk);
#pragma unroll 1
                    for (int c = 0; c < kc; ++c) {
                        if (r0 >= 0) tma_load_2d(dst + 2 * c * kChunk, &map_k, c * 128, r0 * kBlock, bar);
                        if (r1 >= 0) tma_load_2d(dst + (2 * c + 1) * kChunk, &map_k, c * 128, r1 * kBlock, bar);
                    }
#pragma unroll 1
                    for (int c = 0; c < vc; ++c) {
                        if (r0 >= 0) tma_load_2d(dst + v_off + 2 * c * kChunk, &map_v, c * 128, r0 * kBlock, bar);
                        if (r1 >= 0) tma_load_2d(dst + v_off + (2 * c + 1) * kChunk, &map_v, c * 128, r1 * kBlock, bar);
                    }
                }
                // the scales may still be on their way: they follow
                if (j == 0) refer();
                if (lane >> 1 == j) {
                    S.scales[st][lane & 1] = make_float2(ks, vs);
                    if (!(lane & 1)) S.refs[st] = refs;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
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
        // K Q^T of a tile runs `lead` tiles ahead of V^T P^T (whose stages it must leave to the loads).
        const int lead = min(F::kSB / 2, stages - 1);
        int st = 0, phase = 0, st_v = 0, n = 0, done = 0, item = 0;  // tiles whose logits, whose values were issued
        int last = 0;  // first tile of the item before
        uint32_t first = 0;  // bit n % 32: tile n is the first of its item in its set
        uint32_t turns = 0;  // and bit n % 32: its blocks take turns
        uint32_t came = 0;   // bit b: the phase of p_full[b] to wait for
        bool half = false;   // tile `done` has scales far apart, and its first block's values were issued
        bool ok = true;
        const int ksteps = (a.d_qk + 31) / 32;
        auto values = [&]() {  // V^T P^T of tile `done`
            const int set = kSets == 2 ? done & 1 : 0, buf = done & (F::kPB - 1);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.p_full[buf]), (came >> buf) & 1, abort_flag, a.err));
            if (!ok) return;
            tc_fence_after();
            came ^= 1u << buf;
            half = !half && (turns >> (done & 31) & 1);
            const bool fresh = (first >> (done & 31)) & 1;
#pragma unroll 1
            for (int c = 0; c < vc; ++c) {
                const uint64_t da = sw128_desc(sRing + st_v * stage_bytes + v_off + 2 * c * kChunk, 0, 1024);
                const uint64_t db = plain_desc(sP + buf * F::kPBytes, 128, 2048);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    warp_mma_f8(tmem + F::kColO + (set * F::kVCMax + c) * F::kPN, da + k * (4096 >> 4), db + k * (512 >> 4),
                                idesc_f8(F::kPN, 1u, 1u), fresh && k == 0 ? 0u : 1u);
            }
            if (half) {  // the other block's weights follow
                warp_tc_commit(smem_u32(&S.pv_done[buf]));
                first &= ~(1u << (done & 31));
                return;
            }
            warp_tc_commit(smem_u32(&S.empty[st_v]));
            warp_tc_commit(smem_u32(&S.pv_done[buf]));
            if (++st_v == stages) st_v = 0;
            ++done;
        };
        // Waits until the values of the tiles before `least` have been issued and the barrier's phase has ended, and issues
        // the values of any tile whose weights come meanwhile: an item's last would otherwise stand back until the next
        // item's first tiles have landed, and O^T with them.
        auto await = [&](int least, uint32_t bar, uint32_t parity) {
            long long t0 = clock64();
            while (ok && (done < least || !__all_sync(0xFFFFFFFFu, mbar_test(bar, parity)))) {
                if (done == n) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, a.err));
                } else if (__all_sync(0xFFFFFFFFu, mbar_test(smem_u32(&S.p_full[done & (F::kPB - 1)]), (came >> (done & (F::kPB - 1))) & 1))) {
                    values();
                    t0 = clock64();
                } else {
                    const bool late = clock64() - t0 > kWaitCycles;
                    if (late) {
                        *abort_flag = 1;
                        atomicOr(a.err, DSA_FAULT_TIMEOUT);
                    }
                    ok = __all_sync(0xFFFFFFFFu, !late && !*abort_flag);
                }
            }
        };
        for (;; ++item) {
            const int qb = item & 1;
            // (the item before the last must end for this one's queries to come)
            await(last, smem_u32(&S.q_full[qb]), (item >> 1) & 1);
            last = n;
            const int tiles = ok ? S.item[qb].tiles : 0;
            if (!tiles) break;
            ok = __all_sync(0xFFFFFFFFu, item || mbar_wait(smem_u32(&S.q_first), 0, abort_flag, a.err));
            if (!ok) break;
            for (int tile = 0; tile < tiles; ++tile) {
                // this buffer of logits is free then: V^T P^T of tile n - kSB has been issued, after its weights came
                await(n - lead, smem_u32(&S.full[st]), phase);
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < ksteps; ++k) {
                    const uint64_t da = sw128_desc(sRing + st * stage_bytes + (k >> 2) * 2 * kChunk, 0, 1024) + (k & 3) * 2;
                    const uint64_t db = sw128_desc(sQ + (qb * kc + (k >> 2)) * F::kQBytes, 0, 1024) + (k & 3) * 2;
                    warp_mma_f8(tmem + (n & (F::kSB - 1)) * F::kSN, da, db, idesc_f8(F::kSN, 0u, 0u), k ? 1u : 0u);
                }
                warp_tc_commit(smem_u32(&S.s_full[n & (F::kSB - 1)]));
                if (tile + 1 == tiles) warp_tc_commit(smem_u32(&S.q_empty[qb]));
                const uint32_t bit = 1u << (n & 31);
                first = tile < kSets ? first | bit : first & ~bit;
                turns = S.refs[st] & 4 ? turns | bit : turns & ~bit;
                ++n;
                if (++st == stages) st = 0, phase ^= 1;
            }
        }
        while (ok && done < n) values();
        warp_tc_commit(smem_u32(&S.mma_done));  // every product issued so far
        if (lane == 0) mbar_wait_drain(smem_u32(&S.mma_done), 0, a.err);
    } else if (warp >= kWarpQ) {
        // --------------------------------------------------------------------------------- queries
        // Two warps bring the queries of the next item while this one runs (of the first, the softmax's warps do).
        for (int item = 0;; ++item) {
            const int qb = item & 1;
            const bool more = next_piece(a, w, p);
            bool ok = true;
            if (item > 0) {
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
                if (more) split_queries<T, F>(a, w.s, p, S, qb, sQ + qb * kc * F::kQBytes, kc, warp - kWarpQ, F::kQWarps);
            }
            if (lane == 0) {
                if (warp == kWarpQ) {
                    Item it{};
                    if (more) {
                        it.tile0 = p.tile0, it.tiles = p.tile1 - p.tile0, it.len = w.s.len, it.rows = p.rows, it.t = p.t;
                        it.all_see = min(w.s.len, w.s.len - w.s.n + p.row0 / a.G + 1);
                        it.complete = p.tile0 == 0 && p.tile1 == w.s.tiles;
                        if (!it.complete) {
                            const int64_t u0 = p.t - p.tile0, u1 = u0 + w.s.tiles;
                            it.slot = grouped_slot(begin, p.t, blockIdx.x);
                            it.c0 = static_cast<int>(u0 < (1ll << 31) && per < (1ll << 31) ? static_cast<uint32_t>(u0) / static_cast<uint32_t>(per) : u0 / per);
                            it.join_slot = grouped_slot(it.c0 * per, u0, it.c0);
                            it.parts = 2;
                            while ((it.c0 + it.parts) * per < u1) ++it.parts;
                        }
                    }
                    S.item[qb] = it;
                }
                mbar_arrive(smem_u32(&S.q_full[qb]));
            }
            if (!more) break;
        }
        // and then some of the rows that have no positions
        for (int b = blockIdx.x; b < a.B; b += a.ctas) {
            const GroupedSeq none = grouped_seq(a, b, false);
            if (none.tiles) continue;
            for (int64_t i = threadIdx.x - kWarpQ * 32; i < static_cast<int64_t>(none.n) * a.H * a.d_v; i += F::kQWarps * 32) {
                const int64_t at = static_cast<int64_t>(none.q0) * a.H * a.d_v + i;
                store_act(static_cast<T*>(a.out) + at, 0.0f);
                if (i % a.d_v == 0) {
                    if (a.lse) a.lse[at / a.d_v] = -INFINITY;
                    if (a.weights_out) a.row_lse[at / a.d_v] = -INFINITY;
                }
            }
        }
    } else {
        // --------------------------------------------------------------------------------- softmax
        const int set = warp / F::kSetWarps, group = (warp >> 2) % kGroups, quarter = warp & 3;
        const int j = quarter * 32 + lane;  // position of the tile, TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t o_col = lane_base + F::kColO + group * F::kPP * kRW;
        float2* fm = S.fm[warp];
        float* fac = S.fac[warp];
        const int mates = set * kGroups + group;
        int n = set, n_item = 0, st = set, sphase = 0, item = 0, turn = 0, left = 0, asked = 0;  // n: this set's next tile, n_item: the item's first
        uint32_t sent = ~0u;  // bit b: the phase of pv_done[b] that ends with the products of what was last put in buffer b;
        bool ok = true;       // bit 31: 0 while the second block of a tile whose blocks take turns is dealt with
        // The group's four warps meet at a barrier of the hardware, at which they sleep (asking a barrier in memory again and
        // again, four warps slow each other: when this was changed, 2 rows a token went from 108 us to 92). Only the first warp waits for other roles, with
        // its limit; the others take its word, so that all of them go on or none does.
        auto group_sync = [&]() { named_bar_sync(1 + mates, 128); };
        auto group_ask = [&](auto wait) {
            if (quarter == 0) {
                const bool came = __all_sync(0xFFFFFFFFu, wait());
                if (lane == 0) S.go[asked][mates] = came;
            }
            __syncwarp();
            group_sync();
            ok = S.go[asked][mates];
            asked ^= 1;
        };
        if (next_piece(a, w, p)) {
            split_queries<T, F>(a, w.s, p, S, 0, sQ, kc, warp, F::kSoftWarps);
            if (lane == 0) mbar_arrive(smem_u32(&S.q_first));
        }
        for (;; ++item) {
            const int qb = item & 1;
            group_ask([&]() {
                return mbar_wait(smem_u32(&S.q_full[qb]), (item >> 1) & 1, abort_flag, a.err) &&
                       (item || !S.item[0].tiles || mbar_wait(smem_u32(&S.q_first), 0, abort_flag, a.err));
            });
            const Item& it = S.item[qb];
            if (!ok || !it.tiles) break;
            const int n_end = n_item + it.tiles, len = it.len, all_see = it.all_see;
            float l[kRW];
            int v_ref = kLeastRef;  // exponent of what value scales refer to in O^T
            float m = -INFINITY;  // what the weights of row lane % kRW refer to: its maximum so far, or up to kSlack less
#pragma unroll
            for (int r = 0; r < kRW; ++r) l[r] = 0.0f;
            const float f_lane = S.q_factor[qb][group * kRW + lane % kRW];  // lane r: row r's factor (positive)
            const int* seen = S.seen[qb] + group * kRW;
            // the item before this has left O^T and the sets' shares
            bool waited = kSets == 1 || item == 0;
            auto o_left = [&]() { return waited || mbar_wait(smem_u32(&S.o_free), (item - 1) & 1, abort_flag, a.err); };
            const bool any = n < n_end;
            bool fresh = true;
            while (ok && n < n_end) {
                const int tile = it.tile0 + n - n_item;
                group_ask([&]() {
                    return mbar_wait(smem_u32(&S.full[st]), sphase, abort_flag, a.err) &&
                           mbar_wait(smem_u32(&S.s_full[n & (F::kSB - 1)]), (n / F::kSB) & 1, abort_flag, a.err);
                });
                if (!ok) break;
                tc_fence_after();
                const int round = sent >> 31 ^ 1;
                const float2 sc = S.scales[st][quarter >> 1];
                const uint32_t refs = S.refs[st];
                const int valid = refs & 7, pos = tile * kGroupedTile + j;
                const bool there = valid >> (quarter >> 1) & 1 && pos < len, whole = valid == 3 && (tile + 1) * kGroupedTile <= all_see;
                // blocks with scales far apart take turns
                auto turns_now = [&]() { return *static_cast<volatile uint32_t*>(&S.refs[st]) & 4; };
                const bool here = there && (!(valid & 4) || (quarter >> 1) == round);
                if (!whole && group == 0 && !there && !round) {  // what the slot holds must not reach the products: 0 * NaN is NaN
#pragma unroll 1
                    for (int c = 0; c < vc; ++c) {
                        const uint32_t at = sRing + st * stage_bytes + v_off + 2 * c * kChunk + j * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16 * i), "r"(0) : "memory");
                    }
                }
                const float ks = here ? sc.x : 1.0f;
                const int ref = refs >> (round ? 16 : 8) & 255;
                uint32_t* flag = S.flag[turn][mates];
                // The weights are formed against the maxima as they stand. Where a logit passes one by more than kSlack, in
                // any of the group's warps, they are moved up first and the weights formed again.
                bool move = fresh || ref != v_ref, sure = false;
                for (;;) {
                    float s[kRW];
                    load_logits<F::kQP, kRW>(lane_base + (n & (F::kSB - 1)) * F::kSN + group * F::kQP * kRW, ks, s);
                    if (!whole) {
#pragma unroll
                        for (int r = 0; r < kRW; ++r) s[r] = here && pos < seen[r] ? s[r] : -INFINITY;
                    }
                    if (move) {
                        sure = true;
                        // the rows' maxima over the tile: every warp's, then lane r of each warp looks after row r
                        float top = -INFINITY;
#pragma unroll
                        for (int r = 0; r < kRW; ++r) {
                            const float x = warp_max(s[r]);
                            if (lane == r) top = x;
                        }
                        if (lane < kRW) S.red[mates][lane][quarter] = top * f_lane;
                        group_ask([&]() {  // O^T is this set's own, and the products into it have ended
                            constexpr int kBack = kSets == 2 ? 2 : 1;
                            const int back = (round ? n : n - kBack) & (F::kPB - 1);
                            return fresh ? o_left() : mbar_wait(smem_u32(&S.pv_done[back]), (sent >> back) & 1, abort_flag, a.err);
                        });
                        if (!ok) break;
                        if (fresh) waited = true;
                        const float4 t = *reinterpret_cast<const float4*>(S.red[mates][lane % kRW]);
                        const float m_new = fmaxf(fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)), m);
                        const float v_fac = __uint_as_float(static_cast<uint32_t>(max(127 + v_ref - ref, 0)) << 23);
                        v_ref = ref;
                        if (lane < kRW) fac[lane] = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
                        m = m_new;
                        // (a row without positions so far: any logit moves it)
                        if (lane < kRW) fm[lane] = make_float2(f_lane, m == -INFINITY ? 1e30f : -m);
                        __syncwarp();
                        if (!fresh) {
#pragma unroll
                            for (int r = 0; r < kRW; ++r) l[r] *= fac[r];
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < vc; ++c) {
#pragma unroll 1
                                for (int i = 0; i < F::kPP * kRW; i += 8) {
                                    float o[8];
                                    const uint32_t at = o_col + (set * F::kVCMax + c) * F::kPN + i;
                                    load_columns<8>(at, o);
#pragma unroll
                                    for (int r = 0; r < 8; ++r) o[r] *= fac[(i + r) % kRW] * v_fac;
                                    store_columns<8>(at, o);
                                }
                            }
                            tmem_st_wait();
                        }
                        group_sync();  // the maxima have been read
                    }
                    if (a.weights_out && (!turns_now() || (quarter >> 1) == round) && it.t + n - n_item < a.max_tiles) {
                        float* to = a.z + ((it.t + n - n_item) * kRows + group * kRW) * kGroupedTile + j;
#pragma unroll
                        for (int r = 0; r < kRW; ++r)
                            if (group * kRW + r < it.rows) to[r * kGroupedTile] = s[r] * fm[r].x;
                    }
                    float over = -INFINITY;
#pragma unroll
                    for (int r = 0; r < kRW; r += 2) {
                        const float4 g = *reinterpret_cast<const float4*>(fm + r);
                        s[r] = fmaf(s[r], g.x, g.y);
                        s[r + 1] = fmaf(s[r + 1], g.z, g.w);
                        over = fmaxf(over, fmaxf(s[r], s[r + 1]));
                    }
                    if (!sure) {  // (read by the others when they all have their weights)
                        const bool up = __any_sync(0xFFFFFFFFu, over > kSlack);
                        if (lane == 0) flag[quarter] = up;
                    }
                    const float tv = here ? sc.y : 0.0f;
                    const uint32_t p_buf = sP + (n & (F::kPB - 1)) * F::kPBytes + j * 16;
                    constexpr int kRun = kRW < 16 ? 8 : 16;  // rows whose codes stand side by side
#pragma unroll
                    for (int r0 = 0; r0 < kRW; r0 += kRun) {
                        uint32_t parts[kRun / 2][F::kPP];
#pragma unroll
                        for (int i = 0; i < kRun / 2; ++i) {
                            const int r = r0 + 2 * i;
                            s[r] = ex2(s[r]);
                            s[r + 1] = ex2(s[r + 1]);
                            split_pair<kPStep>(s[r] * tv, s[r + 1] * tv, parts[i]);
                        }
#pragma unroll
                        for (int i = 0; i < F::kPP; ++i) {
                            const int col = group * F::kPP * kRW + i * kRW + r0;
                            const uint32_t at = p_buf + (col >> 4) * 2048 + (col & 8);
                            if constexpr (kRun == 8)
                                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(parts[0][i] | parts[1][i] << 16),
                                             "r"(parts[2][i] | parts[3][i] << 16)
                                             : "memory");
                            else
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(parts[0][i] | parts[1][i] << 16),
                                             "r"(parts[2][i] | parts[3][i] << 16), "r"(parts[kRun / 2 - 4][i] | parts[kRun / 2 - 3][i] << 16),
                                             "r"(parts[kRun / 2 - 2][i] | parts[kRun / 2 - 1][i] << 16)
                                             : "memory");
                        }
                    }
                    if (!sure) {
                        __syncwarp();
                        group_sync();
                        const uint4 u = *reinterpret_cast<const uint4*>(flag);
                        if (u.x | u.y | u.z | u.w) {
                            move = true;
                            continue;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kRW; ++r) l[r] += s[r];
                    break;
                }
                if (!ok) break;
                turn ^= 1;
                fresh = false;
                fence_proxy_async_smem();
                tc_fence_before();
                const bool turns = turns_now();  // (the stage may be filled again once the weights are out)
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&S.p_full[n & (F::kPB - 1)]));
                sent ^= 1u << (n & (F::kPB - 1));
                if (turns) {
                    sent ^= 1u << 31;
                    if (!round) continue;  // the tile's other block
                }
                n += kSets;
                st += kSets;
                if (st >= stages) st -= stages, sphase ^= 1;
            }
            if (!ok) break;
            if (!waited) group_ask(o_left);
            if (!ok) break;
            // the item's end: this set's share of it
            const float sum = sum_rows<kRW>(l, lane);
            if (lane < kRW) {
                S.fin_l[qb][set][group * kRW + lane][quarter] = sum;
                S.fin_m[qb][set][group * kRW + lane] = m;
            }
            if (lane == 0) S.fin_unit[qb][set] = any ? __uint_as_float(static_cast<uint32_t>(v_ref) << 23) * (1.0f / kTop) : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.fin));
            const bool complete = it.complete;
            if (kSets == 1 || ((n_end - 1) & 1) == set) {
                // the last tile was this set's: the rows, or their partial
                group_ask([&]() {
                    return mbar_wait(smem_u32(&S.fin), item & 1, abort_flag, a.err) &&
                           mbar_wait(smem_u32(&S.pv_done[(n_end - 1) & (F::kPB - 1)]), (sent >> ((n_end - 1) & (F::kPB - 1))) & 1, abort_flag, a.err);
                });
                if (!ok) break;
                tc_fence_after();
                // lane r: row r's maximum and sum over both sets, and what each set's O^T is to be multiplied by
                const int slot = it.slot, rr = group * kRW + lane % kRW;
                float top = -INFINITY, all = 0.0f, f[kSets];
#pragma unroll
                for (int i = 0; i < kSets; ++i) top = fmaxf(top, S.fin_m[qb][i][rr]);
#pragma unroll
                for (int i = 0; i < kSets; ++i) {
                    const float4 x = *reinterpret_cast<const float4*>(S.fin_l[qb][i][rr]);
                    const float u = S.fin_unit[qb][i];
                    f[i] = top == -INFINITY ? 1.0f : ex2(S.fin_m[qb][i][rr] - top);
                    if (u != 0.0f) all = fmaf((x.x + x.y) + (x.z + x.w), f[i], all);
                    f[i] *= u;
                }
                const float inv = all == 0.0f ? 0.0f : complete ? 1.0f / all : 1.0f;
                const int row_at = S.row_at[qb][rr];
                if (quarter == 0 && lane < kRW && rr < it.rows) {
                    const float lse2 = all == 0.0f ? -INFINITY : top + log2f(all);
                    if (!complete) a.part_ml[slot * kRows + rr] = make_float2(top, all);
                    if (complete && a.lse) a.lse[row_at] = lse2 * 0.6931471805599453f;
                    if (complete && a.weights_out) a.row_lse[row_at] = lse2;
                }
                const int other = kSets == 1 ? 0 : 1 - set;
                const bool both = kSets == 2 && S.fin_unit[qb][other] != 0.0f;
                const float f_own = f[kSets == 1 ? 0 : set] * inv, f_other = f[other] * inv;
#pragma unroll 1
                for (int c = 0; c < vc; ++c) {
                    const int e = c * 128 + j;
                    const uint32_t own_col = o_col + (set * F::kVCMax + c) * F::kPN, other_col = o_col + (other * F::kVCMax + c) * F::kPN;
#pragma unroll 1
                    for (int r0 = 0; r0 < kRW; r0 += 8) {
                        float y[8], x[8];
                        join_parts<F::kPP, kRW>(own_col + r0, y);
                        if (both) join_parts<F::kPP, kRW>(other_col + r0, x);
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            y[r] *= __shfl_sync(0xFFFFFFFFu, f_own, r0 + r);
                            const float fo = __shfl_sync(0xFFFFFFFFu, f_other, r0 + r);
                            if (both) y[r] = fmaf(x[r], fo, y[r]);
                            const int64_t at = __shfl_sync(0xFFFFFFFFu, row_at, r0 + r);
                            const int of_item = group * kRW + r0 + r;
                            if (of_item < it.rows && e < a.d_v) {
                                if (complete) store_act(static_cast<T*>(a.out) + at * a.d_v + e, y[r]);
                                else a.part_o[(static_cast<int64_t>(slot) * kRows + of_item) * a.d_v + e] = y[r];
                            }
                        }
                    }
                }
                tc_fence_before();  // O^T has been read before the next item's first product may overwrite it
                __syncwarp();
                if (lane == 0 && kSets == 2) mbar_arrive(smem_u32(&S.o_free));
                if (!complete) {
                    // The CTA that leaves an item's last partial joins them, in order. (Mostly the one whose share ends in
                    // it, with nothing left to do: the others got theirs out at their shares' begin.)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.left[0]));
                    if (warp == set * F::kSetWarps) {
                        const bool came = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.left[0]), left, abort_flag, a.err));
                        if (lane == 0) {
                            __threadfence();
                            const int shift = 8 * (it.c0 & 3), parts = it.parts;
                            const uint32_t old = came ? atomicAdd(a.arrived + (it.c0 >> 2), 1u << shift) : 0;
                            const bool last = came && static_cast<int>((old >> shift) & 255u) == parts - 1;
                            if (last) atomicSub(a.arrived + (it.c0 >> 2), static_cast<uint32_t>(parts) << shift);  // for the next call
                            __threadfence();
                            S.last_part = last;
                        }
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(smem_u32(&S.left[1]));
                    group_ask([&]() { return mbar_wait(smem_u32(&S.left[1]), left, abort_flag, a.err); });
                    if (!ok) break;
                    if (S.last_part)
                        grouped_join<T, kRows < 32 ? 2 : 4, kRows < 32 ? 4 : 2>(a, S.row_at[qb], it.rows, it.join_slot, it.parts,
                                                                                warp - set * F::kSetWarps, F::kSetWarps);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.q_empty[qb]));
            n_item = n_end;
            if (!complete) left ^= 1;  // (whichever set it was)
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
// of wide values fewer: their parts fill tensor memory (and of wide keys, shared memory). More rows an item read the cache
// fewer times (16 sequences of 8000 on average, 8 heads of 128, 8 query heads each; us): 16 rows a sequence 116 in items of
// 8, 82 in one of 16; 32 rows 145 in items of 16, 107 in one of 32; 64 rows 192 in items of 32, 183 in one of 64; fp32, 16
// rows 126 in items of 8, 92 in one of 16.
int grouped_row_tile(const dsa_grouped_dims& d, int T) {
    const int64_t rows = (static_cast<int64_t>(T) + d.B - 1) / d.B * (d.H / d.H_kv);
    const int most = d.type == DSA_F32 || d.d_v > 128 ? 16 : d.d_qk > 128 ? 32 : 64;
    int tile = 8;
    while (tile < rows && tile < most) tile *= 2;
    return tile;
}

int grouped_ctas(const dsa_grouped_dims&) {
    const int sms = device_sm_count();
    return sms < 240 ? sms : 240;  // (a byte for each in the workspace's first 256)
}

bool launch_grouped_attn(const GroupedArgs& a, cudaStream_t s, int* launches) {
    using namespace gtc;
    bool ok = false;
    if (a.type == DSA_F32) {
        ok = a.row_tile == 8 ? launch_form<float, Form<8, 1, 2, 6, 6, 4>>(a, s) : launch_form<float, Form<8, 2, 1, 6, 6, 2>>(a, s);
    } else {
        switch (a.row_tile) {
            case 8: ok = launch_form<__nv_bfloat16, Form<8, 1, 2, 2, 4, 4>>(a, s); break;
            case 16: ok = launch_form<__nv_bfloat16, Form<16, 1, 2, 2, 4, 4>>(a, s); break;
            case 32: ok = launch_form<__nv_bfloat16, Form<16, 2, 1, 2, 4, 2>>(a, s); break;
            default: ok = launch_form<__nv_bfloat16, Form<16, 4, 1, 2, 4, 2>>(a, s); break;
        }
    }
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
