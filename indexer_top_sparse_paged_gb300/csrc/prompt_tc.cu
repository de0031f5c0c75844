// Dense attention over packed prompts on tcgen05 tensor cores (bf16, d_qk <= 192, d_v <= 128).
//
//   z = sm_scale q k^T over the keys j <= i + lk - lq (causal) or all of them, out = softmax(z) v,
//   lse = log sum exp z; a row without keys gives 0 and -inf.
//
// A CTA takes 256 rows (token, head of the group) of one key head as two query tiles A and B of 128 and
// passes over their keys once, 128 at a time. Tensor memory holds both tiles' logits S (fp32, their bf16
// weights P written over them) and outputs O (fp32). While the softmax of one tile runs on the CUDA
// cores, the tensor pipe works for the other: P_A V, Q_A K, P_B V, Q_B K, ... in that order, where Q_X K
// of the next keys may follow P_X V of the last at once, since the pipe runs in order.
//
// Units of at most 128 rows (single tokens, the end of a prompt) would leave tile B without work and every step
// waiting for the last: there both tiles hold the same rows and take every other key tile, and tile A's warps
// join the two.
//
// Softmax: one thread per row, the running maximum m and sum l in fp32; O is rescaled only when a row's
// maximum has grown by more than 2^8 since the last time (weights then stay below 2^8, and O and l hold
// the same factor). Weights are rounded to bf16 for the product (half a step, 2^-8 of a weight, as the
// values' own); l sums them unrounded, so that lse keeps fp32.
//
// Keys and values arrive by TMA as chunks of 128 rows x 64 columns (16 KB, 128-byte swizzle) in a ring
// shared by both; columns past the width and rows past the tensor read as zeros. Value rows that the
// sequence does not own are zeroed before the product: a weight of 0 would not silence a NaN there.
//
// Roles (384 threads): warps 0-3 softmax and epilogue of tile A, 4-7 of tile B, warps 8 and 9 issue the
// MMAs of tile A and B (two issuers: the tensor pipe takes little work ahead, and one's waits and commits
// would leave it idle), warp 10 loads keys and values, warp 11 hands out the units and loads queries. CTAs are
// persistent and draw units from the plan's list by a counter, late; the next unit's queries and keys arrive,
// and its first products run, while the last one's outputs are written. (Four more warps for the outputs leave
// the softmax 192 registers instead of 208: 304 us, not 297, for 9 prompts with 128 heads.)
//
// The two tiles in turn, the late rescaling and weights that are sent before the last of them is made are ideas
// known from published attention kernels for this kind of GPU; roles, turns, work list and units apart are this file's own.
//
// 8192 tokens, 32 / 8 heads of 128 columns: 398 us back to back (407-414 among other calls), 1380 (1330) TFLOP/s of
// the causal products, 73% (70%) of the measured bf16 rate. Bound by the chain of each tile, logits -> weights -> product, two of which take turns: a pair of
// tiles takes about 2900 cycles and its products 2048 of them. Short prompts pay the filling and draining of that
// chain for every unit (9 prompts of up to 1100 tokens, 128 heads of 192 / 128: 289 us where the bytes take 119).
#include "prompt.cuh"

namespace dsa {
namespace ptc {

constexpr int kThreads = 384;
constexpr int kSoftRegs = 208, kOtherRegs = 80;  // 256 x 208 + 128 x 80 registers of the launch's 384 x 168
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= kThreads * 168, "register shares");
constexpr int kRows = 128;                     // rows of a query tile
constexpr int kKeys = kPromptKeys;             // keys of a key tile
constexpr int kChunk = 128 * 128;              // 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;     // S/P of tile A, B at 0, 128; O at 256, 384
constexpr uint32_t kIdescQK = idesc_f16(128, kKeys, 1u, 0u, 0u);
constexpr uint32_t kIdescPV = idesc_f16(128, 64, 1u, 0u, 1u);
constexpr uint32_t kIdescPV2 = idesc_f16(128, 128, 1u, 0u, 1u);
constexpr int kMaxStages = 12;                 // chunks in the ring, and groups (key or value tiles) in flight
constexpr int kSmemMax = 232448;

// One unit of the work list for one key head.
struct Work {
    int q0, lq, k0, lk, row0, kt0;
    int slot, part, parts;
    int hk;      // key head; -1: no more work
    int nrows;   // rows of the sequence for this head
    int n0, n1;  // key tiles [kt0, n0) of tile A, [kt0, n1) of tile B
    int apart;   // few rows: both tiles hold the same ones, A takes the key tiles kt0, kt0 + 2, ..., B the others
    int pad[2];
};

constexpr int kQueue = 2;            // units handed out and not yet taken up by every role
constexpr int kDrawAhead = 6;        // key tiles of a unit still to come when the next one is drawn
constexpr int kTakers = 11;          // 8 softmax warps, 2 MMA warps, the key loader

struct Ctl {
    Work work[kQueue];
    uint64_t work_full[kQueue], work_free[kQueue];
    uint64_t draw;  // the unit's last tiles are at work: the next unit is drawn
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2][2], o_full[2];  // p_full: the first 96 keys' weights, the rest
    uint64_t turn[2];  // the tensor pipe's next turn belongs to tile A, B
    uint64_t join_full[4], join_free[4];  // tile B's part of a unit apart, by warp: ready, read
    float2 join_ml[kRows];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

// A turn around the kMaxStages group barriers, with the parity of its phase.
struct Turn {
    int i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == kMaxStages) i = 0, phase ^= 1;
    }
    __device__ __forceinline__ void back() {
        if (i-- == 0) i = kMaxStages - 1, phase ^= 1;
    }
};

template <int kQC>
struct Layout {
    static constexpr size_t kOffRing = 2 * static_cast<size_t>(kQC) * kChunk;
    static constexpr int kFit = static_cast<int>((kSmemMax - 1024 - sizeof(Ctl) - kOffRing) / kChunk);
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr size_t kOffCtl = kOffRing + static_cast<size_t>(kStages) * kChunk;
    static constexpr size_t kBytes = 1024 + kOffCtl + sizeof(Ctl);
};

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// A value that is the same in every lane, as the compiler can tell (it may live in a uniform register).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Units are run head group by head group, the heads of a group side by side.
// A whole warp calls (every lane gets the same); hk is -1 past the last unit.
__device__ __forceinline__ Work get_work(const PromptArgs& a, int n_units, int group, int w) {
    Work x;
    PromptUnit u;
    x.hk = -1;
    if (a.self_plan) {
        if (!prompt_self_unit(a, w / a.H_kv, u)) return x;
        x.hk = w % a.H_kv;
    } else {
        if (w >= n_units * a.H_kv) return x;  // n_units * H_kv is below 2^31
        const int per = n_units * group;
        const int g = group == a.H_kv ? 0 : w / per;
        const int heads = min(group, a.H_kv - g * group);
        const int rem = w - g * per;
        const int unit = rem / heads;
        x.hk = g * group + rem - unit * heads;
        u = a.units[unit];
    }
    const int G = a.H / a.H_kv;
    x.nrows = u.lq * G;
    auto tiles = [&](int r0) {
        int n = 0;
        if (r0 < x.nrows)
            n = (prompt_keys_seen(a, (min(x.nrows, r0 + kRows) - 1) / G, u.lq, u.lk) + kKeys - 1) / kKeys;
        return max(u.kt0, min(u.kt1, n));
    };
    x.n0 = tiles(u.row0);
    x.n1 = tiles(u.row0 + kRows);
    x.apart = x.nrows - u.row0 <= kRows && x.n0 - u.kt0 >= 2;
    if (x.apart) x.n1 = x.n0;
    x.q0 = u.q0, x.lq = u.lq, x.k0 = u.k0, x.lk = u.lk, x.row0 = u.row0, x.kt0 = u.kt0;
    x.slot = u.slot, x.part = u.part, x.parts = u.parts;
    return x;
}

template <int kQC, int kVC>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(PromptArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, int q_map, int k_swap, int v_swap) {
    using Lay = Layout<kQC>;
    constexpr int kStages = Lay::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), sRing = smem_u32(smem + Lay::kOffRing);
    Ctl& S = *reinterpret_cast<Ctl*>(smem + Lay::kOffCtl);
    volatile int* abort_flag = &S.abort_flag;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), 2);  // both tiles are done with the group
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&S.q_full[i]), q_map ? 1 : 32);  // TMA, or every lane of the copying warp
            mbar_init(smem_u32(&S.q_free[i]), 1);
            mbar_init(smem_u32(&S.s_full[i]), 1);
            mbar_init(smem_u32(&S.turn[i]), 1);
            mbar_init(smem_u32(&S.p_full[i][0]), 4);
            mbar_init(smem_u32(&S.p_full[i][1]), 4);
            mbar_init(smem_u32(&S.o_full[i]), 1);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(smem_u32(&S.work_full[i]), 1);
            mbar_init(smem_u32(&S.work_free[i]), kTakers);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&S.join_full[i]), 32);
            mbar_init(smem_u32(&S.join_free[i]), 32);
        }
        mbar_init(smem_u32(&S.mma_done), 2);
        mbar_init(smem_u32(&S.draw), 1);
        S.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&S.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    block_sync();
    tc_fence_after();
    const uint32_t tmem = uniform(S.tmem_base);
    griddep_launch_dependents();
    griddep_wait();  // the work list
    const int n_units = a.self_plan ? 0 : a.head->n_units, group = a.self_plan ? 0 : a.head->head_group;
    // The next unit, for every role but the one that hands them out; false: no more, or a wait gave up.
    int turn = 0, turn_phase = 0;
    auto take = [&](Work& k) {
        const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.work_full[turn]), turn_phase, abort_flag, a.err));
        if (!got) return false;
        k = S.work[turn];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.work_free[turn]));
        if (++turn == kQueue) turn = 0, turn_phase ^= 1;
        return k.hk >= 0;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 11) {
            // ------------------------------------------------------------------ units and their queries
            const int G = a.H / a.H_kv;
            int qphase0 = 1, qphase1 = 1, fphase = 1, dphase = 0, slot = 0;
            bool ok = true;
            for (int w = blockIdx.x; ok;) {
                const Work k = get_work(a, n_units, group, w);
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.work_free[slot]), fphase, abort_flag, a.err));
                if (!ok) break;
                if (lane == 0) {
                    S.work[slot] = k;
                    mbar_arrive(smem_u32(&S.work_full[slot]));
                }
                if (++slot == kQueue) slot = 0, fphase ^= 1;
                if (k.hk < 0) break;
    #pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    if ((x ? k.n1 : k.n0) == k.kt0) continue;  // no keys: the tile's queries are not used
                    const int row0 = k.row0 + (k.apart ? 0 : x * kRows);
                    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.q_free[x]), x ? qphase1 : qphase0, abort_flag, a.err));
                    if (!ok) break;
                    if (x) qphase1 ^= 1;
                    else qphase0 ^= 1;
                    const uint32_t dst = sQ + x * kQC * kChunk;
                    if (q_map) {  // 128 / G tokens of G heads; what lies behind the sequence is never used
                        if (lane == 0) {
                            mbar_arrive_expect_tx(smem_u32(&S.q_full[x]), kQC * kChunk);
    #pragma unroll
                            for (int c = 0; c < kQC; ++c)
                                tma_load_3d(dst + c * kChunk, &map_q, c * 64, k.hk * G, k.q0 + row0 / G,
                                            smem_u32(&S.q_full[x]));
                        }
                        continue;
                    }
                    // 16-byte pieces of 128 rows, kPieces to a row; rows and columns past the end are zeros
                    constexpr int kPieces = kQC * 8, kStep = 32 / kPieces;
                    const int piece = lane % kPieces;
                    if (lane < kStep * kPieces) {
                        int r = lane / kPieces;
                        int t = (row0 + r) / G, g = row0 + r - t * G;
                        const uint32_t bytes = piece * 8 < a.d_qk ? 16 : 0;
                        const uint16_t* base = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(k.q0) * a.q_stride_t +
                                               static_cast<int64_t>(k.hk) * G * a.q_stride_h + (bytes ? piece * 8 : 0);
    #pragma unroll 4
                        for (; r < kRows; r += kStep) {
                            const bool in = row0 + r < k.nrows;
                            cp_async16(dst + (piece / 8) * kChunk + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                                       in ? base + t * a.q_stride_t + g * a.q_stride_h : static_cast<const uint16_t*>(a.q),
                                       in ? bytes : 0);
                            g += kStep;
                            while (g >= G) {
                                g -= G;
                                ++t;
                            }
                        }
                    }
                    cp_async_arrive_noinc(smem_u32(&S.q_full[x]));
                }
                if (a.self_plan) {
                    w = 0x7FFFFFFF;  // there is a CTA for every unit
                    continue;
                }
                // The next unit is drawn late, so that CTAs with longer ones draw fewer, yet ahead of this one's end
                // (2048 tokens, 32 / 8 heads: 55 us with two units drawn ahead, 44 so).
                // (This wait lasts as long as the unit, 2^24 tiles at most; what stalls in it gives up by itself.)
                const long long t0 = clock64();
                while (ok && !mbar_try_wait(smem_u32(&S.draw), dphase)) {
                    if (clock64() - t0 > 64 * kWaitCycles) {
                        *abort_flag = 1;
                        atomicOr(a.err, DSA_FAULT_TIMEOUT);
                    }
                    ok = !*abort_flag;
                    __nanosleep(64);
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                dphase ^= 1;
                if (lane == 0) w = gridDim.x + atomicAdd(&a.head->next, 1);
                w = __shfl_sync(0xFFFFFFFFu, w, 0);
            }
            // nothing may still be landing when the CTA exits
            cp_async_wait<0>();
            if (q_map && lane == 0) {  // each tile's last load has this phase
                mbar_wait_drain(smem_u32(&S.q_full[0]), qphase0, a.err);
                mbar_wait_drain(smem_u32(&S.q_full[1]), qphase1, a.err);
            }
        } else if (warp == 10) {
            // --------------------------------------------------------------------------------- TMA
            // a group (a key tile of kQC chunks or a value tile of kVC) fills the ring's next chunks
            // once the groups that held them are released, in order
            int slot = 0, in_use = 0;
            Turn put, freed;
            uint32_t values = 0;  // bit i: the group of barrier i holds values
            bool ok = true;
            int groups = 0;
            auto load = [&](bool value, int head, int row) {
                const int n = value ? kVC : kQC, swap = value ? v_swap : k_swap;
                const CUtensorMap* map = value ? &map_v : &map_k;
                while (ok && in_use + n > kStages) {
                    ok = mbar_wait(smem_u32(&S.empty[freed.i]), freed.phase, abort_flag, a.err);
                    in_use -= (values >> freed.i) & 1 ? kVC : kQC;
                    freed.next();
                }
                if (!ok) return;
                const uint32_t bar = smem_u32(&S.full[put.i]);
                values = (values & ~(1u << put.i)) | (value ? 1u << put.i : 0u);
                mbar_arrive_expect_tx(bar, n * kChunk);
    #pragma unroll
                for (int c = 0; c < 3; ++c) {
                    if (c == n) break;
                    if (swap) tma_load_3d(sRing + slot * kChunk, map, c * 64, row, head, bar);
                    else tma_load_3d(sRing + slot * kChunk, map, c * 64, head, row, bar);
                    if (++slot == kStages) slot = 0;
                }
                in_use += n;
                put.next();
                ++groups;
            };
            for (Work k; ok && take(k);) {
                if (lane == 0) {
                    const int kh = a.k_stride_h ? k.hk : 0, vh = a.v_stride_h ? k.hk : 0;  // a shared head is stored once
                    const int end = max(k.n0, k.n1);
                    // keys run one tile ahead of the values, two where the tiles go apart (see the MMA warps)
                    const int lead = k.apart ? 2 : 1;
                    for (int j = k.kt0; ok && j < min(end, k.kt0 + lead); ++j) load(false, kh, k.k0 + j * kKeys);
                    for (int j = k.kt0; ok && j < end; ++j) {
                        load(true, vh, k.k0 + j * kKeys);
                        if (j + lead < end) load(false, kh, k.k0 + (j + lead) * kKeys);
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
            }
            // nothing may still be landing when the CTA exits
            for (int i = groups < kMaxStages ? groups : kMaxStages; i > 0; --i) {
                put.back();
                mbar_wait_drain(smem_u32(&S.full[put.i]), put.phase, a.err);
            }
        } else {
            // --------------------------------------------------------------------------------- MMA
            // With three key chunks the ring holds little more than what is in use: values go back before the product
            // with the next keys, not after it, and those keys are waited for as late as that, inside the turn
            // (8192 tokens, 192 / 128 columns: 478 us against 589 and 504; with 128 columns the same costs 440 against 410).
            constexpr bool kTight = kQC == 3;
            // The whole warp runs along, one elected lane issues (see warp_mma_ss_x4); what the descriptors and
            // the branches depend on is made uniform by hand where it comes from memory.
            const int x = warp - 8;  // tile
            int slot = 0;            // the ring's next chunk
            Turn got, released;      // its group, the next group to give back
            int qphase = 0, pphase = 0, tphase = 1 - x;  // the first turn is tile A's
            bool ok = true;
            auto next = [&](int s, int n) { return s + n < kStages ? s + n : s + n - kStages; };
            auto wait = [&](const uint64_t* bar, int phase) {
                ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), phase, abort_flag, a.err));
                tc_fence_after();
            };
            auto wait_group = [&] {
                wait(&S.full[got.i], got.phase);
                got.next();
            };
            auto release = [&] {  // once every MMA that this warp has issued is done
                warp_tc_commit(smem_u32(&S.empty[released.i]));
                released.next();
            };
            const uint32_t tS = tmem + kColS + x * 128, tO = tmem + kColO + x * 128;
            const uint64_t dq = sw128_desc(sQ + x * kQC * kChunk, 16, 1024), dk = sw128_desc(sRing, 16, 1024);
            const uint64_t dv = sw128_desc(sRing, kChunk, 1024);
            // While both tiles have work they take turns, so that each tile's product with its weights and the
            // next one with its keys run back to back: interleaved, both tiles' logits would be ready at the
            // same time, and the pipe idle while both softmaxes work.
            auto take_turn = [&](bool both) {
                if (!both) return;
                wait(&S.turn[x], tphase);
                tphase ^= 1;
            };
            auto pass_turn = [&](bool both) {
                if (both && lane == 0) mbar_arrive(smem_u32(&S.turn[x ^ 1]));
                __syncwarp();
            };
            // S = Q K^T with the key chunks from ring slot s on; the turn goes over before the last of them
            auto qk = [&](int s, bool both) {
    #pragma unroll
                for (int c = 0; c < kQC; ++c) {
                    if (c == kQC - 1) pass_turn(both);
                    warp_mma_ss_x4(tS, dq + static_cast<uint64_t>((c * kChunk) >> 4),
                                   dk + static_cast<uint64_t>((next(s, c) * kChunk) >> 4), kIdescQK, c != 0 ? 1u : 0u);
                }
                warp_tc_commit(smem_u32(&S.s_full[x]));
            };
            // O += P V with the value chunks from slot s on, steps [from, from + most) of the `steps` groups of
            // 16 keys that the sequence has there
            auto pv = [&](int from, int most, int s, int steps, bool first) {
                const int n = min(steps - from, most);
                const uint32_t acc = first && from == 0 ? 0u : 1u;
                const uint64_t vd = dv + static_cast<uint64_t>((s * kChunk + from * 2048) >> 4);
                const bool wide = kVC == 2 && s + 1 < kStages;  // side by side in the ring: all columns in one product
    #pragma unroll
                for (int c = 0; c < kVC; ++c) {
                    if (c > 0 && wide) break;
                    const uint64_t vc = wide ? vd : dv + static_cast<uint64_t>((next(s, c) * kChunk + from * 2048) >> 4);
                    const uint32_t o = tO + c * 64, idesc = wide ? kIdescPV2 : kIdescPV;
                    if (n == most) {  // (known where it is called: 8, 6 or 2)
                        if (most > 2) warp_mma_ts_x4(o, tS + from * 8, vc, idesc, acc);
                        if (most == 8) warp_mma_ts_x4(o, tS + 32, vc + 512, idesc, 1u);
                        else warp_mma_ts_x2(o, tS + (from + most - 2) * 8, vc + (most - 2) * 128, idesc, most == 6 ? 1u : acc);
                        continue;
                    }
                    int kk = 0;
                    for (; kk < n; ++kk) warp_mma_ts(o, tS + (from + kk) * 8, vc + kk * 128, idesc, kk ? 1u : acc);
                }
            };
            for (Work k; ok && take(k);) {
                const int k_begin = uniform(k.kt0), lk = uniform(k.lk), n0 = uniform(k.n0), n1 = uniform(k.n1);
                const bool apart = uniform(k.apart) != 0;
                const int n = x ? n1 : n0, end = max(n0, n1);
                if (k_begin >= end) continue;
                if (n > k_begin) {  // a tile without keys only walks the groups
                    wait(&S.q_full[x], qphase);
                    qphase ^= 1;
                    fence_proxy_async_smem();  // queries written by cp.async -> visible to the tensor core
                }
                // Key tile j is this warp's below n, or every other one where the tiles go apart; the groups of
                // the others are walked past. Products with keys run `lead` tiles ahead of those with values.
                const int lead = apart ? 2 : 1, first = k_begin + (apart ? x : 0);
                const int both_end = apart ? k_begin : min(n0, n1);  // [k_begin, both_end): the tiles take turns
                auto mine = [&](int j) { return j < n && (!apart || ((j - first) & 1) == 0); };
                for (int j = k_begin; j < min(end, k_begin + lead); ++j) {
                    wait_group();
                    take_turn(j < both_end);
                    if (!ok) break;
                    if (mine(j)) {
                        qk(slot, j < both_end);
                        if (j + lead >= n) warp_tc_commit(smem_u32(&S.q_free[x]));  // the last product with these queries
                    }
                    slot = next(slot, kQC);
                    release();
                }
                for (int j = k_begin; ok && j < end; ++j) {
                    const int vs = slot, ks = next(slot, kVC);
                    const bool more = j + lead < end, both = j < both_end, own = mine(j), own_next = own && j + lead < n;
                    wait_group();
                    if (more && !kTight) wait_group();
                    if (!ok) break;
                    if (own) {
                        const int valid = min(kKeys, lk - j * kKeys);  // value rows of this sequence
                        const int steps = (valid + 15) / 16;
                        if (valid & 15) {  // the rest of the last step belongs to another sequence, or to nobody
                            for (int c = 0; c < kVC; ++c) {  // (both tiles' warps may write the same zeros)
                                uint4* row = reinterpret_cast<uint4*>(smem + Lay::kOffRing + next(vs, c) * kChunk + valid * 128);
                                for (int i = lane; i < (steps * 16 - valid) * 8; i += 32) row[i] = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        wait(&S.p_full[x][0], pphase);
                        take_turn(both);
                        if (!ok) break;
                        // the last quarter's weights are mostly there by now; if not, the first three go ahead
                        const bool whole = __all_sync(0xFFFFFFFFu, mbar_test(smem_u32(&S.p_full[x][1]), pphase));
                        if (whole) {
                            tc_fence_after();
                            pv(0, 8, vs, steps, j == first);
                        } else {
                            pv(0, 6, vs, steps, j == first);
                            wait(&S.p_full[x][1], pphase);
                            if (!ok) break;
                            pv(6, 2, vs, steps, j == first);
                        }
                        pphase ^= 1;
                        if (!own_next) {
                            pass_turn(both);
                            warp_tc_commit(smem_u32(&S.o_full[x]));
                        }
                    }
                    if (kTight) release();
                    slot = ks;
                    if (more) {
                        if (kTight) wait_group();
                        if (!ok) break;
                        if (own_next) {
                            qk(ks, both);
                            if (j + 2 * lead >= n) warp_tc_commit(smem_u32(&S.q_free[x]));
                        }
                        slot = next(slot, kQC);
                        if (!kTight) release();
                        release();
                    } else if (!kTight) {
                        release();
                    }
                }
            }
            warp_tc_commit(smem_u32(&S.mma_done));
            mbar_wait_drain(smem_u32(&S.mma_done), 0, a.err);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // --------------------------------------------------------------------- softmax + epilogue
        const int x = warp >> 2, r = threadIdx.x & 127;  // tile, row = TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + kColS + x * 128, tO = tmem + lane_base + kColO + x * 128;
        const int G = a.H / a.H_kv;
        const float c2 = a.sm_scale * 1.4426950408889634f;  // logits in powers of two
        int sphase = 0, ophase = 0, jphase = 0;
        bool dead = false;
        for (;;) {
            Work k;
            if (!take(k)) break;
            const int row0 = k.row0 + (k.apart ? 0 : x * kRows), row = row0 + r;
            const int t = row < k.nrows ? row / G : 0, head = k.hk * G + (row < k.nrows ? row - t * G : 0);
            const int end = x ? k.n1 : k.n0;
            const bool any = end > k.kt0;
            const int seen = row < k.nrows ? prompt_keys_seen(a, t, k.lq, k.lk) : 0;
            float m = -INFINITY, l = 0.0f;
            const int first = k.kt0 + (k.apart ? x : 0), step = k.apart ? 2 : 1;
            const bool idle = row0 + (warp & 3) * 32 >= k.nrows;  // none of the warp's rows exist
            // One warp says when the next unit is to be drawn: of the tile that has the last keys.
            const bool last = warp == (k.n1 >= k.n0 ? 4 : 0) && !a.self_plan;
            int late = last ? max(first, end - kDrawAhead) : end;
            if (last && !any && lane == 0) mbar_arrive(smem_u32(&S.draw));
            for (int j = first; j < end; j += step) {
                if (j >= late) {
                    late = end;
                    if (lane == 0) mbar_arrive(smem_u32(&S.draw));
                }
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.s_full[x]), sphase, abort_flag, a.err))) {
                    dead = true;
                    break;
                }
                sphase ^= 1;
                tc_fence_after();
                if (idle) {  // whatever the product makes of these rows is not used
                    __syncwarp();
                    if (lane < 2) mbar_arrive(smem_u32(&S.p_full[x][lane]));
                    continue;
                }
                const int vis = seen - j * kKeys;  // keys of the tile this row sees
                const bool cut = !__all_sync(0xFFFFFFFFu, vis >= kKeys);
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(tS + i * 32, s[i]);
                tmem_ld_wait(s[0], s[1], s[2], s[3]);
                if (cut) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[i][e] = i * 32 + e < vis ? s[i][e] : 0xFF800000u;
                }
                const uint64_t c2c2 = pack2(c2, c2);
                uint64_t ls[4] = {0, 0, 0, 0};  // pairs of sums
                auto weights = [&](int i, uint64_t nn) {  // over columns that have been read
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 z = unpack2(fma2(pack2(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])), c2c2, nn));
                        const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
                        ls[e & 3] = add2(ls[e & 3], pack2(p0, p1));
                        const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
                        pk[e] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    tmem_st16(tS + i * 16, pk);
                };
                auto send = [&](int part) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.p_full[x][part]));
                };
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y0 = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
                    float y1 = fmaxf(__uint_as_float(s[i][2]), __uint_as_float(s[i][3]));
#pragma unroll
                    for (int e = 4; e < 32; e += 4) {
                        y0 = max3(y0, __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
                        y1 = max3(y1, __uint_as_float(s[i][e + 2]), __uint_as_float(s[i][e + 3]));
                    }
                    mx[i] = fmaxf(y0, y1);
                }
                const float mt = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c2;
                const bool need = mt > m + 8.0f;
                if (__any_sync(0xFFFFFFFFu, need)) {
                    const float m_new = need ? mt : m;
                    if (j > first) {  // P V of the last tile is done: its commit came before S's
                        const float alpha = m_new == m ? 1.0f : exp2f(m - m_new);
#pragma unroll 1
                        for (int c = 0; c < 2 * kVC; ++c) {
                            uint32_t v[32];
                            tmem_ld32(tO + c * 32, v);
                            tmem_ld_wait(v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                            tmem_st32(tO + c * 32, v);
                        }
                        l *= alpha;
                    }
                    m = m_new;
                }
                const float neg = m == -INFINITY ? 0.0f : -m;  // no key yet: every weight is 2^-inf = 0
                const uint64_t nn = pack2(neg, neg);
                weights(0, nn);
                weights(1, nn);
                weights(2, nn);
                send(0);  // the product may begin while the last quarter is made
                weights(3, nn);
                send(1);
                const float2 lp = unpack2(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])));
                l += lp.x + lp.y;
            }
            if (any && !dead) {
                dead = !__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.o_full[x]), ophase, abort_flag, a.err));
                ophase ^= 1;
            }
            if (dead) break;
            tc_fence_after();
            if (idle) continue;  // (of a unit apart: in both tiles)
            if (k.apart) {
                if (x == 1) {  // tile B's maximum and sum to A's warp, which finds O in tensor memory
                    S.join_ml[r] = make_float2(m, l);
                    tc_fence_before();
                    mbar_arrive(smem_u32(&S.join_full[warp & 3]));
                    dead = !__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.join_free[warp & 3]), jphase, abort_flag, a.err));
                    jphase ^= 1;
                    if (dead) break;
                    continue;
                }
                dead = !__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&S.join_full[warp & 3]), jphase, abort_flag, a.err));
                jphase ^= 1;
                if (dead) break;
                tc_fence_after();
            }
            float fa = 1.0f, fb = 0.0f;  // out = fa O_A + fb O_B
            if (k.apart) {
                const float2 o = S.join_ml[r];
                const float top = fmaxf(m, o.x);
                fa = m == -INFINITY ? 0.0f : exp2f(m - top);
                fb = o.x == -INFINITY ? 0.0f : exp2f(o.x - top);
                l = l * fa + o.y * fb;
                m = top;
            }
            auto load_o = [&](int c, uint32_t (&v)[32]) {  // columns 32c .. of the row's unnormalised output
                tmem_ld32(tO + c * 32, v);
                tmem_ld_wait(v);
                if (k.apart) {
                    uint32_t u[32];
                    tmem_ld32(tO + 128 + c * 32, u);
                    tmem_ld_wait(u);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * fa + __uint_as_float(u[e]) * fb);
                }
            };
            const bool live = row < k.nrows;
            const int64_t at = (static_cast<int64_t>(k.q0) + t) * a.H + head;  // (token, head)
            if (k.parts == 1) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t* out = static_cast<uint16_t*>(a.out) + at * a.d_v;
                const bool sectors = a.d_v % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
                for (int c = 0; c < 2 * kVC; ++c) {
                    uint32_t v[32] = {};
                    if (any) load_o(c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {  // a whole 32-byte sector a store, where rows allow it
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[e + 2 * i]) * inv,
                                                                           __uint_as_float(v[e + 2 * i + 1]) * inv);
                            o[i] = *reinterpret_cast<const uint32_t*>(&b);
                        }
                        if (live && c * 32 + e + 16 <= a.d_v && sectors) {
                            store_32b(out + c * 32 + e, o);
                        } else {
                            uint4* to = reinterpret_cast<uint4*>(out + c * 32 + e);
                            if (live && c * 32 + e < a.d_v) to[0] = make_uint4(o[0], o[1], o[2], o[3]);
                            if (live && c * 32 + e + 8 < a.d_v) to[1] = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                }
                if (live && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                const int64_t slot0 = static_cast<int64_t>(k.slot) * a.H_kv + static_cast<int64_t>(k.hk) * k.parts;
                const int rr = x * kRows + r;  // row of the partial
                const int64_t prow = (slot0 + k.part) * a.slot_rows + rr;
                if (live) a.part_ml[prow] = make_float2(l == 0.0f ? -INFINITY : m, l);
                float* po = a.part_o + part_at(a, slot0 + k.part, 0, rr);
                const int64_t pitch = a.slot_rows;
#pragma unroll 1
                for (int c = 0; c < 2 * kVC && any; ++c) {
                    uint32_t v[32];
                    load_o(c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (!live || c * 32 + e >= a.d_v) break;  // d_v is a multiple of 8
#pragma unroll
                        for (int i = 0; i < 8; ++i, po += pitch) *po = __uint_as_float(v[e + i]);
                    }
                }
            }
            tc_fence_before();  // O has been read before the next unit's first product may overwrite it
            if (k.apart) mbar_arrive(smem_u32(&S.join_free[warp & 3]));
        }
    }
    tc_fence_before();
    block_sync();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// A map of [tokens][heads][cols] with boxes of `box_tokens` tokens x `box_heads` heads x 64 columns; the
// outer extent is the one of the larger stride (*swap: heads). A stride of 0 between the heads: they share one.
static bool make_map(CUtensorMap* map, const void* base, int cols, int heads, int tokens, int64_t stride_t, int64_t stride_h,
                     int box_heads, int box_tokens, int* swap) {
    if (stride_h == 0) heads = 1;
    if (heads == 1) stride_h = stride_t;
    if (tokens == 1) stride_t = stride_h;
    *swap = stride_h > stride_t ? 1 : 0;
    const uint64_t n[2] = {static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
    const uint64_t st[2] = {static_cast<uint64_t>(stride_h) * 2, static_cast<uint64_t>(stride_t) * 2};
    const uint32_t bx[2] = {static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
    const int i = *swap, j = 1 - i;
    return make_tmap_3d(map, base, {static_cast<uint64_t>(cols), n[i], n[j]}, {st[i], st[j]}, {64, bx[i], bx[j]});
}

struct Maps {
    CUtensorMap q{}, k{}, v{};
    int q_map = 0, k_swap = 0, v_swap = 0;
};

template <int kQC, int kVC>
static bool launch_typed(const PromptArgs& a, const Maps& m, cudaStream_t s) {
    constexpr size_t smem = Layout<kQC>::kBytes;
    static_assert(smem <= kSmemMax && Layout<kQC>::kStages >= 2 * kQC + kVC, "two key tiles and a value tile in flight");
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(prompt_tc_kernel<kQC, kVC>), smem)) return false;
    const int64_t most = static_cast<int64_t>(a.max_units) * a.H_kv;  // below 2^31 (checked by the caller)
    const int grid = static_cast<int>(a.self_plan || most < a.ctas ? most : a.ctas);
    return launch_kernel(!a.self_plan, prompt_tc_kernel<kQC, kVC>, dim3(grid), dim3(kThreads), smem, s, a, m.q, m.k, m.v, m.q_map,
                         m.k_swap, m.v_swap);
}

}  // namespace ptc

bool launch_prompt_tc(const PromptArgs& a, cudaStream_t s, int* launches) {
    ptc::Maps m;
    // without keys no tile is loaded and no map read
    if (a.Tk > 0) {
        if (!ptc::make_map(&m.k, a.k, a.d_qk, a.H_kv, a.Tk, a.k_stride_t, a.k_stride_h, 1, 128, &m.k_swap) ||
            !ptc::make_map(&m.v, a.v, a.d_v, a.H_kv, a.Tk, a.v_stride_t, a.v_stride_h, 1, 128, &m.v_swap))
            return false;
        // A box of 128 / G tokens x G heads is a query tile where G divides 128 and the heads are the inner
        // extent; other groups and orders are copied 16 bytes at a time (4K cycles a tile).
        const int G = a.H / a.H_kv;
        int swap = 0;
        m.q_map = 128 % G == 0 && a.q_stride_t > 0 && a.q_stride_h > 0 &&
                  ptc::make_map(&m.q, a.q, a.d_qk, a.H, a.Tq, a.q_stride_t, a.q_stride_h, G, 128 / G, &swap) && !swap;
    }
    const int qc = (a.d_qk + 63) / 64;
    bool ok;
    if (a.d_v <= 64)
        ok = qc == 1 ? ptc::launch_typed<1, 1>(a, m, s) : qc == 2 ? ptc::launch_typed<2, 1>(a, m, s) : ptc::launch_typed<3, 1>(a, m, s);
    else
        ok = qc == 1 ? ptc::launch_typed<1, 2>(a, m, s) : qc == 2 ? ptc::launch_typed<2, 2>(a, m, s) : ptc::launch_typed<3, 2>(a, m, s);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
