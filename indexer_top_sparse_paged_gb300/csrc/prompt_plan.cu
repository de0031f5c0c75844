// Work list of the prompt attention, made on the device (the host never reads the lengths).
//
// The G = H / H_kv query heads of a key head share its keys, so a sequence of lq tokens gives each key
// head one column of lq * G rows, row r = token r / G, head r % G of the group. A unit is tile_rows of
// them against a range of the key tiles they see; every unit runs once for each key head.
//
// Keys are split when the rows are too few to fill the SMs: with W key tiles over all rows and heads and C
// CTAs, if the longest item has more than 1.25 W / C tiles. Every item is then cut at the multiples of
// s = max(W / f C, a 32nd of the longest, min_tiles); a last part shorter than min_tiles stays with the one
// before. The cuts are the same for all rows of a sequence, so that CTAs that run side by side read the same
// keys (a chunk of 2048 on 32K keys: 0.7 ms where cuts at even shares of all tiles took 1.1). f is 2, so that
// CTAs that are done early find more; on the tensor cores 1 where the items are few, and so cut into parts of one
// length that fill one turn of CTAs (a single token, 64 / 8 heads, on 70K keys: 58 us against 73), or where a
// CTA's share is short beside the cost of a unit (16 tokens on up to 2000 keys: 29 us against 35; on up to 16K keys
// f = 2: 118 us against 125).
// An item of n > s tiles becomes at most ceil(n / s) < 2 n / s parts: fewer than 2 W / s <= 4 C partials.
// Units are listed by falling number of tiles: the last ones to run are the short ones.
//
// One CTA, bound by its latency, much of it instructions that are fetched for the first time: the three passes over
// the items (tiles in all, units of each length, the list) are one loop.
#include "prompt.cuh"

namespace dsa {

constexpr int kPlanThreads = 256;
constexpr int kMaxParts = 32;    // of one item, about: one CTA joins them
constexpr int kBuckets = kPlanThreads;

struct PlanItem {
    int q0, lq, k0, lk, row0, tiles;
};

// Key tiles that rows row0 .. row0 + tile_rows - 1 of a sequence see.
__device__ __forceinline__ int item_tiles(const PromptArgs& a, int G, int lq, int lk, int row0) {
    const int last = min(lq * G, row0 + a.tile_rows) - 1;
    const int seen = a.causal ? min(lk, max(0, lk - lq + last / G + 1)) : lk;
    return (seen + kPromptKeys - 1) / kPromptKeys;
}

// Inclusive sums over the CTA of values of 0 or more, none above `most` (below 2^31): sequences that overlap,
// which some descending entry has let happen, may have more items than the lists were made for.
__device__ __forceinline__ int block_scan(int value, int most, int* warp_sum) {
    unsigned x = min(value, most);
    const unsigned top = most;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x = min(x + y, top);
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = static_cast<int>(x);
    __syncthreads();
    if (warp == 0) {
        unsigned w = lane < kPlanThreads / 32 ? warp_sum[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w = min(w + y, top);
        }
        if (lane < kPlanThreads / 32) warp_sum[lane] = static_cast<int>(w);
    }
    __syncthreads();
    return static_cast<int>(min(x + (warp ? warp_sum[warp - 1] : 0), top));
}

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(PromptArgs a) {
    __shared__ int prefix[kPlanThreads + 1];
    __shared__ int4 seqs[kPlanThreads];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int bucket[kBuckets];
    __shared__ unsigned long long total_tiles;
    __shared__ int most_tiles, most_keys, items, slots, joins, join_rows;
    const int tid = threadIdx.x, G = a.H / a.H_kv, shift = 31 - __clz(a.tile_rows);
    griddep_launch_dependents();  // the attention's prologue may start (it waits for this grid)
    if (tid == 0) {
        total_tiles = 0;
        most_tiles = most_keys = items = slots = joins = join_rows = 0;
    }
    bucket[tid] = 0;
    __syncthreads();
    bool kept = false;  // the thread's item stays in registers, if there are no more than threads
    PlanItem it{};
    bool cut = false;
    int s = 1, longest = 1;
    float per_tile = 0.0f;  // buckets
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        if (pass == 1) {
            const long long work = static_cast<long long>(total_tiles) * a.H_kv;
            cut = a.max_slots > 1 && 4ll * a.ctas * most_tiles > 5 * work;
            const bool once = a.tile_rows == kPromptTcRows && (2ll * items * a.H_kv <= a.ctas || work < 16ll * a.ctas);
            // (rounded up: s >= W / f C bounds the number of partials)
            const float share = static_cast<float>(work) / static_cast<float>(once ? a.ctas : a.shares) * 1.000001f;
            s = max(max(a.min_tiles, static_cast<int>(fminf(share, 1e9f)) + 1), (most_tiles + kMaxParts - 1) / kMaxParts);
            longest = max(1, cut ? min(most_tiles, s + a.min_tiles) : most_tiles);
            per_tile = static_cast<float>(kBuckets - 1) / static_cast<float>(longest);
        } else if (pass == 2) {
            const int x = block_scan(bucket[tid], 0x7FFFFFFF, warp_sum);
            if (tid == kPlanThreads - 1) {
                a.head->n_units = min(x, a.max_units);
                a.head->next = 0;
                // heads whose keys and values (read again by every row tile) fit a part of L2 run side by side
                const float head_bytes = 2.0f * (a.d_qk + a.d_v) * max(1, most_keys);
                a.head->head_group = static_cast<int>(fmaxf(1.0f, fminf(static_cast<float>(a.H_kv), 48.0f * 1048576.0f / head_bytes)));
            }
            bucket[tid] = x - bucket[tid];
            __syncthreads();
        }
        int left = a.max_units;  // items
        for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
            if (a.B > kPlanThreads || pass == 0) {  // up to 256 sequences stay in shared memory
                const int b = b0 + tid;
                int n = 0;
                int4 q = make_int4(0, 0, 0, 0);
                if (b < a.B) {
                    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
                    if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) {
                        atomicOr(a.err, DSA_FAULT_INDEX);
                    } else {
                        q = make_int4(q0, q1 - q0, k0, k1 - k0);
                        n = (q.y * G + a.tile_rows - 1) >> shift;
                    }
                }
                seqs[tid] = q;
                const int x = block_scan(n, left, warp_sum);
                prefix[tid + 1] = x;
                if (tid == 0) prefix[0] = 0;
                __syncthreads();
            }
            const int total = prefix[kPlanThreads], seqs_here = min(kPlanThreads, a.B - b0);
            left -= total;
            for (int i0 = 0; i0 < total; i0 += kPlanThreads) {
                const int i = i0 + tid;
                const bool valid = i < total;
                if (!kept) {
                    it = PlanItem{};
                    if (valid) {
                        int lo = 0, hi = seqs_here - 1;  // the last sequence whose first item is at or before i
                        while (lo < hi) {
                            const int mid = (lo + hi + 1) >> 1;
                            if (prefix[mid] <= i) lo = mid;
                            else hi = mid - 1;
                        }
                        const int4 q = seqs[lo];
                        const int row0 = (i - prefix[lo]) << shift;
                        it = PlanItem{q.x, q.y, q.z, q.w, row0, item_tiles(a, G, q.y, q.w, row0)};
                    }
                    kept = a.B <= kPlanThreads && total <= kPlanThreads;
                }
                if (pass == 0) {
                    const unsigned tiles = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(it.tiles));
                    const int most = __reduce_max_sync(0xFFFFFFFFu, it.tiles), keys = __reduce_max_sync(0xFFFFFFFFu, it.lk);
                    if ((tid & 31) == 0) {
                        atomicAdd(&total_tiles, static_cast<unsigned long long>(tiles));
                        atomicMax(&most_tiles, most);
                        atomicMax(&most_keys, keys);
                    }
                } else if (valid) {
                    const int parts = cut ? max(1, (it.tiles + s - a.min_tiles) / s) : 1;
                    int slot = 0;
                    if (pass == 2 && parts > 1) {
                        slot = atomicAdd(&slots, parts);
                        const int j = atomicAdd(&joins, 1);
                        const int rows = min(a.tile_rows, it.lq * G - it.row0);
                        atomicMax(&join_rows, rows);
                        if (slot + parts <= a.max_slots && j < a.max_slots / 2)
                            a.joins[j] = PromptJoin{it.q0, it.row0, rows, slot, parts, {0, 0, 0}};
                    }
                    for (int p = 0; p < parts; ++p) {
                        const int t0 = p * s, t1 = p == parts - 1 ? it.tiles : t0 + s;
                        const int to = max(0, kBuckets - 1 - static_cast<int>(static_cast<float>(min(t1 - t0, longest)) * per_tile));
                        const int at = atomicAdd(&bucket[to], 1);  // falling number of tiles
                        if (pass == 2 && at < a.max_units && slot + (parts > 1 ? parts : 0) <= a.max_slots)
                            a.units[at] = PromptUnit{it.q0, it.lq, it.k0, it.lk, it.row0, t0, t1, slot, p, parts, {0, 0}};
                    }
                }
            }
            if (tid == 0 && pass == 0) items += total;
            if (a.B > kPlanThreads) __syncthreads();  // the next sequences take their place
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.head->n_joins = min(joins, a.max_slots / 2);
        a.head->join_rows = join_rows;
    }
}
static_assert(kBuckets == kPlanThreads, "the bucket scan takes one bucket per thread");
static_assert((kPromptTcRows & (kPromptTcRows - 1)) == 0 && (kPromptSimtRows & (kPromptSimtRows - 1)) == 0, "rows are shifted");

bool launch_prompt_plan(const PromptArgs& a, cudaStream_t s, int* launches) {
    if (!launch_kernel(false, prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

// Joins the rows whose keys were split: a run of CTAs shares the columns of an item and key head, 8 to a thread
// (a prompt of 1024 tokens, 32 / 8 heads: with one CTA for all columns the call took 60 us, with this 31). In the
// attention kernel itself, by the last part to arrive, it held up the units behind it (16 single tokens over up
// to 16K keys: 195 us, then 127).
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PromptArgs a) {
    griddep_wait();
    const int n = __ldcg(&a.head->n_joins), most = __ldcg(&a.head->join_rows);
    int width = 1;  // threads side by side on the rows
    while (width < most) width *= 2;
    const int per = kJoinThreads / width, runs = ((a.d_v + 7) / 8 + per - 1) / per;  // columns of a CTA / 8, CTAs
    for (int w = blockIdx.x; w < n * a.H_kv * runs; w += gridDim.x) {  // the runs of an item and head side by side
        const int i = w / runs, hk = i % a.H_kv;
        const PromptJoin j = a.joins[i / a.H_kv];
        const int64_t slot0 = static_cast<int64_t>(j.slot) * a.H_kv + static_cast<int64_t>(hk) * j.parts;
        const int c = ((w - i * runs) * per + threadIdx.x / width) * 8, r = threadIdx.x % width;
        if (r >= j.rows || c >= a.d_v) continue;
        if (j.parts <= 4) prompt_join<4, T>(a, slot0, j.parts, j.q0, j.row0, hk, r, c);  // (8: 34 us, not 31, there)
        else prompt_join<8, T>(a, slot0, j.parts, j.q0, j.row0, hk, r, c);  // (4: 129 us, not 126, for the single tokens)
    }
}

bool launch_prompt_join(const PromptArgs& a, cudaStream_t s, int* launches) {
    if (a.max_slots < 2) return true;  // no room to split: the plan does not
    const dim3 grid(a.ctas);  // (twice as many cost calls that split nothing 1 us)
    const bool ok = a.type == DSA_F32
                        ? launch_kernel(true, prompt_join_kernel<float>, grid, dim3(kJoinThreads), 0, s, a)
                        : launch_kernel(true, prompt_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, s, a);
    if (ok) ++*launches;
    return ok;
}

}  // namespace dsa
