// Work list of the prompt attention: the packed sequences' query tiles, found on the device (the host
// never reads the lengths).
//
// The G = H / H_kv query heads of a key head share its keys, so a sequence of lq tokens gives each key
// head one column of lq * G rows, row r = token r / G, head r % G of the group; a tile is kRows of them.
#include "internal.h"

namespace dsa {

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(PromptArgs a) {
    __shared__ int prefix[kPlanThreads + 1];
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.H / a.H_kv;
    int done = 0;  // units written for earlier sequences
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < a.B) {
            const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) atomicOr(a.err, DSA_FAULT_INDEX);
            else n = static_cast<int>((static_cast<int64_t>(q1 - q0) * G + a.tile_rows - 1) / a.tile_rows);
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int w = warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
                if (lane >= o) w += y;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        prefix[tid + 1] = x + (warp ? warp_sum[warp - 1] : 0);
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
        const int total = prefix[kPlanThreads];
        for (int i = tid; i < total && done + i < a.max_units; i += kPlanThreads) {
            int lo = 0, hi = kPlanThreads - 1;  // the last sequence whose first tile is at or before i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            a.units[done + i] = PromptUnit{b0 + lo, i - prefix[lo]};
        }
        done += total;
        __syncthreads();
    }
    if (tid == 0) *a.n_units = min(done, a.max_units);
}

bool launch_prompt_plan(const PromptArgs& a, cudaStream_t s, int* launches) {
    if (!launch_kernel(false, prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
