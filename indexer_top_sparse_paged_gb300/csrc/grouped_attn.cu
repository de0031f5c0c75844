// Attention over the grouped-head cache on the CUDA cores: softmax(sm_scale q k^T) v with keys and values as e4m3 codes,
// one pass over the cached rows with a running maximum and sum (logits in powers of two).
#include "grouped.cuh"

namespace dsa {
namespace gsimt {

constexpr int kThreads = 128;  // thread = position of the tile, then column of the values
constexpr int kRows = 8;

__device__ __forceinline__ float load_act(const float* p) { return *p; }
__device__ __forceinline__ float load_act(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_act(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_act(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) grouped_attn_kernel(GroupedArgs a) {
    __shared__ int64_t warp_sums[kThreads / 32], found[2];
    __shared__ float q_s[kRows][256], p_s[kRows][kGroupedTile], red[kThreads / 32][kRows];
    __shared__ int blk_s[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    auto count = [&](int b) { return grouped_seq_tiles(a, grouped_seq(a, b, blockIdx.x == 0)); };
    int64_t total, base;
    int b;
    find_sequence<kThreads>(a.B, -1, count, &total, &b, &base, warp_sums, found);
    const int64_t per = (total + a.ctas - 1) / a.ctas, begin = per * blockIdx.x, end = min(total, begin + per);
    if (begin >= end) return;
    find_sequence<kThreads>(a.B, begin, count, &total, &b, &base, warp_sums, found);
    const float scale2 = a.sm_scale * 1.4426950408889634f;
    for (int64_t t = begin; t < end;) {
        const GroupedSeq s = grouped_seq(a, b, false);
        const int64_t here = grouped_seq_tiles(a, s);
        if (t - base >= here) {
            base += here;
            ++b;
            continue;
        }
        const int64_t local = t - base;
        const int item = static_cast<int>(local / s.tiles), tile0 = static_cast<int>(local - static_cast<int64_t>(item) * s.tiles);
        const int tile1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), tile0 + (end - t)));
        const int h = item / s.items, row0 = (item - h * s.items) * kRows;
        const int rows = min(kRows, s.n * a.G - row0);
        __syncthreads();
        for (int i = tid; i < kRows * a.d_qk; i += kThreads) {
            const int r = i / a.d_qk, e = i - r * a.d_qk, row = row0 + r;
            float x = 0.0f;
            if (r < rows)
                x = load_act(static_cast<const T*>(a.q) + (s.q0 + row / a.G) * a.q_stride_t + (h * a.G + row % a.G) * a.q_stride_h + e);
            q_s[r][e] = isfinite(x) ? x : NAN;  // (infinite products of both signs would mask positions)
        }
        float m[kRows], l[kRows], acc[kRows][2];
        int seen[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            m[r] = -INFINITY;
            l[r] = acc[r][0] = acc[r][1] = 0.0f;
            seen[r] = r < rows ? s.len - s.n + (row0 + r) / a.G + 1 : 0;
        }
        for (int tile = tile0; tile < tile1; ++tile, ++t) {
            const int pos = tile * kGroupedTile + tid;
            int blk = -1;
            if (pos < s.len) {
                blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + pos / kBlock];
                if (blk < 0 || blk >= a.num_blocks) {
                    blk = -1;
                    if (pos % kBlock == 0) atomicOr(a.err, DSA_FAULT_BLOCK_TABLE);
                }
            }
            __syncthreads();  // q_s is there; the last tile's p_s has been read
            if ((tid & 63) == 0) blk_s[tid >> 6] = blk;
            const int64_t bh = static_cast<int64_t>(blk) * a.H_kv + h;
            float z[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) z[r] = 0.0f;
            if (blk >= 0) {
                const uint4* k = reinterpret_cast<const uint4*>(a.k + (bh * kBlock + pos % kBlock) * a.d_qk);
                for (int e = 0; e < a.d_qk / 16; ++e) {
                    float x[16];
                    e4m3x16_values(k[e], x);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
#pragma unroll
                        for (int r = 0; r < kRows; ++r) z[r] = fmaf(q_s[r][16 * e + i], x[i], z[r]);
                }
            }
            const float f = blk >= 0 ? a.k_scale[bh] * scale2 : 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                z[r] = blk >= 0 && pos < seen[r] ? z[r] * f : -INFINITY;
                float y = z[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, o));
                if (lane == 0) red[warp][r] = y;
            }
            if (a.weights_out && t < a.max_tiles) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) a.z[(t * kGroupedTile + tid) * kRows + r] = z[r];
            }
            __syncthreads();
            const float vs = blk >= 0 ? a.v_scale[bh] : 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float top = fmaxf(fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r])), m[r]);
                const float ref = top == -INFINITY ? 0.0f : top;
                const float old = exp2f(m[r] - ref), p = exp2f(z[r] - ref);
                m[r] = top;
                l[r] = l[r] * old + p;
                acc[r][0] *= old;
                acc[r][1] *= old;
                p_s[r][tid] = p * vs;
            }
            __syncthreads();
            const int valid = min(kGroupedTile, s.len - tile * kGroupedTile);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = tid + c * kThreads;
                if (col >= a.d_v) break;
                for (int j = 0; j < valid; ++j) {
                    const int bj = blk_s[j >> 6];
                    if (bj < 0) continue;
                    const float x = e4m3_to_float(a.v[((static_cast<int64_t>(bj) * a.H_kv + h) * kBlock + (j & 63)) * a.d_v + col]);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) acc[r][c] = fmaf(p_s[r][j], x, acc[r][c]);
                }
            }
        }
        // the item's end: the sums over the block, then the rows or their partial
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float y = l[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
            if (lane == 0) red[warp][r] = y;
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == s.tiles;
        const int slot = grouped_slot(begin, t - (tile1 - tile0), blockIdx.x);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            const float sum = red[0][r] + red[1][r] + red[2][r] + red[3][r];
            const int row = row0 + r;
            const int64_t at = static_cast<int64_t>(s.q0 + row / a.G) * a.H + h * a.G + row % a.G;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = tid + c * kThreads;
                if (col >= a.d_v) break;
                if (whole) store_act(static_cast<T*>(a.out) + at * a.d_v + col, acc[r][c] * inv);
                else a.part_o[(static_cast<int64_t>(slot) * kRows + r) * a.d_v + col] = acc[r][c];
            }
            if (tid == 0) {
                const float lse2 = sum == 0.0f ? -INFINITY : m[r] + log2f(sum);
                if (!whole) a.part_ml[slot * kRows + r] = make_float2(m[r], sum);
                if (whole && a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
                if (whole && a.weights_out) a.row_lse[at] = lse2;
            }
        }
    }
}

}  // namespace gsimt

int grouped_row_tile(const dsa_grouped_dims&, int) { return gsimt::kRows; }
int grouped_ctas(const dsa_grouped_dims&) { return 4 * device_sm_count(); }

bool launch_grouped_attn(const GroupedArgs& a, cudaStream_t s, int* launches) {
    auto* kernel = a.type == DSA_F32 ? gsimt::grouped_attn_kernel<float> : gsimt::grouped_attn_kernel<__nv_bfloat16>;
    if (!launch_kernel(false, kernel, dim3(a.ctas), dim3(gsimt::kThreads), 0, s, a)) return false;
    ++*launches;
    return true;
}

}  // namespace dsa
