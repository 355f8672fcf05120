// Joins the partials of a pass that split every row's keys over n_chunks CTAs or
// warps (attn_cross, attn_extend): for each token and head,
//   out = sum_c 2^(lse_c - m) o_c / sum_c 2^(lse_c - m),  m = max_c lse_c,
// with o_c normalised and lse_c in log2 units (-infinity: a chunk without keys,
// whose o_c is not written).
#pragma once

#include "attn_decode.cuh"

#include <type_traits>

namespace rc_dec {

struct SplitMerge {
    const float* part_o;    // [tokens][q_heads][n_chunks][D]
    const float* part_lse;  // [tokens][q_heads][n_chunks]
    int32_t n_chunks;
    const int32_t* qo_indptr;
    int32_t max_q;          // row b's tokens: blockIdx.x = b * max_q + token
    int64_t max_rows;
    int32_t q_heads;
    __nv_bfloat16* out;
    float* lse;
    const int32_t* err;
};

constexpr int kSplitMergeWarps = 8;

// W warps per (token, head), each taking every W-th chunk; blockIdx.y is a group
// of kSplitMergeWarps / W heads.  Bound by latency: a row's first eight chunks
// are read while their log-sum-exps are on their way.
template <int D, int W>
__global__ void __launch_bounds__(32 * kSplitMergeWarps) split_merge_kernel(const SplitMerge p) {
    constexpr int V = D / 32, R = 8, HEADS = kSplitMergeWarps / W;
    using Vec = typename std::conditional<V == 4, float4, float2>::type;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, slot = (threadIdx.x >> 5) / W;
    const int b = blockIdx.x / p.max_q, token = blockIdx.x % p.max_q, h = blockIdx.y * HEADS + slot;
    const int qo0 = p.qo_indptr[b], nq = p.qo_indptr[b + 1] - qo0;
    grid_dep_wait();
    // a row that the pass refused has no partials, nor any after one that gave
    // up on a bounded wait
    if (nq > p.max_q || qo0 < 0 || (int64_t)qo0 + nq > p.max_rows || token >= nq) return;
    if (p.err && (*reinterpret_cast<const volatile int32_t*>(p.err) & rc::kErrTimeout)) return;
    const bool live = h < p.q_heads;
    const int64_t row = (int64_t)(qo0 + token) * p.q_heads + (live ? h : 0);
    const float* pl = p.part_lse + row * p.n_chunks;
    const Vec* po = reinterpret_cast<const Vec*>(p.part_o + row * p.n_chunks * D) + lane;
    float m = -INFINITY, wsum = 0.f, acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    const int n = live ? p.n_chunks : 0;
    for (int c0 = warp; c0 < n; c0 += R * W) {
        float l2[R];
        Vec v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = c0 + i * W;
            l2[i] = c < n ? pl[c] : -INFINITY;
            if (c < n) v[i] = po[(int64_t)c * 32];
        }
        float mb = m;
#pragma unroll
        for (int i = 0; i < R; ++i) mb = fmaxf(mb, l2[i]);
        if (mb == -INFINITY) continue;
        const float a = m == -INFINITY ? 0.f : rc::fast_exp2(m - mb);
        wsum *= a;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= a;
        m = mb;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float wi = l2[i] == -INFINITY ? 0.f : rc::fast_exp2(l2[i] - m);
            if (wi == 0.f) continue;
            wsum += wi;
            const float* x = reinterpret_cast<const float*>(&v[i]);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += wi * x[k];
        }
    }
    if constexpr (W > 1) {  // the warps' sums, joined in their order
        __shared__ float sM[kSplitMergeWarps], sW[kSplitMergeWarps];
        __shared__ __align__(16) float sA[kSplitMergeWarps][D];
        const int me = slot * W + warp;
        if (lane == 0) {
            sM[me] = m;
            sW[me] = wsum;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sA[me][lane * V + k] = acc[k];
        __syncthreads();
        if (warp != 0) return;
        m = -INFINITY;
        wsum = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) m = fmaxf(m, sM[me + i]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float e = sM[me + i] == -INFINITY ? 0.f : rc::fast_exp2(sM[me + i] - m);
            if (e == 0.f) continue;
            wsum += e * sW[me + i];
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += e * sA[me + i][lane * V + k];
        }
    }
    if (!live) return;
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + row * D) + lane * (V / 2);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) out[k] = rc::pack_bf16(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    if (p.lse && lane == 0) p.lse[row] = rc::log2_sum(m, wsum) * rc::kLn2;
}

// As the pass's programmatic dependent: its blocks start as that pass's leave
// and wait for its end inside.  Rows in many chunks get eight warps a head (200
// tokens of 16 heads in 9 chunks: 31 us with eight, 27 with one).
template <int D>
cudaError_t launch_split_merge(const SplitMerge& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * kSplitMergeWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int w = p.n_chunks <= 16 ? 1 : 8;
    const int heads = kSplitMergeWarps / w;
    cfg.gridDim = dim3((unsigned)p.max_rows, (p.q_heads + heads - 1) / heads);
    return w == 1 ? cudaLaunchKernelEx(&cfg, split_merge_kernel<D, 1>, p)
                  : cudaLaunchKernelEx(&cfg, split_merge_kernel<D, 8>, p);
}

}  // namespace rc_dec
