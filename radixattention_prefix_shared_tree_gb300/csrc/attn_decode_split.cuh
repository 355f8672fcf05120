// The table pass of attn_decode over bf16 and E4M3 pools (and of attn_cross
// with few queries over them).
#pragma once

#include "attn_decode.cuh"

namespace rc_dec {

// Decode with one warp per item (request b, KV head, key chunk).  Each warp
// streams its keys through a private ring of 16-key tiles (one m16 tile of
// the swapped product) with cp.async, synchronising with __syncwarp only, so
// the warps of an SM overlap each other's load latency and epilogues freely.
constexpr int kWarpKeys = 16;
constexpr int kWarpsPerCta = 14;  // one CTA per SM (14 x 16 KB + the CTA's 1 KB reserve fit; seven CTAs of
constexpr int kCtasPerSm = 1;     // two warps would not): 2128 resident warps, the 2048 (row, KV head) items
                                  // of a 256-row GQA-8 batch in one wave

// Per-warp ring: S stages of one 16-key tile each (K then V, then for an FP8
// pool the tile's 16 K scales and 16 V scales); a stage is refilled as soon
// as its tile is reduced, so S tiles are in flight while the warp waits.
template <bool FP8>
__host__ __device__ constexpr int warp_stages() { return FP8 ? 3 : 2; }
template <int D, bool FP8>
__host__ __device__ constexpr int tile_bytes() { return kWarpKeys * D * (FP8 ? 1 : 2); }
template <int D, bool FP8>
__host__ __device__ constexpr int stage_bytes() { return 2 * tile_bytes<D, FP8>() + (FP8 ? 2 * kWarpKeys * 4 : 0); }
template <int D, bool FP8>
__host__ __device__ constexpr int warp_smem_bytes() {  // the K/V ring only (Q and slot ids in registers)
    return warp_stages<FP8>() * stage_bytes<D, FP8>();
}
template <int D, bool FP8>
__host__ __device__ constexpr int dec_smem_bytes() {
    return kWarpsPerCta * warp_smem_bytes<D, FP8>();
}

template <int D, int G, bool FUSED, bool FP8, bool CROSS = false>
__global__ void __launch_bounds__(32 * kWarpsPerCta, kCtasPerSm) decode_split_kernel(const DecParams p, int n_items) {
    constexpr int ESZ = FP8 ? 1 : 2;                // bytes per K/V element
    constexpr int CH = D * ESZ / 16;                // 16-byte chunks per row
    constexpr int KS = D / 16;
    constexpr int PER = kWarpKeys * CH / 32;        // chunks per lane per matrix
    constexpr int S = warp_stages<FP8>();
    constexpr int TILE_BYTES = tile_bytes<D, FP8>();
    constexpr int STAGE_BYTES = stage_bytes<D, FP8>();
    static_assert(kWarpKeys == 16, "slot ids: one lane per key");
    static_assert(!FP8 || D == 128, "FP8 pools: head_dim 128");
    // the epilogue reuses the ring: [8][D] fp32 outputs plus the merge scratch
    static_assert(warp_smem_bytes<D, FP8>() >= epilogue_bytes<D, G>(), "epilogue scratch");
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g_lane = lane >> 2, t_lane = lane & 3;
    // the next step's cascade kernel (launched as this grid's dependent) may
    // take SMs as they free up: it waits for this grid's end itself
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int it = blockIdx.x * kWarpsPerCta + warp;
    if (it >= n_items) {
        grid_dep_wait();
        return;
    }
    unsigned char* wbase = smem + warp * warp_smem_bytes<D, FP8>();

    const Item w = decode_item<G, FUSED, CROSS>(p, it, lane);
    const int kvh = w.kvh, b = w.b, L = w.L, k0 = w.k0, count = w.count;
    if (CROSS && w.ncol == 0) {
        grid_dep_wait();
        return;
    }
    if (!FUSED && count == 0) {
        grid_dep_wait();
        empty_partial<G, CROSS>(p, w, lane);
        return;
    }
    const int32_t* keys = p.table + w.row0 + k0;
    const int n_tiles = (count + kWarpKeys - 1) / kWarpKeys;
    // fused epilogue: the cascade partials this row folds in; the row offsets
    // of the first 32 (lane j: partial j) are read now, ahead of the main loop
    // (the segment tables are the caller's inputs, not the cascade's output)
    SegParts seg{0, 0};
    if (FUSED && p.req_seg_indptr) {
        seg.e0 = p.req_seg_indptr[b];
        seg.n_parts = (p.req_seg_indptr[b + 1] - seg.e0) * p.seg_chunks;
    }
    const int64_t first_row = seg.row(p, lane);
    // attn_decode_append: the row's last key (position L-1) is the step's new
    // token.  The warp whose keys hold it gathers it from k_new/v_new and
    // writes it to its pool slot (lanes 0..CH-1 the K row, CH..2CH-1 the V row).
    const int new_at = (!FP8 && p.k_new && L > 0 && L - 1 >= k0 && L - 1 < k0 + count) ? L - 1 - k0 : -1;
    if (new_at >= 0) {
        const int slot = keys[new_at];
        if (slot < 0 || (int64_t)slot >= p.n_slots) {
            if (lane == 0) rc::flag_error(p.err, rc::kErrBadSlot);
        } else if (lane < 2 * CH) {
            const int c = lane % CH;
            const int64_t off = ((int64_t)slot * p.kv_heads + kvh) * D + c * 8;
            const int64_t src = ((int64_t)b * p.kv_heads + kvh) * D + c * 8;
            if (lane < CH)
                *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.pool_k) + off) =
                    *reinterpret_cast<const uint4*>(p.k_new + src);
            else
                *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.pool_v) + off) =
                    *reinterpret_cast<const uint4*>(p.v_new + src);
        }
    }

    // Slot ids are prefetched into registers one tile ahead: lane l (and
    // l + 16) holds the slot of key l of a tile.
    auto slot_of = [&](int t) -> int {
        const int key = t * kWarpKeys + (lane & 15);
        return (t < n_tiles && key < count) ? __ldg(keys + key) : 0;
    };
    // a request's own keys are read once per step: they should not push the
    // shared prefix (read by the cascade kernel every step) out of L2
    const uint64_t pol = rc::l2_policy_evict_first();
    auto issue = [&](int t, int tslots) {
        if (t < n_tiles) {
            unsigned char* sK = wbase + (t % S) * STAGE_BYTES;
            unsigned char* sV = sK + TILE_BYTES;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int lin = i * 32 + lane;
                const int r = lin / CH, c = lin % CH;
                const int slot = __shfl_sync(0xffffffffu, tslots, r);
                uint32_t bytes = 16;
                const unsigned char* bk = reinterpret_cast<const unsigned char*>(p.pool_k);
                const unsigned char* bv = reinterpret_cast<const unsigned char*>(p.pool_v);
                int64_t row = 0;
                if (t * kWarpKeys + r >= count) bytes = 0;
                else if (t * kWarpKeys + r == new_at) {  // the appended key, straight from its source
                    bk = reinterpret_cast<const unsigned char*>(p.k_new);
                    bv = reinterpret_cast<const unsigned char*>(p.v_new);
                    row = b;
                } else if (slot < 0 || (int64_t)slot >= p.n_slots) {
                    rc::flag_error(p.err, rc::kErrBadSlot);
                    bytes = 0;
                } else {
                    row = slot;
                }
                const int64_t roff = (row * p.kv_heads + kvh) * (D * ESZ) + c * 16;
                rc::cp_async16(rc::smem_u32(sK + rc::swz<CH>(r, c)), bk + roff, bytes, pol);
                rc::cp_async16(rc::smem_u32(sV + rc::swz<CH>(r, c)), bv + roff, bytes, pol);
            }
            if constexpr (FP8) {  // lanes 0-15: K scale of key lane, 16-31: V scale of key lane-16
                const int r = lane & 15;
                const bool ok = t * kWarpKeys + r < count && tslots >= 0 && (int64_t)tslots < p.n_slots;
                const float* src = (lane < 16 ? p.k_scale : p.v_scale) + (ok ? (int64_t)tslots * p.kv_heads + kvh : 0);
                rc::cp_async4(rc::smem_u32(sV + TILE_BYTES + lane * 4), src, ok ? 4u : 0u);
            }
        }
    };
    // prologue: slot ids of tiles 0 and 1, K/V of tile 0, and the Q operand
    // fragments straight from global memory (head g_lane of this KV head's
    // group, zero for g_lane >= G; two bf16 per register, as ldmatrix would
    // give them)
    // Tiles t..t+S-1 are in flight while the warp waits for tile t; tile
    // t+S goes into tile t's stage as soon as tile t has been reduced.
    int cur = slot_of(S), nxt;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        issue(i, slot_of(i));
        rc::cp_async_commit();
    }
    uint32_t qb[KS][2];
    {
        const bool hv = g_lane < (CROSS ? w.ncol : G);
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.q + w.qrow<G, CROSS>(p, hv ? g_lane : 0) * D);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (FP8) {
                // f16 operands, and k-step ks takes dims 16ks+4t..16ks+4t+3 of
                // this lane's K words (see below): the same dims of Q
                qb[ks][0] = hv ? rc::bf16x2_to_f16x2(__ldg(qrow + ks * 8 + 2 * t_lane)) : 0u;
                qb[ks][1] = hv ? rc::bf16x2_to_f16x2(__ldg(qrow + ks * 8 + 2 * t_lane + 1)) : 0u;
            } else {
                qb[ks][0] = hv ? __ldg(qrow + ks * 8 + t_lane) : 0u;
                qb[ks][1] = hv ? __ldg(qrow + ks * 8 + 4 + t_lane) : 0u;
            }
        }
    }
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    // FP8: O and l are in units of 2^unit_f (rc::scale_unit), until a V scale of
    // unit_limit or more
    float unit_f = rc::kUnitMin, unit_limit = rc::pow2(rc::kUnitMin + 6);

    for (int t = 0; t < n_tiles; ++t) {
        rc::cp_async_wait<S - 1>();  // tile t landed (later tiles may still be in flight)
        __syncwarp();
        nxt = slot_of(t + S + 1);
        const unsigned char* sK = wbase + (t % S) * STAGE_BYTES;
        const unsigned char* sV = sK + TILE_BYTES;
        const float* sSc = reinterpret_cast<const float*>(sV + TILE_BYTES);  // FP8: K scales, then V scales
        // S^T (16 keys x 8 heads) = K Q^T, even and odd k-steps in two
        // accumulators (two independent chains of MMAs)
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        {
            float s2[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (FP8) {
                // A fragment from E4M3 words: row g (and g+8), 16-byte chunk ks,
                // word t_lane = dims 16ks+4t..+3; the k-step's columns 2t, 2t+1
                // take the word's first two dims, 2t+8, 2t+9 the last two
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(sK + rc::swz<CH>(g_lane, ks) + 4 * t_lane);
                    const uint32_t w1 =
                        *reinterpret_cast<const uint32_t*>(sK + rc::swz<CH>(g_lane + 8, ks) + 4 * t_lane);
                    uint32_t a0, a1, a2, a3;
                    rc::e4m3x4_to_f16x4(w0, a0, a2);
                    rc::e4m3x4_to_f16x4(w1, a1, a3);
                    rc::mma_f16_16816(ks & 1 ? s2 : s, a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
                }
            } else {
                const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t a0, a1, a2, a3;
                    rc::ldmatrix_x4(rc::smem_u32(sK + rc::swz<CH>(key, ks * 2 + (lane >> 4))), a0, a1, a2, a3);
                    rc::mma_bf16_16816(ks & 1 ? s2 : s, a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += s2[i];
            if constexpr (FP8) {  // code products times the keys' scales
                const float k_lo = sSc[g_lane], k_hi = sSc[g_lane + 8];
                s[0] *= k_lo;
                s[1] *= k_lo;
                s[2] *= k_hi;
                s[3] *= k_hi;
            }
        }
        const int key_lo = t * kWarpKeys + g_lane;
        const bool v_lo = key_lo < count, v_hi = key_lo + 8 < count;
        s[0] = v_lo ? s[0] * p.scale_log2 : -INFINITY;
        s[1] = v_lo ? s[1] * p.scale_log2 : -INFINITY;
        s[2] = v_hi ? s[2] * p.scale_log2 : -INFINITY;
        s[3] = v_hi ? s[3] * p.scale_log2 : -INFINITY;
        // Online softmax with a lazy reference: exponentials are taken
        // against m_run, which moves (rescaling O and l) only when a head's
        // max grows past it by more than 2^8 -- the terms stay below 2^8, and
        // most tiles skip the 32 multiplies of the rescale.
        float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
        float alpha[2] = {1.f, 1.f};
        bool grow = false;
        float vs_lo = 0.f, vs_hi = 0.f;  // FP8: V scales of keys g and g+8
        if constexpr (FP8) {
            vs_lo = sSc[kWarpKeys + g_lane], vs_hi = sSc[kWarpKeys + g_lane + 8];
            grow = fmaxf(fabsf(vs_lo), fabsf(vs_hi)) >= unit_limit;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
            if (mx[j] > m_run[j] + 8.f) {
                alpha[j] = rc::fast_exp2(m_run[j] - mx[j]);  // 0 while nothing was seen
                m_run[j] = mx[j];
                grow = true;
            }
        }
        // (-0: the one zero whose addition is no instruction)
        const float mu0 = (m_run[0] == -INFINITY ? 0.f : m_run[0]) + (FP8 ? unit_f : -0.f);
        const float mu1 = (m_run[1] == -INFINITY ? 0.f : m_run[1]) + (FP8 ? unit_f : -0.f);
        float p0 = rc::fast_exp2(s[0] - mu0), p1 = rc::fast_exp2(s[1] - mu1);
        float p2 = rc::fast_exp2(s[2] - mu0), p3 = rc::fast_exp2(s[3] - mu1);
        if (__any_sync(0xffffffffu, grow)) {
            l_run[0] *= alpha[0];
            l_run[1] *= alpha[1];
            if constexpr (FP8) {
                const int unit = (int)unit_f, u = rc::scale_unit(__reduce_max_sync(
                                                  0xffffffffu, max(rc::abs_bits(vs_lo), rc::abs_bits(vs_hi))));
                if (u > unit) {
                    for (float* x : {&l_run[0], &l_run[1], &alpha[0], &alpha[1], &p0, &p1, &p2, &p3})
                        *x = rc::to_unit(*x, unit, u);
                    unit_f = (float)u;
                    unit_limit = rc::pow2(u + 6);
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                o[i][0] *= alpha[0];
                o[i][1] *= alpha[1];
                o[i][2] *= alpha[0];
                o[i][3] *= alpha[1];
            }
        }
        l_run[0] += p0 + p2;
        l_run[1] += p1 + p3;
        if constexpr (FP8) {
            // P times the values' scales (f16), then O^T += V^T P^T with V^T
            // built from E4M3 bytes: this lane reads 16-byte chunk g of keys
            // 2t, 2t+1, 2t+8, 2t+9 (dims 16g..16g+15); product mt uses dims
            // 16g+2mt (row g) and 16g+2mt+1 (row g+8), paired across keys
            // with a byte permute
            const uint32_t pb0 = rc::movmatrix_trans(rc::pack_f16(p0 * vs_lo, p1 * vs_lo));
            const uint32_t pb1 = rc::movmatrix_trans(rc::pack_f16(p2 * vs_hi, p3 * vs_hi));
            const uint4 w0 = *reinterpret_cast<const uint4*>(sV + rc::swz<CH>(2 * t_lane, g_lane));
            const uint4 w1 = *reinterpret_cast<const uint4*>(sV + rc::swz<CH>(2 * t_lane + 1, g_lane));
            const uint4 w8 = *reinterpret_cast<const uint4*>(sV + rc::swz<CH>(2 * t_lane + 8, g_lane));
            const uint4 w9 = *reinterpret_cast<const uint4*>(sV + rc::swz<CH>(2 * t_lane + 9, g_lane));
            const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
            const uint32_t x8[4] = {w8.x, w8.y, w8.z, w8.w}, x9[4] = {w9.x, w9.y, w9.z, w9.w};
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                rc::e4m3x4_to_f16x4(rc::prmt(x0[mt >> 1], x1[mt >> 1], sel), a0, a1);
                rc::e4m3x4_to_f16x4(rc::prmt(x8[mt >> 1], x9[mt >> 1], sel), a2, a3);
                rc::mma_f16_16816(o[mt], a0, a1, a2, a3, pb0, pb1);
            }
        } else {
            // P to bf16, V's type (one product takes one type); the denominator
            // keeps the fp32 terms
            const uint32_t pb0 = rc::movmatrix_trans(rc::pack_bf16(p0, p1));
            const uint32_t pb1 = rc::movmatrix_trans(rc::pack_bf16(p2, p3));
            const int key = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                uint32_t a0, a1, a2, a3;
                rc::ldmatrix_x4_trans(rc::smem_u32(sV + rc::swz<CH>(key, mt * 2 + ((lane >> 3) & 1))), a0, a1, a2,
                                      a3);
                rc::mma_bf16_16816(o[mt], a0, a1, a2, a3, pb0, pb1);
            }
        }
        __syncwarp();  // every lane has read tile t: its stage takes tile t+S
        issue(t + S, cur);
        rc::cp_async_commit();
        cur = nxt;
    }
    rc::cp_async_wait<0>();
    __syncwarp();

    // ---------------------------------------------------------- epilogue
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 4);
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 8);
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 16);
    }
    // this warp's normalised output per (head, dim) into its (now free) ring
    float* sE = reinterpret_cast<float*>(wbase);           // [8][D]
    float* sOwn = sE + 8 * D;                               // [8] log2-sum-exp per head
    const float inv0 = l_run[0] > 0.f ? 1.f / l_run[0] : 0.f;
    const float inv1 = l_run[1] > 0.f ? 1.f / l_run[1] : 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
        // accumulator rows g and g+8 of product mt: dims d0 and d1
        const int d0 = FP8 ? 16 * g_lane + 2 * mt : mt * 16 + g_lane;
        const int d1 = FP8 ? d0 + 1 : d0 + 8;
        sE[(2 * t_lane) * D + d0] = o[mt][0] * inv0;
        sE[(2 * t_lane + 1) * D + d0] = o[mt][1] * inv1;
        sE[(2 * t_lane) * D + d1] = o[mt][2] * inv0;
        sE[(2 * t_lane + 1) * D + d1] = o[mt][3] * inv1;
    }
    if (g_lane == 0) {
        if constexpr (FP8) m_run[0] += unit_f, m_run[1] += unit_f;
        sOwn[2 * t_lane] = rc::log2_sum(m_run[0], l_run[0]);
        sOwn[2 * t_lane + 1] = rc::log2_sum(m_run[1], l_run[1]);
    }
    __syncwarp();
    decode_epilogue<D, G, FUSED, CROSS>(p, w, sE, sOwn, seg, first_row, lane);
}

}  // namespace rc_dec
