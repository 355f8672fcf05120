// The table pass of attn_decode over a 4-bit pool (and of attn_cross with few
// queries over one): E2M1 codes with a scale byte per 16 of them.
//
//   out[c] = sum_j softmax_j(scale q[c].K[j]) V[j],   K[j], V[j] = code * scale
//
// One warp per item (request, KV head, key chunk) with a private ring of
// 32-key tiles in shared memory, filled by cp.async.  A key's row is 72 bytes
// at D = 128 (64 of codes, 8 of scales) against 256 in bf16, so at HBM speed a
// tile lasts half as many cycles per key as the bf16 pass has, and the pass is
// bound by instruction issue as much as by HBM.  What that decides:
//  * code times scale is exactly an f16 value, so both products run on f16
//    mma.sync with the values themselves and the softmax sees no scales;
//  * the order of the head's dims inside the products is free as long as both
//    operands agree: lane t of a group takes D/4 consecutive dims of K (one
//    16-byte load per key), lane group g D/8 consecutive dims of V (one 8-byte
//    load per key), so a lane's codes share one or two block scales;
//  * V's operand pairs two keys per register: the nibbles of two keys are
//    interleaved before they are widened (half a logic instruction per pair
//    instead of a byte permute each);
//  * 32 keys per tile share one round of max shuffles and one rescale test.
#pragma once

#include "attn_decode.cuh"
#include "tc.cuh"

namespace rc_dec {

namespace fp4 {

constexpr int kKeys = 32;          // keys per tile: a lane's slot id each
constexpr int kWarps = 16;         // per CTA
constexpr int kStages = 3;

template <int D>
__host__ __device__ constexpr int code_bytes() { return D / 2; }
template <int D>
__host__ __device__ constexpr int scale_bytes() { return D / 16; }
template <int D>
__host__ __device__ constexpr int stage_bytes() { return 2 * kKeys * (code_bytes<D>() + scale_bytes<D>()); }
template <int D>
__host__ __device__ constexpr int warp_bytes() { return kStages * stage_bytes<D>(); }
template <int D>
__host__ __device__ constexpr int smem_bytes() { return kWarps * warp_bytes<D>(); }

// 4- or 8-byte asynchronous copy (block scales); src_bytes = 0 writes zeros.
template <int N>
RC_DEV void cp_async_small(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes), "n"(N)
                 : "memory");
}

// Shared-memory row of V's key m (0..31): inside each 16 keys the even ones
// come first, so that the four key pairs that lanes read together lie in
// neighbouring rows.
RC_DEV int v_row(int m) { return (m & 16) | ((m & 14) >> 1) | ((m & 1) << 3); }
// D = 128: 16-byte chunk c of V's row r sits at chunk c ^ v_swz(r); with it an
// 8-byte read of four rows' neighbouring halves touches every bank once.
template <int D>
RC_DEV int v_swz(int r) { return D == 128 ? (r & 2) : 0; }

}  // namespace fp4

template <int D, int NC, bool FUSED, bool CROSS>
__global__ void __launch_bounds__(32 * fp4::kWarps, 1) decode_fp4_kernel(const DecParams p, int n_items) {
    using namespace fp4;
    static_assert(D == 128 || D == 64, "head_dim");
    constexpr int KS = D / 16;                 // k-steps of S, m-tiles of O
    constexpr int CB = code_bytes<D>(), SB = scale_bytes<D>();
    constexpr int CPR = CB / 16;               // 16-byte chunks per row
    constexpr int RPI = 32 / CPR;              // rows one instruction copies
    constexpr int STAGE = stage_bytes<D>();
    static_assert(warp_bytes<D>() >= epilogue_bytes<D, NC>(), "epilogue scratch");
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g_lane = lane >> 2, t_lane = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int it = blockIdx.x * kWarps + warp;
    if (it >= n_items) {
        grid_dep_wait();
        return;
    }
    unsigned char* wbase = smem + warp * warp_bytes<D>();
    const Item w = decode_item<NC, FUSED, CROSS>(p, it, lane);
    if (CROSS && w.ncol == 0) {
        grid_dep_wait();
        return;
    }
    if (!FUSED && w.count == 0) {
        grid_dep_wait();
        empty_partial<CROSS>(p, w, lane);
        return;
    }
    const int count = w.count;
    const int32_t* keys = p.table + w.row0 + w.k0;
    const int n_tiles = (count + kKeys - 1) / kKeys;
    SegParts seg{0, 0};
    if (FUSED && !CROSS && p.req_seg_indptr) {
        seg.e0 = p.req_seg_indptr[w.b];
        seg.n_parts = (p.req_seg_indptr[w.b + 1] - seg.e0) * p.seg_chunks;
    }
    const int64_t first_row = seg.row(p, lane);

    // Lane l holds the slot id of key l of a tile: -1 past the end and for an
    // id outside the pool (flagged), whose row then reads as zeros.
    auto slot_of = [&](int t) -> int {
        const int key = t * kKeys + lane;
        if (key >= count) return -1;
        const int s = __ldg(keys + key);
        if (s < 0 || (int64_t)s >= p.n_slots) {
            rc::flag_error(p.err, rc::kErrBadSlot);
            return -1;
        }
        return s;
    };
    const uint64_t pol = rc::l2_policy_evict_first();  // a request's own keys are read once per step
    const unsigned char* kc = reinterpret_cast<const unsigned char*>(p.pool_k) + (int64_t)w.kvh * CB + (lane % CPR) * 16;
    const unsigned char* vc = reinterpret_cast<const unsigned char*>(p.pool_v) + (int64_t)w.kvh * CB + (lane % CPR) * 16;
    const int64_t row_stride = (int64_t)p.kv_heads * CB;
    const uint32_t sbase = rc::smem_u32(wbase);
    auto issue = [&](int t, int slot) {
        if (t < n_tiles) {
            const uint32_t st = sbase + (t % kStages) * STAGE;
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
                const int r = i * RPI + lane / CPR;
                const int s = __shfl_sync(0xffffffffu, slot, r);
                const int64_t off = (int64_t)(s < 0 ? 0 : s) * row_stride;
                const uint32_t bytes = s < 0 ? 0u : 16u;
                const int vr = v_row(r);
                rc::cp_async16(st + r * CB + (lane % CPR) * 16, kc + off, bytes, pol);
                rc::cp_async16(st + kKeys * CB + vr * CB + ((lane % CPR) ^ v_swz<D>(vr)) * 16, vc + off, bytes, pol);
            }
            const int64_t soff = ((int64_t)(slot < 0 ? 0 : slot) * p.kv_heads + w.kvh) * SB;
            const uint32_t sb = slot < 0 ? 0u : (uint32_t)SB;
            cp_async_small<SB>(st + 2 * kKeys * CB + lane * SB, p.k_bscale + soff, sb);
            cp_async_small<SB>(st + 2 * kKeys * CB + kKeys * SB + lane * SB, p.v_bscale + soff, sb);
        }
    };
    int cur = slot_of(kStages), nxt;
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
        issue(i, slot_of(i));
        rc::cp_async_commit();
    }
    // Q operand (f16): k-step ks of lane t covers dims t D/4 + 4 ks .. + 3
    uint32_t qb[KS][2];
    {
        const bool hv = g_lane < w.ncol;
        const uint4* qrow = reinterpret_cast<const uint4*>(p.q + w.qrow<CROSS>(hv ? g_lane : 0) * D + t_lane * (D / 4));
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            const uint4 x = hv ? __ldg(qrow + j) : make_uint4(0, 0, 0, 0);
            qb[2 * j][0] = rc::bf16x2_to_f16x2(x.x);
            qb[2 * j][1] = rc::bf16x2_to_f16x2(x.y);
            qb[2 * j + 1][0] = rc::bf16x2_to_f16x2(x.z);
            qb[2 * j + 1][1] = rc::bf16x2_to_f16x2(x.w);
        }
    }
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

    for (int t = 0; t < n_tiles; ++t) {
        rc::cp_async_wait<kStages - 1>();
        __syncwarp();
        nxt = slot_of(t + kStages + 1);
        const unsigned char* sK = wbase + (t % kStages) * STAGE;
        const unsigned char* sV = sK + kKeys * CB;
        const unsigned char* sKs = sV + kKeys * CB;
        const unsigned char* sVs = sKs + kKeys * SB;
        float s[2][4];  // [16 keys][key g head 2t, head 2t+1; key g+8 ...]
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r0 = half * 16 + g_lane, r1 = r0 + 8;
            uint32_t x0[KS / 2], x1[KS / 2], s0[2], s1[2];
            if constexpr (D == 128) {
                const uint4 a = *reinterpret_cast<const uint4*>(sK + r0 * CB + t_lane * 16);
                const uint4 b = *reinterpret_cast<const uint4*>(sK + r1 * CB + t_lane * 16);
                x0[0] = a.x, x0[1] = a.y, x0[2] = a.z, x0[3] = a.w;
                x1[0] = b.x, x1[1] = b.y, x1[2] = b.z, x1[3] = b.w;
                const uint32_t u0 = *reinterpret_cast<const uint16_t*>(sKs + r0 * SB + 2 * t_lane);
                const uint32_t u1 = *reinterpret_cast<const uint16_t*>(sKs + r1 * SB + 2 * t_lane);
                s0[0] = rc::scale_pair<0, 0>(u0), s0[1] = rc::scale_pair<1, 1>(u0);
                s1[0] = rc::scale_pair<0, 0>(u1), s1[1] = rc::scale_pair<1, 1>(u1);
            } else {
                const uint2 a = *reinterpret_cast<const uint2*>(sK + r0 * CB + t_lane * 8);
                const uint2 b = *reinterpret_cast<const uint2*>(sK + r1 * CB + t_lane * 8);
                x0[0] = a.x, x0[1] = a.y;
                x1[0] = b.x, x1[1] = b.y;
                s0[0] = s0[1] = rc::scale_pair<0, 0>(sKs[r0 * SB + t_lane]);
                s1[0] = s1[1] = rc::scale_pair<0, 0>(sKs[r1 * SB + t_lane]);
            }
            float e[4] = {0.f, 0.f, 0.f, 0.f}, f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {  // a word: two k-steps
                const int sc = j / (KS / 4);
                uint32_t a0, a2, c0, c2, a1, a3, c1, c3;
                rc::e2m1x8_to_f16x8(x0[j], a0, a2, c0, c2);
                rc::e2m1x8_to_f16x8(x1[j], a1, a3, c1, c3);
                rc::mma_f16_16816(e, rc::mul_f16x2(a0, s0[sc]), rc::mul_f16x2(a1, s1[sc]), rc::mul_f16x2(a2, s0[sc]),
                                  rc::mul_f16x2(a3, s1[sc]), qb[2 * j][0], qb[2 * j][1]);
                rc::mma_f16_16816(f, rc::mul_f16x2(c0, s0[sc]), rc::mul_f16x2(c1, s1[sc]), rc::mul_f16x2(c2, s0[sc]),
                                  rc::mul_f16x2(c3, s1[sc]), qb[2 * j + 1][0], qb[2 * j + 1][1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[half][i] = (e[i] + f[i]) * p.scale_log2;
        }
        if (t == n_tiles - 1) {  // keys past the end (their codes are zeros)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int k = t * kKeys + half * 16 + g_lane;
                if (k >= count) s[half][0] = s[half][1] = -INFINITY;
                if (k + 8 >= count) s[half][2] = s[half][3] = -INFINITY;
            }
        }
        // Online softmax with a lazy reference, as in the bf16 table pass: it
        // moves only when a column's max grows past it by more than 2^8.
        float alpha[2] = {1.f, 1.f};
        bool grow = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(fmaxf(s[0][j], s[0][j + 2]), fmaxf(s[1][j], s[1][j + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (mx > m_run[j] + 8.f) {
                alpha[j] = tc::ex2(m_run[j] - mx);  // 0 while nothing was seen
                m_run[j] = mx;
                grow = true;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
            l_run[0] *= alpha[0];
            l_run[1] *= alpha[1];
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                o[i][0] *= alpha[0];
                o[i][1] *= alpha[1];
                o[i][2] *= alpha[0];
                o[i][3] *= alpha[1];
            }
        }
        const float mu0 = m_run[0] == -INFINITY ? 0.f : m_run[0];
        const float mu1 = m_run[1] == -INFINITY ? 0.f : m_run[1];
        uint32_t pb[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float p0 = tc::ex2(s[half][0] - mu0), p1 = tc::ex2(s[half][1] - mu1);
            const float p2 = tc::ex2(s[half][2] - mu0), p3 = tc::ex2(s[half][3] - mu1);
            l_run[0] += p0 + p2;
            l_run[1] += p1 + p3;
            // P to f16 (11 bits, at most 2^8): the denominator keeps the fp32 terms
            pb[half][0] = rc::movmatrix_trans(rc::pack_f16(p0, p1));
            pb[half][1] = rc::movmatrix_trans(rc::pack_f16(p2, p3));
        }
        // O^T += V^T P^T: lane group g holds dims g D/8 .. of keys 2t, 2t+1,
        // 2t+8, 2t+9; product mt takes dims g D/8 + 2 mt (row g) and + 1
        // (row g + 8): the two nibbles of byte mt
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t x[4][KS / 4], sc[2];
            uint32_t sb[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int m = half * 16 + 2 * t_lane + (k & 1) + (k >> 1) * 8;
                const int r = v_row(m);
                if constexpr (D == 128) {
                    const uint2 v = *reinterpret_cast<const uint2*>(sV + r * CB + (((g_lane >> 1) ^ v_swz<D>(r)) * 16) +
                                                                    (g_lane & 1) * 8);
                    x[k][0] = v.x, x[k][1] = v.y;
                    sb[k] = sVs[m * SB + g_lane];
                } else {
                    x[k][0] = *reinterpret_cast<const uint32_t*>(sV + r * CB + g_lane * 4);
                    sb[k] = sVs[m * SB + (g_lane >> 1)];
                }
            }
            sc[0] = (sb[0] | (sb[1] << 16)) << 7;
            sc[1] = (sb[2] | (sb[3] << 16)) << 7;
#pragma unroll
            for (int j = 0; j < KS / 4; ++j) {
                uint32_t a[2][2][4];  // [key pair][dim parity][byte]
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t u = x[2 * k][j], v = x[2 * k + 1][j];
                    const uint32_t lo = (u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u);
                    const uint32_t hi = ((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u);
                    rc::e2m1x8_to_f16x8(lo, a[k][0][0], a[k][0][1], a[k][0][2], a[k][0][3]);
                    rc::e2m1x8_to_f16x8(hi, a[k][1][0], a[k][1][1], a[k][1][2], a[k][1][3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rc::mma_f16_16816(o[4 * j + i], rc::mul_f16x2(a[0][0][i], sc[0]), rc::mul_f16x2(a[0][1][i], sc[0]),
                                      rc::mul_f16x2(a[1][0][i], sc[1]), rc::mul_f16x2(a[1][1][i], sc[1]), pb[half][0],
                                      pb[half][1]);
            }
        }
        __syncwarp();  // every lane has read tile t: its stage takes tile t + kStages
        issue(t + kStages, cur);
        rc::cp_async_commit();
        cur = nxt;
    }
    rc::cp_async_wait<0>();
    __syncwarp();

#pragma unroll
    for (int j = 0; j < 2; ++j) {
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 4);
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 8);
        l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], 16);
    }
    float* sE = reinterpret_cast<float*>(wbase);
    float* sOwn = sE + 8 * D;
    const float inv0 = l_run[0] > 0.f ? 1.f / l_run[0] : 0.f;
    const float inv1 = l_run[1] > 0.f ? 1.f / l_run[1] : 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
        const int d0 = g_lane * (D / 8) + 2 * mt;
        *reinterpret_cast<float2*>(sE + (2 * t_lane) * D + d0) = make_float2(o[mt][0] * inv0, o[mt][2] * inv0);
        *reinterpret_cast<float2*>(sE + (2 * t_lane + 1) * D + d0) = make_float2(o[mt][1] * inv1, o[mt][3] * inv1);
    }
    // a NaN sum (a key whose block holds NaN) weighs as +infinity, so that the
    // merge turns the row into NaN instead of skipping the partial
    auto lse2 = [](float m, float l) { return l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : INFINITY; };
    if (g_lane == 0) {
        sOwn[2 * t_lane] = lse2(m_run[0], l_run[0]);
        sOwn[2 * t_lane + 1] = lse2(m_run[1], l_run[1]);
    }
    __syncwarp();
    decode_epilogue<D, NC, FUSED, CROSS>(p, w, sE, sOwn, seg, first_row, lane);
}

}  // namespace rc_dec
