// The table pass of attn_decode over a 4-bit pool (and of attn_cross with few
// queries over one): E2M1 codes with a scale byte per 16 of them.
//
//   out[c] = sum_j softmax_j(scale q[c].K[j]) V[j],   K[j], V[j] = code * scale
//
// A warp works on one KV head and a stretch of 32-key tiles: whole rows (FUSED),
// or an equal run of all rows' tiles laid end to end, whose parts
// merge_runs_kernel joins.  The tiles come by cp.async into a two-stage ring,
// four neighbouring heads' together where there are that many (COOP).  A key's
// row is 72 bytes at D = 128 (64 of codes, 8 of scales) against 256 in bf16, so
// HBM gives a tile fewer cycles than its instructions take: at 256 rows of
// 512-5119 keys, 8 KV heads, the pass takes 160 us and the merge behind it 6, the
// pass's loads alone 131 and its arithmetic alone 132; 123 would be HBM's copy
// rate.  What that decides:
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
// Measured and left out at that size (against 166 us with the merge): a third
// stage 169, eight warps a CTA 179, five or six CTAs per SM 211 and 251
// (registers spill).
#pragma once

#include "attn_decode.cuh"
#include "tc.cuh"

#include <type_traits>

namespace rc_dec {

namespace fp4 {

constexpr int kKeys = 32;          // keys per tile: a lane's slot id each
constexpr int kWarps = 4;          // per CTA
constexpr int kCtasPerSm = 4;      // 16 warps' rings and registers fill an SM
constexpr int kStages = 2;

template <int D>
__host__ __device__ constexpr int code_bytes() { return D / 2; }
template <int D>
__host__ __device__ constexpr int scale_bytes() { return D / 16; }
template <int D>
__host__ __device__ constexpr int stage_bytes() { return 2 * kKeys * (code_bytes<D>() + scale_bytes<D>()); }
// One head's part of a stage that the CTA's warps fill together: padded so that
// neighbouring heads' copies land in different banks.
template <int D>
__host__ __device__ constexpr int head_bytes() { return stage_bytes<D>() + code_bytes<D>(); }
template <int D, bool COOP>
__host__ __device__ constexpr int warp_bytes() { return kStages * (COOP ? head_bytes<D>() : stage_bytes<D>()); }
template <int D, bool COOP>
__host__ __device__ constexpr int smem_bytes() { return kWarps * warp_bytes<D, COOP>(); }

// How the split pass divides a batch: all rows' keys, 32 to a tile, laid end to
// end and cut into equal runs of tiles, one run per group of kv_heads warps (a
// warp per KV head).  Every warp then has the same work whatever the rows'
// lengths, and a row has one partial per run that touches it.  Run g's part of
// row b goes to partial slot g + b: runs and rows both only move forward, so
// no two parts share a sum, and a row's slots are consecutive.
// At most as many runs as fit the SMs at once, of at least kMinTiles tiles.
constexpr int kMinTiles = 2;
inline int groups(int64_t batch, int64_t kv_heads, int64_t max_len, int64_t sms) {
    const int64_t resident = (int64_t)kWarps * kCtasPerSm * sms / kv_heads;
    const int64_t tiles = batch * ((max_len + kKeys - 1) / kKeys);
    const int64_t most = (tiles + kMinTiles - 1) / kMinTiles;
    const int64_t g = resident < most ? resident : most;
    return (int)(g < 1 ? 1 : g);
}
// The runs of a batch of so many tiles, given the most there may be.
RC_DEV int64_t runs_of(int64_t tiles, int most) {
    const int64_t r = (tiles + kMinTiles - 1) / kMinTiles;
    return r < most ? r : most;
}
// One warp per (row, KV head) and no merge: rows of three tiles at most (their
// merge would take longer: 4 rows of 96 keys 9.8 us in runs), or short ones
// and enough of them that a warp each fills most of the SMs.
inline bool whole_rows(int64_t batch, int64_t kv_heads, int64_t max_len, int64_t sms) {
    return max_len <= 3 * kKeys ||
           (2 * batch * kv_heads >= (int64_t)kWarps * kCtasPerSm * sms && max_len <= 512);
}

// Shared-memory row of V's key m (0..31): inside each 16 keys the even ones
// come first, so that the four key pairs that lanes read together lie in
// neighbouring rows.
RC_DEV int v_row(int m) { return (m & 16) | ((m & 14) >> 1) | ((m & 1) << 3); }
// D = 128: 16-byte chunk c of V's row r sits at chunk c ^ v_swz(r); with it an
// 8-byte read of four rows' neighbouring halves touches every bank once.
template <int D>
RC_DEV int v_swz(int r) { return D == 128 ? (r & 2) : 0; }

constexpr int kMergeWarps = 8;

}  // namespace fp4

// FUSED: one item per warp, result written (and the row's cascade partials
// folded in) by its epilogue.  Otherwise the equal runs described above.
//
// COOP (kv_heads a multiple of 4): a CTA's four warps are four neighbouring
// heads of the same keys and fill their ring together, a key's four code rows
// as one 256-byte read and its four scale blocks as one 32-byte read (D = 128).
// Apart, every warp reads 64 and 8 bytes of them, and the number of requests,
// not their bytes, bounds the loads: at 256 rows of 512-5119 keys the loads
// alone took 152 us against 123 without the scales' eight-byte reads.  Other
// head counts keep a ring per warp.  A call over those rows: 8 KV heads 169 us
// together, 315 apart, 4 heads 94 and 124; 3 heads, apart, 99 us, 2 heads 56, one
// head 45 (floors 46, 31 and 15).
template <int D, int NC, bool FUSED, bool CROSS, bool COOP>
__global__ void __launch_bounds__(32 * fp4::kWarps, fp4::kCtasPerSm) decode_fp4_kernel(const DecParams p, int n_items) {
    using namespace fp4;
    static_assert(D == 128 || D == 64, "head_dim");
    constexpr int KS = D / 16;                 // k-steps of S, m-tiles of O
    constexpr int CB = code_bytes<D>(), SB = scale_bytes<D>();
    constexpr int CPR = CB / 16;               // 16-byte chunks per row
    constexpr int RPI = 32 / CPR;              // rows one instruction copies
    constexpr int HS = head_bytes<D>();
    constexpr int STAGE = COOP ? kWarps * HS : stage_bytes<D>();  // bytes from a warp's stage to its next
    constexpr int AHEAD = COOP ? kStages - 1 : kStages;           // tiles in flight at a tile's start
    static_assert(warp_bytes<D, COOP>() >= epilogue_bytes<D, NC>(), "epilogue scratch");
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g_lane = lane >> 2, t_lane = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int it = blockIdx.x * kWarps + warp;
    if (it >= n_items) {
        grid_dep_wait();
        return;
    }
    // this warp's first stage, and (once all warps are done with theirs) its scratch
    unsigned char* wbase = smem + warp * (COOP ? HS : warp_bytes<D, COOP>());
    unsigned char* scratch = smem + warp * warp_bytes<D, COOP>();
    Item w;
    SegParts seg{0, 0};
    int64_t first_row = 0;
    // !FUSED: this warp's run of tiles [run, run_end), the row it stands in
    // and the first tile of that row
    int64_t run = 0, run_end = 1, row_tile = 0;
    int group = 0, row_tiles = 0;
    bool waited = false;
    if constexpr (FUSED) {
        w = decode_item<NC, FUSED, CROSS>(p, it, lane);
        if (CROSS && w.ncol == 0) {
            grid_dep_wait();
            return;
        }
        if (!CROSS && p.req_seg_indptr) {
            seg.e0 = p.req_seg_indptr[w.b];
            seg.n_parts = (p.req_seg_indptr[w.b + 1] - seg.e0) * p.seg_chunks;
        }
        first_row = seg.row(p, lane);
    } else {
        w.kvh = it % p.kv_heads;
        group = it / p.kv_heads;
        int64_t tiles = 0;  // of the whole batch
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            RowKeys r = row_keys<CROSS>(p, b0 + lane);
            if (r.bad && it == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            tiles += (r.L + kKeys - 1) / kKeys;
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, k);
        const int64_t runs = runs_of(tiles, p.n_chunks);
        if (group >= runs) {
            grid_dep_wait();
            return;
        }
        run = group * tiles / runs;
        run_end = (group + 1) * tiles / runs;
        w.b = -1;
        for (int b0 = 0; w.b < 0 && b0 < p.batch; b0 += 32) {  // the row that holds tile `run`
            const int n = (row_keys<CROSS>(p, b0 + lane).L + kKeys - 1) / kKeys;
            int64_t incl = n;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, k);
                if (lane >= k) incl += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, run < row_tile + incl);
            if (m) {
                const int src = __ffs(m) - 1;
                w.b = b0 + src;
                row_tile += __shfl_sync(0xffffffffu, incl - n, src);
            } else {
                row_tile += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
    }
    const float sc = fmaxf(fabsf(p.scale_log2), 1e-30f);
    const uint64_t pol = rc::l2_policy_evict_first();  // a request's own keys are read once per step
    const uint32_t row_codes = (uint32_t)p.kv_heads * CB, row_scales = (uint32_t)p.kv_heads * SB;
    const uint32_t n_slots = (uint32_t)min(p.n_slots, (int64_t)0x7fffffff);  // at least 1 (checked by the host)
    // Code copy i of this thread is chunk c of key i * RPI + r: of this warp's
    // head, or (COOP) of the CTA's head c / CPR.  Its place moves by a constant
    // with i: RPI rows of K, and the same rows' places in V.  Scale copies: key
    // `sr`, head offset `sh`.
    const int r = COOP ? threadIdx.x / (kWarps * CPR) : lane / CPR;
    const int c = COOP ? threadIdx.x % (kWarps * CPR) : lane % CPR;
    const int sr = COOP ? threadIdx.x / kWarps : lane, sh = COOP ? threadIdx.x % kWarps : 0;
    const int kvh0 = COOP ? w.kvh - warp : w.kvh;
    const unsigned char* kc = reinterpret_cast<const unsigned char*>(p.pool_k) + (int64_t)kvh0 * CB + c * 16;
    const unsigned char* vc = reinterpret_cast<const unsigned char*>(p.pool_v) + (int64_t)kvh0 * CB + c * 16;
    const uint8_t* ksc = p.k_bscale + (int64_t)(kvh0 + sh) * SB;
    const uint8_t* vsc = p.v_bscale + (int64_t)(kvh0 + sh) * SB;
    const uint32_t ring = rc::smem_u32(COOP ? smem : wbase);
    const int vr0 = v_row(r);
    const uint32_t kdst = ring + (c / CPR) * HS + r * CB + (c % CPR) * 16;
    const uint32_t vdst = ring + (c / CPR) * HS + kKeys * CB + vr0 * CB + ((c % CPR) ^ v_swz<D>(vr0)) * 16;
    const uint32_t sdst = ring + sh * HS + 2 * kKeys * CB + sr * SB;

    while (run < run_end && (FUSED || (w.b >= 0 && w.b < p.batch))) {
    if constexpr (FUSED) {
        run = run_end;
    } else {  // the part of row w.b that lies in the run
        const RowKeys rk = row_keys<CROSS>(p, w.b);
        row_tiles = (rk.L + kKeys - 1) / kKeys;
        const int64_t lo = run - row_tile;
        if (lo >= row_tiles) {  // the run goes on in the next row
            row_tile += row_tiles;
            ++w.b;
            continue;
        }
        const int64_t n = min((int64_t)row_tiles - lo, run_end - run);
        w.row0 = rk.row0;
        w.ncol = CROSS ? rk.ncol : NC;
        w.qrow0 = CROSS ? (int64_t)rk.qo0 * p.q_heads + w.kvh * p.group : 0;
        w.k0 = (int)lo * kKeys;
        w.count = (int)min((int64_t)rk.L - w.k0, n * kKeys);
        if (lane == 0 && w.kvh == 0) {  // for the merge: the runs that touch the row
            if (lo == 0) p.row_runs[2 * w.b] = group;
            if (lo + n == row_tiles) p.row_runs[2 * w.b + 1] = group;
        }
        run += n;
    }
    const int count = w.count;
    const int32_t* keys = p.table + w.row0 + w.k0;
    const int n_tiles = (count + kKeys - 1) / kKeys;
    // Lane l holds the slot id of key l of a tile, -1 past the end.  It is read
    // one tile before its copies are issued and looked at only then, so the
    // load's latency is never waited for.
    auto slot_of = [&](int t) -> int {
        const int key = t * kKeys + lane;
        return key < count ? __ldg(keys + key) : -1;
    };
    auto issue = [&](int t, int slot) {
        if (t >= n_tiles) return;
        const uint32_t st = (t % kStages) * STAGE;
        // past the end, and for an id outside the pool (flagged), the scales
        // are zeros, so the row reads as zeros whatever its codes: slot 0's
        const bool ok = (uint32_t)slot < n_slots;
        if (!ok && t * kKeys + lane < count) rc::flag_error(p.err, rc::kErrBadSlot);
        const int id = ok ? slot : 0;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
            const int s = __shfl_sync(0xffffffffu, id, i * RPI + r);
            const uint64_t off = (uint64_t)(uint32_t)s * row_codes;
            rc::cp_async16(kdst + st + i * RPI * CB, kc + off, 16u, pol);
            rc::cp_async16(vdst + st + v_row(i * RPI) * CB, vc + off, 16u, pol);
        }
        const int sid = COOP ? __shfl_sync(0xffffffffu, ok ? slot : -1, sr) : ok ? slot : -1;
        const uint64_t soff = (uint64_t)(uint32_t)max(sid, 0) * row_scales;
        const uint32_t sb = sid >= 0 ? (uint32_t)SB : 0u;
        rc::cp_async_small<SB>(sdst + st, ksc + soff, sb);
        rc::cp_async_small<SB>(sdst + st + kKeys * SB, vsc + soff, sb);
    };
    {
        int first[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) first[i] = slot_of(i);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            issue(i, first[i]);
            rc::cp_async_commit();
        }
    }
    int cur = slot_of(AHEAD), nxt;
    // Q operand (f16): k-step ks of lane t covers dims t D/4 + 4 ks .. + 3.  The
    // scale's sign goes into Q, so that the largest score is the largest
    // scaled one; a scale of 0 becomes one too small to matter, which keeps a
    // masked score (-infinity) what it is.
    uint32_t qb[KS][2];
    {
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        const bool hv = g_lane < w.ncol;
        const uint4* qrow = reinterpret_cast<const uint4*>(p.q + w.qrow<NC, CROSS>(p, hv ? g_lane : 0) * D + t_lane * (D / 4));
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            uint4 x = hv ? __ldg(qrow + j) : make_uint4(0, 0, 0, 0);
            x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
            qb[2 * j][0] = rc::bf16x2_to_f16x2(x.x);
            qb[2 * j][1] = rc::bf16x2_to_f16x2(x.y);
            qb[2 * j + 1][0] = rc::bf16x2_to_f16x2(x.z);
            qb[2 * j + 1][1] = rc::bf16x2_to_f16x2(x.w);
        }
    }
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY};
    float2 l_run = make_float2(0.f, 0.f);

    for (int t = 0; t < n_tiles; ++t) {
        rc::cp_async_wait<AHEAD - 1>();
        nxt = slot_of(t + AHEAD + 1);
        if constexpr (COOP) {  // tile t is everyone's, and everyone is done with tile t - 1: refill its stage
            __syncthreads();
            issue(t + AHEAD, cur);
            rc::cp_async_commit();
        } else {
            __syncwarp();
        }
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
            s[half][0] = s[half][1] = s[half][2] = s[half][3] = 0.f;
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {  // a word: two k-steps
                const int bl = j / (KS / 4);
                uint32_t a0, a2, c0, c2, a1, a3, c1, c3;
                rc::e2m1x8_to_f16x8(x0[j], a0, a2, c0, c2);
                rc::e2m1x8_to_f16x8(x1[j], a1, a3, c1, c3);
                rc::mma_f16_16816(s[half], rc::mul_f16x2(a0, s0[bl]), rc::mul_f16x2(a1, s1[bl]), rc::mul_f16x2(a2, s0[bl]),
                                  rc::mul_f16x2(a3, s1[bl]), qb[2 * j][0], qb[2 * j][1]);
                rc::mma_f16_16816(s[half], rc::mul_f16x2(c0, s0[bl]), rc::mul_f16x2(c1, s1[bl]), rc::mul_f16x2(c2, s0[bl]),
                                  rc::mul_f16x2(c3, s1[bl]), qb[2 * j + 1][0], qb[2 * j + 1][1]);
            }
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
            mx *= sc;
            if (mx > m_run[j] + 8.f) {
                alpha[j] = tc::ex2(m_run[j] - mx);  // 0 while nothing was seen
                m_run[j] = mx;
                grow = true;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
            l_run.x *= alpha[0];
            l_run.y *= alpha[1];
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                o[i][0] *= alpha[0];
                o[i][1] *= alpha[1];
                o[i][2] *= alpha[0];
                o[i][3] *= alpha[1];
            }
        }
        const float2 nmu = make_float2(m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]);
        uint32_t pb[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 x = tc::ffma2(make_float2(s[half][2 * k], s[half][2 * k + 1]), sc, nmu);
                const float2 e = make_float2(tc::ex2(x.x), tc::ex2(x.y));
                l_run = tc::fadd2(l_run, e);
                // P to f16 (11 bits, at most 2^8): the denominator keeps the fp32 terms
                pb[half][k] = rc::movmatrix_trans(rc::pack_f16(e.x, e.y));
            }
        // O^T += V^T P^T: lane group g holds dims g D/8 .. of keys 2t, 2t+1,
        // 2t+8, 2t+9; product mt takes dims g D/8 + 2 mt (row g) and + 1
        // (row g + 8): the two nibbles of byte mt
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t x[4][KS / 4], vs[2];
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
            vs[0] = (sb[0] | (sb[1] << 16)) << 7;
            vs[1] = (sb[2] | (sb[3] << 16)) << 7;
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
                    rc::mma_f16_16816(o[4 * j + i], rc::mul_f16x2(a[0][0][i], vs[0]), rc::mul_f16x2(a[0][1][i], vs[0]),
                                      rc::mul_f16x2(a[1][0][i], vs[1]), rc::mul_f16x2(a[1][1][i], vs[1]), pb[half][0],
                                      pb[half][1]);
            }
        }
        if constexpr (!COOP) {
            __syncwarp();  // every lane has read tile t: its stage takes tile t + kStages
            issue(t + AHEAD, cur);
            rc::cp_async_commit();
        }
        cur = nxt;
    }
    rc::cp_async_wait<0>();
    if constexpr (COOP) __syncthreads();
    else __syncwarp();

#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
        l_run.x += __shfl_xor_sync(0xffffffffu, l_run.x, k);
        l_run.y += __shfl_xor_sync(0xffffffffu, l_run.y, k);
    }
    float* sE = reinterpret_cast<float*>(scratch);
    float* sOwn = sE + 8 * D;
    const float inv0 = l_run.x > 0.f ? 1.f / l_run.x : 0.f;
    const float inv1 = l_run.y > 0.f ? 1.f / l_run.y : 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
        const int d0 = g_lane * (D / 8) + 2 * mt;
        *reinterpret_cast<float2*>(sE + (2 * t_lane) * D + d0) = make_float2(o[mt][0] * inv0, o[mt][2] * inv0);
        *reinterpret_cast<float2*>(sE + (2 * t_lane + 1) * D + d0) = make_float2(o[mt][1] * inv1, o[mt][3] * inv1);
    }
    if (g_lane == 0) {
        sOwn[2 * t_lane] = rc::log2_sum(m_run[0], l_run.x);
        sOwn[2 * t_lane + 1] = rc::log2_sum(m_run[1], l_run.y);
    }
    __syncwarp();
    if constexpr (FUSED) {
        decode_epilogue<D, NC, FUSED, CROSS>(p, w, sE, sOwn, seg, first_row, lane);
    } else {
        // the partials belong to the preceding grid until it has ended
        if (!waited) grid_dep_wait();
        waited = true;
        const int64_t idx = ((int64_t)(group + w.b) * p.kv_heads + w.kvh) * NC;
        for (int c = 0; c < w.ncol; ++c)
            for (int d = lane; d < D; d += 32) p.part_o[(idx + c) * D + d] = sE[c * D + d];
        if (lane < w.ncol) p.part_lse[idx + lane] = sOwn[lane];
        if constexpr (COOP) __syncthreads();  // the ring is refilled next
        else __syncwarp();
    }
    }
    if (!FUSED && !waited) grid_dep_wait();
}

// Joins the partials of the split pass, W warps per (row, head) (CROSS: per
// (token, head)), each taking every W-th partial: the row's cascade segments
// first, then the runs that touch it.  Rows with few partials get one warp,
// long rows in many runs eight.  blockIdx.x is the row (CROSS: row * max_q +
// token); blockIdx.y a group of kMergeWarps / W heads.
template <int D, bool CROSS, int W>
__global__ void __launch_bounds__(32 * fp4::kMergeWarps) merge_runs_kernel(const DecParams p) {
    constexpr int V = D / 32;  // a lane's neighbouring columns
    constexpr int HEADS = fp4::kMergeWarps / W;
    using Vec = typename std::conditional<V == 4, float4, float2>::type;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, slot = (threadIdx.x >> 5) / W;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int b = CROSS ? blockIdx.x / p.max_q : blockIdx.x, token = CROSS ? blockIdx.x % p.max_q : 0;
    const int h = blockIdx.y * HEADS + slot;
    const RowKeys r = row_keys<CROSS>(p, b);
    const int s0 = !CROSS && p.req_seg_indptr ? p.req_seg_indptr[b] : 0;
    int n_seg = !CROSS && p.req_seg_indptr ? (p.req_seg_indptr[b + 1] - s0) * p.seg_chunks : 0;
    // The runs that touch the row: up to 32 rows from the lengths, ahead of the
    // wait; beyond, as the split pass noted them.
    int g0 = 0, g1 = -1;
    if (p.batch <= 32) {
        const int n = (row_keys<CROSS>(p, lane).L + fp4::kKeys - 1) / fp4::kKeys;
        int64_t incl = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, k);
            if (lane >= k) incl += v;
        }
        const int64_t tiles = __shfl_sync(0xffffffffu, incl, 31), end = __shfl_sync(0xffffffffu, incl, b);
        const int64_t first = end - __shfl_sync(0xffffffffu, n, b), runs = fp4::runs_of(tiles, p.n_chunks);
        if (r.L > 0) {  // run g begins at tile g * tiles / runs: tile x lies in the last that begins by x
            g0 = (int)(((first + 1) * runs - 1) / tiles);
            g1 = (int)((end * runs - 1) / tiles);
        }
    }
    grid_dep_wait();
    const bool live = h < p.q_heads && (!CROSS || token * p.group < r.ncol);
    if (W == 1 && !live) return;
    // a cascade kernel that gave up on a bounded wait left its partials unwritten
    if (n_seg && p.err && (*reinterpret_cast<volatile int32_t*>(p.err) & rc::kErrTimeout)) n_seg = 0;
    if (p.batch > 32 && r.L > 0) g0 = p.row_runs[2 * b], g1 = p.row_runs[2 * b + 1];
    const int n_all = live ? n_seg + g1 - g0 + 1 : 0;
    const int kvh = h / p.group, nc = CROSS ? 8 : p.group, col = token * p.group + h % p.group;
    // lane l looks up the l-th of a round of 32 and its log-sum-exp; all lanes
    // read the rows, eight at a time, the first eight while the log-sum-exps
    // are still on their way (a segment chunk without keys has an unwritten
    // row and no weight); against a running maximum
    constexpr int R = 8;
    float m = -INFINITY, wsum = 0.f, acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    for (int j0 = warp; j0 < n_all; j0 += 32 * W) {
        const int j = j0 + lane * W;
        const bool in_seg = j < n_seg;
        int64_t row = 0;
        if (in_seg)
            row = ((int64_t)p.req_seg_pos[s0 + j / p.seg_chunks] * p.q_heads + h) * p.seg_chunks + j % p.seg_chunks;
        else if (j < n_all)
            row = ((int64_t)(g0 + b + j - n_seg) * p.kv_heads + kvh) * nc + col;
        const float l2 = j < n_all ? (in_seg ? p.seg_lse : p.part_lse)[row] : -INFINITY;
        const float* src = (in_seg ? p.seg_o : p.part_o) + row * D;
        const int nb = min(32, (n_all - j0 + W - 1) / W);
        Vec v[R];
        auto read = [&](int i0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float* s = reinterpret_cast<const float*>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), min(i0 + i, nb - 1)));
                if (i0 + i < nb) v[i] = reinterpret_cast<const Vec*>(s)[lane];
            }
        };
        read(0);
        float mb = fmaxf(m, l2);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, k));
        if (mb == -INFINITY) continue;
        const float a = m == -INFINITY ? 0.f : rc::fast_exp2(m - mb);
        wsum *= a;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= a;
        m = mb;
        const float wt = l2 == -INFINITY ? 0.f : rc::fast_exp2(l2 - m);
        for (int i0 = 0; i0 < nb; i0 += R) {
            if (i0 > 0) read(i0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float wi = i0 + i < nb ? __shfl_sync(0xffffffffu, wt, i0 + i) : 0.f;
                if (wi == 0.f) continue;
                wsum += wi;
                const float* x = reinterpret_cast<const float*>(&v[i]);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += wi * x[k];
            }
        }
    }
    if constexpr (W > 1) {  // the warps' sums, joined in their order
        __shared__ float sM[fp4::kMergeWarps], sW[fp4::kMergeWarps];
        __shared__ __align__(16) float sA[fp4::kMergeWarps][D];
        const int me = slot * W + warp;
        if (lane == 0) {
            sM[me] = m;
            sW[me] = wsum;
        }
        Vec v;
        float* x = reinterpret_cast<float*>(&v);
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = acc[k];
        reinterpret_cast<Vec*>(sA[me])[lane] = v;
        __syncthreads();
        if (warp != 0 || !live) return;
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
            const Vec u = reinterpret_cast<const Vec*>(sA[me + i])[lane];
            const float* y = reinterpret_cast<const float*>(&u);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += e * y[k];
        }
    }
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
    const int64_t orow = CROSS ? (int64_t)(r.qo0 + token) * p.q_heads + h : (int64_t)b * p.q_heads + h;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (V / 2);
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(rc::pack_bf16(acc[0] * inv, acc[1] * inv),
                                                    rc::pack_bf16(acc[2] * inv, acc[3] * inv));
    else
        *out = rc::pack_bf16(acc[0] * inv, acc[1] * inv);
    if (p.lse && lane == 0) p.lse[orow] = rc::log2_sum(m, wsum) * rc::kLn2;
}

// rows: batch rows, or (CROSS) their tokens; as the split pass's programmatic
// dependent, so that its blocks start as that pass's leave.
template <int D, bool CROSS>
cudaError_t launch_merge_runs(const DecParams& p, int64_t rows, cudaStream_t st) {
    const int64_t parts = (p.n_chunks + (int64_t)p.batch) / p.batch;  // of a row, on average
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * fp4::kMergeWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int w = parts <= 8 ? 1 : 8;
    const int heads = fp4::kMergeWarps / w;
    cfg.gridDim = dim3((unsigned)rows, (p.q_heads + heads - 1) / heads);
    return w == 1 ? cudaLaunchKernelEx(&cfg, merge_runs_kernel<D, CROSS, 1>, p)
                  : cudaLaunchKernelEx(&cfg, merge_runs_kernel<D, CROSS, 8>, p);
}

}  // namespace rc_dec
