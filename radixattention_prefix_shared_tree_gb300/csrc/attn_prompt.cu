// attn_prompt: attention over whole prompts, packed one after the other.
//
//   out_i = sum_{j <= i} softmax_j(s q_i . k_j) v_j      within one prompt,
//
// query head h on KV head h / G.  Unlike attn_extend there is no pool and no slot
// table: a prompt's keys lie side by side as the projection left them, so tiles
// come by TMA, an instruction for 64 columns of 32 rows (of Q: of the whole tile).
//
// A unit is 256 query rows of one KV head of one prompt: two tiles of M = 128, each
// TPT = 128 / G tokens x the G heads of the group, so that every K/V tile in shared
// memory serves both.  Per 128-key tile and query tile q
//     S_q = Q_q K^T  (128 x 128 x D),  P_q = 2^(s S_q - m),  O_q += P_q V  (128 x D x 128)
// with S, P (bf16) and O in tensor memory, 512 columns in all.  D = 128 leaves room for
// one S a query tile, and P goes over it; D = 64 has columns for a P of its own, and a
// tile's next S is computed as soon as its softmax has read this one.
// P goes to the tensor core in halves of 64 keys: O += P V starts on the first while the
// second is computed.  At the edge the products end at the last key that a token of the
// tile sees (in steps of 16), and copies at the last that one of the unit sees (of 32).
//
// Twelve warps: 0-3 and 4-7 the softmax and the results of query tile 0 and 1 (a thread
// a row), 8 the copies, 9 and 10 the products of query tile 0 and 1 (one elected lane),
// 11 the units and the guard of V (below).  One warp for both tiles' products spent
// 1,900 cycles and more on a tile's 1,024 cycles of them, as it looks after eight
// barriers in turn; two, each with its own tile's, let the two tiles fall out of step, so
// that one's products run under the other's softmax.  CTAs are persistent, one an SM;
// unit u+1's copies and its first product run while unit u's rows are written.
//
// Measured: 3 prompts of 9,000 to 14,000 tokens, 32/8 heads of 128: 1,690 to 1,860 us from GPU to
// GPU, 1,460 to 1,610 TFLOP/s of the products a causal mask leaves, bound by the tensor core (cuBLAS
// keeps up 1,725).  One of 2,049, 64/8 heads: 69 us.  256 prompts of 128 to 512: 508 us, 3.3
// TB/s, bound by the chain of a unit (loads, two to five tiles, rows out).  12 of 375 to 1,500,
// 16 heads of 64: 58.5 us.  At the 168 registers that twelve warps leave each thread, head
// dimension 64 spills 36 bytes a thread, 128 52.
// Tried and slower: results by four warps of their own with TMA stores (sixteen warps:
// 556 us for the short prompts), a softmax of two passes over S instead of 128 scores in
// registers (2,145 us for the long ones), a lock around a tile's products (528 us for the
// short ones), one warp for both tiles' products (531, 1,874 and 62.4 us), rows written
// straight from registers or a fifth stage of K and V (1,900 us and more for the long
// ones: what ends sooner brings the two tiles into step, and then both wait for the tensor
// core and leave it idle together).
//
// Order of the units: by their number of keys, largest first (all prompts' last
// blocks, so to speak, then those before), which evens out the end of the grid
// for any mix of lengths; the KV heads of one block are neighbours.
//
// What a weight of zero meets: scores are masked by selection, so a NaN or an
// infinity in K behind the causal edge has no effect.  In V it would (0 x inf), so
// the guard warp looks over the tiles at the edge before they are used: rows behind
// the prompt's end (the next prompt's) become zeros, non-finite values of its later
// tokens too, and the results' warps then add those to the rows that do attend to them.

#include "tma.cuh"

namespace {

constexpr int TM = 128, QT = 2, TN = 128;
constexpr int BOX = 32;         // rows of K or V a copy
constexpr int UNITS = 4;        // units known ahead
constexpr int NB_CACHE = 2048;  // prompts whose block counts are kept in shared memory
constexpr int FEW = 1024;            // prompts that are looked through again for every unit
constexpr int MAX_BATCH = 1 << 20;  // every CTA goes through the prompts, about 8 ms each time with so many
constexpr int THREADS = 384;
constexpr int COPY_WARP = 8, MMA_WARP = 9, UNIT_WARP = 11;
constexpr int READERS = 11;  // warps that read a unit: all but its writer
constexpr uint32_t kWaitIter = 1u << 24;

struct PromptParams {
    const int32_t* indptr;
    int32_t batch, n_tokens;
    int32_t q_heads, kv_heads, group, tpt;
    float scale_log2;
    const __nv_bfloat16* v;  // for the rows that attend to a non-finite value
    int64_t v_stride;
    __nv_bfloat16* out;
    float* lse;
    int32_t* err;
};

struct Unit {
    int32_t first;  // the prompt's first token in the packed rows
    int32_t len;    // its tokens; < 0: no more units
    int32_t t0;     // the unit's first token within the prompt
    int32_t kvh;
};

template <int D>
__host__ __device__ constexpr int stages() { return D == 128 ? 4 : 8; }
template <int D>
__host__ __device__ constexpr int n_bars() { return 10 * QT + 4 * stages<D>() + 3 * UNITS; }
template <int D>
__host__ __device__ constexpr int smem_bytes() {
    return QT * TM * D * 2 + stages<D>() * TN * D * 2 + 8 * 2048 + NB_CACHE * 4 + UNITS * (int)sizeof(Unit) + UNITS * 4 +
           n_bars<D>() * 8 + 16 + 1024;  // (the last for the alignment of the tiles)
}

RC_DEV int n_blocks(const PromptParams& p, int b, int tpc) {
    const int a = __ldg(p.indptr + b), e = __ldg(p.indptr + b + 1);
    if (a < 0 || e < a || e > p.n_tokens) return -1;
    return (int)(((int64_t)e - a + tpc - 1) / tpc);
}

using tc::ex2;
using tc::fadd2;
using tc::ffma2;
using tc::max3;
using tc::mbar_arrive;

// MANY: more prompts than FEW.  (An instance of its own, because what the units' warp does and where
// its code lies moves the two query tiles against each other: with both ways in one, 3 prompts of 9,000
// to 14,000 took 6 % longer, 12 of 375 to 1,500 5 %.)
template <int D, bool MANY>
__global__ void __launch_bounds__(THREADS, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PromptParams p) {
    constexpr int NS = stages<D>();
    constexpr int BLK = TN * 128;        // bytes of one 64-column block
    constexpr int TILE = TN * D * 2;     // bytes of a K, V or Q tile
    constexpr uint32_t idS = tc::idesc_bf16(TM, TN, false), idPV = tc::idesc_bf16(TM, D, true);
    constexpr bool OWN_P = D == 64;      // P has columns of its own
    constexpr int P_COL = OWN_P ? QT * TN : 0, P_STEP = OWN_P ? TN / 2 : TN;  // columns of P_0, from P_0 to P_1
    constexpr int O_COL = QT * TN + (OWN_P ? QT * TN / 2 : 0);
    static_assert(O_COL + QT * D <= 512, "tensor memory");
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (rc::smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sQ = smem;
    unsigned char* sKV = sQ + QT * TILE;
    unsigned char* sOut = sKV + NS * TILE;                      // 2 KB a softmax warp
    int32_t* sNB = reinterpret_cast<int32_t*>(sOut + 8 * 2048);
    Unit* sUnit = reinterpret_cast<Unit*>(sNB + NB_CACHE);
    int32_t* sBad = reinterpret_cast<int32_t*>(sUnit + UNITS);  // the unit's V had non-finite values at the edge
    uint64_t* bar = reinterpret_cast<uint64_t*>(sBad + UNITS);
    uint64_t* q_full = bar;                    // [QT] 1 + bytes
    uint64_t* q_empty = q_full + QT;           // [QT] 1 (commit)
    uint64_t* kv_full = q_empty + QT;          // [NS] 1 + bytes
    uint64_t* kv_empty = kv_full + NS;         // [NS] 2 (a commit, or an arrival, of both product warps)
    uint64_t* edge_full = kv_empty + NS;       // [NS] 1 + bytes, instead of kv_full for a V tile at the causal edge
    uint64_t* v_ok = edge_full + NS;           // [NS] 1: the guard has seen it
    uint64_t* s_full = v_ok + NS;              // [QT] 1 (commit)
    uint64_t* s_read = s_full + QT;            // [QT] 4: S is in the softmax warps' registers (OWN_P)
    uint64_t* p_full = s_read + QT;            // [QT][2] 4 (the tile's softmax warps): 64 keys of P
    uint64_t* pv_done = p_full + 2 * QT;           // [QT] 1 (commit): of every tile (OWN_P)
    uint64_t* o_done = pv_done + QT;           // [QT] 1 (commit): the unit's last P V
    uint64_t* o_free = o_done + QT;            // [QT] 4: O is in the softmax warps' registers
    uint64_t* unit_full = o_free + QT;         // [UNITS] 1
    uint64_t* unit_empty = unit_full + UNITS;  // [UNITS] READERS
    uint64_t* guarded = unit_empty + UNITS;    // [UNITS] 1: the unit's edge tiles are all seen
    uint64_t* drained = guarded + UNITS;       // [QT] 1: products in flight when a wait gave up
    uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + QT);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = p.group, tpt = p.tpt, tpc = QT * tpt;
    // a wait gave up in an earlier CTA: the results are void
    const int gave_up = p.err && (*reinterpret_cast<volatile int32_t*>(p.err) & rc::kErrTimeout);
    if (warp == MMA_WARP) {
        if (lane == 0) {
            for (int i = 0; i < QT; ++i) {
                tc::mbar_init(&q_full[i], 1);
                tc::mbar_init(&q_empty[i], 1);
                tc::mbar_init(&s_full[i], 1);
                tc::mbar_init(&s_read[i], 4);
                tc::mbar_init(&p_full[2 * i], 4);
                tc::mbar_init(&p_full[2 * i + 1], 4);
                tc::mbar_init(&pv_done[i], 1);
                tc::mbar_init(&o_done[i], 1);
                tc::mbar_init(&o_free[i], 4);
                tc::mbar_init(&drained[i], 1);
            }
            for (int i = 0; i < NS; ++i) {
                tc::mbar_init(&kv_full[i], 1);
                tc::mbar_init(&kv_empty[i], 2);
                tc::mbar_init(&edge_full[i], 1);
                tc::mbar_init(&v_ok[i], 1);
            }
            for (int i = 0; i < UNITS; ++i) {
                tc::mbar_init(&unit_full[i], 1);
                tc::mbar_init(&unit_empty[i], READERS);
                tc::mbar_init(&guarded[i], 1);
            }
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(tslot, 512);
        tc::tmem_relinquish();
    } else if (warp == COPY_WARP) {
        if (lane == 0) {
            tma::prefetch_map(&map_q);
            tma::prefetch_map(&map_k);
            tma::prefetch_map(&map_v);
        }
    } else if (warp < COPY_WARP) {
        const int t = tid;
        for (int b = t; b < min(p.batch, NB_CACHE); b += 32 * COPY_WARP) {
            const int n = n_blocks(p, b, tpc);
            if (n < 0 && blockIdx.x == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            sNB[b] = max(n, 0);
        }
        if (blockIdx.x == 0)
            for (int b = NB_CACHE + t; b < p.batch; b += 32 * COPY_WARP)
                if (n_blocks(p, b, tpc) < 0) rc::flag_error(p.err, rc::kErrBadSlot);
    }
    tc::fence_before();
    const int leave = __syncthreads_or(gave_up);
    tc::fence_after();
    const uint32_t tbase = *tslot;
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(b, parity, kWaitIter)) && ok;
        return ok;
    };
    // A V tile at the unit's causal edge, which some of its tokens do not see whole.
    // Its copy completes on a barrier that only the guard waits for, and the
    // products wait for the guard: a parity tells two phases apart, not three, so
    // every barrier's phases are all waited for by whoever waits at all.
    auto at_edge = [&](const Unit& u, int t) { return (t + 1) * TN - 1 > u.t0; };
    // tiles of 128 keys that query tile q of unit u attends to (0: no rows)
    auto tiles = [&](const Unit& u, int q) {
        const int t = u.t0 + q * tpt;
        return t < u.len ? (min(t + tpt, u.len) + TN - 1) / TN : 0;
    };

    if (leave) {
        // nothing is on its way yet
    } else if (warp < 8) {
        // ========================================================= softmax
        const int q = warp >> 2, r = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + q * TN + lane_off, tO = tbase + O_COL + q * D + lane_off;
        const uint32_t tP = tbase + P_COL + q * P_STEP + lane_off;
        const int r_tok = r / G, r_head = r - r_tok * G;
        const float sc = p.scale_log2;
        uint32_t ps = 0, po = 0, pp = 1;  // phases of s_full, o_done, pv_done
        for (int i = 0; ok; ++i) {
            const int slot = i % UNITS, ph = (i / UNITS) & 1;
            if (!wait(&unit_full[slot], ph)) break;
            const Unit u = sUnit[slot];
            if (u.len < 0) break;
            const int n = tiles(u, q);
            const int tok = u.t0 + q * tpt + r_tok;
            const bool valid = r_tok < tpt && tok < u.len;
            const int lim = tok + 1;  // (rows without a token run along, on what their tile holds)
            const int warp_lim = __shfl_sync(0xffffffffu, lim, 0);
            float m_used = -INFINITY, l_run = 0.f;
            for (int t = 0; t < n; ++t) {
                if (!wait(&s_full[q], ps)) break;
                ps ^= 1;
                tc::fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_ld32_issue(tS + c * 32, s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_ld_wait(s[c]);
                if constexpr (OWN_P) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_read[q]);
                }
                const int kb = t * TN;
                if (__builtin_expect(kb + TN > warp_lim, 0)) {  // the causal edge (a branch of the whole warp)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int seen = min(max(lim - kb - c * 32, 0), 32);
                        const uint32_t keep = (uint32_t)((1ull << seen) - 1ull);
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[c][j] = keep & (1u << j) ? s[c][j] : 0xff800000u;
                    }
                }
                auto f = [&](int j) { return __uint_as_float(s[j >> 5][j & 31]); };
                float m8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m8[k] = f(k);
#pragma unroll
                    for (int j = 8; j < 120; j += 16) m8[k] = max3(m8[k], f(k + j), f(k + j + 8));
                    m8[k] = fmaxf(m8[k], f(k + 120));
                }
                const float mt = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sc;
                const bool grow = mt > m_used + 8.f;
                const bool rescale = grow && m_used != -INFINITY;
                if constexpr (OWN_P) {  // the last tile's P has been read, and O is stable
                    if (!wait(&pv_done[q], pp)) break;
                    pp ^= 1;
                    tc::fence_after();
                }
                if (__builtin_expect(__any_sync(0xffffffffu, rescale), 0)) {
                    // O is stable (without OWN_P: S(t) is done, and P(t-1).V was issued before it)
                    const float a = rescale ? ex2(m_used - mt) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tc::tmem_ld32_issue(tO + c * 32, o);
                        tc::tmem_ld_wait(o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
                        tc::tmem_st32_issue(tO + c * 32, o);
                    }
                    tc::tmem_st_wait();
                }
                if (grow) {
                    l_run *= ex2(m_used - mt);  // 0 while nothing was seen
                    m_used = mt;
                }
                const float nmu = m_used == -INFINITY ? 0.f : -m_used;
                float2 ls[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = ffma2(make_float2(f(c * 32 + 2 * j), f(c * 32 + 2 * j + 1)), sc, nmu);
                        const float2 e = make_float2(ex2(x.x), ex2(x.y));
                        ls[j & 3] = fadd2(ls[j & 3], e);
                        // P to V's type, as every product here takes one type: bf16 keeps 8 bits
                        // of a weight; their sum keeps the fp32 terms
                        pk[j] = rc::pack_bf16(e.x, e.y);
                    }
                    tc::tmem_st16_issue(tP + c * 16, pk);
                    if (c & 1) {
                        tc::tmem_st_wait();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[2 * q + c / 2]);
                    }
                }
                const float2 l01 = fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3]));
                l_run += l01.x + l01.y;
            }
            if (!ok) break;
            if (n > 0) {
                // ---- normalised rows out.  All of O is read first, so that the next
                // unit's P.V may start; rows go through 2 KB a warp, 32 columns at a
                // time, so that a store instruction writes runs of 64 bytes.
                if (!wait(&o_done[q], po)) break;
                po ^= 1;
                tc::fence_after();
                uint32_t o[D / 32][32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tc::tmem_ld32_issue(tO + c * 32, o[c]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tc::tmem_ld_wait(o[c]);
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[q]);
                if (!wait(&guarded[slot], ph)) break;
                if (__builtin_expect(sBad[slot] && valid, 0)) {  // rare: values that the guard took out of V, for the rows that see them
                    for (int j = u.t0 + 1; j <= tok; ++j) {
                        const __nv_bfloat16* vr = p.v + (int64_t)(u.first + j) * p.v_stride + (int64_t)u.kvh * D;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const float x = __bfloat162float(vr[c * 32 + k]);
                                if (!isfinite(x)) o[c][k] = __float_as_uint(__uint_as_float(o[c][k]) + x);
                            }
                    }
                }
                const float inv = l_run > 0.f ? 1.f / l_run : l_run;  // (NaN stays)
                const int64_t row = (int64_t)(u.first + tok) * p.q_heads + u.kvh * G + r_head;
                const int64_t mine = valid ? row : -1;
                unsigned char* stg = sOut + warp * 2048;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    auto x = [&](int k) { return __uint_as_float(o[c][k]) * inv; };
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) * 16)) =
                            make_uint4(rc::pack_bf16(x(8 * k), x(8 * k + 1)), rc::pack_bf16(x(8 * k + 2), x(8 * k + 3)),
                                       rc::pack_bf16(x(8 * k + 4), x(8 * k + 5)), rc::pack_bf16(x(8 * k + 6), x(8 * k + 7)));
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int lr = k * 8 + (lane >> 2), ch = lane & 3;
                        const uint4 w = *reinterpret_cast<const uint4*>(stg + lr * 64 + ((ch ^ ((lr >> 1) & 3)) * 16));
                        const int64_t to = __shfl_sync(0xffffffffu, mine, lr);
                        if (to >= 0) reinterpret_cast<uint4*>(p.out + to * D)[c * 4 + ch] = w;
                    }
                    __syncwarp();
                }
                if (p.lse && valid) p.lse[row] = rc::log2_sum(m_used, l_run) * rc::kLn2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&unit_empty[slot]);
        }
        if constexpr (OWN_P)  // (no arrival may come when the CTA has left)
            if (ok) wait(&pv_done[q], pp);
        if (!ok) rc::flag_error(p.err, rc::kErrTimeout);
    } else if (warp == COPY_WARP) {
        // ========================================================== copies
        const bool lead = tc::elect_one();
        int st = 0, ph = 1;         // the next load's stage, and the parity of the wait for it (its first use waits for nothing)
        uint32_t pq[QT] = {1, 1};   // likewise of Q's tiles
        int loads = 0, q_loads[QT] = {0, 0};
        uint32_t used[2] = {0, 0}, kind = 0;  // per stage: parity of the next use of kv_full, edge_full; which was last
        const uint32_t q_bytes = (uint32_t)(tpt * G) * D * 2;
        for (int i = 0; ok; ++i) {
            const int slot = i % UNITS;
            if (!wait(&unit_full[slot], (i / UNITS) & 1)) break;
            const Unit u = sUnit[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&unit_empty[slot]);
            if (u.len < 0) break;
            const int nq[QT] = {tiles(u, 0), tiles(u, 1)};
            const int n = max(nq[0], nq[1]);
            auto load_q = [&](int q) {
                if (nq[q] == 0 || !wait(&q_empty[q], pq[q])) return;
                pq[q] ^= 1;
                ++q_loads[q];
                if (lead) {
                    tma::expect(&q_full[q], q_bytes);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma::load3(sQ + q * TILE + c * BLK, &map_q, &q_full[q], c * 64, u.kvh * G, u.first + u.t0 + q * tpt);
                }
            };
            // Q_0, K(0), Q_1, V(0), K(1), ...: the first product of query tile 0 waits for
            // nothing of the unit before but that tile's own last product
            load_q(0);
            for (int t = 0; t < 2 * n && ok; ++t) {
                if (t == 1) load_q(1);
                if (!ok) break;
                if (!wait(&kv_empty[st], ph)) break;
                ++loads;
                const bool edge = (t & 1) && at_edge(u, t >> 1);
                used[edge] ^= 1u << st;
                kind = (kind & ~(1u << st)) | ((edge ? 1u : 0u) << st);
                uint64_t* full = edge ? &edge_full[st] : &kv_full[st];
                if (lead) {  // only the rows that the unit's tokens look at (in steps of BOX)
                    const int rows = min(TN, (min(u.t0 + tpc, u.len) - (t >> 1) * TN + BOX - 1) / BOX * BOX);
                    tma::expect(full, rows * D * 2);
                    for (int r = 0; r < rows; r += BOX)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma::load3(sKV + st * TILE + c * BLK + r * 128, t & 1 ? &map_v : &map_k, full, c * 64, u.kvh,
                                       u.first + (t >> 1) * TN + r);
                }
                if (++st == NS) st = 0, ph ^= 1;
            }
        }
        // nothing may be on its way to this CTA's memory when it leaves: neither
        // copies nor the tensor core's arrivals (after a wait that gave up, the copies)
        if (!ok) rc::flag_error(p.err, rc::kErrTimeout);
        __syncwarp();
        const bool fine = ok;
        for (int k = 0; k < min(loads, NS); ++k) {
            const int last = loads - 1 - k, s = last % NS;
            const int e = (kind >> s) & 1;
            if (fine) tc::mbar_wait(&kv_empty[s], (last / NS) & 1, kWaitIter);
            else tc::mbar_wait(e ? &edge_full[s] : &kv_full[s], ((used[e] >> s) & 1) ^ 1, kWaitIter);
        }
        for (int q = 0; q < QT; ++q)
            if (q_loads[q] > 0) tc::mbar_wait(fine ? &q_empty[q] : &q_full[q], (q_loads[q] - 1) & 1, kWaitIter);
    } else if (warp < UNIT_WARP) {
        // ======================================================== products
        const int q = warp - MMA_WARP;
        const bool lead = tc::elect_one();
        const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
        constexpr uint32_t STEP = TILE / 16;
        const tc::Desc qd = tma::desc_sw128(rc::smem_u32(sQ + q * TILE), 16);
        const tc::Desc kd = tma::desc_sw128(rc::smem_u32(sKV), 16);
        const tc::Desc vd = tma::desc_sw128(rc::smem_u32(sKV), BLK);
        const uint32_t tS = tb + q * TN, tP = tb + P_COL + q * P_STEP, tO = tb + O_COL + q * D;
        const uint32_t a_kv_full = rc::smem_u32(kv_full), a_kv_empty = rc::smem_u32(kv_empty), a_v_ok = rc::smem_u32(v_ok),
                       a_q_full = rc::smem_u32(q_full + q), a_q_empty = rc::smem_u32(q_empty + q),
                       a_s_full = rc::smem_u32(s_full + q), a_s_read = rc::smem_u32(s_read + q),
                       a_p_full = rc::smem_u32(p_full + 2 * q), a_pv_done = rc::smem_u32(pv_done + q),
                       a_o_done = rc::smem_u32(o_done + q), a_o_free = rc::smem_u32(o_free + q);
        int st = 0;  // the stage of the unit's K(0)
        uint32_t pk = 0, pv = 0;  // phases of kv_full and v_ok, a bit a stage
        uint32_t pq = 0, pp = 0, pf = 1, pr = 1;  // of q_full, p_full, o_free, s_read
        auto need = [&](uint32_t at, uint32_t parity) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait_at(at, parity, kWaitIter)) && ok;
            return ok;
        };
        auto need_kv = [&](int s, bool edge) {
            const bool there = need((edge ? a_v_ok : a_kv_full) + s * 8, ((edge ? pv : pk) >> s) & 1);
            if (edge) pv ^= 1u << s;
            else pk ^= 1u << s;
            return there;
        };
        auto pass = [&](int s, bool edge) {  // a tile that this query tile does not look at
            if (!need_kv(s, edge)) return;
            if (lane == 0) mbar_arrive(&kv_empty[s]);
            __syncwarp();
        };
        for (int i = 0; ok; ++i) {
            const int slot = i % UNITS;
            if (!wait(&unit_full[slot], (i / UNITS) & 1)) break;
            Unit u = sUnit[slot];
            u.len = __shfl_sync(0xffffffffu, u.len, 0);  // (the same in all lanes)
            u.t0 = __shfl_sync(0xffffffffu, u.t0, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&unit_empty[slot]);
            if (u.len < 0) break;
            const int n = max(tiles(u, 0), tiles(u, 1)), mine = tiles(u, q);
            const int keys = min(u.t0 + (q + 1) * tpt, u.len);
            auto k_stage = [&](int t) { return (st + 2 * t) % NS; };
            // S(t) = Q K(t)^T, over as many keys (in steps of 16) as the tile's last token sees
            auto ready_s = [&](int t) {
                if (!need_kv(k_stage(t), false)) return false;
                if (t == 0) {
                    if (!need(a_q_full, pq)) return false;
                    pq ^= 1;
                }
                if constexpr (OWN_P) {
                    if (!need(a_s_read, pr)) return false;
                    pr ^= 1;
                }
                return true;
            };
            auto issue_s = [&](int t) {
                const int s = k_stage(t);
                const uint32_t wide = min(TN, (keys - t * TN + 15) & ~15);
                const uint32_t id = (idS & ~(0x3fu << 17)) | ((wide >> 3) << 17);  // N of the product
                const uint32_t klo = kd.lo + s * STEP;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * (BLK / 16) + (k % 4) * 2;
                    tc::mma_bf16_h(tS, qd.lo + off, qd.hi, klo + off, kd.hi, id, k > 0 ? 1u : 0u);
                }
                tc::commit_at(a_s_full);
                tc::commit_at(a_kv_empty + s * 8);
                if (t + 1 == mine) tc::commit_at(a_q_empty);
            };
            // half h of P V(t): 64 keys
            auto issue_pv = [&](int t, int vs, int h) {
                const int steps = min(TN, keys - t * TN + 15) / 16;
                const uint32_t plo = tP + h * 32, vlo = vd.lo + vs * STEP + h * 4 * (2048 / 16);
                const uint32_t add = t > 0 || h > 0 ? 1u : 0u;
                if (steps == TN / 16) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_bf16_ts_h(tO, plo + k * 8, vlo + k * (2048 / 16), vd.hi, idPV, k > 0 ? 1u : add);
                } else {
#pragma unroll 1
                    for (int k = 0; k < min(steps - h * 4, 4); ++k)
                        tc::mma_bf16_ts_h(tO, plo + k * 8, vlo + k * (2048 / 16), vd.hi, idPV, k > 0 ? 1u : add);
                }
                if (h == 0) return;
                tc::commit_at(a_kv_empty + vs * 8);
                if (OWN_P) tc::commit_at(a_pv_done);
                if (t + 1 == mine) tc::commit_at(a_o_done);
            };
            if (mine > 0) {
                if (!ready_s(0)) break;
                tc::fence_after();
                if (lead) issue_s(0);
                __syncwarp();
            } else {
                pass(st, false);
            }
            for (int t = 0; t < n && ok; ++t) {
                const int vs = (st + 2 * t + 1) % NS;
                const bool edge = at_edge(u, t), more = t + 1 < mine;
                if (t >= mine) {
                    pass(vs, edge);
                    if (t + 1 < n) pass(k_stage(t + 1), false);
                    continue;
                }
                if constexpr (OWN_P)
                    if (more) {
                        if (!ready_s(t + 1)) break;
                        tc::fence_after();
                        if (lead) issue_s(t + 1);
                        __syncwarp();
                    }
                if (!need_kv(vs, edge)) break;
                if (t == 0) {
                    if (!need(a_o_free, pf)) break;
                    pf ^= 1;
                }
                if (!need(a_p_full, pp)) break;
                tc::fence_after();
                if (lead) issue_pv(t, vs, 0);
                __syncwarp();
                if constexpr (!OWN_P)
                    if (more && !ready_s(t + 1)) break;
                if (!need(a_p_full + 8, pp)) break;
                pp ^= 1;
                tc::fence_after();
                if (lead) {
                    issue_pv(t, vs, 1);
                    if (!OWN_P && more) issue_s(t + 1);
                }
                __syncwarp();
                if (!more && t + 1 < n) pass(k_stage(t + 1), false);
            }
            st = (st + 2 * n) % NS;
        }
        if (!ok) {
            if (lead) {
                rc::flag_error(p.err, rc::kErrTimeout);
                tc::commit(&drained[q]);
            }
            tc::mbar_wait(&drained[q], 0, kWaitIter);  // the products read tiles and write TMEM
        }
        __syncwarp();
    } else {
        // ================================================= units, guard of V
        auto blocks = [&](int b) { return b < NB_CACHE ? sNB[b] : max(n_blocks(p, b, tpc), 0); };
        int most = 0;
        int64_t total = 0;
        for (int b = lane; b < p.batch; b += 32) {
            const int x = blocks(b);
            most = max(most, x);
            total += x;
        }
        most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        // blocks number `lev` (from 0) of the prompts that have one; `above`: blocks of higher numbers
        int lev = most, have = 0;
        int64_t above = 0;
        auto count = [&](int l) {
            int c = 0;
            for (int b = lane; b < p.batch; b += 32) c += blocks(b) > l;
            return (int)__reduce_add_sync(0xffffffffu, c);
        };
        // MANY: looked through from the start for every unit, thousands of prompts would take longer
        // than their work (5,000 of one token, 8 heads of 64: 3,360 us, 1,180 as here; a million, 2
        // heads: 76 ms).  A level's prompts are gone through once, from b0 on, where its last unit was
        // found, with `before` of its blocks in front; and counted once for all levels down to `low`,
        // the next smaller number of blocks that a prompt has.
        [[maybe_unused]] int low = most, b0 = 0, before = 0;
        [[maybe_unused]] auto count_down = [&] {
            int c = 0, next = 0;
#pragma unroll 8
            for (int b = lane; b < p.batch; b += 32) {
                const int x = blocks(b);
                c += x > lev;
                next = max(next, x > lev ? 0 : x);
            }
            have = (int)__reduce_add_sync(0xffffffffu, c);
            low = __reduce_max_sync(0xffffffffu, next);
        };
        auto find = [&](int64_t u) -> Unit {  // (u rises from call to call)
            Unit x{0, -1, 0, 0};
            const int64_t pos = u / p.kv_heads;
            if (pos >= total) return x;
            while (pos >= above + have) {
                above += have;
                --lev;
                if constexpr (MANY) {
                    b0 = before = 0;
                    if (lev < low) count_down();
                } else {
                    have = count(lev);
                }
            }
            if constexpr (!MANY) b0 = before = 0;
            int rank = (int)(pos - above) - before;
            for (;; b0 += 32) {
                const unsigned m = __ballot_sync(0xffffffffu, b0 + lane < p.batch && blocks(b0 + lane) > lev);
                const int c = __popc(m);
                if (rank < c) {
                    x.first = b0 + __fns(m, 0, rank + 1);
                    break;
                }
                rank -= c;
                if constexpr (MANY) before += c;
            }
            const int b = x.first;
            x.first = __ldg(p.indptr + b);
            x.len = __ldg(p.indptr + b + 1) - x.first;
            x.t0 = lev * tpc;
            x.kvh = (int)(u % p.kv_heads);
            return x;
        };
        auto publish = [&](int i, const Unit& x) {
            const int slot = i % UNITS;
            if (i >= UNITS && !wait(&unit_empty[slot], ((i / UNITS) & 1) ^ 1)) return;
            if (lane == 0) {
                sUnit[slot] = x;
                sBad[slot] = 0;
                mbar_arrive(&unit_full[slot]);
            }
            __syncwarp();
        };
        int st = 0;
        uint32_t pe = 0;  // phases of edge_full, a bit a stage
        // this CTA's k-th unit: forth and back through the CTAs, so that no CTA has the
        // largest of every round (2,049 tokens, 64/8 heads: 76 -> 69 us)
        auto unit_at = [&](int k) { return (int64_t)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
        Unit cur = find(unit_at(0));
        publish(0, cur);
        for (int i = 0; ok && cur.len >= 0; ++i) {
            const int slot = i % UNITS;
            const Unit nxt = find(unit_at(i + 1));
            publish(i + 1, nxt);
            if (!ok) break;
            const int n = max(tiles(cur, 0), tiles(cur, 1));
            for (int t = 0; t < n && ok; ++t) {
                if (++st == NS) st = 0;  // K(t)
                const int kb = t * TN;
                if (at_edge(cur, t)) {
                    if (!wait(&edge_full[st], (pe >> st) & 1)) break;
                    pe ^= 1u << st;
                    unsigned char* tile = sKV + st * TILE;
                    // rows that some of the unit's tokens do not see, and rows that are not the
                    // prompt's, as far as the products go
                    const int keys = min(cur.t0 + tpc, cur.len), end = min(TN, (keys - kb + 15) & ~15);
                    const int r0 = max(cur.t0 + 1 - kb, 0), r1 = max(min(keys - kb, TN), r0);
                    __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
                    const __nv_bfloat162 zero = acc;
                    auto look = [&](const uint4& w) {  // 0, or NaN from an infinity or a NaN on
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[j]), zero, acc);
                    };
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4* rows = reinterpret_cast<const uint4*>(tile + c * BLK);
                        int k = r0 * 8 + lane;
                        for (; k + 96 < r1 * 8; k += 128) {
                            const uint4 w0 = rows[k], w1 = rows[k + 32], w2 = rows[k + 64], w3 = rows[k + 96];
                            look(w0), look(w1), look(w2), look(w3);
                        }
                        for (; k < r1 * 8; k += 32) look(rows[k]);
                        for (k = r1 * 8 + lane; k < end * 8; k += 32)
                            reinterpret_cast<uint4*>(tile + c * BLK)[k] = make_uint4(0, 0, 0, 0);
                    }
                    const bool here = __any_sync(0xffffffffu, __hisnan(acc.x) || __hisnan(acc.y));
                    if (here) {
                        for (int c = 0; c < D / 64; ++c)
                            for (int k = r0 * 8 + lane; k < r1 * 8; k += 32) {
                                uint16_t* x = reinterpret_cast<uint16_t*>(tile + c * BLK + k * 16);
                                for (int j = 0; j < 8; ++j)
                                    if ((x[j] & 0x7f80u) == 0x7f80u) x[j] = 0;
                            }
                        if (lane == 0) sBad[slot] = 1;
                    }
                    if (here || r1 < end) tc::fence_proxy_async();  // this lane's zeros, before the tensor core reads the tile
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_ok[st]);
                }
                if (++st == NS) st = 0;  // V(t)
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&guarded[slot]);
            __syncwarp();
            cur = nxt;
        }
        if (!ok && lane == 0) rc::flag_error(p.err, rc::kErrTimeout);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc::fence_after();
        tc::tmem_dealloc(tbase, 512);
    }
}

template <int D, bool MANY>
cudaError_t launch(const CUtensorMap (&m)[3], const PromptParams& p, int grid, cudaStream_t st) {
    cudaError_t e = rc_host::ensure_smem<attn_prompt_kernel<D, MANY>>(smem_bytes<D>());
    if (e != cudaSuccess) return e;
    attn_prompt_kernel<D, MANY><<<grid, THREADS, smem_bytes<D>(), st>>>(m[0], m[1], m[2], p);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch(const CUtensorMap (&m)[3], const PromptParams& p, int grid, cudaStream_t st) {
    return p.batch > FEW ? launch<D, true>(m, p, grid, st) : launch<D, false>(m, p, grid, st);
}

}  // namespace

bool rc_host::rows_map(CUtensorMap* map, const void* base, int64_t tokens, int32_t heads, int32_t dim, int64_t stride,
                       int32_t box_heads, int32_t box_tokens) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" rc_status attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const int32_t* indptr, int32_t batch, int64_t n_tokens, int32_t q_heads,
                                 int32_t kv_heads, int32_t head_dim, float sm_scale, void* out, float* lse, int32_t* err,
                                 rc_stream_t stream) {
    if (batch < 0 || n_tokens < 0 || n_tokens > 0x7fffffff || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads ||
        head_dim <= 0)
        return RC_ERR_ARG;
    if (!(sm_scale > 0.f)) return RC_ERR_ARG;  // the largest score has to be the largest scaled one
    const int G = q_heads / kv_heads;
    if ((head_dim != 64 && head_dim != 128) || G > TM || batch > MAX_BATCH) return RC_ERR_UNSUPPORTED;
    // reads may overlap (a broadcast row would have stride 0), but a map's strides may not be zero
    const int64_t q_row = (int64_t)q_heads * head_dim, kv_row = (int64_t)kv_heads * head_dim;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || ((q_stride | k_stride | v_stride) & 7) ||
        (q_stride | k_stride | v_stride) >= ((int64_t)1 << 38))
        return RC_ERR_ARG;
    if (batch == 0 || n_tokens == 0) return RC_OK;
    if (!q || !k || !v || !indptr || !out) return RC_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(out)) & 15)
        return RC_ERR_ARG;
    const int64_t out_bytes = n_tokens * q_row * 2, lse_bytes = n_tokens * q_heads * 4;
    for (int i = 0; i < 3; ++i) {  // other units may still read what this one's rows would go over
        const void* const in = i == 0 ? q : i == 1 ? k : v;
        const int64_t stride = i == 0 ? q_stride : i == 1 ? k_stride : v_stride, row = i == 0 ? q_row : kv_row;
        if (rc_host::overlap(out, out_bytes, in, n_tokens, stride * 2, row * 2) ||
            rc_host::overlap(lse, lse_bytes, in, n_tokens, stride * 2, row * 2))
            return RC_ERR_ARG;
    }
    const int64_t ip = ((int64_t)batch + 1) * 4;
    if (rc_host::overlap(out, out_bytes, indptr, 1, ip, ip) || rc_host::overlap(lse, lse_bytes, indptr, 1, ip, ip) ||
        rc_host::overlap(lse, lse_bytes, out, 1, out_bytes, out_bytes))
        return RC_ERR_ARG;
    PromptParams p{};
    p.indptr = indptr;
    p.batch = batch;
    p.n_tokens = (int32_t)n_tokens;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = G;
    p.tpt = TM / G;
    p.scale_log2 = sm_scale * rc::kLog2e;
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.v_stride = v_stride;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.err = err;
    CUtensorMap m[3];
    if (!rc_host::rows_map(&m[0], q, n_tokens, q_heads, head_dim, q_stride, G, p.tpt) ||
        !rc_host::rows_map(&m[1], k, n_tokens, kv_heads, head_dim, k_stride, 1, BOX) ||
        !rc_host::rows_map(&m[2], v, n_tokens, kv_heads, head_dim, v_stride, 1, BOX))
        return RC_ERR_CUDA;
    // at most this many units: a block for every tpc tokens, and one more a prompt
    const int64_t units = ((n_tokens + QT * p.tpt - 1) / (QT * p.tpt) + batch) * kv_heads;
    const int grid = (int)(units < rc_host::sm_count() ? units : rc_host::sm_count());
    cudaStream_t st = (cudaStream_t)stream;
    return rc_host::launch_status(head_dim == 128 ? launch<128>(m, p, grid, st) : launch<64>(m, p, grid, st));
}
