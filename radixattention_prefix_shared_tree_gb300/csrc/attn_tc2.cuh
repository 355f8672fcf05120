// Many query rows over one gathered key list on tcgen05, warp-specialized:
// the kernel body of attn_extend (new tokens over their cached prefix, causal
// among themselves) and of the cascade step of attn_decode (a shared segment
// read once for every request below it).
//
// A CTA owns 256 query rows of one KV head -- two M=128 tiles, each (128/G
// tokens or requests) x (the G query heads of that KV head) -- so every K/V
// tile it gathers feeds both.  Eight softmax warps, NP producers (two for a
// bf16 pool, three for codes) and one for the tensor core, with fixed roles:
//   warps 0-3 and 4-7  softmax of query tile 0 and 1: one thread per row /
//                      TMEM lane; read S from TMEM, write P (bf16) back over
//                      it, rescale the row's O in TMEM when its max grows by
//                      more than 2^8; at the end normalise O and write it out;
//   warps 8..8+NP-1    producers, warp 8+i of the tiles t = i mod NP: gather
//                      K/V rows by slot id with 16-byte cp.async into a
//                      5-stage ring (no-swizzle operand layout), each lane's
//                      copies arriving on the stage's mbarrier when they
//                      land (their first tiles' before the set-up barrier);
//   warp 8+NP          issues every MMA (one elected lane of the converged
//                      warp) and owns TMEM.
// Per 64-key tile and query tile q:  S_q = Q_q K^T (M=128, N=64, K=D) into
// one of two S buffers, O_q += P_q V (M=128, N=D, K=64) with P read from
// tensor memory.  The next tile's S products are issued before this tile's
// P.V, so the tensor core works while the softmax warps run, and the softmax
// of tile t+1 does not wait for P.V of tile t (only a rescale of O does).
// TMEM: query tile q uses columns [256q, 256q+256): S buffers at +0 and +64
// (P over their first 32 columns), O at +128.  The tensor core runs one
// thread's MMAs in issue order, so S(t+2) overwrites P(t) only after P(t).V
// has read it.  All hand-offs are mbarriers; every wait is bounded and a wait
// that gives up flags RC_ERR_TIMEOUT.  The MMA warp builds each
// operand's descriptor once and steps it along K with 32-bit adds, and the
// producers' copies of a row carry their offsets as immediates, so neither
// spends issue slots on address arithmetic.
//
// FP8 pool (E4M3 codes, one fp32 scale per (slot, KV head) row): the products
// run in f16 (every E4M3 value is an f16 value; the bf16 queries convert
// exactly within f16's range).  The producers load codes with plain 16-byte
// loads, widen them to f16 in registers and store the operand tiles
// themselves (then fence to the async proxy and arrive), along with the
// tile's 64 K and 64 V scales; the softmax scales S by the K scales and folds
// the V scales into P, against a reference that keeps the products within f16's
// normal numbers (rc::scale_unit).  The ring has 4 stages (the scales take the
// room of the fifth).
//
// 4-bit pool (E2M1 codes, one scale byte per 16 of them): code times scale is
// itself an f16 value, so the stages hold the pool's exact values and the
// softmax is the bf16 pool's, with P in f16.  All three producers widen every
// tile (Fp4Feed), from codes that cp.async brought two tiles ahead; 4 stages.
//
// Cross attention (kCross): extend without the causal edge, every token of
// row z seeing all of the row's keys; with few rows of long keys the keys are
// split over seg_chunks CTAs that leave partials, as the cascade does.  So does
// extend over a 4-bit pool with few tokens.
#pragma once

#include "mq_attn.cuh"
#include "tc.cuh"

#include <type_traits>

namespace rc_tc2 {

constexpr int QT = 2;          // query tiles per CTA
constexpr int TM = 128;        // rows per query tile
constexpr int ROWS = QT * TM;  // query rows per CTA
constexpr int TN = 64;         // keys per tile
constexpr int NS_BF16 = 5;     // K/V stages
constexpr int NS_FP8 = 4;
constexpr int NS_FP4 = 4;
// Producer warps: two keep up with bf16 tiles, which they copy asynchronously; a
// third one measured no faster.  Codes pass through their registers, and two
// warps took longer over a tile than its products take.
template <int FMT>
__host__ __device__ constexpr int producers() { return FMT == rc::kFmtBf16 ? 2 : 3; }
template <int FMT>
__host__ __device__ constexpr int threads() { return 32 * (8 + producers<FMT>() + 1); }
constexpr uint32_t kWaitIter = 1u << 24;
template <int FMT>
__host__ __device__ constexpr int stages() {
    return FMT == rc::kFmtFp8 ? NS_FP8 : FMT == rc::kFmtFp4 ? NS_FP4 : NS_BF16;
}
template <int FMT>
__host__ __device__ constexpr int n_bars() { return 1 + 2 * stages<FMT>() + 4 + 4 + 2 + 1; }

// 4-bit pool: every producer warp takes every NP-th group of eight keys of every
// tile.  Its part of a tile as the pool holds it (K codes, V codes, K scales, V
// scales of RAW_ROWS keys), and how many of those it has on their way or at hand.
constexpr int RAW_ROWS = 8 * ((TN / 8 + 2) / 3);
template <int D>
__host__ __device__ constexpr int raw_bytes() { return 2 * RAW_ROWS * (D / 2 + D / 16); }
constexpr int RAW = 2;
template <int D, int FMT = rc::kFmtBf16>
__host__ __device__ constexpr int smem_bytes() {
    return QT * TM * D * 2 + stages<FMT>() * 2 * TN * D * 2 +
           (FMT == rc::kFmtFp8   ? stages<FMT>() * (2 * TN + 1) * 4
            : FMT == rc::kFmtFp4 ? producers<FMT>() * RAW * raw_bytes<D>()
                                 : 0) +
           n_bars<FMT>() * 8 + 16;
}

// The cascade path reads FP8 pools too.
inline constexpr bool fp8_cascade_supported() { return true; }

using tc::ex2;
using tc::fadd2;
using tc::ffma2;
using tc::max3;
using tc::mbar_arrive;

// The 4-bit pool's producer warps.  All of them widen every tile together: a
// stage is held from the start of its widening until P.V has read it, and one
// warp's ~2200 cycles for a tile were a third of that.  Codes and scales come by
// cp.async into the warp's own RAW parts, two tiles ahead, and are widened
// from there into the operand stage.  Every value is exact in f16.
template <int D, int NP>
struct Fp4Feed {
    static_assert(NP == 3 && TN == 64, "groups of eight keys per warp");
    static constexpr int CB = D / 2, SB = D / 16, CH = D / 8;
    static constexpr int CPR = CB / 16;        // 16-byte chunks per row
    static constexpr int RPI = 32 / CPR;       // rows one instruction copies
    const rc::MQParams& p;
    const int32_t* keys;
    int key_count, n_tiles, kvh, wi, lane;
    unsigned char* raw;
    uint32_t n_slots;
    uint64_t pol;

    // the tile's key of this warp's row r: groups wi, wi + NP, ...
    RC_DEV int key_of(int r) const { return ((r >> 3) * NP + wi) * 8 + (r & 7); }
    // chunk c of row r lies at chunk c ^ swz(r): eight rows' equal chunks then
    // touch every bank once
    RC_DEV static int swz(int r) { return D == 128 ? (r >> 1) & 3 : (r >> 2) & 1; }
    // whether row `lane` of this warp's part of tile t is a key (none of a tile past the last)
    RC_DEV bool has(int t) const {
        return lane < RAW_ROWS && key_of(lane) < TN && t * TN + key_of(lane) < key_count;
    }
    // lane r: the slot id of row r's key (-1 where there is none, which `has`
    // tells apart from a table entry of -1)
    RC_DEV int id_of(int t) const { return has(t) ? __ldg(keys + t * TN + key_of(lane)) : -1; }
    RC_DEV void fetch(int t, int id) const {
        if (t < n_tiles) {
            const uint32_t dst = rc::smem_u32(raw) + (t % RAW) * raw_bytes<D>();
            const int c = lane % CPR;
            const bool live = (uint32_t)id < n_slots;
            if (!live && has(t)) rc::flag_error(p.err, rc::kErrBadSlot);
            const int safe = live ? id : 0;
#pragma unroll
            for (int i = 0; i < (RAW_ROWS + RPI - 1) / RPI; ++i) {
                const int r = i * RPI + lane / CPR;
                const int s = __shfl_sync(0xffffffffu, safe, r & 31);
                const int64_t off = ((int64_t)s * p.kv_heads + kvh) * CB + c * 16;
                const uint32_t d = dst + r * CB + ((c ^ swz(r)) * 16);
                if (RAW_ROWS % RPI == 0 || r < RAW_ROWS) {
                    rc::cp_async16(d, reinterpret_cast<const unsigned char*>(p.pool_k) + off, 16u, pol);
                    rc::cp_async16(d + RAW_ROWS * CB, reinterpret_cast<const unsigned char*>(p.pool_v) + off, 16u, pol);
                }
            }
            if (lane < RAW_ROWS) {  // zero scales: past the end, and for a slot outside the pool
                const int64_t off = ((int64_t)safe * p.kv_heads + kvh) * SB;
                const uint32_t d = dst + 2 * RAW_ROWS * CB + lane * SB;
                rc::cp_async_small<SB>(d, p.k_bscale + off, live ? (uint32_t)SB : 0u);
                rc::cp_async_small<SB>(d + RAW_ROWS * SB, p.v_bscale + off, live ? (uint32_t)SB : 0u);
            }
        }
        rc::cp_async_commit();
    }
    // 32 codes under two scales per lane: eight neighbouring lanes hold eight
    // keys' equal chunks, so a 16-byte f16 store of theirs is 128 contiguous
    // bytes
    RC_DEV void widen(unsigned char* dst, const unsigned char* codes, const unsigned char* scales) const {
        constexpr int KPI = 32 / (D / 32);
        const int krow = lane & (KPI - 1), cq = lane / KPI;
#pragma unroll
        for (int i = 0; i < (RAW_ROWS + KPI - 1) / KPI; ++i) {
            const int r = i * KPI + krow, key = key_of(r);
            if (r >= RAW_ROWS || key >= TN) continue;
            const uint4 w = *reinterpret_cast<const uint4*>(codes + r * CB + ((cq ^ swz(r)) * 16));
            const uint32_t c = *reinterpret_cast<const uint16_t*>(scales + r * SB + 2 * cq);
            const uint32_t s0 = rc::scale_pair<0, 0>(c), s1 = rc::scale_pair<1, 1>(c);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 8 codes: f16 chunk 4 cq + k
                uint4 f;
                rc::e2m1x8_to_f16x8(x[k], f.x, f.y, f.z, f.w);
                const uint32_t sc = k < 2 ? s0 : s1;
                f.x = rc::mul_f16x2(f.x, sc);
                f.y = rc::mul_f16x2(f.y, sc);
                f.z = rc::mul_f16x2(f.z, sc);
                f.w = rc::mul_f16x2(f.w, sc);
                *reinterpret_cast<uint4*>(dst + tc::cm_offset(key, 4 * cq + k, CH)) = f;
            }
        }
    }
    // tile t from its raw part into the operand stage at dst
    RC_DEV void put(int t, unsigned char* dst) const {
        const unsigned char* src = raw + (t % RAW) * raw_bytes<D>();
        widen(dst, src, src + 2 * RAW_ROWS * CB);
        widen(dst + TN * D * 2, src + RAW_ROWS * CB, src + 2 * RAW_ROWS * CB + RAW_ROWS * SB);
    }
};

template <int D, int G, rc::MQMode MODE, int FMT = rc::kFmtBf16>
__global__ void __launch_bounds__(threads<FMT>(), 1) attn_tc2_kernel(const rc::MQParams p) {
    constexpr bool FP8 = FMT == rc::kFmtFp8, FP4 = FMT == rc::kFmtFp4;
    constexpr bool F16 = FP8 || FP4;             // operands in f16, widened from codes
    static_assert(!FP8 || D == 128, "FP8 pools: head_dim 128");
    constexpr int NP = producers<FMT>(), MMA_WARP = 8 + NP, THREADS = threads<FMT>();
    constexpr int NS = stages<FMT>();
    constexpr int kBars = n_bars<FMT>();
    constexpr int CH = D / 8;
    constexpr int TPC = ROWS / G;               // tokens (or requests) per CTA
    constexpr int KV_BYTES = TN * D * 2;
    constexpr uint32_t SB = CH * 128;            // bytes between 8-row groups of Q/K/V tiles
    constexpr uint32_t idS = F16 ? tc::idesc_f16(TM, TN, false) : tc::idesc_bf16(TM, TN, false);
    constexpr uint32_t idPV = F16 ? tc::idesc_f16(TM, D, true) : tc::idesc_bf16(TM, D, true);
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* sQ = smem;                                  // [QT][128 rows][D]
    unsigned char* sKV = sQ + QT * TM * D * 2;                 // [NS][K, V]
    float* sScale = reinterpret_cast<float*>(sKV + NS * 2 * KV_BYTES);  // FP8: [NS][K scales, V scales]
    float* sUnit = sScale + NS * 2 * TN;                                 // FP8: [NS] the unit of the V scales
    unsigned char* sRaw = sKV + NS * 2 * KV_BYTES;                       // FP4: [NP][RAW] tiles of codes and scales
    uint64_t* bar = reinterpret_cast<uint64_t*>(sKV + NS * 2 * KV_BYTES +
                                                (FP8 ? NS * (2 * TN + 1) * 4 : FP4 ? NP * RAW * raw_bytes<D>() : 0));
    uint64_t* q_full = bar + 0;              // count 8 (softmax warps)
    uint64_t* kv_full = bar + 1;             // [NS], count 32 (the lanes of the tile's producer warp; FP4: of all)
    uint64_t* kv_empty = bar + 1 + NS;       // [NS], count 1 (MMA commit)
    uint64_t* s_full = bar + 1 + 2 * NS;     // [QT][2], count 1
    uint64_t* p_full = s_full + 4;           // [QT][2] (one per S buffer), count 4 (the tile's softmax warps)
    uint64_t* o_done = p_full + 4;           // [QT], count 1
    uint64_t* drained = o_done + QT;         // count 1: products in flight when a wait gave up
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + kBars);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int kvh = blockIdx.y, z = blockIdx.z;
    int blk = blockIdx.x;
    // cascade: launched as the programmatic dependent of whatever precedes it
    // on the stream (the previous step's table pass), so its CTAs take SMs as
    // that grid drains; nothing is read before that grid has finished.  The
    // table pass of this call is in turn this grid's dependent: it may start
    // once every CTA here has begun (it waits for this grid's end before
    // reading the partials).
    // (early: the wait and the trigger move to just before the first global
    // write, see MQParams::early; the table pass then still launches only
    // after the preceding grid has finished)
    if constexpr (MODE == rc::MQMode::kCascade) {
        if (!p.early) {
            asm volatile("griddepcontrol.wait;\n" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
        }
    }
    // cascade: this CTA's segment, key chunk and the segment's chunk count.
    // With a compact grid (seg_items > 0) blockIdx.x is the item: one warp
    // walks the segments 32 at a time, each lane counting its segment's
    // (key chunk, row block) items, and a warp scan finds the segment that
    // holds this item (chunk-major inside a segment).
    int c_seg = 0, c_chunk = 0, c_nch = 1;
    if constexpr (MODE == rc::MQMode::kCascade) {
        if (p.seg_items > 0) {
            __shared__ int s_map[4];
            if (threadIdx.x < 32) {
                const int ln = threadIdx.x;
                const int target = blockIdx.x;
                int base = 0, found = -1, f_chunk = 0, f_blk = 0, f_nch = 1;
                for (int s0 = 0; s0 < p.n_seg && found < 0; s0 += 32) {
                    const int sg = s0 + ln;
                    int items = 0, rb = 1, ch = 1;
                    if (sg < p.n_seg) {
                        const int rows = p.seg_row_indptr[sg + 1] - p.seg_row_indptr[sg];
                        const int len = p.seg_indptr[sg + 1] - p.seg_indptr[sg];
                        rb = rows > 0 ? (rows + TPC - 1) / TPC : 1;
                        ch = len > 0 ? min((len + p.seg_chunk - 1) / p.seg_chunk, p.seg_chunks) : 1;
                        items = rows > 0 ? ch * rb : 0;
                    }
                    int incl = items;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, incl, o);
                        if (ln >= o) incl += v;
                    }
                    const int excl = base + incl - items;
                    const unsigned m = __ballot_sync(0xffffffffu, items > 0 && target >= excl && target < excl + items);
                    if (m) {
                        const int src = __ffs(m) - 1;
                        const int j = target - __shfl_sync(0xffffffffu, excl, src);
                        const int rb_s = __shfl_sync(0xffffffffu, rb, src);
                        f_nch = __shfl_sync(0xffffffffu, ch, src);
                        found = s0 + src;
                        f_chunk = j / rb_s;
                        f_blk = j % rb_s;
                    }
                    base += __shfl_sync(0xffffffffu, incl, 31);
                }
                if (ln == 0) {
                    s_map[0] = found;
                    s_map[1] = f_chunk;
                    s_map[2] = f_blk;
                    s_map[3] = f_nch;
                }
            }
            __syncthreads();
            if (s_map[0] < 0) {  // more items than the segments hold: the host arrays differ
                if (threadIdx.x == 0) rc::flag_error(p.err, rc::kErrBadSlot);
                return;
            }
            c_seg = s_map[0];
            c_chunk = s_map[1];
            blk = s_map[2];
            c_nch = s_map[3];
        } else {
            c_seg = z / p.seg_chunks;
            c_chunk = z % p.seg_chunks;
            c_nch = p.seg_chunks;
        }
    }
    const int tok0 = blk * TPC;

    // ---- this CTA's rows and keys (uniform)
    int n_rows_tok, key_count, prefix = 0, qo0, chunk = 0;
    const int32_t* keys;
    if constexpr (MODE == rc::MQMode::kExtend) {
        const int b = z / p.seg_chunks;
        chunk = z % p.seg_chunks;
        qo0 = p.qo_indptr[b];
        n_rows_tok = p.qo_indptr[b + 1] - qo0;
        const int L = p.len[b];
        prefix = L - n_rows_tok;
        const int64_t row0 = p.start[b];
        if (p.seg_chunks > 1 && (n_rows_tok > p.max_q || qo0 < 0 || (int64_t)qo0 + n_rows_tok > p.max_rows)) {
            if (tid == 0) rc::flag_error(p.err, rc::kErrBadSlot);  // more tokens than the partials have room for
            return;
        }
        if (tok0 >= n_rows_tok) return;
        if (row0 < 0 || prefix < 0 || row0 + L > p.table_len || (p.seg_chunks > 1 && L > p.max_len)) {
            if (tid == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            if (p.seg_chunks > 1)  // (the merge reads what is written here)
                for (int i = tid; i < min(n_rows_tok - tok0, TPC) * G; i += THREADS)
                    p.part_lse[((int64_t)(qo0 + tok0 + i / G) * p.q_heads + kvh * G + i % G) * p.seg_chunks + chunk] =
                        -INFINITY;
            return;
        }
        const int k0 = chunk * p.seg_chunk;
        prefix -= k0;  // the first token's position, counted from the chunk's first key
        keys = p.table + row0 + k0;
        key_count = prefix + min(n_rows_tok, tok0 + TPC);
        if (p.seg_chunks > 1) {
            key_count = min(key_count, p.seg_chunk);
            if (key_count <= 0) {  // none of these tokens sees a key of the chunk
                for (int i = tid; i < min(n_rows_tok - tok0, TPC) * G; i += THREADS)
                    p.part_lse[((int64_t)(qo0 + tok0 + i / G) * p.q_heads + kvh * G + i % G) * p.seg_chunks + chunk] =
                        -INFINITY;
                return;
            }
        }
    } else if constexpr (MODE == rc::MQMode::kCross) {
        const int b = z / p.seg_chunks;
        chunk = z % p.seg_chunks;
        qo0 = p.qo_indptr[b];
        n_rows_tok = p.qo_indptr[b + 1] - qo0;
        // more tokens than the caller's bounds (they size the grid and the
        // partials): none of the row's is computed
        if (n_rows_tok > p.max_q || qo0 < 0 || (int64_t)qo0 + n_rows_tok > p.max_rows) {
            if (tid == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            return;
        }
        if (tok0 >= n_rows_tok) return;
        const int64_t row0 = p.start[b];
        int L = p.len[b];
        if (row0 < 0 || L < 0 || row0 + L > p.table_len || L > p.max_len) {  // not read: as an empty row
            if (tid == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            L = 0;
        }
        const int k0 = chunk * p.seg_chunk;
        keys = p.table + row0 + k0;
        key_count = min(L - k0, p.seg_chunk);
        if (key_count <= 0) {  // nothing to attend to: a zero output, or an empty partial
            for (int i = tid; i < min(n_rows_tok - tok0, TPC) * G; i += THREADS) {
                const int64_t r = (int64_t)(qo0 + tok0 + i / G) * p.q_heads + kvh * G + i % G;
                if (p.seg_chunks > 1) {
                    p.part_lse[r * p.seg_chunks + chunk] = -INFINITY;
                } else {
                    for (int c = 0; c < CH; ++c)
                        reinterpret_cast<uint4*>(p.out + r * D)[c] = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[r] = -INFINITY;
                }
            }
            return;
        }
    } else {
        const int seg = c_seg;
        chunk = c_chunk;
        qo0 = p.seg_row_indptr[seg];
        n_rows_tok = p.seg_row_indptr[seg + 1] - qo0;
        const int k0 = chunk * p.seg_chunk;
        keys = p.seg_slots + p.seg_indptr[seg] + k0;
        key_count = min(p.seg_indptr[seg + 1] - p.seg_indptr[seg] - k0, p.seg_chunk);
        if (tok0 >= n_rows_tok) return;
        // compact grid: no CTA runs past the segment's last chunk, so its
        // first chunk's CTA marks those partials empty for its rows
        if (p.seg_items > 0 && !p.early && chunk == 0 && c_nch < p.seg_chunks && tid < ROWS) {
            const int tk = tok0 + tid / G;
            if (tk < n_rows_tok)
                for (int c = c_nch; c < p.seg_chunks; ++c)
                    p.part_lse[((int64_t)(qo0 + tk) * p.q_heads + kvh * G + (tid % G)) * p.seg_chunks + c] = -INFINITY;
        }
        if (key_count <= 0) {  // segment shorter than this chunk: an empty partial
            if (p.early) {
                asm volatile("griddepcontrol.wait;\n" ::: "memory");
                asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
                if (p.seg_items > 0 && chunk == 0 && tid < ROWS) {
                    const int tk = tok0 + tid / G;
                    if (tk < n_rows_tok)
                        for (int c = c_nch; c < p.seg_chunks; ++c)
                            p.part_lse[((int64_t)(qo0 + tk) * p.q_heads + kvh * G + (tid % G)) * p.seg_chunks + c] =
                                -INFINITY;
                }
            }
            if (tid < ROWS) {
                const int tk = tok0 + tid / G;
                if (tk < n_rows_tok)
                    p.part_lse[((int64_t)(qo0 + tk) * p.q_heads + kvh * G + (tid % G)) * p.seg_chunks + chunk] =
                        -INFINITY;
            }
            return;
        }
    }
    // a wait gave up in an earlier CTA: the results are void (looked at at the
    // set-up barrier)
    const int gave_up = p.err && (*reinterpret_cast<volatile int32_t*>(p.err) & rc::kErrTimeout);
    const int n_tiles = (key_count + TN - 1) / TN;
    // query tiles with at least one valid row
    const int n_qt = min(QT, ((min(n_rows_tok - tok0, TPC) * G) + TM - 1) / TM);

    // set-up by the MMA warp, which has no loads of its own on their way (the
    // fence would wait for them)
    if (warp == MMA_WARP) {
        if (lane == 0) {
            tc::mbar_init(q_full, 8);
            for (int s = 0; s < NS; ++s) {
                tc::mbar_init(&kv_full[s], FP4 ? 32 * NP : 32);
                tc::mbar_init(&kv_empty[s], 1);
            }
            for (int i = 0; i < 4; ++i) {
                tc::mbar_init(&s_full[i], 1);
                tc::mbar_init(&p_full[i], 4);
            }
            for (int q = 0; q < QT; ++q) {
                tc::mbar_init(&o_done[q], 1);
            }
            tc::mbar_init(drained, 1);
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(tslot, 512);
        tc::tmem_relinquish();
    }
    // Producers: their first tiles' copies go out before the set-up barrier, which
    // their latency then overlaps (a stage's first use waits for nothing).
    // Keys here are shared: by the CTAs of the other row blocks, and (a cached
    // prefix) by later steps -- keep them in L2.
    const uint64_t pol = rc::l2_policy_evict_last();
    const int t0 = warp - 8;  // this producer's first tile
    auto load_ids = [&](int t, int (&sl)[2]) {
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
            const int key = t * TN + lane + 32 * h2;
            sl[h2] = (t < n_tiles && key < key_count) ? __ldg(keys + key) : -1;
        }
    };
    auto copy_tile = [&](int t, const int (&sl)[2]) {  // bf16 pool: tile t into its stage
        // lane -> (key within an 8-key group, 16-byte column within a group of 4)
        const int klo = lane & 7, csub = lane >> 3;
        unsigned char* sK = sKV + (t % NS) * 2 * KV_BYTES;
        unsigned char* sV = sK + KV_BYTES;
#pragma unroll
        for (int kg = 0; kg < TN / 8; ++kg) {
            const int key = kg * 8 + klo;
            int slot = __shfl_sync(0xffffffffu, sl[kg >> 2], (kg & 3) * 8 + klo);
            uint32_t bytes = 16;
            if (t * TN + key >= key_count) { slot = 0; bytes = 0; }
            else if (slot < 0 || (int64_t)slot >= p.n_slots) {
                rc::flag_error(p.err, rc::kErrBadSlot);
                slot = 0;
                bytes = 0;
            }
            // chunks c = 4 cg + csub: 512 bytes apart in the stage, 64 in the row
            const int64_t base = ((int64_t)slot * p.kv_heads + kvh) * D + csub * 8;
            const uint32_t off = tc::cm_offset(key, csub, CH);
            rc::cp_async16_run<512, 64>(rc::smem_u32(sK) + off, p.pool_k + base, bytes, pol,
                                        std::make_integer_sequence<int, CH / 4>{});
            rc::cp_async16_run<512, 64>(rc::smem_u32(sV) + off, p.pool_v + base, bytes, pol,
                                        std::make_integer_sequence<int, CH / 4>{});
        }
    };
    const Fp4Feed<D, 3> feed{p, keys, key_count, n_tiles, kvh, t0, lane, sRaw + (FP4 ? t0 * RAW * raw_bytes<D>() : 0),
                             (uint32_t)min(p.n_slots, (int64_t)0x7fffffff), pol};
    int feed_id = -1, sl[2] = {-1, -1};
    if (warp >= 8 && warp < MMA_WARP) {
        if constexpr (FP4) {
            int first[RAW];
#pragma unroll
            for (int i = 0; i < RAW; ++i) first[i] = feed.id_of(i);
            feed_id = feed.id_of(RAW);
#pragma unroll
            for (int i = 0; i < RAW; ++i) feed.fetch(i, first[i]);
        } else {
            load_ids(t0, sl);
            if constexpr (!F16)
                if (t0 < n_tiles) copy_tile(t0, sl);
        }
    }
    uint4 qv[F16 ? CH : 1];
    if (warp < 8) {
        // Q rows of query tile warp/4, issued first so that their latency
        // overlaps the set-up.  The row indices (cascade: a gather through
        // seg_rows) are all loaded before the first copy is issued.
        const int q = warp >> 2, r = tid & 127;
        unsigned char* sQq = sQ + q * TM * D * 2;
        int64_t qrow[CH];
        bool qok[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int gi = r + 128 * i;
            const int rr = (gi & 7) + 8 * (gi / (8 * CH));
            const int qr = q * TM + rr;
            const int tk = tok0 + qr / G;
            const int h = kvh * G + (qr % G);
            qok[i] = tk < n_rows_tok;
            if constexpr (MODE != rc::MQMode::kCascade) qrow[i] = (int64_t)(qo0 + tk) * p.q_heads + h;
            else qrow[i] = qok[i] ? (int64_t)__ldg(p.seg_rows + qo0 + tk) * p.q_heads + h : 0;
            if (!qok[i]) qrow[i] = 0;
        }
        if constexpr (F16) {  // f16 operand: loaded here, converted and stored after the barrier
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = ((r + 128 * i) >> 3) % CH;
                qv[i] = qok[i] ? __ldg(reinterpret_cast<const uint4*>(p.q + qrow[i] * D + c * 8)) : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int gi = r + 128 * i;
                const int rr = (gi & 7) + 8 * (gi / (8 * CH));
                const int c = (gi >> 3) % CH;
                rc::cp_async16(rc::smem_u32(sQq + tc::cm_offset(rr, c, CH)), p.q + qrow[i] * D + c * 8,
                               qok[i] ? 16u : 0u);
            }
            rc::cp_async_commit();
        }
    }
    tc::fence_before();
    const int leave = __syncthreads_or(gave_up);
    tc::fence_after();
    const uint32_t tbase = *tslot;
    if (leave) {  // all threads alike (the word can change between two threads' reads)
        rc::cp_async_wait<0>();
        __syncthreads();
        if (warp == MMA_WARP) tc::tmem_dealloc(tbase, 512);
        return;
    }
    bool ok = true;

    if (warp < 8) {
        // ================================================= softmax warpgroups
        const int q = warp >> 2;             // query tile
        const int r = tid & 127;             // row within the tile = TMEM lane
        const int row = q * TM + r;          // row within the CTA
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tq = tbase + q * 256 + lane_off;
        if constexpr (F16) {
            unsigned char* sQq = sQ + q * TM * D * 2;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int gi = r + 128 * i;
                const int rr = (gi & 7) + 8 * (gi / (8 * CH));
                const int c = (gi >> 3) % CH;
                *reinterpret_cast<uint4*>(sQq + tc::cm_offset(rr, c, CH)) =
                    make_uint4(rc::bf16x2_to_f16x2(qv[i].x), rc::bf16x2_to_f16x2(qv[i].y),
                               rc::bf16x2_to_f16x2(qv[i].z), rc::bf16x2_to_f16x2(qv[i].w));
            }
        }
        rc::cp_async_wait<0>();  // this thread's Q chunks (issued before the set-up)
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);

        const int r_tok = tok0 + row / G;
        const bool row_valid = r_tok < n_rows_tok;
        int lim;
        if constexpr (MODE == rc::MQMode::kExtend) lim = row_valid ? prefix + r_tok + 1 : 0;
        else lim = row_valid ? key_count : 0;
        const float sc = p.scale_log2;
        float m_used = -INFINITY, l_run = 0.f;
        float unit = 0.f;  // FP8: O and l are in units of 2^unit (rc::scale_unit)
        if (q < n_qt) {
            for (int t = 0; t < n_tiles && ok; ++t) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[q * 2 + (t & 1)], (t >> 1) & 1, kWaitIter));
                tc::fence_after();
                const uint32_t tS = tq + (t & 1) * TN;
                uint32_t sa[32], sb[32];
                tc::tmem_ld32_issue(tS, sa);
                tc::tmem_ld32_issue(tS + 32, sb);
                tc::tmem_ld_wait(sa);
                tc::tmem_ld_wait(sb);
                float s[TN];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    s[j] = __uint_as_float(sa[j]);
                    s[32 + j] = __uint_as_float(sb[j]);
                }
                const float* tsc = sScale + (t % NS) * 2 * TN;  // FP8: this tile's K then V scales
                float u = 0.f;                                  // and their unit
                if constexpr (FP8) {
                    // the producer's scale stores are visible once its arrival
                    // on the stage is (that phase completed before S(t) ran)
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_full[t % NS], (t / NS) & 1, kWaitIter)) && ok;
#pragma unroll
                    for (int j = 0; j < TN; ++j) s[j] *= tsc[j];
                    u = sUnit[t % NS];
                    if (t == 0) unit = u;
                }
                const int kb = t * TN;
                if (kb + TN > lim) {  // the causal edge or the end of the keys
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        if (kb + j >= lim) s[j] = -INFINITY;
                }
                float m8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m8[i] = max3(s[i], s[8 + i], s[16 + i]);
                    m8[i] = max3(m8[i], s[24 + i], s[32 + i]);
                    m8[i] = max3(m8[i], s[40 + i], s[48 + i]);
                    m8[i] = fmaxf(m8[i], s[56 + i]);
                }
                const float mraw = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                const float mt = mraw * sc;  // sc > 0: the max of the scaled row
                const bool grow = mt > m_used + 8.f;
                const bool rescale_o = grow && m_used != -INFINITY;
                const bool larger = FP8 && u > unit;  // all rows alike: a tile of a larger unit than O's
                if (larger || __any_sync(0xffffffffu, rescale_o)) {
                    // O must be stable: the previous tile's P.V has completed
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_done[q], (t - 1) & 1, kWaitIter)) && ok;
                    tc::fence_after();
                    float a = rescale_o ? ex2(m_used - mt) : 1.f;
                    if (larger) {
                        a = rc::to_unit(a, (int)unit, (int)u);
                        l_run = rc::to_unit(l_run, (int)unit, (int)u);
                        unit = u;
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tc::tmem_ld32_issue(tq + 128 + c * 32, v);
                        tc::tmem_ld_wait(v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * a);
                        tc::tmem_st32_issue(tq + 128 + c * 32, v);
                    }
                    tc::tmem_st_wait();
                }
                if (grow) {
                    l_run *= ex2(m_used - mt);  // 0 while nothing was seen
                    m_used = mt;
                }
                const float nmu = (m_used == -INFINITY ? 0.f : -m_used) - (FP8 ? unit : 0.f);
                uint32_t pk[32];
                float2 ls[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 x = ffma2(make_float2(s[2 * i], s[2 * i + 1]), sc, nmu);
                    const float2 e = make_float2(ex2(x.x), ex2(x.y));
                    ls[i & 3] = fadd2(ls[i & 3], e);
                    // P to the type of V's operand (one product takes one type): bf16
                    // keeps 8 bits of a weight, f16 11; the sum keeps the fp32 terms
                    if constexpr (FP8) pk[i] = rc::pack_f16(e.x * tsc[TN + 2 * i], e.y * tsc[TN + 2 * i + 1]);
                    else if constexpr (FP4) pk[i] = rc::pack_f16(e.x, e.y);
                    else pk[i] = rc::pack_bf16(e.x, e.y);
                }
                // P (bf16) over the first half of this S buffer: the A operand of P.V
                tc::tmem_st32_issue(tS, pk);
                const float2 l01 = fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3]));
                l_run += l01.x + l01.y;
                tc::tmem_st_wait();
                // Last tile: see P(n-2).V done before handing over P(n-1), while
                // o_done can only be at phase n-2 or n-1 (a parity wait tells
                // two phases apart, not three; S(n-1) guarantees P(n-3).V).
                if (t == n_tiles - 1 && t > 0) {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_done[q], (t - 1) & 1, kWaitIter)) && ok;
                    tc::fence_after();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[q * 2 + (t & 1)]);
            }
            // the last P.V: o_done is at phase n-1 or n here
            if (ok && n_tiles > 0)
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_done[q], (n_tiles - 1) & 1, kWaitIter));
            tc::fence_after();
        }
        if (!ok) rc::flag_error(p.err, rc::kErrTimeout);
        if constexpr (MODE == rc::MQMode::kCascade) {
            if (p.early) {  // the partials below are what the preceding grid read
                asm volatile("griddepcontrol.wait;\n" ::: "memory");
                asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
                if (p.seg_items > 0 && chunk == 0 && c_nch < p.seg_chunks) {
                    const int tk = tok0 + tid / G;  // tid < ROWS here
                    if (tk < n_rows_tok)
                        for (int c = c_nch; c < p.seg_chunks; ++c)
                            p.part_lse[((int64_t)(qo0 + tk) * p.q_heads + kvh * G + (tid % G)) * p.seg_chunks + c] =
                                -INFINITY;
                }
            }
        }
        // ---- epilogue: normalised O rows and their log-sum-exp.  Each thread
        // has a row; it goes out through the warp's 8 KB of its own query
        // tile's Q (free once the tile's last P.V is done, since every S
        // product was issued before it), so that a store instruction writes
        // whole rows: a row's 16-byte chunks XOR-swizzled by the row, so that
        // neither side meets a bank twice.  (Straight from the registers every
        // instruction would touch 32 rows, one tag each: 2.6 us a CTA.)
        if (q < n_qt) {
            const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
            const float lse2 = rc::log2_sum(FP8 ? m_used + unit : m_used, l_run);
            const bool whole = MODE != rc::MQMode::kCascade && p.seg_chunks == 1;
            unsigned char* stg = sQ + warp * 32 * D * 2;
            // n 16-byte chunks of every row of the warp, staged, to row `rw` of dst
            // (its rows `stride` 16-byte units apart)
            auto write_rows = [&](auto n_, uint4* dst, int64_t stride, int64_t extra) {
                constexpr int N = decltype(n_)::value;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int lr = i * (32 / N) + lane / N, c = lane % N;
                    const uint4 v = *reinterpret_cast<const uint4*>(stg + lr * N * 16 + ((c ^ (lr & 7)) * 16));
                    const int cr = q * TM + (warp & 3) * 32 + lr, tk = tok0 + cr / G;  // row within the CTA, its token
                    if (!ok || tk >= n_rows_tok) continue;
                    uint4* d = dst + ((int64_t)(qo0 + tk) * p.q_heads + kvh * G + cr % G) * stride + extra + c;
                    if (whole && !p.out_wide) {  // out aligned to 8 bytes only
                        reinterpret_cast<uint2*>(d)[0] = make_uint2(v.x, v.y);
                        reinterpret_cast<uint2*>(d)[1] = make_uint2(v.z, v.w);
                    } else {
                        *d = v;
                    }
                }
                __syncwarp();
            };
            if (whole) {
                constexpr int N = D / 8;
#pragma unroll 1
                for (int c0 = 0; c0 < D / 32; ++c0) {
                    uint32_t v[32];
                    tc::tmem_ld32_issue(tq + 128 + c0 * 32, v);
                    tc::tmem_ld_wait(v);
                    auto x = [&](int i) { return __uint_as_float(v[i]) * inv; };
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(stg + lane * N * 16 + (((c0 * 4 + k) ^ (lane & 7)) * 16)) =
                            make_uint4(rc::pack_bf16(x(8 * k), x(8 * k + 1)), rc::pack_bf16(x(8 * k + 2), x(8 * k + 3)),
                                       rc::pack_bf16(x(8 * k + 4), x(8 * k + 5)), rc::pack_bf16(x(8 * k + 6), x(8 * k + 7)));
                }
                write_rows(std::integral_constant<int, N>{}, reinterpret_cast<uint4*>(p.out), N, 0);
            } else {  // fp32 partials, 32 columns (128 bytes a row) at a time
#pragma unroll 1
                for (int c0 = 0; c0 < D / 32; ++c0) {
                    uint32_t v[32];
                    tc::tmem_ld32_issue(tq + 128 + c0 * 32, v);
                    tc::tmem_ld_wait(v);
                    auto x = [&](int i) { return __uint_as_float(v[i]) * inv; };
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4*>(stg + lane * 128 + ((k ^ (lane & 7)) * 16)) =
                            make_float4(x(4 * k), x(4 * k + 1), x(4 * k + 2), x(4 * k + 3));
                    write_rows(std::integral_constant<int, 8>{}, reinterpret_cast<uint4*>(p.part_o),
                               (int64_t)p.seg_chunks * D / 4, (int64_t)chunk * D / 4 + c0 * 8);
                }
            }
            if (ok && row_valid) {
                const int h = kvh * G + (row % G);
                if (whole) {
                    if (p.lse) p.lse[(int64_t)(qo0 + r_tok) * p.q_heads + h] = lse2 * rc::kLn2;
                } else {
                    p.part_lse[((int64_t)(qo0 + r_tok) * p.q_heads + h) * p.seg_chunks + chunk] = lse2;
                }
            }
        }
    } else if (warp < MMA_WARP) {
        // ============================================== producers (NP warps)
        // warp 8+i loads the tiles t = i mod NP, each as far ahead as free
        // stages allow (completion is signalled on the stage's barrier by the
        // copies themselves), reading the slot ids of its next tile one tile
        // ahead.
        if constexpr (FP4) {
            int s = 0, ph = 1;  // stage, and the parity of the wait for it (its first use waits for nothing)
            for (int t = 0; t < n_tiles && ok; ++t) {
                const int ahead = feed.id_of(t + RAW + 1);
                if (t >= NS) ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_empty[s], ph, kWaitIter));
                if (!ok) break;
                rc::cp_async_wait<RAW - 1>();
                __syncwarp();
                feed.put(t, sKV + s * 2 * KV_BYTES);
                tc::fence_proxy_async();  // this lane's stores, before the tensor core reads them
                mbar_arrive(&kv_full[s]);
                __syncwarp();  // every lane has read the raw tile
                feed.fetch(t + RAW, feed_id);
                feed_id = ahead;
                if (++s == NS) s = 0, ph ^= 1;
            }
        }
        int sl_next[2];
        for (int t = FP4 ? n_tiles : t0; t < n_tiles && ok; t += NP) {
            const int s = t % NS;
            load_ids(t + NP, sl_next);
            if (t >= NS) ok = __all_sync(0xffffffffu, tc::mbar_wait(&kv_empty[s], ((t / NS) + 1) & 1, kWaitIter));
            if (!ok) break;
            unsigned char* sK = sKV + s * 2 * KV_BYTES;
            unsigned char* sV = sK + KV_BYTES;
            if constexpr (FP8) {
                const int klo = lane & 7, csub = lane >> 3;
                // 16 E4M3 codes per load (8 keys x 64 bytes per instruction,
                // so the 16-byte f16 stores of 8 keys are 128 contiguous bytes);
                // the K and V loads of the tile are all in flight together
                uint4 w2[2][TN / 8][2];
#pragma unroll
                for (int kg = 0; kg < TN / 8; ++kg) {
                    const int key = kg * 8 + klo;
                    int slot = __shfl_sync(0xffffffffu, sl[kg >> 2], (kg & 3) * 8 + klo);
                    bool live = t * TN + key < key_count;
                    if (live && (slot < 0 || (int64_t)slot >= p.n_slots)) {
                        rc::flag_error(p.err, rc::kErrBadSlot);
                        live = false;
                    }
                    const int64_t base = ((int64_t)(live ? slot : 0) * p.kv_heads + kvh) * D;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const unsigned char* src = reinterpret_cast<const unsigned char*>(m ? p.pool_v : p.pool_k);
#pragma unroll
                        for (int cg = 0; cg < 2; ++cg)
                            w2[m][kg][cg] = live ? __ldg(reinterpret_cast<const uint4*>(src + base + (cg * 4 + csub) * 16))
                                                 : make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    unsigned char* dst = m ? sV : sK;
                    auto& w = w2[m];
#pragma unroll
                    for (int kg = 0; kg < TN / 8; ++kg) {
                        const int key = kg * 8 + klo;
#pragma unroll
                        for (int cg = 0; cg < 2; ++cg) {
                            const int c8 = cg * 4 + csub;  // 16-code chunk: f16 chunks 2*c8, 2*c8+1
                            const uint4 x = w[kg][cg];
                            uint4 f0, f1;
                            rc::e4m3x4_to_f16x4(x.x, f0.x, f0.y);
                            rc::e4m3x4_to_f16x4(x.y, f0.z, f0.w);
                            rc::e4m3x4_to_f16x4(x.z, f1.x, f1.y);
                            rc::e4m3x4_to_f16x4(x.w, f1.z, f1.w);
                            *reinterpret_cast<uint4*>(dst + tc::cm_offset(key, 2 * c8, CH)) = f0;
                            *reinterpret_cast<uint4*>(dst + tc::cm_offset(key, 2 * c8 + 1, CH)) = f1;
                        }
                    }
                }
                float* tsc = sScale + s * 2 * TN;
                uint32_t top = 0;  // the bits of the largest V scale
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    const int key = lane + 32 * h2;
                    const int slot = sl[h2];
                    const bool live = t * TN + key < key_count && slot >= 0 && (int64_t)slot < p.n_slots;
                    const int64_t row = (int64_t)(live ? slot : 0) * p.kv_heads + kvh;
                    tsc[key] = live ? __ldg(p.k_scale + row) : 0.f;
                    const float vs = live ? __ldg(p.v_scale + row) : 0.f;
                    tsc[TN + key] = vs;
                    top = max(top, rc::abs_bits(vs));
                }
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) sUnit[s] = (float)rc::scale_unit(top);
                tc::fence_proxy_async();  // this lane's stores, before the tensor core reads them
                mbar_arrive(&kv_full[s]);
            }
            if constexpr (!F16) {
                if (t > t0) copy_tile(t, sl);  // (the first went out before the set-up)
                // each lane arrives on the stage's barrier when its copies have
                // landed; the warp goes on to the next tile at once
                tc::cp_async_mbar_arrive(&kv_full[s]);
            }
            sl[0] = sl_next[0];
            sl[1] = sl_next[1];
        }
        rc::cp_async_wait<0>();  // nothing in flight when the warp leaves
        if (!ok) rc::flag_error(p.err, rc::kErrTimeout);
    } else {
        // ================================================= MMA (warp 8+NP)
        // The whole warp runs the loop and one elected lane issues, so that the
        // descriptors (built once per operand, stepped along K by 32-bit adds)
        // stay in uniform registers, where the instruction wants them: from a
        // lane of its own each product cost ~85 cycles to issue against the
        // ~53 (N = 64) and 64 (N = 128) that it runs.  A barrier's state is asked
        // for before the products ahead of its use are issued, which hides
        // the answer's ~60 cycles behind them.
        const bool lead = tc::elect_one();
        const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
        const int nt = __shfl_sync(0xffffffffu, n_tiles, 0), nq = __shfl_sync(0xffffffffu, n_qt, 0);
        const tc::Desc qd = tc::desc_halves(rc::smem_u32(sQ), 128, SB);
        const tc::Desc kd = tc::desc_halves(rc::smem_u32(sKV), 128, SB);
        const tc::Desc vd = tc::desc_halves(rc::smem_u32(sKV + KV_BYTES), SB, 128);
        constexpr uint32_t STEP = 2 * KV_BYTES / 16;  // from a stage to the next
        auto issue_s = [&](int t, int st) {
            const uint32_t klo = kd.lo + st * STEP, ds = tb + (t & 1) * TN;
#pragma unroll
            for (int q = 0; q < QT; ++q) {
                if (q < nq && lead) {
                    const uint32_t qlo = qd.lo + q * (TM * D * 2 / 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc::mma_bf16_h(ds + q * 256, qlo + k * 16, qd.hi, klo + k * 16, kd.hi, idS, k > 0 ? 1u : 0u);
                    tc::commit(&s_full[q * 2 + (t & 1)]);
                }
            }
        };
        // waits for a phase that `asked` may have seen complete already
        auto wait = [&](uint32_t asked, uint64_t* bar_, uint32_t parity) {
            ok = __all_sync(0xffffffffu, asked != 0 || tc::mbar_wait(bar_, parity, kWaitIter));
            tc::fence_after();
        };
        wait(0, q_full, 0);
        if (ok && nt > 0) {
            wait(0, &kv_full[0], 0);
            if constexpr (!F16) tc::fence_proxy_async();  // the rows came by cp.async; the tensor core reads them
            if (ok) issue_s(0, 0);
        }
        int st = 0, ph = 0;                // tile t's stage, and how often it was used before (parity)
        for (int t = 0; t < nt && ok; ++t) {
            const int st1 = st + 1 == NS ? 0 : st + 1, ph1 = st + 1 == NS ? ph ^ 1 : ph;
            if (t + 1 < nt) {  // next tile's S products first: they run during this softmax
                wait(0, &kv_full[st1], ph1);
                if constexpr (!F16) tc::fence_proxy_async();
                if (!ok) break;
            }
            uint32_t asked = tc::mbar_test(&p_full[t & 1], (t >> 1) & 1);
            if (t + 1 < nt) issue_s(t + 1, st1);
            const uint32_t vlo = vd.lo + st * STEP, acc = t > 0 ? 1u : 0u;
#pragma unroll
            for (int q = 0; q < QT; ++q) {
                if (q >= nq || !ok) break;
                wait(asked, &p_full[q * 2 + (t & 1)], (t >> 1) & 1);
                if (!ok) break;
                if (q + 1 < nq) asked = tc::mbar_test(&p_full[(q + 1) * 2 + (t & 1)], (t >> 1) & 1);
                const uint32_t pt = tb + q * 256 + (t & 1) * TN;  // P(t) in TMEM, 8 columns per 16 keys
                if (lead) {
#pragma unroll
                    for (int j = 0; j < TN / 16; ++j)
                        tc::mma_bf16_ts_h(tb + q * 256 + 128, pt + j * 8, vlo + j * (2 * SB / 16), vd.hi, idPV,
                                          j > 0 ? 1u : acc);
                    tc::commit(&o_done[q]);
                }
            }
            // the stage is free once everything issued so far is done (a last use
            // has nobody to tell, and the CTA must not leave an arrival behind)
            if (lead && t + NS < nt) tc::commit(&kv_empty[st]);
            st = st1;
            ph = ph1;
        }
        if (!ok) {
            if (lead) {
                rc::flag_error(p.err, rc::kErrTimeout);
                tc::commit(drained);
            }
            tc::mbar_wait(drained, 0, kWaitIter);  // the products read stages and write TMEM
        }
        __syncwarp();
    }
    if constexpr (MODE == rc::MQMode::kCascade) {
        if (p.early) {  // every thread of the CTA has waited and triggered before it leaves
            asm volatile("griddepcontrol.wait;\n" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc::fence_after();
        tc::tmem_dealloc(tbase, 512);
    }
}

}  // namespace rc_tc2
