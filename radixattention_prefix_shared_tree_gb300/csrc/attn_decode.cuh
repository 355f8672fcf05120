// What the table passes of attn_decode and attn_cross share (attn_decode.cu,
// attn_decode_fp4.cuh, attn_cross.cu): their parameters, the item a warp
// works on, and the epilogue that writes its result or folds in the row's
// cascade partials.
#pragma once

#include "common.cuh"

namespace rc_dec {

constexpr int kDecKeys = 64;    // chunk sizes are multiples of this

struct DecParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* pool_k;
    const __nv_bfloat16* pool_v;
    int64_t n_slots;
    int32_t kv_heads, q_heads;
    float scale_log2;
    int32_t* err;
    const int32_t* table;
    const int32_t* start;
    const int32_t* len;
    int64_t table_len;
    int32_t chunk;       // keys per CTA
    int32_t n_chunks;    // max chunks per request (partial stride)
    float* part_o;       // [B][Hq][n_chunks][D]      (unfused)
    float* part_lse;     // [B][Hq][n_chunks]
    // fused epilogue: combine with the cascade partials and write the result
    const float* seg_o;  // [total_seg_rows][Hq][seg_chunks][D]
    const float* seg_lse;
    const int32_t* req_seg_indptr;  // NULL: no cascade
    const int32_t* req_seg_pos;
    int32_t seg_chunks;
    __nv_bfloat16* out;
    float* lse;
    // attn_decode_append: each row's last key comes from here and is stored
    const __nv_bfloat16* k_new;  // [B][kv_heads][D] or NULL
    const __nv_bfloat16* v_new;
    // FP8 pool: pool_k / pool_v hold E4M3 codes, these the per-row scales
    const float* k_scale;  // [n_slots][kv_heads]
    const float* v_scale;
    // 4-bit pool: E2M1 codes, and their block scales
    const uint8_t* k_bscale;  // [n_slots][kv_heads][D / 16]
    const uint8_t* v_bscale;
    // cross attention: row b's queries are tokens qo_indptr[b] .. [b+1), and
    // the caller's bounds on a row's tokens, all tokens and a row's keys
    const int32_t* qo_indptr;
    int32_t group;       // query heads per KV head
    // 4-bit pool, split rows: n_chunks is the number of runs and part_o is
    // [runs + batch][kv_heads][columns][D] (attn_decode_fp4.cuh)
    int32_t batch;
    int32_t* row_runs;   // [batch][2]: first and last run that touch the row
    int32_t max_q;
    int32_t max_len;
    int64_t max_rows;
};

// Wait until the grid this one depends on programmatically (the cascade
// kernel) has finished and its writes are visible; returns at once when the
// grid was launched without that dependency.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// One warp's work: columns 0..ncol-1 (query rows) over keys [k0, k0 + count)
// of request b's table row, for one KV head.  Decode: the columns are the G
// query heads of the KV head.  CROSS: NC columns at most, the (token, head)
// pairs of the request's tokens, token-major.
struct Item {
    int b, kvh, chunk, ncol, L, k0, count;
    int64_t row0;        // the row's first entry in the table
    int64_t qrow0;       // CROSS: flat (token, head) row of column 0
    template <int NC, bool CROSS>
    RC_DEV int64_t qrow(const DecParams& p, int c) const {  // column c's
        return CROSS ? qrow0 + (int64_t)(c / p.group) * p.q_heads + c % p.group
                     : (int64_t)b * p.q_heads + kvh * NC + c;
    }
};

// Item `it` of the grid; L = 0 and a flagged error where the row is outside
// the table.  CROSS: ncol = 0 where there is nothing to write.
template <int NC, bool FUSED, bool CROSS>
RC_DEV Item decode_item(const DecParams& p, int it, int lane) {
    Item w;
    w.kvh = it % p.kv_heads;
    const int rest = it / p.kv_heads;
    w.chunk = rest % p.n_chunks;
    w.b = rest / p.n_chunks;
    w.row0 = p.start[w.b];
    w.L = p.len[w.b];
    bool bad = w.row0 < 0 || w.L < 0 || w.row0 + w.L > p.table_len;
    if constexpr (CROSS) {
        const int qo0 = p.qo_indptr[w.b], nq = p.qo_indptr[w.b + 1] - qo0;
        const bool bad_q = nq > p.max_q || qo0 < 0 || (int64_t)qo0 + nq > p.max_rows;
        w.ncol = bad_q || nq <= 0 ? 0 : nq * p.group;
        w.qrow0 = (int64_t)qo0 * p.q_heads + w.kvh * p.group;
        if (bad_q && lane == 0 && w.kvh == 0 && w.chunk == 0) rc::flag_error(p.err, rc::kErrBadSlot);
        bad = bad || w.L > p.max_len;
    } else {
        w.ncol = NC;
        w.qrow0 = 0;
    }
    if (bad) {  // row outside the table: read nothing
        if (lane == 0 && w.kvh == 0 && w.chunk == 0) rc::flag_error(p.err, rc::kErrBadSlot);
        w.L = 0;
    }
    if (!CROSS && FUSED && lane == 0 && w.kvh == 0 && w.L > p.chunk) rc::flag_error(p.err, rc::kErrBadSlot);
    w.k0 = w.chunk * p.chunk;
    w.count = max(0, min(w.L - w.k0, p.chunk));
    return w;
}

// Row b's keys (and, CROSS, its tokens) as the 4-bit pool's passes and their
// merge read them: L = 0 for a row that is not there, lies outside the table
// or (CROSS) exceeds the caller's bounds or has no tokens; decode reads a row
// longer than max_len up to it.
struct RowKeys {
    int64_t row0;
    int L, qo0, ncol;
    bool bad;
};
template <bool CROSS>
RC_DEV RowKeys row_keys(const DecParams& p, int b) {
    RowKeys r{0, 0, 0, 0, false};
    if (b >= p.batch) return r;
    r.row0 = __ldg(p.start + b);
    r.L = __ldg(p.len + b);
    r.bad = r.row0 < 0 || r.L < 0 || r.row0 + r.L > p.table_len || r.L > p.max_len;
    if constexpr (CROSS) {
        r.qo0 = __ldg(p.qo_indptr + b);
        const int nq = __ldg(p.qo_indptr + b + 1) - r.qo0;
        const bool bad_q = nq > p.max_q || r.qo0 < 0 || (int64_t)r.qo0 + nq > p.max_rows;
        r.ncol = bad_q || nq < 0 ? 0 : nq * p.group;
        if (r.bad || r.ncol == 0) r.L = 0;
        r.bad = r.bad || bad_q;
    } else if (r.bad) {
        const bool too_long = r.row0 >= 0 && r.L > p.max_len && r.row0 + r.L <= p.table_len;
        r.L = too_long ? p.max_len : 0;
    }
    return r;
}

// A split item without keys: decode leaves its partial unwritten (the merge
// goes by the row's length), cross marks its columns' partials empty.
template <int NC, bool CROSS>
RC_DEV void empty_partial(const DecParams& p, const Item& w, int lane) {
    if constexpr (CROSS)
        if (lane < w.ncol) p.part_lse[w.qrow<NC, CROSS>(p, lane) * p.n_chunks + w.chunk] = -INFINITY;
}

// The cascade partials a row folds in: entries e0.. of req_seg_pos, n_parts
// of them (chunks included).
struct SegParts {
    int e0, n_parts;
    RC_DEV int64_t row(const DecParams& p, int j) const {
        return j < n_parts ? (int64_t)p.req_seg_pos[e0 + j / p.seg_chunks] * p.q_heads * p.seg_chunks +
                                 (j % p.seg_chunks)
                           : 0;
    }
};

// Bytes of a warp's shared memory that the epilogue uses: [8][D] outputs,
// [8] log-sum-exps, and the fold's row offsets and log-sum-exps.
template <int D, int NC>
__host__ __device__ constexpr int epilogue_bytes() { return 8 * D * 4 + 32 + 32 * 8 + NC * 32 * 4 + NC * 8; }

// Writes the item's result: sE [8][D] this warp's normalised outputs per
// column, sOwn [8] their log2-sum-exps, both in the warp's shared memory.
template <int D, int NC, bool FUSED, bool CROSS>
RC_DEV void decode_epilogue(const DecParams& p, const Item& w, float* sE, float* sOwn, const SegParts& seg,
                            int64_t first_row, int lane) {
    const int kvh = w.kvh, n_parts = seg.n_parts;
    // The cascade kernel, when there is one, may still be running (this
    // grid is its programmatic dependent): wait for it before reading its
    // partials, and in any case before leaving, so that the end of this grid
    // implies the end of both.
    grid_dep_wait();
    if constexpr (!FUSED) {
        for (int h = 0; h < w.ncol; ++h) {
            const int64_t idx = w.qrow<NC, CROSS>(p, h) * p.n_chunks + w.chunk;
            for (int d = lane; d < D; d += 32) p.part_o[idx * D + d] = sE[h * D + d];
            if (lane == 0) p.part_lse[idx] = sOwn[h];
        }
    } else {
        // the row's whole table part is here: fold in its cascade partials
        // (every chunk of every segment it reads; partial j of head h sits at
        // row seg.row(j) + (kvh * NC + h) * seg_chunks).  Partials come in
        // batches of 32: lane j loads partial j's log-sum-exps in one
        // round, then every lane loads the batch's rows in a second round
        // (all independent loads), merged online against a running max.
        constexpr int kPB = 32;
        int64_t* sRow = reinterpret_cast<int64_t*>(sOwn + 8);   // [kPB]
        float* sL = reinterpret_cast<float*>(sRow + kPB);         // [NC][kPB]
        const int sc = p.seg_chunks;
        float m_h[NC], w_h[NC], acc[NC][D / 32];
#pragma unroll
        for (int h = 0; h < NC; ++h) {
            m_h[h] = sOwn[h];
            w_h[h] = sOwn[h] == -INFINITY ? 0.f : 1.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) acc[h][k] = m_h[h] == -INFINITY ? 0.f : sE[h * D + lane + 32 * k];
        }
        // none after a cascade kernel gave up on a bounded wait (unwritten)
        const int n_use = (p.err && (*reinterpret_cast<volatile int32_t*>(p.err) & rc::kErrTimeout)) ? 0 : n_parts;
        for (int j0 = 0; j0 < n_use; j0 += kPB) {
            const int nb = min(kPB, n_use - j0);
            const int64_t my_row = j0 == 0 ? first_row : seg.row(p, j0 + lane);
            if (lane < nb) {
                sRow[lane] = my_row;
#pragma unroll
                for (int h = 0; h < NC; ++h) sL[h * kPB + lane] = p.seg_lse[my_row + (int64_t)(kvh * NC + h) * sc];
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < NC; ++h) {
                float mb = m_h[h];
                for (int j = 0; j < nb; ++j) mb = fmaxf(mb, sL[h * kPB + j]);
                if (mb == -INFINITY) continue;   // nothing yet for this head
                const float a = m_h[h] == -INFINITY ? 0.f : rc::fast_exp2(m_h[h] - mb);
                w_h[h] *= a;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) acc[h][k] *= a;
                m_h[h] = mb;
            }
#pragma unroll 4
            for (int j = 0; j < nb; ++j) {
                const int64_t row = sRow[j];
#pragma unroll
                for (int h = 0; h < NC; ++h) {
                    const float l2 = sL[h * kPB + j];
                    const float wj = l2 == -INFINITY ? 0.f : rc::fast_exp2(l2 - m_h[h]);
                    w_h[h] += wj;
                    const float* src = p.seg_o + (row + (int64_t)(kvh * NC + h) * sc) * D + lane;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        const float v = src[32 * k];
                        acc[h][k] += wj == 0.f ? 0.f : wj * v;
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < NC; ++h) {
            if (CROSS && h >= w.ncol) break;
            const int64_t orow = w.qrow<NC, CROSS>(p, h);
            const float inv = w_h[h] > 0.f ? 1.f / w_h[h] : 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                p.out[orow * D + lane + 32 * k] = __float2bfloat16_rn(acc[h][k] * inv);
            if (p.lse && lane == 0) p.lse[orow] = rc::log2_sum(m_h[h], w_h[h]) * rc::kLn2;
        }
    }
}

}  // namespace rc_dec
