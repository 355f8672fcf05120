// attn_cross: every new token of a row attends to all of the row's keys, an
// encoder's states held in the pool and read through the slot table.
//
//   out[i] = sum_j softmax_j(scale q[i].K[j]) V[j]   over all keys j of row b
//
// No causal edge and no relation between a row's tokens and its keys, so the
// same K/V serve any number of tokens.  Two forms, by the (token, head) pairs
// that share a K/V head, max_q * q_heads / kv_heads:
//  * at most 8: bound by the K/V read once; the decode table pass, one warp
//    per (row, KV head, key chunk) with the pairs as its columns (32 rows of
//    1500 bf16 keys, 16 KV heads of 64: 38.2 us a call, 5.15 TB/s);
//  * more: the tcgen05 kernel of attn_extend without the causal edge, 256
//    pairs per CTA, bound by the hand-offs of its tiles (6 rows of 900-1024
//    tokens over 4095 4-bit keys, 32 heads over 8 of 128: 328 us a call, 1160
//    TFLOP/s); where its grid would leave SMs idle the keys are split over CTAs.
// Split keys leave normalised partials that a merge joins (attn_split_merge.cuh,
// or for the 4-bit table pass merge_runs_kernel).

#include "attn_decode_fp4.cuh"
#include "attn_decode_split.cuh"
#include "attn_split_merge.cuh"
#include "attn_tc2.cuh"

namespace {

using namespace rc_dec;

// The n = 8 side of the table pass's products.  At 8 pairs, 8 KV heads of 128 and
// 1500 keys a call takes, in the table pass and in the many-row kernel: 32 rows
// 42 and 69 us (bf16), 32 and 80 (E4M3), 40 and 54 (4 bits); 8 rows 22 and 24, 19
// and 27, 21 and 21; one row 17 and 14, 15 and 15, 13 and 13.
constexpr int kFewColumns = 8;

struct CrossPlan {
    bool few = false, runs = false;  // runs: the 4-bit table pass over equal runs of keys
    int chunk = 0, n_chunks = 1;
    size_t part_o = 0, part_lse = 0, row_runs = 0, total = 0;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

rc_status plan_cross(const rc_attn_desc* d, int32_t batch, int32_t max_q, int32_t max_len, CrossPlan* pl) {
    const rc_pool_desc& P = d->pool;
    const int hkv = P.kv_heads;
    if (hkv <= 0 || d->q_heads <= 0 || d->q_heads % hkv) return RC_ERR_ARG;
    const int G = d->q_heads / hkv;
    const int64_t sms = rc_host::sm_count();
    const int64_t cols = (int64_t)max_q * G;
    pl->few = cols <= kFewColumns;
    int64_t splits = 1, step;
    int64_t unit = kDecKeys;         // chunks are multiples of this many keys
    if (pl->few) {  // one wave of warps, at least two 16-key tiles each
        const int64_t base = (int64_t)batch * hkv;
        if (base > 0 && base < 8 * sms) splits = kWarpsPerCta * sms / base;
        step = unit = 2 * kWarpKeys;
    } else {  // one CTA per SM, at least two 64-key tiles each
        const int64_t grid = ((cols + rc_tc2::ROWS - 1) / rc_tc2::ROWS) * hkv * batch;
        if (grid > 0 && grid < sms) splits = sms / grid;
        step = 2 * rc_tc2::TN;
    }
    const int64_t most = max_len > 0 ? (max_len + step - 1) / step : 1;
    splits = splits < 1 ? 1 : splits > most ? most : splits;
    int64_t chunk = max_len > 0 ? (max_len + splits - 1) / splits : kDecKeys;
    chunk = (chunk + unit - 1) / unit * unit;
    if (chunk > 0x7fffffc0) return RC_ERR_ARG;
    pl->chunk = (int)chunk;
    pl->n_chunks = max_len > 0 ? (int)((max_len + chunk - 1) / chunk) : 1;
    pl->runs = pl->few && rc_host::pool_format(P) == rc::kFmtFp4 && !fp4::whole_rows(batch, hkv, max_len, sms);
    if (pl->few && rc_host::pool_format(P) == rc::kFmtFp4) {
        pl->chunk = max_len > 0 ? max_len : 1;
        pl->n_chunks = pl->runs ? fp4::groups(batch, hkv, max_len, sms) : 1;
    }
    if (pl->runs) {
        const size_t parts = ((size_t)pl->n_chunks + batch) * hkv * kFewColumns;
        pl->part_o = align256(parts * P.head_dim_v * sizeof(float));
        pl->part_lse = align256(parts * sizeof(float));
        pl->row_runs = align256((size_t)batch * 2 * sizeof(int32_t));
    } else if (pl->n_chunks > 1) {
        // room for `splits` chunks, which some max_len up to this one has:
        // n_chunks, after rounding, falls as max_len passes a unit
        const size_t rows = (size_t)batch * max_q * d->q_heads * splits;
        pl->part_o = align256(rows * P.head_dim_v * sizeof(float));
        pl->part_lse = align256(rows * sizeof(float));
    }
    pl->total = pl->part_o + pl->part_lse + pl->row_runs;
    return RC_OK;
}

rc_status check_pool(const rc_attn_desc* d) {
    const rc_pool_desc& P = d->pool;
    if (!P.k || P.kv_heads <= 0 || d->q_heads <= 0 || d->q_heads % P.kv_heads) return RC_ERR_ARG;
    if (P.mla || P.head_dim_k != P.head_dim_v || (P.head_dim_k != 128 && P.head_dim_k != 64))
        return RC_ERR_UNSUPPORTED;
    const int G = d->q_heads / P.kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return RC_ERR_UNSUPPORTED;
    if (!P.v) return RC_ERR_ARG;
    const int fmt = rc_host::pool_format(P);
    if (fmt == rc::kFmtFp8) {
        if (P.head_dim_k != 128) return RC_ERR_UNSUPPORTED;
        if (!P.k_scale || !P.v_scale) return RC_ERR_ARG;
    }
    if (fmt == rc::kFmtFp4) return rc_host::check_fp4(P);
    return RC_OK;
}

template <auto Kernel, int WARPS, bool RUNS = false>
cudaError_t launch_few(const DecParams& p, int smem, int batch, cudaStream_t st) {
    cudaError_t e = rc_host::ensure_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
    const int n_items = RUNS ? p.kv_heads * p.n_chunks : batch * p.kv_heads * p.n_chunks;
    Kernel<<<(n_items + WARPS - 1) / WARPS, 32 * WARPS, smem, st>>>(p, n_items);
    return cudaGetLastError();
}

template <int D, int FMT, bool FUSED>
cudaError_t few(const DecParams& p, int batch, cudaStream_t st) {
    if constexpr (FMT == rc::kFmtFp4)
        return p.kv_heads % fp4::kWarps == 0
                   ? launch_few<decode_fp4_kernel<D, kFewColumns, FUSED, true, true>, fp4::kWarps, !FUSED>(
                         p, fp4::smem_bytes<D, true>(), batch, st)
                   : launch_few<decode_fp4_kernel<D, kFewColumns, FUSED, true, false>, fp4::kWarps, !FUSED>(
                         p, fp4::smem_bytes<D, false>(), batch, st);
    else
        return launch_few<decode_split_kernel<D, kFewColumns, FUSED, FMT == rc::kFmtFp8, true>, kWarpsPerCta>(
            p, dec_smem_bytes<D, FMT == rc::kFmtFp8>(), batch, st);
}

template <int D, int G, int FMT>
cudaError_t many_group(const rc::MQParams& p, int batch, int max_q, cudaStream_t st) {
    constexpr int smem = rc_tc2::smem_bytes<D, FMT>();
    cudaError_t e = rc_host::ensure_smem<rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kCross, FMT>>(smem);
    if (e != cudaSuccess) return e;
    constexpr int TPC = rc_tc2::ROWS / G;
    dim3 grid((max_q + TPC - 1) / TPC, p.kv_heads, batch * p.seg_chunks);
    rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kCross, FMT><<<grid, rc_tc2::threads<FMT>(), smem, st>>>(p);
    return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t many(int G, const rc::MQParams& p, int batch, int max_q, cudaStream_t st) {
    switch (G) {
        case 1: return many_group<D, 1, FMT>(p, batch, max_q, st);
        case 2: return many_group<D, 2, FMT>(p, batch, max_q, st);
        case 4: return many_group<D, 4, FMT>(p, batch, max_q, st);
        default: return many_group<D, 8, FMT>(p, batch, max_q, st);
    }
}

template <int D, int FMT>
cudaError_t run(const CrossPlan& pl, int G, const DecParams& dp, const rc::MQParams& mp, int batch, int max_q,
                cudaStream_t st) {
    if (!pl.few) return many<D, FMT>(G, mp, batch, max_q, st);
    return pl.n_chunks == 1 && !pl.runs ? few<D, FMT, true>(dp, batch, st) : few<D, FMT, false>(dp, batch, st);
}

}  // namespace

extern "C" rc_status attn_cross_workspace(const rc_attn_desc* desc, int32_t batch, int32_t max_q, int32_t max_len,
                                          size_t* bytes) {
    if (!desc || !bytes || batch < 0 || max_q < 0 || max_len < 0) return RC_ERR_ARG;
    const rc_pool_desc& P = desc->pool;
    if (P.mla) return RC_ERR_UNSUPPORTED;
    CrossPlan pl;
    const rc_status s = plan_cross(desc, batch, max_q, max_len, &pl);
    if (s != RC_OK) return s;
    *bytes = pl.total;
    return RC_OK;
}

extern "C" rc_status attn_cross(const rc_attn_desc* desc, const void* q, const int32_t* qo_indptr,
                                const rc_kv_table* kv, int32_t batch, int32_t max_q, void* out, float* lse, void* ws,
                                size_t ws_bytes, rc_stream_t stream) {
    if (!desc || !kv || batch < 0 || max_q < 0 || kv->max_len < 0) return RC_ERR_ARG;
    rc_status s = check_pool(desc);
    if (s != RC_OK) return s;
    if (!(desc->sm_scale > 0.f)) return RC_ERR_ARG;  // the largest score has to be the largest scaled one
    if (batch == 0 || max_q == 0) return RC_OK;
    if (!q || !qo_indptr || !out || !kv->slots || !kv->start || !kv->len) return RC_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return RC_ERR_ARG;
    CrossPlan pl;
    s = plan_cross(desc, batch, max_q, kv->max_len, &pl);
    if (s != RC_OK) return s;
    if (pl.total > 0 && (!ws || ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(ws) & 255))) return RC_ERR_ARG;
    const rc_pool_desc& P = desc->pool;
    const int fmt = rc_host::pool_format(P);
    const int G = desc->q_heads / P.kv_heads;
    const int64_t max_rows = (int64_t)batch * max_q;
    // grid limits: blocks in x for the table pass and the merge, z for the many-row kernel
    if ((int64_t)batch * P.kv_heads * pl.n_chunks > 0x7fffffff || max_rows > 0x7fffffff) return RC_ERR_ARG;
    if (pl.runs && desc->q_heads > 65535) return RC_ERR_UNSUPPORTED;
    if (!pl.few && ((int64_t)batch * pl.n_chunks > 65535 || P.kv_heads > 65535)) return RC_ERR_UNSUPPORTED;
    unsigned char* w = static_cast<unsigned char*>(ws);
    float* part_o = reinterpret_cast<float*>(w);
    float* part_lse = reinterpret_cast<float*>(w + pl.part_o);
    const float* k_scale = fmt == rc::kFmtFp8 ? P.k_scale : nullptr;
    const float* v_scale = fmt == rc::kFmtFp8 ? P.v_scale : nullptr;
    const uint8_t* k_bscale = fmt == rc::kFmtFp4 ? P.k_bscale : nullptr;
    const uint8_t* v_bscale = fmt == rc::kFmtFp4 ? P.v_bscale : nullptr;
    DecParams dp{};
    rc::MQParams mp{};
    dp.q = mp.q = static_cast<const __nv_bfloat16*>(q);
    dp.pool_k = mp.pool_k = static_cast<const __nv_bfloat16*>(P.k);
    dp.pool_v = mp.pool_v = static_cast<const __nv_bfloat16*>(P.v);
    dp.n_slots = mp.n_slots = P.n_slots;
    dp.kv_heads = mp.kv_heads = P.kv_heads;
    dp.q_heads = mp.q_heads = desc->q_heads;
    dp.scale_log2 = mp.scale_log2 = desc->sm_scale * rc::kLog2e;
    dp.err = mp.err = P.err;
    dp.qo_indptr = mp.qo_indptr = qo_indptr;
    dp.table = mp.table = kv->slots;
    dp.start = mp.start = kv->start;
    dp.len = mp.len = kv->len;
    dp.table_len = mp.table_len = kv->table_len;
    dp.out = mp.out = static_cast<__nv_bfloat16*>(out);
    dp.lse = mp.lse = lse;
    mp.out_wide = 1;
    dp.part_o = mp.part_o = part_o;
    dp.part_lse = mp.part_lse = part_lse;
    dp.chunk = mp.seg_chunk = pl.chunk;
    dp.n_chunks = mp.seg_chunks = pl.n_chunks;
    dp.k_scale = mp.k_scale = k_scale;
    dp.v_scale = mp.v_scale = v_scale;
    dp.k_bscale = mp.k_bscale = k_bscale;
    dp.v_bscale = mp.v_bscale = v_bscale;
    dp.max_q = mp.max_q = max_q;
    dp.max_len = mp.max_len = kv->max_len;
    dp.max_rows = mp.max_rows = max_rows;
    dp.group = G;
    dp.batch = batch;
    dp.row_runs = reinterpret_cast<int32_t*>(w + pl.part_o + pl.part_lse);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    const bool wide = P.head_dim_k == 128;
    if (fmt == rc::kFmtFp4)
        e = wide ? run<128, rc::kFmtFp4>(pl, G, dp, mp, batch, max_q, st)
                 : run<64, rc::kFmtFp4>(pl, G, dp, mp, batch, max_q, st);
    else if (fmt == rc::kFmtFp8)
        e = run<128, rc::kFmtFp8>(pl, G, dp, mp, batch, max_q, st);
    else
        e = wide ? run<128, rc::kFmtBf16>(pl, G, dp, mp, batch, max_q, st)
                 : run<64, rc::kFmtBf16>(pl, G, dp, mp, batch, max_q, st);
    if (e != cudaSuccess) return RC_ERR_CUDA;
    if (pl.n_chunks == 1 && !pl.runs) return RC_OK;
    if (pl.runs)
        return rc_host::launch_status(wide ? launch_merge_runs<128, true>(dp, max_rows, st)
                                           : launch_merge_runs<64, true>(dp, max_rows, st));
    const rc_dec::SplitMerge m{part_o, part_lse, pl.n_chunks, qo_indptr, max_q, max_rows, desc->q_heads,
                               static_cast<__nv_bfloat16*>(out), lse, P.err};
    e = wide ? launch_split_merge<128>(m, st) : launch_split_merge<64>(m, st);
    return rc_host::launch_status(e);
}
