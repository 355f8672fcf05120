// attn_extend: prefill of the new (uncached) tokens of each request over its
// cached prefix.  In inference-notes note 49, section 2, request 2 reuses the
// shared system prompt and "only Q2" has to be computed; in the SageMaker LMI
// article's prefill phase all of those tokens are processed at once.  Token i
// of request b sits at position len[b] - n_b + i of its slot-table row and
// attends causally to positions 0..itself, prefix included.
//
// The kernel body is attn_tc2.cuh: a CTA owns 256 query rows = (256/G new
// tokens) x (the G query heads of one KV head) in two M=128 tiles, so each
// gathered K/V row serves every head of its group and both tiles; both
// products run on tcgen05 with the accumulators in TMEM, with producer,
// MMA and softmax warps; bf16 output written directly (no split, no
// workspace).

#include "attn_split_merge.cuh"
#include "attn_tc2.cuh"
#include "common.cuh"

namespace {

template <int D, int G, int FMT>
cudaError_t launch_extend(const rc::MQParams& p, int batch, int max_q, int kv_heads, cudaStream_t st) {
    constexpr int smem = rc_tc2::smem_bytes<D, FMT>();
    cudaError_t e = rc_host::ensure_smem<rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kExtend, FMT>>(smem);
    if (e != cudaSuccess) return e;
    constexpr int TPC = rc_tc2::ROWS / G;
    dim3 grid((max_q + TPC - 1) / TPC, kv_heads, batch * p.seg_chunks);
    rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kExtend, FMT><<<grid, rc_tc2::threads<FMT>(), smem, st>>>(p);
    return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t dispatch(int G, const rc::MQParams& p, int batch, int max_q, int kv_heads, cudaStream_t st, bool* ok) {
    *ok = true;
    switch (G) {
        case 1: return launch_extend<D, 1, FMT>(p, batch, max_q, kv_heads, st);
        case 2: return launch_extend<D, 2, FMT>(p, batch, max_q, kv_heads, st);
        case 4: return launch_extend<D, 4, FMT>(p, batch, max_q, kv_heads, st);
        case 8: return launch_extend<D, 8, FMT>(p, batch, max_q, kv_heads, st);
        default: *ok = false; return cudaSuccess;
    }
}

// Over a 4-bit pool (the other formats' calls never ask for a workspace and stay
// whole), a grid that would leave most SMs idle splits the keys, at least four
// tiles a CTA, where there are enough of them to pay for the
// merge (1 row of 8 tokens over 4,000 keys: 57 us whole, 12 split; 4 rows of 40
// over 340: 12.3 whole, 14.1 split; over 1,040: 22.4 and 16.3).
constexpr int kSplitKeys = 512;
struct ExtendPlan {
    int chunk = 0, n_chunks = 1;
    size_t part_o = 0, total = 0;
    size_t bound = 0;  // the largest total of any max_len up to this one
};

ExtendPlan plan_extend(const rc_attn_desc* d, int32_t batch, int32_t max_q, int32_t max_len) {
    ExtendPlan pl;
    const rc_pool_desc& P = d->pool;
    if (rc_host::pool_format(P) != rc::kFmtFp4 || P.kv_heads <= 0 || max_len < kSplitKeys || batch <= 0 ||
        max_q <= 0)
        return pl;
    const int64_t G = d->q_heads / P.kv_heads;
    const int64_t grid = ((max_q * G + rc_tc2::ROWS - 1) / rc_tc2::ROWS) * P.kv_heads * batch;
    const int64_t most = (max_len + 4 * rc_tc2::TN - 1) / (4 * rc_tc2::TN);
    int64_t splits = rc_host::sm_count() / (grid > 0 ? grid : 1);
    splits = splits < most ? splits : most;
    const int64_t max_rows = (int64_t)batch * max_q;
    if (splits < 2 || batch * splits > 65535 || max_rows > 0x7fffffff) return pl;
    const int64_t chunk = (max_len + splits - 1) / splits;
    pl.chunk = (int)((chunk + rc_tc2::TN - 1) / rc_tc2::TN * rc_tc2::TN);
    pl.n_chunks = (max_len + pl.chunk - 1) / pl.chunk;
    if (pl.n_chunks < 2) return ExtendPlan();
    const size_t rows = (size_t)max_rows * d->q_heads * pl.n_chunks;
    auto bytes = [&](size_t n) { return (n * sizeof(float) + 255) & ~size_t(255); };
    pl.part_o = bytes(rows * P.head_dim_v);
    pl.total = pl.part_o + bytes(rows);
    const size_t most_rows = (size_t)max_rows * d->q_heads * splits;  // n_chunks, rounded, can fall as max_len grows
    pl.bound = bytes(most_rows * P.head_dim_v) + bytes(most_rows);
    return pl;
}

}  // namespace

extern "C" rc_status attn_extend_workspace(const rc_attn_desc* desc, int32_t batch, int32_t max_q,
                                           int32_t max_len, size_t* bytes) {
    if (!desc || !bytes || batch < 0 || max_q < 0 || max_len < 0) return RC_ERR_ARG;
    *bytes = plan_extend(desc, batch, max_q, max_len).bound;
    return RC_OK;
}

extern "C" rc_status attn_extend(const rc_attn_desc* desc, const void* q, const int32_t* qo_indptr,
                                 const rc_kv_table* kv, int32_t batch, int32_t max_q, void* out, float* lse,
                                 void* ws, size_t ws_bytes, rc_stream_t stream) {
    if (!desc || !kv || batch < 0 || max_q < 0) return RC_ERR_ARG;
    if (batch == 0 || max_q == 0) return RC_OK;
    if (!q || !qo_indptr || !out || !kv->slots || !kv->start || !kv->len || !desc->pool.k) return RC_ERR_ARG;
    const rc_pool_desc& P = desc->pool;
    if (P.kv_heads <= 0 || desc->q_heads <= 0 || desc->q_heads % P.kv_heads) return RC_ERR_ARG;
    if (P.mla || !P.v || P.head_dim_v != P.head_dim_k) return RC_ERR_UNSUPPORTED;
    const int fmt = rc_host::pool_format(P);
    const bool fp8 = fmt == rc::kFmtFp8;
    if (fp8 && P.head_dim_k != 128) return RC_ERR_UNSUPPORTED;
    if (fp8 && (!P.k_scale || !P.v_scale)) return RC_ERR_ARG;
    if (fmt == rc::kFmtFp4) {
        const rc_status s = rc_host::check_fp4(P);
        if (s != RC_OK) return s;
        if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return RC_ERR_ARG;
    }
    if (!(desc->sm_scale > 0.f)) return RC_ERR_ARG;  // scores are masked, and their largest taken, before they are scaled
    rc::MQParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pool_k = static_cast<const __nv_bfloat16*>(P.k);
    p.pool_v = static_cast<const __nv_bfloat16*>(P.v);
    p.n_slots = P.n_slots;
    p.kv_heads = P.kv_heads;
    p.q_heads = desc->q_heads;
    p.scale_log2 = desc->sm_scale * rc::kLog2e;
    p.err = P.err;
    p.qo_indptr = qo_indptr;
    p.table = kv->slots;
    p.start = kv->start;
    p.len = kv->len;
    p.table_len = kv->table_len;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.out_wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    p.k_scale = fp8 ? P.k_scale : nullptr;
    p.v_scale = fp8 ? P.v_scale : nullptr;
    p.k_bscale = fmt == rc::kFmtFp4 ? P.k_bscale : nullptr;
    p.v_bscale = fmt == rc::kFmtFp4 ? P.v_bscale : nullptr;
    // without a workspace, or with one too small, every row's keys stay with one CTA
    ExtendPlan pl = plan_extend(desc, batch, max_q, kv->max_len);
    if (pl.n_chunks > 1 && (!ws || ws_bytes < pl.total)) pl = ExtendPlan();
    if (pl.n_chunks > 1 && (reinterpret_cast<uintptr_t>(ws) & 255)) return RC_ERR_ARG;
    const int64_t max_rows = (int64_t)batch * max_q;
    p.seg_chunk = pl.chunk;
    p.seg_chunks = pl.n_chunks;
    p.max_q = max_q;
    p.max_len = kv->max_len;
    p.max_rows = max_rows;
    p.part_o = static_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + pl.part_o);
    const int G = desc->q_heads / P.kv_heads;
    bool ok = false;
    cudaError_t e = cudaSuccess;
    cudaStream_t st = (cudaStream_t)stream;
    if (fmt == rc::kFmtFp4) {
        e = P.head_dim_k == 128 ? dispatch<128, rc::kFmtFp4>(G, p, batch, max_q, P.kv_heads, st, &ok)
                                : dispatch<64, rc::kFmtFp4>(G, p, batch, max_q, P.kv_heads, st, &ok);
    } else if (fp8) {
        e = dispatch<128, rc::kFmtFp8>(G, p, batch, max_q, P.kv_heads, st, &ok);
    } else if (P.head_dim_k == 128) {
        e = dispatch<128, rc::kFmtBf16>(G, p, batch, max_q, P.kv_heads, st, &ok);
    } else if (P.head_dim_k == 64) {
        e = dispatch<64, rc::kFmtBf16>(G, p, batch, max_q, P.kv_heads, st, &ok);
    }
    if (!ok) return RC_ERR_UNSUPPORTED;
    if (e != cudaSuccess || pl.n_chunks == 1) return rc_host::launch_status(e);
    const rc_dec::SplitMerge m{p.part_o, p.part_lse, pl.n_chunks, qo_indptr, max_q, max_rows, desc->q_heads, p.out, lse,
                               P.err};
    return rc_host::launch_status(P.head_dim_k == 128 ? rc_dec::launch_split_merge<128>(m, st)
                                                      : rc_dec::launch_split_merge<64>(m, st));
}
