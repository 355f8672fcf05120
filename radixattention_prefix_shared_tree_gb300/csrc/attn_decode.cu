// attn_decode: one new token per request attends to its whole cached context,
// read through the request's slot table (decode phase of the SageMaker LMI
// article; the K/V come from the radix-tree cache of inference-notes note 49,
// section 2).  Memory-bound: every K/V row of the context is read once per KV
// head per step, so the design goal is to stream rows at HBM speed.
//
//  1. cascade pass (when the batch shares prefixes): each shared segment is
//     read once for all rows below it by the tcgen05 many-row kernel
//     (attn_tc2.cuh), one partial per (row, head, segment, key chunk).
//  2. table pass: one warp per item (request, KV head[, key chunk]).  The G
//     query heads of the KV head share each K/V row (grouped-query head
//     grouping).  Each warp gathers its keys by slot with 16-byte cp.async
//     into its own two-stage ring of 16-key tiles; the products run on
//     mma.sync with the keys on the M side and the G heads on the N side (so
//     G = 4 or 8 wastes at most half of an n8 tile instead of 12 of 16 rows),
//     and P moves from accumulator to operand layout with movmatrix.  With
//     one chunk per row the warp's epilogue folds in the row's cascade
//     partials and writes the output (fused); otherwise it writes a
//     normalised partial and its log-sum-exp per (request, head, chunk).
//  3. merge pass (split rows only): per (request, head), combine all
//     partials by log-sum-exp.

#include "attn_decode_fp4.cuh"
#include "attn_decode_split.cuh"
#include "attn_tc2.cuh"
#include "common.cuh"

namespace {

using namespace rc_dec;

// Combine every partial of (request, head): cascade segments (all chunks)
// then the chunks of the request's own table row.
template <int D>
__global__ void __launch_bounds__(32) merge_kernel(const float* __restrict__ tail_o,
                                                   const float* __restrict__ tail_lse, int32_t n_chunks,
                                                   int32_t chunk, const int32_t* __restrict__ len,
                                                   const float* __restrict__ seg_o,
                                                   const float* __restrict__ seg_lse, int32_t seg_chunks,
                                                   const int32_t* __restrict__ req_seg_indptr,
                                                   const int32_t* __restrict__ req_seg_pos, int32_t q_heads,
                                                   const int32_t* __restrict__ start, int64_t table_len,
                                                   __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                                                   int32_t* err) {
    constexpr int PER = D / 32;
    const int bh = blockIdx.x;
    const int b = bh / q_heads, h = bh % q_heads;
    const int lane = threadIdx.x;
    // launched as the split pass's programmatic dependent: let the next
    // kernel launch, then wait for the split pass (and through it the
    // cascade) before reading anything they wrote
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    grid_dep_wait();
    const int64_t row0 = start[b];
    const int L = len[b];
    // a row the split pass rejected (outside the table) wrote no partials
    int nc = (row0 < 0 || L < 0 || row0 + L > table_len) ? 0 : (L + chunk - 1) / chunk;
    if (nc > n_chunks) {  // len[b] above the caller's max_len: the split pass skipped keys
        if (lane == 0 && h == 0) rc::flag_error(err, rc::kErrBadSlot);
        nc = n_chunks;
    }
    // a cascade kernel that gave up on a bounded wait (or met the flag of an
    // earlier one) left its partials unwritten: use none of them
    const bool casc_ok = !(err && (*reinterpret_cast<volatile int32_t*>(err) & rc::kErrTimeout));
    const int s0 = req_seg_indptr && casc_ok ? req_seg_indptr[b] : 0;
    const int ns = req_seg_indptr && casc_ok ? req_seg_indptr[b + 1] - s0 : 0;
    // partials j < ns * seg_chunks: cascade (segment entry j / seg_chunks,
    // chunk j % seg_chunks); then the nc chunks of the row's own table part.
    // Batches of 32: lane j loads partial j's log-sum-exp (one round), then
    // every lane reads the batch's rows (independent loads), merged online.
    const int n_all = ns * seg_chunks + nc;
    __shared__ float sL[32];
    __shared__ const float* sSrc[32];
    float m = -INFINITY, wsum = 0.f;
    float acc[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) acc[j] = 0.f;
    for (int j0 = 0; j0 < n_all; j0 += 32) {
        const int nb = min(32, n_all - j0);
        if (lane < nb) {
            const int j = j0 + lane;
            int64_t row;
            const float* base;
            const float* lbase;
            if (j < ns * seg_chunks) {
                row = ((int64_t)req_seg_pos[s0 + j / seg_chunks] * q_heads + h) * seg_chunks + j % seg_chunks;
                base = seg_o;
                lbase = seg_lse;
            } else {
                row = (int64_t)bh * n_chunks + (j - ns * seg_chunks);
                base = tail_o;
                lbase = tail_lse;
            }
            sL[lane] = lbase[row];
            sSrc[lane] = base + row * D;
        }
        __syncwarp();
        float mb = m;
        for (int j = 0; j < nb; ++j) mb = fmaxf(mb, sL[j]);
        if (mb != -INFINITY) {
            const float a = m == -INFINITY ? 0.f : rc::fast_exp2(m - mb);
            wsum *= a;
#pragma unroll
            for (int k = 0; k < PER; ++k) acc[k] *= a;
            m = mb;
#pragma unroll 4
            for (int j = 0; j < nb; ++j) {
                const float l2 = sL[j];
                if (l2 == -INFINITY) continue;
                const float w = rc::fast_exp2(l2 - m);
                wsum += w;
                const float* src = sSrc[j] + lane;
#pragma unroll
                for (int k = 0; k < PER; ++k) acc[k] += w * src[32 * k];
            }
        }
        __syncwarp();
    }
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) out[(int64_t)bh * D + lane + 32 * j] = __float2bfloat16_rn(acc[j] * inv);
    if (lse && lane == 0) lse[bh] = rc::log2_sum(m, wsum) * rc::kLn2;
}

// ------------------------------------------------------------------ planning
struct DecodePlan {
    int chunk = 0, n_chunks = 0;        // table part: keys per CTA, CTAs per row
    int seg_chunk = 0, seg_chunks = 0;  // cascade: keys per CTA, CTAs per segment
    bool fused = false;                 // one CTA per (row, KV head): no merge pass
    size_t tail_o = 0, tail_lse = 0, row_runs = 0, seg_o = 0, seg_lse = 0, total = 0;
    size_t bound = 0;                   // the largest total of any max_len up to this one
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

rc_status plan_decode(const rc_attn_desc* d, int32_t batch, int32_t max_len, const rc_cascade* casc,
                      DecodePlan* pl) {
    if (!d || batch < 0 || max_len < 0) return RC_ERR_ARG;
    const int hkv = d->pool.kv_heads;
    if (hkv <= 0 || d->q_heads <= 0 || d->q_heads % hkv) return RC_ERR_ARG;
    const int dv = d->pool.head_dim_v;
    const int64_t sms = rc_host::sm_count();
    // Table part: one warp per (row, KV head) when that already gives every
    // SM eight warps (the merge is then fused); otherwise split the keys so
    // that the items just fill one wave of CTAs (a warp's time grows with its
    // tiles, about 2.5 us per 16 keys when the gather saturates HBM, so the
    // wave's longest item sets the call), down to 64 keys per chunk.
    const int64_t base = (int64_t)batch * hkv;
    const bool is_fp4 = rc_host::pool_format(d->pool) == rc::kFmtFp4;
    int64_t splits = 1;
    if (base < 8 * sms) {
        splits = base > 0 ? (kWarpsPerCta * sms) / base : 1;
        const int64_t max_splits = max_len > 0 ? (max_len + kDecKeys - 1) / kDecKeys : 1;
        if (splits > max_splits) splits = max_splits;
        if (splits < 1) splits = 1;
    }
    int64_t chunk = max_len > 0 ? (max_len + splits - 1) / splits : kDecKeys;
    chunk = (chunk + kDecKeys - 1) / kDecKeys * kDecKeys;
    pl->chunk = (int)chunk;
    pl->n_chunks = max_len > 0 ? (int)((max_len + chunk - 1) / chunk) : 1;
    pl->fused = pl->n_chunks == 1;
    if (is_fp4) {  // whole rows, or equal runs of the batch's keys (n_chunks of them)
        pl->fused = fp4::whole_rows(batch, hkv, max_len, sms);
        pl->chunk = max_len > 0 ? max_len : 1;
        pl->n_chunks = pl->fused ? 1 : fp4::groups(batch, hkv, max_len, sms);
    }
    // Cascade part: split each segment's keys so that the grid fills the SMs
    // once (one CTA per SM: a second, partial wave would double the time),
    // and in any case so that no CTA takes more than about kSegKeys keys: a
    // CTA's time grows with its tiles, and with many segments (a grid of
    // several waves anyway) a long one would otherwise run all its keys in
    // one CTA while the short ones finish early.  Chunks past a segment's end
    // are empty CTAs that leave at once.
    constexpr int64_t kSegKeys = 512;
    pl->seg_chunk = 0;
    pl->seg_chunks = 1;
    if (casc && casc->n_seg > 0 && casc->max_seg_len > 0) {
        const int G = d->q_heads / hkv;
        const int64_t row_blocks = (casc->max_seg_rows * (int64_t)G + rc_tc2::ROWS - 1) / rc_tc2::ROWS;
        const int64_t cbase = (int64_t)casc->n_seg * row_blocks * hkv;
        int64_t sc = cbase > 0 ? sms / cbase : 1;
        const int64_t sc_len = (casc->max_seg_len + kSegKeys - 1) / kSegKeys;
        if (sc < sc_len) sc = sc_len;
        const int64_t sc_max = (casc->max_seg_len + 255) / 256;
        if (sc > sc_max) sc = sc_max;
        if (sc < 1) sc = 1;
        int64_t len = (casc->max_seg_len + sc - 1) / sc;
        len = (len + rc_tc2::TN - 1) / rc_tc2::TN * rc_tc2::TN;
        pl->seg_chunk = (int)len;
        pl->seg_chunks = (int)((casc->max_seg_len + len - 1) / len);
    }
    const size_t rows = (size_t)batch * d->q_heads;
    pl->tail_o = pl->fused ? 0 : align256(rows * pl->n_chunks * dv * sizeof(float));
    pl->tail_lse = pl->fused ? 0 : align256(rows * pl->n_chunks * sizeof(float));
    if (is_fp4 && !pl->fused) {
        const size_t parts = ((size_t)pl->n_chunks + batch) * d->q_heads;
        pl->tail_o = align256(parts * dv * sizeof(float));
        pl->tail_lse = align256(parts * sizeof(float));
        pl->row_runs = align256((size_t)batch * 2 * sizeof(int32_t));
    }
    const size_t srows = casc && casc->n_seg > 0 ? (size_t)casc->total_seg_rows * d->q_heads * pl->seg_chunks : 0;
    pl->seg_o = align256(srows * dv * sizeof(float));
    pl->seg_lse = align256(srows * sizeof(float));
    pl->total = pl->tail_o + pl->tail_lse + pl->row_runs + pl->seg_o + pl->seg_lse;
    // Chunks are rounded up to kDecKeys keys, so n_chunks can fall as max_len
    // grows; `splits`, which it reaches at some max_len up to this one, cannot.
    // (A 4-bit pool's runs only grow.)
    pl->bound = pl->total;
    if (!is_fp4 && !pl->fused)
        pl->bound += align256(rows * splits * dv * sizeof(float)) - pl->tail_o +
                     align256(rows * splits * sizeof(float)) - pl->tail_lse;
    if (pl->total == 0) pl->total = 256;
    if (pl->bound == 0) pl->bound = 256;
    return RC_OK;
}

// after_cascade: launched as the programmatic dependent of the cascade kernel
// just queued on the stream, so that its CTAs start on SMs the cascade leaves
// free and as cascade CTAs finish, instead of after the whole cascade grid.
// RUNS: a warp per (run, KV head) instead of (row, KV head, chunk).
template <auto Kernel, int WARPS, bool RUNS = false>
cudaError_t launch_table(const DecParams& p, int smem, int batch, int kv_heads, cudaStream_t st, bool after_cascade) {
    cudaError_t e = rc_host::ensure_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
    const int n_items = RUNS ? kv_heads * p.n_chunks : batch * kv_heads * p.n_chunks;
    const int grid = (n_items + WARPS - 1) / WARPS;
    if (!after_cascade) {
        Kernel<<<grid, 32 * WARPS, smem, st>>>(p, n_items);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, Kernel, p, n_items);
}

template <int D, int G, bool FUSED, int FMT>
cudaError_t launch_split(const DecParams& p, int batch, int kv_heads, cudaStream_t st, bool after_cascade) {
    if constexpr (FMT == rc::kFmtFp4)
        return kv_heads % fp4::kWarps == 0
                   ? launch_table<decode_fp4_kernel<D, G, FUSED, false, true>, fp4::kWarps, !FUSED>(
                         p, fp4::smem_bytes<D, true>(), batch, kv_heads, st, after_cascade)
                   : launch_table<decode_fp4_kernel<D, G, FUSED, false, false>, fp4::kWarps, !FUSED>(
                         p, fp4::smem_bytes<D, false>(), batch, kv_heads, st, after_cascade);
    else
        return launch_table<decode_split_kernel<D, G, FUSED, FMT == rc::kFmtFp8>, kWarpsPerCta>(
            p, dec_smem_bytes<D, FMT == rc::kFmtFp8>(), batch, kv_heads, st, after_cascade);
}

template <int D, int G, int FMT>
cudaError_t launch_cascade(const rc::MQParams& p0, const rc_cascade* c, int kv_heads, cudaStream_t st) {
    constexpr int smem = rc_tc2::smem_bytes<D, FMT>();
    cudaError_t e = rc_host::ensure_smem<rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kCascade, FMT>>(smem);
    if (e != cudaSuccess) return e;
    constexpr int TPC = rc_tc2::ROWS / G;
    rc::MQParams p = p0;
    dim3 grid((c->max_seg_rows + TPC - 1) / TPC, kv_heads, c->n_seg * p.seg_chunks);
    p.n_seg = c->n_seg;
    p.seg_items = 0;
    if (c->host_seg_indptr && c->host_seg_row_indptr) {
        // one CTA per non-empty (segment, key chunk, row block), counted the
        // way the kernel counts them from the device arrays
        int64_t items = 0;
        for (int s = 0; s < c->n_seg; ++s) {
            const int64_t rows = (int64_t)c->host_seg_row_indptr[s + 1] - c->host_seg_row_indptr[s];
            const int64_t len = (int64_t)c->host_seg_indptr[s + 1] - c->host_seg_indptr[s];
            if (rows <= 0) continue;
            int64_t ch = len > 0 ? (len + p.seg_chunk - 1) / p.seg_chunk : 1;
            if (ch > p.seg_chunks) ch = p.seg_chunks;
            items += ch * ((rows + TPC - 1) / TPC);
        }
        if (items > 0 && items <= 0x7fffffff) {
            grid = dim3((unsigned)items, kv_heads, 1);
            p.seg_items = (int32_t)items;
        }
    }
    // programmatic dependent of the previous kernel on the stream (the kernel
    // waits for it before reading anything)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(rc_tc2::threads<FMT>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // Reading ahead of the previous grid's end pays while the grid's CTAs all run
    // at once (256 few-shot rows: 41.0 us a decode call against 46.3).  The second
    // wave of a larger grid would hold the table pass back until its keys are
    // through (64 agents, 224 CTAs: 53.9 us a call, with it 1.2 more).
    if ((int64_t)grid.x * grid.y * grid.z > rc_host::sm_count()) p.early = 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rc_tc2::attn_tc2_kernel<D, G, rc::MQMode::kCascade, FMT>, p);
}

template <int D, int G, int FMT>
cudaError_t run_gqa(const DecParams& dp, const rc::MQParams& mp, const rc_cascade* casc, bool fused, int batch,
                    int kv_heads, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    const bool with_cascade = casc && casc->n_seg > 0 && casc->max_seg_rows > 0;
    if (with_cascade) e = launch_cascade<D, G, FMT>(mp, casc, kv_heads, st);
    if (e != cudaSuccess) return e;
    return fused ? launch_split<D, G, true, FMT>(dp, batch, kv_heads, st, with_cascade)
                 : launch_split<D, G, false, FMT>(dp, batch, kv_heads, st, with_cascade);
}

template <int D, int FMT>
cudaError_t dispatch_group(int G, const DecParams& dp, const rc::MQParams& mp, const rc_cascade* casc, bool fused,
                           int batch, int kv_heads, cudaStream_t st, bool* ok) {
    *ok = true;
    switch (G) {
        case 1: return run_gqa<D, 1, FMT>(dp, mp, casc, fused, batch, kv_heads, st);
        case 2: return run_gqa<D, 2, FMT>(dp, mp, casc, fused, batch, kv_heads, st);
        case 4: return run_gqa<D, 4, FMT>(dp, mp, casc, fused, batch, kv_heads, st);
        case 8: return run_gqa<D, 8, FMT>(dp, mp, casc, fused, batch, kv_heads, st);
        default: *ok = false; return cudaSuccess;
    }
}

}  // namespace

extern "C" rc_status attn_decode_workspace(const rc_attn_desc* desc, int32_t batch, int32_t max_len,
                                           const rc_cascade* cascade, size_t* bytes) {
    if (!bytes) return RC_ERR_ARG;
    if (desc && desc->pool.mla) {
        if (batch < 0 || max_len < 0 || desc->q_heads <= 0) return RC_ERR_ARG;
        if (cascade && cascade->n_seg > 0) return RC_ERR_UNSUPPORTED;
        *bytes = rc_host::mla_workspace_bound(batch, desc->q_heads, max_len);
        return RC_OK;
    }
    DecodePlan pl;
    rc_status s = plan_decode(desc, batch, max_len, cascade, &pl);
    if (s != RC_OK) return s;
    *bytes = pl.bound;
    return RC_OK;
}

namespace {

// early: the kernel queued just before is the previous step's table pass
// (see MQParams::early)
rc_status decode_impl(const rc_attn_desc* desc, const void* q, const void* k_new, const void* v_new,
                      const rc_kv_table* kv, int32_t batch, const rc_cascade* casc, void* out, float* lse, void* ws,
                      size_t ws_bytes, rc_stream_t stream, bool early = false) {
    if (!desc || !kv || batch < 0) return RC_ERR_ARG;
    if (batch == 0) return RC_OK;
    if (!q || !out || !kv->slots || !kv->start || !kv->len || !desc->pool.k) return RC_ERR_ARG;
    const bool use_casc = casc && casc->n_seg > 0;
    if (desc->pool.mla) {  // one latent KV head: its own kernel (attn_decode_mla.cu)
        if (k_new || desc->pool.kv_fp8) return RC_ERR_UNSUPPORTED;
        if (use_casc) return RC_ERR_UNSUPPORTED;
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return RC_ERR_ARG;
        return rc_host::mla_decode(desc, q, kv, batch, out, lse, ws, ws_bytes, (cudaStream_t)stream);
    }
    DecodePlan pl;
    rc_status s = plan_decode(desc, batch, kv->max_len, use_casc ? casc : nullptr, &pl);
    if (s != RC_OK) return s;
    if (!ws || ws_bytes < pl.total) return RC_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return RC_ERR_ARG;
    if (use_casc && (!casc->seg_slots || !casc->seg_indptr || !casc->seg_row_indptr || !casc->seg_rows ||
                     !casc->req_seg_indptr || !casc->req_seg_pos))
        return RC_ERR_ARG;
    // the cascade masks scores and takes their largest before it scales them
    if (use_casc && !(desc->sm_scale > 0.f)) return RC_ERR_ARG;
    const rc_pool_desc& P = desc->pool;
    const int D = P.head_dim_k;
    if (P.mla || P.head_dim_v != D || !P.v) return RC_ERR_UNSUPPORTED;
    const int fmt = rc_host::pool_format(P);
    const bool fp8 = fmt == rc::kFmtFp8;
    if (fp8) {  // E4M3 pool: the table pass and the cascade read codes and scales
        if (D != 128 || k_new) return RC_ERR_UNSUPPORTED;
        if (!P.k_scale || !P.v_scale) return RC_ERR_ARG;
        if (use_casc && !rc_tc2::fp8_cascade_supported()) return RC_ERR_UNSUPPORTED;
    }
    if (fmt == rc::kFmtFp4) {
        if (k_new) return RC_ERR_UNSUPPORTED;
        s = rc_host::check_fp4(P);
        if (s != RC_OK) return s;
        if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return RC_ERR_ARG;
        if (desc->sm_scale != desc->sm_scale) return RC_ERR_ARG;  // (a negative one is turned into Q)
    }
    const int G = desc->q_heads / P.kv_heads;
    unsigned char* w = static_cast<unsigned char*>(ws);
    unsigned char* ws_seg = w + pl.tail_o + pl.tail_lse + pl.row_runs;
    float* seg_o = reinterpret_cast<float*>(ws_seg);
    float* seg_lse = reinterpret_cast<float*>(ws_seg + pl.seg_o);
    DecParams dp{};
    dp.q = static_cast<const __nv_bfloat16*>(q);
    dp.pool_k = static_cast<const __nv_bfloat16*>(P.k);
    dp.pool_v = static_cast<const __nv_bfloat16*>(P.v);
    dp.n_slots = P.n_slots;
    dp.kv_heads = P.kv_heads;
    dp.q_heads = desc->q_heads;
    dp.scale_log2 = desc->sm_scale * rc::kLog2e;
    dp.err = P.err;
    dp.table = kv->slots;
    dp.start = kv->start;
    dp.len = kv->len;
    dp.table_len = kv->table_len;
    dp.chunk = pl.chunk;
    dp.n_chunks = pl.n_chunks;
    dp.part_o = reinterpret_cast<float*>(w);
    dp.part_lse = reinterpret_cast<float*>(w + pl.tail_o);
    dp.seg_o = seg_o;
    dp.seg_lse = seg_lse;
    dp.req_seg_indptr = use_casc ? casc->req_seg_indptr : nullptr;
    dp.req_seg_pos = use_casc ? casc->req_seg_pos : nullptr;
    dp.seg_chunks = pl.seg_chunks;
    dp.out = static_cast<__nv_bfloat16*>(out);
    dp.lse = lse;
    dp.k_new = static_cast<const __nv_bfloat16*>(k_new);
    dp.v_new = static_cast<const __nv_bfloat16*>(v_new);
    dp.k_scale = fp8 ? P.k_scale : nullptr;
    dp.v_scale = fp8 ? P.v_scale : nullptr;
    dp.k_bscale = fmt == rc::kFmtFp4 ? P.k_bscale : nullptr;
    dp.v_bscale = fmt == rc::kFmtFp4 ? P.v_bscale : nullptr;
    dp.group = G;
    dp.batch = batch;
    dp.max_len = kv->max_len;
    dp.row_runs = reinterpret_cast<int32_t*>(w + pl.tail_o + pl.tail_lse);
    rc::MQParams mp{};
    mp.q = dp.q;
    mp.pool_k = dp.pool_k;
    mp.pool_v = dp.pool_v;
    mp.n_slots = dp.n_slots;
    mp.kv_heads = dp.kv_heads;
    mp.q_heads = dp.q_heads;
    mp.scale_log2 = dp.scale_log2;
    mp.err = dp.err;
    mp.k_scale = dp.k_scale;
    mp.v_scale = dp.v_scale;
    mp.k_bscale = dp.k_bscale;
    mp.v_bscale = dp.v_bscale;
    if (use_casc) {
        mp.seg_slots = casc->seg_slots;
        mp.seg_indptr = casc->seg_indptr;
        mp.seg_row_indptr = casc->seg_row_indptr;
        mp.seg_rows = casc->seg_rows;
        mp.part_o = seg_o;
        mp.part_lse = seg_lse;
        mp.seg_chunk = pl.seg_chunk;
        mp.seg_chunks = pl.seg_chunks;
        mp.early = early ? 1 : 0;
    }
    cudaStream_t st = (cudaStream_t)stream;
    bool ok = false;
    cudaError_t e = cudaSuccess;
    const rc_cascade* cc = use_casc ? casc : nullptr;
    if (fmt == rc::kFmtFp4) {
        if (D == 128) e = dispatch_group<128, rc::kFmtFp4>(G, dp, mp, cc, pl.fused, batch, P.kv_heads, st, &ok);
        else e = dispatch_group<64, rc::kFmtFp4>(G, dp, mp, cc, pl.fused, batch, P.kv_heads, st, &ok);
    } else if (fp8) {
        e = dispatch_group<128, rc::kFmtFp8>(G, dp, mp, cc, pl.fused, batch, P.kv_heads, st, &ok);
    } else if (D == 128) {
        e = dispatch_group<128, rc::kFmtBf16>(G, dp, mp, cc, pl.fused, batch, P.kv_heads, st, &ok);
    } else if (D == 64) {
        e = dispatch_group<64, rc::kFmtBf16>(G, dp, mp, cc, pl.fused, batch, P.kv_heads, st, &ok);
    }
    if (!ok) return RC_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return RC_ERR_CUDA;
    if (pl.fused) return RC_OK;
    if (fmt == rc::kFmtFp4)
        return rc_host::launch_status(D == 128 ? launch_merge_runs<128, false>(dp, batch, st)
                                               : launch_merge_runs<64, false>(dp, batch, st));
    const int32_t* ri = use_casc ? casc->req_seg_indptr : nullptr;
    const int32_t* rp = use_casc ? casc->req_seg_pos : nullptr;
    const unsigned nbh = (unsigned)batch * desc->q_heads;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
    // the merge is the split pass's programmatic dependent (it waits for it
    // inside), so its CTAs start as the split pass's leave
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nbh);
    cfg.blockDim = dim3(32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (D == 128)
        e = cudaLaunchKernelEx(&cfg, merge_kernel<128>, (const float*)dp.part_o, (const float*)dp.part_lse,
                               dp.n_chunks, dp.chunk, dp.len, (const float*)seg_o, (const float*)seg_lse,
                               pl.seg_chunks, ri, rp, desc->q_heads, dp.start, dp.table_len, o, lse, P.err);
    else
        e = cudaLaunchKernelEx(&cfg, merge_kernel<64>, (const float*)dp.part_o, (const float*)dp.part_lse,
                               dp.n_chunks, dp.chunk, dp.len, (const float*)seg_o, (const float*)seg_lse,
                               pl.seg_chunks, ri, rp, desc->q_heads, dp.start, dp.table_len, o, lse, P.err);
    return rc_host::launch_status(e);
}

}  // namespace

extern "C" rc_status attn_decode(const rc_attn_desc* desc, const void* q, const rc_kv_table* kv, int32_t batch,
                                 const rc_cascade* casc, void* out, float* lse, void* ws, size_t ws_bytes,
                                 rc_stream_t stream) {
    return decode_impl(desc, q, nullptr, nullptr, kv, batch, casc, out, lse, ws, ws_bytes, stream);
}

extern "C" rc_status attn_decode_append(const rc_attn_desc* desc, const void* q, const void* k_new,
                                        const void* v_new, const rc_kv_table* kv, int32_t batch,
                                        const rc_cascade* casc, void* out, float* lse, void* ws, size_t ws_bytes,
                                        rc_stream_t stream) {
    if (!k_new || !v_new) return RC_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return RC_ERR_ARG;
    return decode_impl(desc, q, k_new, v_new, kv, batch, casc, out, lse, ws, ws_bytes, stream);
}

extern "C" rc_status attn_decode_steps(const rc_attn_desc* desc, const rc_kv_table* kv, int32_t batch,
                                       const rc_cascade* casc, const rc_decode_step* steps, int32_t n_steps,
                                       void* ws, size_t ws_bytes, rc_stream_t stream, int32_t* n_done) {
    if (n_done) *n_done = 0;
    if (!desc || !kv || n_steps < 0 || (n_steps > 0 && !steps)) return RC_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    for (int32_t i = 0; i < n_steps; ++i) {
        const rc_decode_step& s = steps[i];
        if (s.ev_begin && cudaEventRecord((cudaEvent_t)s.ev_begin, st) != cudaSuccess) return RC_ERR_CUDA;
        rc_kv_table t = *kv;
        t.len = s.len;
        t.max_len = s.max_len;
        rc_status r;
        if (s.store_slots) {
            r = kv_store(&desc->pool, s.store_slots, s.k_new, s.v_new, batch, nullptr, nullptr, stream);
            if (r == RC_OK) r = attn_decode(desc, s.q, &t, batch, casc, s.out, s.lse, ws, ws_bytes, stream);
        } else if (s.k_new) {
            if ((reinterpret_cast<uintptr_t>(s.k_new) | reinterpret_cast<uintptr_t>(s.v_new)) & 15 || !s.v_new) {
                r = RC_ERR_ARG;
            } else {
                // after an append step with no event in between, the kernel queued
                // last is that step's table pass (or its merge): this step's
                // cascade may read before waiting for it
                const rc_decode_step* pv = i > 0 ? &steps[i - 1] : nullptr;
                const bool early = pv && pv->k_new && !pv->store_slots && !pv->ev_end && !s.ev_begin;
                r = decode_impl(desc, s.q, s.k_new, s.v_new, &t, batch, casc, s.out, s.lse, ws, ws_bytes, stream,
                                early);
            }
        } else {
            r = attn_decode(desc, s.q, &t, batch, casc, s.out, s.lse, ws, ws_bytes, stream);
        }
        if (r != RC_OK) return r;
        if (s.ev_end && cudaEventRecord((cudaEvent_t)s.ev_end, st) != cudaSuccess) return RC_ERR_CUDA;
        if (n_done) *n_done = i + 1;
    }
    return RC_OK;
}

// ---------------------------------------------------------------------------
// Allocation-free variant.  The split partials go to a file-scope device
// array instead of a caller workspace.  In host code the array's name is only
// a host-side stand-in, so its device address is looked up once per device
// (with that device current) and passed to the kernels like any workspace.

#include <mutex>

namespace {

static __device__ __align__(256) unsigned char rc_decode_scratch[RC_STATIC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
void* g_scratch_ptr[kMaxDevices] = {nullptr};
std::mutex g_scratch_mu;

rc_status scratch_for_current_device(void** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RC_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return RC_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, rc_decode_scratch) != cudaSuccess || !p) return RC_ERR_CUDA;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return RC_OK;
}

}  // namespace

extern "C" rc_status attn_decode_static(const rc_attn_desc* desc, const void* q, const rc_kv_table* kv,
                                        int32_t batch, const rc_cascade* casc, void* out, float* lse,
                                        rc_stream_t stream) {
    if (!desc || !kv || batch < 0) return RC_ERR_ARG;
    if (batch == 0) return RC_OK;
    const rc_cascade* cc = casc && casc->n_seg > 0 ? casc : nullptr;  // as attn_decode plans it
    size_t need = 0;  // of this very call, not of every smaller max_len
    rc_status s = RC_OK;
    if (desc->pool.mla) {
        if (kv->max_len < 0 || desc->q_heads <= 0) return RC_ERR_ARG;
        if (cc) return RC_ERR_UNSUPPORTED;
        need = rc_host::mla_workspace(batch, desc->q_heads, kv->max_len);
    } else {
        DecodePlan pl;
        s = plan_decode(desc, batch, kv->max_len, cc, &pl);
        if (s != RC_OK) return s;
        need = pl.total;
    }
    if (need > (size_t)RC_STATIC_SCRATCH_BYTES) return RC_ERR_SCRATCH;
    void* ws = nullptr;
    s = scratch_for_current_device(&ws);
    if (s != RC_OK) return s;
    return attn_decode(desc, q, kv, batch, casc, out, lse, ws, (size_t)RC_STATIC_SCRATCH_BYTES, stream);
}
