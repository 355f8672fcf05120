// kv_load: rows of the pool, in whatever type it holds them, as dense bf16.
//
//   out[i] = bf16(code * scale)   over the rows of slot slots[i]
//
// (bf16 and latent pools: the rows as they are.)  Pure data movement: each row is
// read once and written once, so HBM bounds it.  A thread takes 16 values, which
// are 32 bytes of output (one 256-bit store where the arrays are aligned to it; two
// 16-byte stores, each half a sector wide per lane, otherwise), 8 bytes of E2M1
// codes with their scale byte, or 16 of E4M3 codes; consecutive lanes take
// consecutive values.  A warp takes UN runs of 32 such units, all loads before the
// first use: one while all threads run at once, which is the shorter way for few tokens, two
// beyond (8 KV heads of 128, 1, 2, 4 and 8 of them, a call among others: 27 tokens of E4M3 2.75,
// 3.2, 3.4 and 4.4 us, 60,001 of 4 bits 60.7, 53.3, 57.5 and 67.5).
// Measured (from a graph): 60,001 tokens, 8 KV heads of 128, 4 bits 51.1 us, 6.2 TB/s of what is
// read and written (a copy does 6.8), E4M3 57.8, bf16 73.5, latent rows 23.0; 1,792 tokens of
// E4M3 3.7 us, of which 0.8 is an empty launch's: the slot, then code and scale, then the store
// wait for one another.

#include "common.cuh"

namespace {

constexpr int kThreads = 128;

struct LoadParams {
    const void* pool[2];          // K, V
    const float* scale[2];        // E4M3
    const uint8_t* bscale[2];     // 4 bits
    __nv_bfloat16* out[2];
    int64_t stride[2];            // elements between tokens
    int64_t n_slots;
    const int32_t* slots;
    int32_t n, kv_heads;
    int32_t units[2];             // units a token of K and of V (0: not asked for)
    int32_t* err;
};

struct Word8 {
    uint32_t w[8];
};

template <bool WIDE>
RC_DEV void store32(void* dst, const Word8& x) {
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(x.w[0]), "r"(x.w[1]),
                     "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
    }
}

// a pair of f16 to a pair of bf16 after a product in fp32
RC_DEV uint32_t scaled_pair(uint32_t h2, float s) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    return rc::pack_bf16(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
}

// CH: units a head row (D / 16)
template <int CH, int FMT, int UN, bool WIDE>
__global__ void __launch_bounds__(kThreads) load_kernel(const LoadParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int per = p.units[0] + p.units[1];
    const int64_t first = warp * (32 * UN);
    const int64_t t0 = first / per;
    const int rest = (int)(first - t0 * per);
    Word8 x[UN];
    float s[UN];
    int tok[UN], unit[UN], which[UN], slot[UN];
    bool live[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const int e = rest + 32 * i + lane, dt = e / per;
        unit[i] = e - dt * per;
        which[i] = unit[i] >= p.units[0];
        if (which[i]) unit[i] -= p.units[0];
        live[i] = t0 + dt < p.n;
        tok[i] = live[i] ? (int)(t0 + dt) : 0;
        slot[i] = __ldg(p.slots + tok[i]);
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const bool ok = slot[i] >= 0 && (int64_t)slot[i] < p.n_slots;
        if (live[i] && !ok) rc::flag_error(p.err, rc::kErrBadSlot);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i].w[k] = 0u;
        s[i] = 0.f;
        if (!live[i] || !ok) continue;  // a slot outside the pool reads as zeros
        const int64_t at = (int64_t)slot[i] * p.kv_heads * CH + unit[i];  // 16-value units into the pool
        const unsigned char* src = static_cast<const unsigned char*>(which[i] ? p.pool[1] : p.pool[0]);
        if constexpr (FMT == rc::kFmtBf16) {
            const uint4* q = reinterpret_cast<const uint4*>(src + at * 32);
            const uint4 a = __ldg(q), b = __ldg(q + 1);
            x[i] = Word8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
        } else if constexpr (FMT == rc::kFmtFp8) {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(src + at * 16));
            x[i].w[0] = a.x, x[i].w[1] = a.y, x[i].w[2] = a.z, x[i].w[3] = a.w;
            s[i] = __ldg((which[i] ? p.scale[1] : p.scale[0]) + at / CH);
        } else {
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(src + at * 8));
            x[i].w[0] = a.x, x[i].w[1] = a.y;
            x[i].w[2] = __ldg((which[i] ? p.bscale[1] : p.bscale[0]) + at);
        }
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        Word8 y = x[i];
        if constexpr (FMT == rc::kFmtFp8) {  // code x scale rounded to fp32, then to bf16
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t lo, hi;
                rc::e4m3x4_to_f16x4(x[i].w[k], lo, hi);
                y.w[2 * k] = scaled_pair(lo, s[i]);
                y.w[2 * k + 1] = scaled_pair(hi, s[i]);
            }
        } else if constexpr (FMT == rc::kFmtFp4) {  // code x scale has at most six significant bits: exact
            const float sc = __half2float(__ushort_as_half((unsigned short)(x[i].w[2] << 7)));
            uint32_t h[8];
            rc::e2m1x8_to_f16x8(x[i].w[0], h[0], h[1], h[2], h[3]);
            rc::e2m1x8_to_f16x8(x[i].w[1], h[4], h[5], h[6], h[7]);
#pragma unroll
            for (int k = 0; k < 8; ++k) y.w[k] = scaled_pair(h[k], sc);
        }
        if (live[i])
            store32<WIDE>((which[i] ? p.out[1] : p.out[0]) + tok[i] * (which[i] ? p.stride[1] : p.stride[0]) +
                              (int64_t)unit[i] * 16,
                          y);
    }
}

template <int CH, int FMT>
rc_status launch(const LoadParams& p, cudaStream_t st) {
    const int64_t units = (int64_t)p.n * (p.units[0] + p.units[1]);
    const bool few = units <= (int64_t)rc_host::sm_count() * 2048;
    const int a_block = kThreads * (few ? 1 : 2);
    const int64_t blocks = (units + a_block - 1) / a_block;
    if (blocks > 0x7fffffff) return RC_ERR_ARG;
    bool wide = true;
    for (int a = 0; a < 2; ++a)
        if (p.units[a] && ((reinterpret_cast<uintptr_t>(p.out[a]) & 31) || p.stride[a] % 16)) wide = false;
    auto* const kernel = few ? wide ? load_kernel<CH, FMT, 1, true> : load_kernel<CH, FMT, 1, false>
                             : wide ? load_kernel<CH, FMT, 2, true> : load_kernel<CH, FMT, 2, false>;
    kernel<<<(unsigned)blocks, kThreads, 0, st>>>(p);
    return rc_host::launch_status(cudaGetLastError());
}

}  // namespace

extern "C" rc_status kv_load(const rc_pool_desc* pool, const int32_t* slots, int32_t n, void* k_out, int64_t k_stride,
                             void* v_out, int64_t v_stride, rc_stream_t stream) {
    if (!pool || n < 0 || !pool->k || pool->kv_heads <= 0 || pool->head_dim_k <= 0 || pool->n_slots <= 0) return RC_ERR_ARG;
    const int fmt = rc_host::pool_format(*pool);
    const int D = pool->head_dim_k;
    if (pool->mla) {
        if (fmt != rc::kFmtBf16 || pool->kv_heads != 1 || D != 576) return RC_ERR_UNSUPPORTED;
        if (v_out) return RC_ERR_ARG;  // V is K's first columns
    } else {
        if (pool->head_dim_v != D || (D != 128 && D != 64)) return RC_ERR_UNSUPPORTED;
        if (fmt == rc::kFmtFp8 && D != 128) return RC_ERR_UNSUPPORTED;
        if (!pool->v) return RC_ERR_ARG;
    }
    if (fmt == rc::kFmtFp8 && (!pool->k_scale || !pool->v_scale)) return RC_ERR_ARG;
    if (fmt == rc::kFmtFp4) {
        const rc_status s = rc_host::check_fp4(*pool);
        if (s != RC_OK) return s;
    }
    if (n > 0 && !k_out && !v_out) return RC_ERR_ARG;  // (no rows: an empty tensor's address may be NULL)
    const int64_t row = (int64_t)pool->kv_heads * D;
    if (row > (1 << 24)) return RC_ERR_UNSUPPORTED;
    if ((k_out && (k_stride < row || k_stride % 8)) || (v_out && (v_stride < row || v_stride % 8))) return RC_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(pool->k) | reinterpret_cast<uintptr_t>(pool->v) | reinterpret_cast<uintptr_t>(k_out) |
         reinterpret_cast<uintptr_t>(v_out)) & 15)
        return RC_ERR_ARG;
    if (n == 0) return RC_OK;
    if (!slots) return RC_ERR_ARG;
    const int64_t rows = pool->n_slots * pool->kv_heads;
    const int64_t bytes = fmt == rc::kFmtBf16 ? rows * D * 2 : fmt == rc::kFmtFp8 ? rows * D : rows * D / 2;
    for (int i = 0; i < 2; ++i) {  // other blocks may still read what these rows would go over
        const void* const out = i ? v_out : k_out;
        const int64_t stride = (i ? v_stride : k_stride) * 2;
        auto over = [&](const void* in, int64_t size) { return rc_host::overlap(in, size, out, n, stride, row * 2); };
        if (over(slots, (int64_t)n * 4) || over(pool->k, bytes) || (!pool->mla && over(pool->v, bytes))) return RC_ERR_ARG;
        if (fmt == rc::kFmtFp8 && (over(pool->k_scale, rows * 4) || over(pool->v_scale, rows * 4))) return RC_ERR_ARG;
        if (fmt == rc::kFmtFp4 && (over(pool->k_bscale, rows * D / 16) || over(pool->v_bscale, rows * D / 16))) return RC_ERR_ARG;
    }
    LoadParams p{};
    p.pool[0] = pool->k;
    p.pool[1] = pool->v;
    p.scale[0] = pool->k_scale;
    p.scale[1] = pool->v_scale;
    if (fmt == rc::kFmtFp4) {
        p.bscale[0] = pool->k_bscale;
        p.bscale[1] = pool->v_bscale;
    }
    p.out[0] = static_cast<__nv_bfloat16*>(k_out);
    p.out[1] = static_cast<__nv_bfloat16*>(v_out);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.n_slots = pool->n_slots;
    p.slots = slots;
    p.n = n;
    p.kv_heads = pool->kv_heads;
    p.units[0] = k_out ? (int)(row / 16) : 0;
    p.units[1] = v_out ? (int)(row / 16) : 0;
    p.err = pool->err;
    cudaStream_t st = (cudaStream_t)stream;
    if (pool->mla) return launch<36, rc::kFmtBf16>(p, st);
    if (fmt == rc::kFmtFp8) return launch<8, rc::kFmtFp8>(p, st);
    if (fmt == rc::kFmtFp4) return D == 128 ? launch<8, rc::kFmtFp4>(p, st) : launch<4, rc::kFmtFp4>(p, st);
    return D == 128 ? launch<8, rc::kFmtBf16>(p, st) : launch<4, rc::kFmtBf16>(p, st);
}
