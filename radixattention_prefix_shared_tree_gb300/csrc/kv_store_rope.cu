// kv_store_rope: append new tokens' K and V to the pool with the position
// rotation of K (and of Q) applied on the way; and kv_store for a 4-bit pool
// (the same kernel without a rotation).
//
//   (y_a, y_b) = (x_a cos - x_b sin, x_b cos + x_a sin)
//
// over the pairs (a, b) of the rotated columns, in fp32 with one rounding per
// product and sum, then one rounding to the type the pool holds.  Pure data
// movement: each K, V and Q value is read once and written once, so HBM bounds
// large calls and launch latency small ones.  A thread holds 16 values of one
// head row, two 16-byte chunks chosen so that both halves of every rotated
// pair are its own (no exchange between threads, and Q may be rotated in
// place); consecutive lanes hold consecutive chunks, so a warp reads and writes
// whole rows.  With 64 or 128 columns a lane meets the same columns in every
// row, so it keeps their cosines and sines in registers for all its rows.

#include "tc.cuh"

#include <type_traits>

namespace {

constexpr int kWarps = 4;  // per block

struct StoreParams {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;   // NULL: latent pool
    const __nv_bfloat16* q;   // NULL: no queries
    __nv_bfloat16* q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;  // elements between tokens
    const int32_t* slots;
    const int32_t* positions; // [n], or with axes [axes][n]
    const float* cos_sin;     // [max_pos][rot]: cosines, then sines
    int32_t axes;
    uint32_t pair_axis[18];   // axes > 1: two bits a pair, a byte to the four pairs of a 16-byte group of cosines
    int32_t max_pos, rot, offset;
    int32_t n, kv_heads, q_heads;
    void* pool_k;
    void* pool_v;
    float* k_scale;
    float* v_scale;
    uint8_t* k_bscale;
    uint8_t* v_bscale;
    int64_t n_slots;
    int32_t* table;
    const int32_t* table_pos;
    int32_t* err;
    int32_t slices;    // warps per token
    int32_t per_slice; // units (thread's 16 values) per warp, a multiple of 32
};

RC_DEV void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
RC_DEV uint4 pack(const float (&x)[8]) {
    return make_uint4(rc::pack_bf16(x[0], x[1]), rc::pack_bf16(x[2], x[3]), rc::pack_bf16(x[4], x[5]),
                      rc::pack_bf16(x[6], x[7]));
}
RC_DEV uint32_t abs_bits_max(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

// Scale byte of a block whose largest magnitude has the bits `amax`: amax / 6
// rounded to 5 exponent and 3 mantissa bits (nearest, ties to even), at most
// 10240; 0xff (a NaN) for a block with a non-finite value.
RC_DEV uint32_t block_scale(uint32_t amax) {
    if (amax >= 0x7f800000u) return 0xffu;
    const float raw = fminf(__fdiv_rn(__uint_as_float(amax), 6.f), 10240.f);
    if (raw < 6.103515625e-05f) return (uint32_t)__float2int_rn(raw * 131072.f);  // below 2^-14: steps of 2^-17
    uint32_t u = __float_as_uint(raw);
    u += 0x7ffffu + ((u >> 20) & 1u);
    return (u >> 20) - 896u;  // exponent bias 127 -> 15
}
RC_DEV float block_scale_value(uint32_t byte) {
    return byte < 8u ? (float)byte * 7.62939453125e-06f : __uint_as_float((byte + 896u) << 20);
}
// Eight E2M1 codes, x[0] in the low nibble: nearest of x / s, ties to even, at most 6
// in magnitude.  The borders between codes are T = 1/4, 3/4, .. 5, three bits, and s has
// four: T s is exact, so an x that is not T s is a step of fp32 away from it at least,
// and its quotient, rounded to fp32, is not T either.  So any quotient good to a step
// decides as the exact one does, if it is T where x = T s: q of 12 bits, whose product
// with s is exact, plus the remainder (exact, too) over s.  (16 divisions a thread
// instead: 46.6 us for 9,001 tokens of 8 KV and 32 query heads of 128, against 43.9.)
RC_DEV uint32_t e2m1_codes(const float (&x)[8], uint32_t byte) {
    if (byte == 0u || byte == 0xffu) return 0u;
    const float s = block_scale_value(byte), r = __frcp_rn(s);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = make_float2(x[i], x[i + 1]);
        float2 q = tc::fmul2(v, r);
        q.x = __uint_as_float(__float_as_uint(q.x) & 0xfffff000u);
        q.y = __uint_as_float(__float_as_uint(q.y) & 0xfffff000u);
        const float2 z = tc::ffma2(tc::ffma2(q, -s, v), r, q);
        y[i] = copysignf(z.x, v.x), y[i + 1] = copysignf(z.y, v.y);  // (of -0 too)
    }
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}\n"
        : "=r"(d)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return d;
}
// Eight E4M3 codes of x / scale, x[0] in the low byte.
RC_DEV uint2 e4m3_codes(const float (&x)[8], float scale) {
    const bool some = scale > 0.f;  // otherwise a row of zeros and NaNs: as it is
    const float by = some ? scale : 1.f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], by), __fdiv_rn(x[2 * i + 1], by)),
                                        __NV_SATFINITE, __NV_E4M3);
    const uint2 c = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    return some ? c : make_uint2(rc::e4m3_only_nans(c.x), rc::e4m3_only_nans(c.y));
}

// U: units per head row (D / 16).  ROT 0: no rotation; 1: pairs half the
// rotated width apart; 2: neighbouring pairs.  AXES: a pair's angle is that of its
// own axis' position (image and video tokens: a row, a column and a frame); four
// pairs of one axis still take one 16-byte load of cosines and one of sines.
template <int U, int FMT, int ROT, int UN, bool AXES>
__global__ void __launch_bounds__(32 * kWarps) store_rope_kernel(const StoreParams p) {
    constexpr int D = 16 * U, CH = 2 * U;
    constexpr bool FIXED = 32 % U == 0;  // a lane's unit is the same in every row
    const int lane = threadIdx.x & 31;
    const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int t = (int)(item / p.slices), slice = (int)(item % p.slices);
    if (t >= p.n) return;
    const int k_rows = p.kv_heads, v_rows = p.v ? p.kv_heads : 0;
    const int units = (k_rows + v_rows + (p.q ? p.q_heads : 0)) * U;
    const int begin = slice * p.per_slice, end = min(begin + p.per_slice, units);
    const int slot = __ldg(p.slots + t);
    const bool slot_ok = slot >= 0 && (int64_t)slot < p.n_slots;
    int pos = 0;
    if constexpr (ROT != 0) {
        pos = __ldg(p.positions + t);
        if (pos < 0 || pos >= p.max_pos) {  // no angles for it: the token is left out
            if (slice == 0 && lane == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            return;
        }
    }
    int pos1 = pos, pos2 = pos, pos3 = pos;
    if constexpr (AXES) {
        pos1 = __ldg(p.positions + p.n + (int64_t)t);
        if (p.axes > 2) pos2 = __ldg(p.positions + 2 * (int64_t)p.n + t);
        if (p.axes > 3) pos3 = __ldg(p.positions + 3 * (int64_t)p.n + t);
        if (min(min(pos1, pos2), pos3) < 0 || max(max(pos1, pos2), pos3) >= p.max_pos) {
            if (slice == 0 && lane == 0) rc::flag_error(p.err, rc::kErrBadSlot);
            return;
        }
    }
    if (slice == 0 && lane == 0) {
        if (!slot_ok) rc::flag_error(p.err, rc::kErrBadSlot);
        else if (p.table) p.table[__ldg(p.table_pos + t)] = slot;
    }
    const bool in_place = p.q_out == p.q && p.q_out_stride == p.q_stride;
    const int rot_ch = p.rot / 8, off_ch = p.offset / 8;  // the rotated chunks: off_ch .. off_ch + rot_ch - 1
    const float* angles = p.cos_sin + (int64_t)pos * p.rot;

    // unit u's chunks, whether they turn, and (ROT 1) the pair's angle index
    auto chunks = [&](int u, int& c0, int& c1, bool& r0, bool& r1) {
        if constexpr (ROT == 1) {
            if (u < rot_ch / 2) {
                c0 = off_ch + u;
                c1 = c0 + rot_ch / 2;
                r0 = r1 = true;
            } else {  // the columns beside the rotated ones, likewise in two halves
                const int i = u - rot_ch / 2, j = i + (CH - rot_ch) / 2;
                c0 = i < off_ch ? i : i + rot_ch;
                c1 = j < off_ch ? j : j + rot_ch;
                r0 = r1 = false;
            }
        } else {
            c0 = u;
            c1 = u + U;
            r0 = ROT == 2 && c0 >= off_ch && c0 < off_ch + rot_ch;
            r1 = ROT == 2 && c1 >= off_ch && c1 < off_ch + rot_ch;
        }
    };
    // ROT 1: cs = 8 cosines, sn = 8 sines of the pairs; ROT 2: the first four of
    // each belong to chunk c0, the others to c1
    float cs[8], sn[8];
    auto load_angles = [&](int u, int c0, int c1, bool r0, bool r1) {
        const float4* c4 = reinterpret_cast<const float4*>(angles);
        const int half = p.rot / 8;  // float4s to the sines
        const int i0 = ROT == 1 ? 2 * u : c0 - off_ch, i1 = ROT == 1 ? 2 * u + 1 : c1 - off_ch;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 a = z, b = z, c = z, d = z;
        if constexpr (AXES) {
            auto group = [&](int i, float4& cos4, float4& sin4) {  // pairs 4i .. 4i + 3
                const uint32_t ax = (p.pair_axis[i >> 2] >> ((i & 3) * 8)) & 255u;
                auto row = [&](uint32_t k) {
                    const int at = k == 0 ? pos : k == 1 ? pos1 : k == 2 ? pos2 : pos3;
                    return p.cos_sin + (int64_t)at * p.rot + 4 * i;
                };
                if (ax == (ax & 3u) * 0x55u) {
                    const float4* r4 = reinterpret_cast<const float4*>(row(ax & 3u));
                    cos4 = __ldg(r4);
                    sin4 = __ldg(r4 + half);
                } else {
                    const float *ra = row(ax & 3u), *rb = row((ax >> 2) & 3u), *rc_ = row((ax >> 4) & 3u), *rd = row(ax >> 6);
                    const int to_sin = 4 * half;
                    cos4 = make_float4(__ldg(ra), __ldg(rb + 1), __ldg(rc_ + 2), __ldg(rd + 3));
                    sin4 = make_float4(__ldg(ra + to_sin), __ldg(rb + to_sin + 1), __ldg(rc_ + to_sin + 2),
                                       __ldg(rd + to_sin + 3));
                }
            };
            if (r0) group(i0, a, c);
            if (r1) group(i1, b, d);
        } else {
            if (r0) a = __ldg(c4 + i0);
            if (r1) b = __ldg(c4 + i1);
            if (r0) c = __ldg(c4 + half + i0);
            if (r1) d = __ldg(c4 + half + i1);
        }
        cs[0] = a.x, cs[1] = a.y, cs[2] = a.z, cs[3] = a.w, cs[4] = b.x, cs[5] = b.y, cs[6] = b.z, cs[7] = b.w;
        sn[0] = c.x, sn[1] = c.y, sn[2] = c.z, sn[3] = c.w, sn[4] = d.x, sn[5] = d.y, sn[6] = d.z, sn[7] = d.w;
    };
    auto turn = [](float& a, float& b, float c, float s) {  // no contraction: one rounding each
        const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
        a = x;
    };
    // what unit e of the token is: its row's source and head, its chunks, whether
    // they turn, and whether they are read at all
    struct Unit {
        const uint4* src;
        int head, u, c0, c1;
        bool live, is_k, is_q, r0, r1, t0, t1;
    };
    int fc0 = 0, fc1 = 0;
    bool fr0 = false, fr1 = false;
    if constexpr (FIXED) {
        chunks(lane % U, fc0, fc1, fr0, fr1);
        if constexpr (ROT != 0) load_angles(lane % U, fc0, fc1, fr0, fr1);
    }

    auto unit = [&](int e) -> Unit {
        Unit m;
        m.live = e < end;
        const int row = e / U;
        m.u = FIXED ? lane % U : e - row * U;
        m.c0 = fc0, m.c1 = fc1, m.r0 = fr0, m.r1 = fr1;
        if constexpr (!FIXED) chunks(m.u, m.c0, m.c1, m.r0, m.r1);
        m.is_k = row < k_rows;
        m.is_q = row >= k_rows + v_rows;
        m.head = m.is_k ? row : m.is_q ? row - k_rows - v_rows : row - k_rows;
        if (!m.is_k && !m.is_q) m.r0 = m.r1 = false;  // V is stored as it is
        const __nv_bfloat16* s = m.is_q ? p.q + (int64_t)t * p.q_stride
                                        : m.is_k ? p.k + (int64_t)t * p.k_stride : p.v + (int64_t)t * p.v_stride;
        m.src = reinterpret_cast<const uint4*>(s + (int64_t)m.head * D);
        const bool keep = m.is_q && in_place;  // columns that stay as they are need no copy
        m.t0 = m.live && !(keep && !m.r0);
        m.t1 = m.live && !(keep && !m.r1);
        return m;
    };

    // UN units per lane at a time, all their loads before the first is used
    for (int e0 = begin; e0 < end; e0 += 32 * UN) {
        uint4 w0[UN], w1[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const Unit m = unit(e0 + 32 * i + lane);
            const uint4 z = make_uint4(0, 0, 0, 0);
            w0[i] = m.t0 ? m.src[m.c0] : z;
            w1[i] = m.t1 ? m.src[m.c1] : z;
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            if (e0 + 32 * i >= end) break;  // (uniform)
            const Unit m = unit(e0 + 32 * i + lane);
            float x0[8], x1[8];
            if constexpr (ROT != 0 || FMT != rc::kFmtBf16) {
                unpack(w0[i], x0);
                unpack(w1[i], x1);
                if constexpr (ROT != 0 && !FIXED)
                    if (m.r0 || m.r1) load_angles(m.u, m.c0, m.c1, m.r0, m.r1);
                if constexpr (ROT == 1) {
                    if (m.r0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) turn(x0[j], x1[j], cs[j], sn[j]);
                    }
                }
                if constexpr (ROT == 2) {
                    if (m.r0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) turn(x0[2 * j], x0[2 * j + 1], cs[j], sn[j]);
                    }
                    if (m.r1) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) turn(x1[2 * j], x1[2 * j + 1], cs[4 + j], sn[4 + j]);
                    }
                }
                if (m.r0) w0[i] = pack(x0);
                if (m.r1) w1[i] = pack(x1);
            }
            if (m.is_q) {
                uint4* d4 = reinterpret_cast<uint4*>(p.q_out + (int64_t)t * p.q_out_stride + (int64_t)m.head * D);
                if (m.t0) d4[m.c0] = w0[i];
                if (m.t1) d4[m.c1] = w1[i];
            }
            const bool put = m.live && !m.is_q && slot_ok;
            const int64_t prow = (int64_t)(slot_ok ? slot : 0) * p.kv_heads + m.head;
            if constexpr (FMT == rc::kFmtBf16) {
                uint4* d4 = reinterpret_cast<uint4*>(m.is_k ? p.pool_k : p.pool_v) + prow * CH;
                if (put) {
                    d4[m.c0] = w0[i];
                    d4[m.c1] = w1[i];
                }
            } else if constexpr (FMT == rc::kFmtFp8) {  // 8 lanes hold a row
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(fabsf(x0[j]), fabsf(x1[j])));
#pragma unroll
                for (int j = 1; j < U; j <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, j));
                const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
                if (put) {
                    uint2* d2 = reinterpret_cast<uint2*>(m.is_k ? p.pool_k : p.pool_v) + prow * CH;
                    d2[m.c0] = e4m3_codes(x0, scale);
                    d2[m.c1] = e4m3_codes(x1, scale);
                    if (m.u == 0) (m.is_k ? p.k_scale : p.v_scale)[prow] = scale;
                }
            } else {  // a block of 16 is the chunk of this lane and the next: chunks 2i and 2i + 1
                uint32_t a0 = abs_bits_max(x0), a1 = abs_bits_max(x1);
                a0 = max(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
                a1 = max(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
                if (put) {
                    const uint32_t b0 = block_scale(a0), b1 = block_scale(a1);
                    uint32_t* d1 = reinterpret_cast<uint32_t*>(m.is_k ? p.pool_k : p.pool_v) + prow * CH;
                    d1[m.c0] = e2m1_codes(x0, b0);
                    d1[m.c1] = e2m1_codes(x1, b1);
                    if (!(lane & 1)) {
                        uint8_t* bs = (m.is_k ? p.k_bscale : p.v_bscale) + prow * U;
                        bs[m.c0 / 2] = (uint8_t)b0;
                        bs[m.c1 / 2] = (uint8_t)b1;
                    }
                }
            }
        }
    }
}

// Warps of the kernel that the GPU holds at once (the occupancy does not depend on the call).
template <int U, int FMT, int ROT, int UN, bool AXES>
int64_t resident() {
    static const int an_sm = [] {
        int blocks = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, store_rope_kernel<U, FMT, ROT, UN, AXES>, 32 * kWarps, 0) !=
            cudaSuccess)
            blocks = 0;
        return blocks > 0 ? blocks * kWarps : 16;
    }();
    return (int64_t)an_sm * rc_host::sm_count();
}

template <int U, int FMT, int ROT, bool AXES = false>
rc_status launch(StoreParams& p, cudaStream_t st) {
    const int units = (p.kv_heads * (p.v ? 2 : 1) + (p.q ? p.q_heads : 0)) * U;
    // A warp takes one 32-unit pass of its token while that keeps the grid within a few
    // waves.  Beyond, it takes several, which share the token's positions and angles, with
    // the loads of some of them on their way together.
    const int passes = (units + 31) / 32;
    int cut = passes, ahead = 1;  // warps a token, of as many passes each as any other; passes ahead
    if (passes > 1 && (int64_t)p.n * passes > (int64_t)rc_host::sm_count() * 64) {
        auto warps_of = [&](int most) { return (passes + most - 1) / most; };
        if constexpr (U == 36) {
            // Latent rows: 4 and 4 (1,023 tokens of 128 query heads: 56 us, 60 with 2 ahead), but with
            // several axes a unit's angles take registers too (9,001 tokens of 16: 130 us, 86 with 2 ahead).
            cut = warps_of(4);
            ahead = AXES ? 2 : 4;
        } else {
            // 4 to 12 passes a warp, whatever takes the fewest waves of passes.  A token's first
            // loads (slot, position, angles, values, one after the other) cost a warp about as
            // much as six passes, seven with several axes (8 KV and 32 query heads of 128 into
            // an 8-bit pool, 6 against 12 passes a warp: 1,200 tokens 9.9 and 12.6 us, 2,100 17.0
            // and 14.6, 9,001 51.4 and 43.7).  Three passes' loads are ahead (80 to 100 registers a
            // thread, 20 to 24 warps an SM; with six ahead 120 and 16: 9,001 tokens 57.6 us), or all
            // of four, where as many warps find room (811 tokens 8.5 us, 9.1 with three).
            int64_t least = INT64_MAX;
            auto weigh = [&](int c, int un, int64_t room, int more) {
                const int64_t cost = (((int64_t)p.n * c + room - 1) / room) * ((passes + c - 1) / c + (AXES ? 7 : 6) + more);
                if (cost <= least) least = cost, cut = c, ahead = un;
            };
            for (int c = warps_of(12); c <= warps_of(AXES ? 6 : 4); ++c) {
                const bool four = !AXES && (passes + c - 1) / c == 4;
                weigh(c, 3, resident<U, FMT, ROT, 3, AXES>(), four ? 3 : 0);
                if constexpr (!AXES)
                    if (four) weigh(c, 4, resident<U, FMT, ROT, 4, AXES>(), 0);
            }
            // Six ahead into a bf16 pool while all warps run at once even so (1,100 tokens 7.0 us,
            // 7.3 with three; into an 8-bit pool 10.0 and 9.8).
            if constexpr (FMT == rc::kFmtBf16 && !AXES) {
                const int per = (passes + cut - 1) / cut;
                if (ahead == 3 && per > 4 && per <= 6 && (int64_t)p.n * cut <= resident<U, FMT, ROT, 6, AXES>()) ahead = 6;
            }
        }
    }
    p.per_slice = 32 * ((passes + cut - 1) / cut);
    p.slices = (units + p.per_slice - 1) / p.per_slice;
    const int64_t warps = (int64_t)p.n * p.slices;
    const int64_t blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return RC_ERR_ARG;
    auto go = [&](auto un) { store_rope_kernel<U, FMT, ROT, un(), AXES><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(p); };
    if (ahead == 1) go(std::integral_constant<int, 1>());
    else if constexpr (U == 36) go(std::integral_constant<int, AXES ? 2 : 4>());
    else if (ahead == 3) go(std::integral_constant<int, 3>());
    else if constexpr (!AXES) {
        if (ahead == 4) go(std::integral_constant<int, 4>());
        else if constexpr (FMT == rc::kFmtBf16) go(std::integral_constant<int, 6>());
    }
    return rc_host::launch_status(cudaGetLastError());
}

template <int U, int FMT>
rc_status launch_rot(StoreParams& p, int rot, cudaStream_t st) {
    if (rot == 1) return p.axes > 1 ? launch<U, FMT, 1, true>(p, st) : launch<U, FMT, 1>(p, st);
    if (rot == 2) return p.axes > 1 ? launch<U, FMT, 2, true>(p, st) : launch<U, FMT, 2>(p, st);
    if constexpr (FMT == rc::kFmtFp4) return launch<U, FMT, 0>(p, st);
    return RC_ERR_ARG;
}

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

}  // namespace

// kv_store on a 4-bit pool: the store kernel without rotation and queries.
rc_status rc_host::store_fp4(const rc_pool_desc* pool, const int32_t* slots, const void* k_new, const void* v_new,
                             int32_t n, int32_t* table, const int32_t* table_pos, cudaStream_t st) {
    const rc_status s = check_fp4(*pool);
    if (s != RC_OK) return s;
    if (!v_new || !aligned16(k_new) || !aligned16(v_new)) return RC_ERR_ARG;
    StoreParams p{};
    p.k = static_cast<const __nv_bfloat16*>(k_new);
    p.v = static_cast<const __nv_bfloat16*>(v_new);
    p.k_stride = p.v_stride = (int64_t)pool->kv_heads * pool->head_dim_k;
    p.slots = slots;
    p.n = n;
    p.kv_heads = pool->kv_heads;
    p.pool_k = pool->k;
    p.pool_v = pool->v;
    p.k_bscale = pool->k_bscale;
    p.v_bscale = pool->v_bscale;
    p.n_slots = pool->n_slots;
    p.table = table;
    p.table_pos = table_pos;
    p.err = pool->err;
    return pool->head_dim_k == 128 ? launch_rot<8, rc::kFmtFp4>(p, 0, st) : launch_rot<4, rc::kFmtFp4>(p, 0, st);
}

extern "C" rc_status kv_store_rope(const rc_pool_desc* pool, const rc_rope_desc* rope, const int32_t* slots,
                                   const int32_t* positions, const void* k_new, int64_t k_stride, const void* v_new,
                                   int64_t v_stride, int32_t n, const void* q, int64_t q_stride, int32_t q_heads,
                                   void* q_out, int64_t q_out_stride, int32_t* table, const int32_t* table_pos,
                                   rc_stream_t stream) {
    if (!pool || !rope || n < 0 || !pool->k || pool->kv_heads <= 0 || pool->head_dim_k <= 0) return RC_ERR_ARG;
    const int fmt = rc_host::pool_format(*pool);
    const int D = pool->head_dim_k;
    if (pool->mla) {
        if (fmt != rc::kFmtBf16 || pool->kv_heads != 1 || D != 576) return RC_ERR_UNSUPPORTED;
    } else {
        if (pool->head_dim_v != D || (D != 128 && D != 64)) return RC_ERR_UNSUPPORTED;
        if (fmt == rc::kFmtFp8 && D != 128) return RC_ERR_UNSUPPORTED;
    }
    if (rope->rot_dim <= 0 || rope->offset < 0 || (int64_t)rope->offset + rope->rot_dim > D || rope->max_pos < 0)
        return RC_ERR_ARG;
    if (rope->rot_dim % 32 || rope->offset % 16) return RC_ERR_UNSUPPORTED;
    if (rope->n_axes < 0 || rope->n_axes > 4 || (rope->n_axes > 1 && !rope->pair_axis)) return RC_ERR_ARG;
    if (n == 0) return RC_OK;
    if (!rope->cos_sin || !slots || !positions || !k_new) return RC_ERR_ARG;
    if ((table == nullptr) != (table_pos == nullptr)) return RC_ERR_ARG;
    if (!pool->mla && (!pool->v || !v_new)) return RC_ERR_ARG;
    if (fmt == rc::kFmtFp8 && (!pool->k_scale || !pool->v_scale)) return RC_ERR_ARG;
    if (fmt == rc::kFmtFp4) {
        const rc_status s = rc_host::check_fp4(*pool);
        if (s != RC_OK) return s;
    }
    if ((q == nullptr) != (q_out == nullptr)) return RC_ERR_ARG;
    if (q && (q_heads <= 0 || q_heads > 65536)) return RC_ERR_ARG;
    const void* v = pool->mla ? nullptr : v_new;
    const int64_t q_row = (int64_t)q_heads * D;
    if (!aligned16(pool->k) || !aligned16(pool->v) || !aligned16(k_new) || !aligned16(v) || !aligned16(q) ||
        !aligned16(q_out) || !aligned16(rope->cos_sin))
        return RC_ERR_ARG;
    // reads may overlap (a broadcast row has stride 0); written rows may not
    if (k_stride % 8 || k_stride < 0 || (v && (v_stride % 8 || v_stride < 0)) ||
        (q && (q_stride % 8 || q_stride < 0 || q_out_stride % 8 || q_out_stride < q_row)))
        return RC_ERR_ARG;
    StoreParams p{};
    p.axes = rope->n_axes;
    if (rope->n_axes > 1)
        for (int j = 0; j < rope->rot_dim / 2; ++j) {
            if (rope->pair_axis[j] >= rope->n_axes) return RC_ERR_ARG;
            p.pair_axis[j / 16] |= (uint32_t)rope->pair_axis[j] << (2 * (j % 16));
        }
    p.k = static_cast<const __nv_bfloat16*>(k_new);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.slots = slots;
    p.positions = positions;
    p.cos_sin = rope->cos_sin;
    p.max_pos = rope->max_pos;
    p.rot = rope->rot_dim;
    p.offset = rope->offset;
    p.n = n;
    p.kv_heads = pool->kv_heads;
    p.q_heads = q_heads;
    p.pool_k = pool->k;
    p.pool_v = pool->v;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    if (fmt == rc::kFmtFp4) {
        p.k_bscale = pool->k_bscale;
        p.v_bscale = pool->v_bscale;
    }
    p.n_slots = pool->n_slots;
    p.table = table;
    p.table_pos = table_pos;
    p.err = pool->err;
    const int rot = rope->interleaved ? 2 : 1;
    cudaStream_t st = (cudaStream_t)stream;
    if (pool->mla) return launch_rot<36, rc::kFmtBf16>(p, rot, st);
    if (fmt == rc::kFmtFp8) return launch_rot<8, rc::kFmtFp8>(p, rot, st);
    if (fmt == rc::kFmtFp4)
        return D == 128 ? launch_rot<8, rc::kFmtFp4>(p, rot, st) : launch_rot<4, rc::kFmtFp4>(p, rot, st);
    return D == 128 ? launch_rot<8, rc::kFmtBf16>(p, rot, st) : launch_rot<4, rc::kFmtBf16>(p, rot, st);
}
