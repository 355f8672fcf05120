// Beam search: beam_select (the best continuations over a request's beams and the
// vocabulary) and beam_reorder (rows of slot tables or token histories follow
// their parents).
//
//   score(w, v) = s_w + (x_wv - lse_w),   lse_w = m_w + log sum_v 2^((x_wv - m_w) log2 e)
//
// The logits are read once from HBM, by one cluster of CTAs a request: HBM bounds
// large calls, launch and the stages' latency small ones.  A CTA takes a beam's row, or
// a piece of it (of more beams than CTAs in the cluster, several rows in turn).  Streaming over it, a
// thread keeps the running maximum, a compensated sum of exponentials relative to
// it, and the maximum of every few words that it reads.  Within a beam the score rises
// with the logit, so the row's best n_out logits are wanted, and they are found
// without a sort of the row: the row is cut into 32 (above n_out = 32, 64) sets, the
// n_out-th largest of the sets' maxima is a bar that at least n_out elements reach
// and hardly more do (n_out = 16: 22 of any number), and only the words whose maximum
// reaches it are read again (from L2).  What reaches the bar is ranked by counting.
// The first CTA of the cluster ranks the rows' lists together.  Measured: 64 requests of
// 8 beams, 32,000 fp32 logits, n_out 16, 20.2 us (3.2 TB/s); 1 x 4 x 32,000 bf16, 7.0 us; 200 x 4 x
// 32,003 bf16, 21.7 us (2.4 TB/s): a row's stages wait for one another (barriers and loads are
// most of the stalls), and at 64 registers a thread an SM has 1,024 threads to fill the gaps.
// beam_reorder, 200 x 4 rows of 2,000 columns: 4.0 us.
//
// Ties: equal scores go to the lowest (beam, token).  A logit and its token make one
// 64-bit key (the logit's order above, the token's complement below), so no two are
// equal and no order of collecting them matters.  Between the beams scores of two
// 32-bit words rank, because beams' near scores decide which one lives and fp32's step at
// a score of 10 is 1e-6; 64-bit arithmetic takes about 100 cycles an operation here.  They are
// as good as the log-sum-exps in them: 2^-20 (fp32 arguments and results of ex2, a thread's
// sums and its factor expf(m - top)), 1.6e-7 at most as measured, so nearer scores of two beams may come
// in either order.  Within a beam the order is exact.

#include "tc.cuh"

#include <cfloat>

namespace {

constexpr int kMaxBeams = 32, kMaxOut = 64, kMaxCluster = 8, kWideCluster = 16;
constexpr int UN = 2;             // words a thread has on their way (4, with three CTAs an SM instead of four: 64 x 8 rows
                                  // of 32,000 fp32 took a quarter longer)
constexpr int kBlocks = 8;        // runs of groups whose maxima are kept, at most
constexpr int kKeys = 1024, kPairs = 1024;

struct SelectParams {
    const void* logits;
    int64_t stride;  // elements between rows
    int32_t batch, beams, vocab, n_out;
    const float* scores;
    const uint8_t* done;
    int32_t end_token;
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
    uint8_t* out_done;
    int32_t* err;
    int32_t cluster;
    int32_t threads;  // a CTA
    int32_t pieces;   // CTAs a beam; with more beams than CTAs 1, and a CTA takes every cluster-th beam
    int32_t words, each;  // 16-byte words of a row and of a piece
    int32_t blocks;   // of a piece
    int32_t per;      // groups a block
};

// A logit and its token: the logit's order in the upper half, the token's complement
// in the lower one; 0 is none.
using Key = uint64_t;
// A number as the unevaluated sum of two words, the second at most half a step of the first.
struct Two {
    float hi, lo;
};
struct Part {  // a piece's maximum and sum of 2^((x - m) log2 e)
    uint64_t m;
    uint64_t s;  // a Two
};

// Dynamic shared memory: blocks' maxima (later the candidates' scores), what the rows' CTAs send.
struct Layout {
    int in_parts, in_lists, bytes;
    __host__ __device__ Layout(const SelectParams& p) {
        const int lists = p.beams * p.pieces;
        const int maxima = p.blocks * p.threads * 4, scores = lists * p.n_out * 8;
        in_parts = maxima > scores ? maxima : scores;
        in_lists = in_parts + lists * (int)sizeof(Part);
        bytes = in_lists + lists * p.n_out * (int)sizeof(Key);
    }
};

// Floats as whole numbers of the same order; 0 lies below all of them.
RC_DEV uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 as 0: they are equal)
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
RC_DEV float unordered(uint32_t u) { return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u); }
RC_DEV Key make_key(float x, int token) { return ((uint64_t)ordered(x) << 32) | (uint32_t)~token; }
RC_DEV float key_logit(Key k) { return unordered((uint32_t)(k >> 32)); }
RC_DEV int key_token(Key k) { return (int)~(uint32_t)k; }
RC_DEV Two two_sum(float a, float b) {  // exact (Knuth)
    const float z = a + b, v = z - a;
    return {z, (a - (z - v)) + (b - v)};
}
RC_DEV Two add(Two a, Two b) {
    const Two h = two_sum(a.hi, b.hi);
    return two_sum(h.hi, h.lo + (a.lo + b.lo));
}
RC_DEV uint64_t words(Two x) { return ((uint64_t)__float_as_uint(x.hi) << 32) | __float_as_uint(x.lo); }
RC_DEV Two from_words(uint64_t u) { return {__uint_as_float((uint32_t)(u >> 32)), __uint_as_float((uint32_t)u)}; }
// What lies below 53 bits goes, as in 64-bit arithmetic: it decides among logits that are masked with
// their type's lowest value (10^38), whose scores are then equal in all beams.
RC_DEV Two as_64(Two y) {
    if (!(fabsf(y.lo) > fabsf(y.hi) * 1.1102230246251565e-16f)) y.lo = 0.f;
    return y;
}
// The score (x - lse) + s as a whole number of the same order, above 0.
RC_DEV uint64_t score_key(float x, Two lse, float s) {
    Two y = two_sum(x, -lse.hi);
    y = add({y.hi, y.lo}, {s, -lse.lo});
    if (!(fabsf(y.hi) < INFINITY)) y = {-INFINITY, 0.f};  // (logits 10^38 apart)
    y = as_64(y);
    return ((uint64_t)ordered(y.hi) << 32) | ordered(y.lo);
}
RC_DEV float key_score(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
// log of x >= 1 to about 2^-24: 2^k f with 1 <= f < 2.
RC_DEV Two log_two(Two x) {
    const int e = (int)(__float_as_uint(x.hi) >> 23) - 127;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23), f = x.hi * down, k = (float)e;
    // log 2 in two parts, the first of 16 bits, so that its product with k is exact
    return add({k * 0.693145751953125f, 0.f}, two_sum(logf(f), k * 1.42860682030942e-06f + __fdividef(x.lo * down, f)));
}

RC_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
RC_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
RC_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
// Into the same place of the cluster's first CTA (cs 1: its own).
RC_DEV void send(int cs, void* to, uint64_t v) {
    if (cs == 1) {
        *static_cast<uint64_t*>(to) = v;
        return;
    }
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(a) : "r"(rc::smem_u32(to)));
    asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(a), "l"(v) : "memory");
}

// Logits of one 16-byte word.
template <typename T>
struct Word;
template <>
struct Word<__nv_bfloat16> {
    static constexpr int E = 8;
    static RC_DEV float get(const uint4& w, int e) {
        const uint32_t u = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
    }
};
template <>
struct Word<float> {
    static constexpr int E = 4;
    static RC_DEV float get(const uint4& w, int e) {
        return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
    }
};

// 16 of the 32 bytes a, b, from byte 4 Q + bits / 8 on.
template <int Q>
RC_DEV uint4 cut(const uint4& a, const uint4& b, int bits) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return make_uint4(__funnelshift_r(w[Q], w[Q + 1], bits), __funnelshift_r(w[Q + 1], w[Q + 2], bits),
                      __funnelshift_r(w[Q + 2], w[Q + 3], bits), __funnelshift_r(w[Q + 3], w[Q + 4], bits));
}
RC_DEV uint4 cut(const uint4& a, const uint4& b, int bytes) {
    const int bits = (bytes & 3) * 8;
    switch (bytes >> 2) {
        case 0: return cut<0>(a, b, bits);
        case 1: return cut<1>(a, b, bits);
        case 2: return cut<2>(a, b, bits);
        default: return cut<3>(a, b, bits);
    }
}

// Words [w0, w1) of a row, word i the tokens i E .. i E + E - 1.  A row that starts `shift`
// bytes into a 16-byte unit (rows of an odd vocabulary) is read in aligned units,
// `units` in all, and its words are cut out of neighbouring ones: the sums then do not
// depend on where a row lies, and equal beams get equal scores.
struct Run {
    const uint4* row;
    int shift;
    int units, w0, w1, vocab;
};
template <typename T>
RC_DEV void elements(const Run& r, const uint4& word, int at, float (&x)[Word<T>::E]) {
    constexpr int E = Word<T>::E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = Word<T>::get(word, e);
    if (at >= r.w1 || at * (int64_t)E + E > r.vocab) {  // the row's end may lie inside a word
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (at >= r.w1 || at * (int64_t)E + e >= r.vocab) x[e] = -INFINITY;
    }
}

// One pass over the run: this thread's maximum m and sum of 2^((x - m) log2 e), and its
// maxima of the blocks.  Q < 0: the row lies on a 16-byte boundary, otherwise it starts
// 4 Q bytes, or 4 Q + 2, behind one.  (The difference x - m is exact near m, and
// stays in range where logits are masked with their type's lowest value.)
template <typename T, int Q, int TH>
RC_DEV void stream_run(const Run& r, int per, float* maxima, float& m_out, float& s_out) {
    constexpr int E = Word<T>::E, kThreads = TH, kGroup = TH * UN;
    constexpr bool CUT = Q >= 0;
    static_assert(UN == 2, "two partial sums");
    constexpr float kNone = -INFINITY;
    const int t = threadIdx.x, lane = t & 31, bits = (r.shift & 3) * 8;
    float m = kNone, sum = 0.f, carry = 0.f, block = kNone;
    int left = per;
    uint4 next[UN], over[CUT ? UN : 1];
    auto load = [&](int w) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int at = w + i * kThreads + t;
            const bool in = CUT ? at <= r.w1 && at < r.units : at < r.w1;  // (and the unit behind the run's last word)
            next[i] = in ? __ldcs(r.row + at) : make_uint4(0, 0, 0, 0);
            if constexpr (CUT) over[i] = lane == 31 && at < r.w1 && at + 1 < r.units ? __ldcs(r.row + at + 1) : make_uint4(0, 0, 0, 0);
        }
    };
    load(r.w0);
    for (int w = r.w0; w < r.w1; w += kGroup) {
        float x[UN][E], top = kNone;
        uint4 raw[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            raw[i] = next[i];
            if constexpr (CUT) {
                uint4 b;
                b.x = __shfl_down_sync(0xffffffffu, raw[i].x, 1);
                if (Q > 1 || E > 4) b.y = __shfl_down_sync(0xffffffffu, raw[i].y, 1);
                if (Q > 2 || E > 4) b.z = __shfl_down_sync(0xffffffffu, raw[i].z, 1);
                if (Q > 3 || E > 4) b.w = __shfl_down_sync(0xffffffffu, raw[i].w, 1);
                raw[i] = cut<CUT ? Q : 0>(raw[i], lane == 31 ? over[i] : b, bits);
            }
        }
        load(w + kGroup);  // on its way meanwhile
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            elements<T>(r, raw[i], w + i * kThreads + t, x[i]);
#pragma unroll
            for (int e = 0; e < E; e += 2) top = tc::max3(top, x[i][e], x[i][e + 1]);
        }
        if (top > m) {
            if (m != kNone) {
                const float a = tc::ex2((m - top) * rc::kLog2e);
                sum *= a;
                carry *= a;
            }
            m = top;
        }
        const float2 ref = m == kNone ? make_float2(0.f, 0.f) : make_float2(-m, -m);
        float2 part[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            part[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 y = tc::fmul2(tc::fadd2(make_float2(x[i][e], x[i][e + 1]), ref), rc::kLog2e);
                part[i] = tc::fadd2(part[i], make_float2(tc::ex2(y.x), tc::ex2(y.y)));
            }
        }
        const float2 all = tc::fadd2(part[0], part[1]);
        const float y = (all.x + all.y) - carry, z = sum + y;  // compensated
        carry = (z - sum) - y;
        sum = z;
        block = fmaxf(block, top);
        if (--left == 0 || w + kGroup >= r.w1) {
            *maxima = block;
            maxima += kThreads;
            block = kNone;
            left = per;
        }
    }
    m_out = m;
    s_out = sum - carry;
}

// This thread's words of one block again: f(logit, token).
template <typename T, int TH, typename F>
RC_DEV void block_again(const Run& r, int per, int block, int t, F f) {
    constexpr int E = Word<T>::E, kThreads = TH, kGroup = TH * UN;
    for (int g = block * per; g < (block + 1) * per; ++g) {
        const int w = r.w0 + g * kGroup + t;
        uint4 raw[UN], over[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int at = w + i * kThreads;
            raw[i] = at < r.w1 ? __ldg(r.row + at) : make_uint4(0, 0, 0, 0);
            over[i] = r.shift && at < r.w1 && at + 1 < r.units ? __ldg(r.row + at + 1) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int at = w + i * kThreads;
            float x[E];
            elements<T>(r, r.shift ? cut(raw[i], over[i], r.shift) : raw[i], at, x);
#pragma unroll
            for (int e = 0; e < E; ++e) f(x[e], at * E + e);
        }
    }
}

// f(logit, token) for thread t's elements of group g that reach the bar.  They are marked first:
// a warp's threads have them in different places, and would come to f one by one.
template <typename T, int TH, typename F>
RC_DEV void reaching(const Run& r, int g, int t, float bar, F f) {
    constexpr int E = Word<T>::E, kThreads = TH, kGroup = TH * UN;
    const int w = r.w0 + g * kGroup + t;
    uint4 raw[UN], over[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const int at = w + i * kThreads;
        raw[i] = at < r.w1 ? __ldg(r.row + at) : make_uint4(0, 0, 0, 0);
        over[i] = r.shift && at < r.w1 && at + 1 < r.units ? __ldg(r.row + at + 1) : make_uint4(0, 0, 0, 0);
    }
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        float x[E];
        if (r.shift) raw[i] = cut(raw[i], over[i], r.shift);
        elements<T>(r, raw[i], w + i * kThreads, x);
#pragma unroll
        for (int e = 0; e < E; ++e) hits |= (x[e] >= bar ? 1u : 0u) << (i * E + e);
    }
    while (hits) {
        const int e = __ffs(hits) - 1;
        hits &= hits - 1;
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < UN * E; ++j)
            if (j == e) x = Word<T>::get(raw[j / E], j % E);
        f(x, (w + e / E * kThreads) * E + e % E);
    }
}

// The n-th largest (from 0) of the lanes' values (with TWO of both of each), -infinity if there is none.
template <bool TWO>
RC_DEV float nth_of_lanes(float a0, float a1, int n, int lane) {
    int above0 = 0, above1 = 0;
#pragma unroll
    for (int l = 0; l < 32; ++l) {
        const float o0 = __shfl_sync(0xffffffffu, a0, l);
        above0 += o0 > a0 || (o0 == a0 && l < lane);
        if constexpr (TWO) {
            const float o1 = __shfl_sync(0xffffffffu, a1, l);
            above0 += o1 > a0;
            above1 += (o0 >= a1) + (o1 > a1 || (o1 == a1 && l < lane));
        }
    }
    const unsigned who0 = __ballot_sync(0xffffffffu, above0 == n);
    if (who0) return __shfl_sync(0xffffffffu, a0, __ffs(who0) - 1);
    if constexpr (TWO) {
        const unsigned who1 = __ballot_sync(0xffffffffu, above1 == n);
        if (who1) return __shfl_sync(0xffffffffu, a1, __ffs(who1) - 1);
    }
    return -INFINITY;
}

template <typename T, bool TWO, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) beam_select_kernel(const SelectParams p) {
    constexpr int kThreads = TH, kWarps = TH / 32, kGroup = TH * UN;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Key s_keys[kKeys];
    __shared__ uint16_t s_pairs[kPairs];
    __shared__ float s_top[kThreads];
    __shared__ Two s_sum[kWarps];
    __shared__ Key s_best[kWarps];
    __shared__ Two s_lse[kMaxBeams];
    __shared__ float s_score[kMaxBeams];
    __shared__ uint8_t s_kind[kMaxBeams];  // 0: to be read, 1: finished, 2: none of its continuations counts
    __shared__ int s_n_pairs, s_n_keys;
    const Layout lay(p);
    float* maxima = reinterpret_cast<float*>(smem);
    Part* in_parts = reinterpret_cast<Part*>(smem + lay.in_parts);
    Key* in_lists = reinterpret_cast<Key*>(smem + lay.in_lists);
    const int cs = p.cluster, rank = cs > 1 ? (int)cluster_rank() : 0;
    const int b = blockIdx.x / cs, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int W = p.beams, K = p.n_out;
    if (cs > 1) cluster_arrive();  // before anything goes to the first CTA's memory, it has to run
    auto read_kinds = [&] {
        if (t >= W) return;
        const float s = __ldg(p.scores + (int64_t)b * W + t);
        const uint8_t over = p.done ? __ldg(p.done + (int64_t)b * W + t) : 0;
        s_score[t] = s;
        const bool fin = fabsf(s) < INFINITY;
        s_kind[t] = !fin ? 2 : over ? 1 : 0;
        if (rank == 0 && !fin && !(s < 0.f)) rc::flag_error(p.err, rc::kErrBadSlot);  // a NaN or +infinity
    };
    bool waited = cs == 1;
    for (int w = rank / p.pieces; w < W; w += cs / p.pieces) {
        const int list = w * p.pieces + rank % p.pieces;
        const T* row = static_cast<const T*>(p.logits) + ((int64_t)b * W + w) * p.stride;
        Run r;
        r.shift = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        r.row = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row) - r.shift);
        r.vocab = p.vocab;
        r.units = (int)((r.shift + (int64_t)p.vocab * (int)sizeof(T) + 15) / 16);
        r.w0 = min(p.words, p.each * (rank % p.pieces));
        r.w1 = min(p.words, r.w0 + p.each);
#pragma unroll
        for (int i = 0; i < UN; ++i)  // the first words on their way to L2, while the scores are read
            if (r.w0 + i * kThreads + t < r.w1)
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(r.row + r.w0 + i * kThreads + t));
        if (w != rank / p.pieces) __syncthreads();  // the last row's counts have been read
        else read_kinds();
        if (t == 0) s_n_pairs = s_n_keys = 0;
        __syncthreads();
        if (s_kind[w] != 0) continue;
        float m, s;
        switch (r.shift ? r.shift >> 2 : -1) {
            case -1: stream_run<T, -1, TH>(r, p.per, maxima + t, m, s); break;
            case 0: stream_run<T, 0, TH>(r, p.per, maxima + t, m, s); break;
            case 1: stream_run<T, 1, TH>(r, p.per, maxima + t, m, s); break;
            case 2: stream_run<T, 2, TH>(r, p.per, maxima + t, m, s); break;
            default: stream_run<T, 3, TH>(r, p.per, maxima + t, m, s);
        }
        s_top[t] = m;
        __syncthreads();
        // ---- the bar: lane l's set is what the threads of that lane have read (every warp
        // finds it: by one, with a barrier more, a call of 64 x 8 rows took 1 us longer)
        float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; k += 2) {
            a0 = fmaxf(a0, s_top[k * 32 + lane]);
            a1 = fmaxf(a1, s_top[k * 32 + 32 + lane]);
        }
        float bar = nth_of_lanes<TWO>(TWO ? a0 : fmaxf(a0, a1), a1, K - 1, lane);
        bar = fmaxf(bar, -FLT_MAX);  // (a logit of -infinity is none)
        const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(fmaxf(a0, a1))));
        const int blocks = ((r.w1 - r.w0 + kGroup - 1) / kGroup + p.per - 1) / p.per;
        uint32_t which = 0;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k)
            if (k < blocks) which |= (maxima[k * kThreads + t] >= bar ? 1u : 0u) << k;
        while (which) {
            const int k = __ffs(which) - 1, at = atomicAdd(&s_n_pairs, 1);
            which &= which - 1;
            if (at < kPairs) s_pairs[at] = (uint16_t)(k * kThreads + t);
        }
        __syncthreads();
        // ---- what reaches it
        const int n_pairs = s_n_pairs;
        if (n_pairs <= kPairs)
            for (int i = t; i < n_pairs * p.per; i += kThreads) {  // a thread a group: their loads go together
                const int pair = s_pairs[i / p.per];
                reaching<T, TH>(r, pair / kThreads * p.per + i % p.per, pair % kThreads, bar, [&](float x, int token) {
                    const int at = atomicAdd(&s_n_keys, 1);
                    if (at < kKeys) s_keys[at] = make_key(x, token);
                });
            }
        // (meanwhile) the sum: threads' parts relative to the largest
        Two sum{m == -INFINITY ? s : s * expf(m - top), 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum = add(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
        if (lane == 0) s_sum[warp] = sum;
        if (!waited) cluster_wait();
        waited = true;
        __syncthreads();
        if (warp == kWarps - 1) {  // (the first warps rank)
            Two all = s_sum[lane % kWarps];
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1)
                all = add(all, {__shfl_xor_sync(0xffffffffu, all.hi, o), __shfl_xor_sync(0xffffffffu, all.lo, o)});
            if (lane == 0) {
                send(cs, &in_parts[list].m, (uint64_t)__float_as_uint(top));
                send(cs, &in_parts[list].s, words(all));
            }
        }
        Key* to = in_lists + list * K;
        const int n_keys = s_n_keys;
        if (n_pairs <= kPairs && n_keys <= kKeys) {  // ranked by counting
            for (int i = t; i < n_keys; i += kThreads) {
                const Key mine = s_keys[i];
                int above = 0;
#pragma unroll 8
                for (int j = 0; j < n_keys; ++j) above += s_keys[j] > mine;
                if (above < K) send(cs, to + above, mine);
            }
            for (int i = n_keys + t; i < K; i += kThreads) send(cs, to + i, 0);
        } else {
            // more than there is room for (many equal logits): one after the other, the largest below the last.
            // K passes over the row: with all but five logits at fp32's lowest value 64 x 8 x 32,000, K = 16, takes
            // 294 us (20 with them at -infinity), 200 x 4 x 32,003 bf16, K = 64, 1.6 ms
            Key last = ~0ull;
            for (int k = 0; k < K; ++k) {
                Key best = 0;
                if (last)
                    for (int i = 0; i < blocks; ++i)
                        block_again<T, TH>(r, p.per, i, t, [&](float x, int token) {
                            const Key key = x >= bar ? make_key(x, token) : 0;
                            if (key < last && key > best) best = key;
                        });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const Key other = __shfl_xor_sync(0xffffffffu, (unsigned long long)best, o);
                    best = other > best ? other : best;
                }
                __syncthreads();
                if (lane == 0) s_best[warp] = best;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWarps; ++i) best = s_best[i] > best ? s_best[i] : best;
                if (t == 0) send(cs, to + k, best);
                last = best;
            }
        }
    }
    if (cs > 1) {
        if (!waited) cluster_wait();
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // ---- every beam's log-sum-exp
    if (t < W) {
        Two lse{0.f, 0.f};
        if (s_kind[t] == 0) {
            float m = -INFINITY;
            Two s{0.f, 0.f};
            for (int k = 0; k < p.pieces; ++k) m = fmaxf(m, __uint_as_float((uint32_t)in_parts[t * p.pieces + k].m));
            for (int k = 0; k < p.pieces; ++k) {
                const float x = __uint_as_float((uint32_t)in_parts[t * p.pieces + k].m);
                const Two y = from_words(in_parts[t * p.pieces + k].s);
                const float a = x == -INFINITY ? 1.f : expf(x - m);  // (1 where it is the largest: exact)
                s = add(s, {y.hi * a, y.lo * a});
            }
            const bool odd = !(m < INFINITY) || !(s.hi < INFINITY);  // an infinity or a NaN: no distribution
            if (odd) rc::flag_error(p.err, rc::kErrBadSlot);
            if (odd || m == -INFINITY) s_kind[t] = 2;
            else lse = as_64(add({m, 0.f}, log_two(s)));
        }
        s_lse[t] = lse;
    }
    __syncthreads();
    // ---- the rows' lists together
    uint64_t* score = reinterpret_cast<uint64_t*>(smem);
    const int lists = W * p.pieces, n = lists * K;
    int count = 0;
    for (int i = t; i < n; i += kThreads) {
        const int list = i / K, w = list / p.pieces;
        Key key = in_lists[i];
        if (s_kind[w] == 1) key = i % K == 0 && list % p.pieces == 0 ? make_key(0.f, p.end_token) : 0;
        if (s_kind[w] == 2) key = 0;
        in_lists[i] = key;
        score[i] = key ? score_key(key_logit(key), s_lse[w], s_score[w]) : 0;
        count += key != 0;
    }
    auto put = [&](int k, int list, Key key, uint64_t value) {
        const int64_t to = (int64_t)b * K + k;
        const int w = list / p.pieces, token = key_token(key);
        p.out_scores[to] = key_score(value);
        p.out_tokens[to] = token;
        p.out_parents[to] = w;
        if (p.out_done) p.out_done[to] = s_kind[w] == 1 || token == p.end_token;
    };
    auto none = [&](int k) {  // fewer continuations than asked for
        const int64_t to = (int64_t)b * K + k;
        p.out_scores[to] = -INFINITY;
        p.out_tokens[to] = 0;
        p.out_parents[to] = 0;
        if (p.out_done) p.out_done[to] = 0;
    };
    if (n <= kThreads) {  // ranked by counting; equals by their lists, which rise with the beam and the token
        count = __syncthreads_count(count);  // (a thread has one candidate at most here)
        if (t < n && score[t]) {
            int above = 0;
            const uint64_t mine = score[t];
            const int w0 = warp * 32, w1 = min(w0 + 32, n);  // (equals count before the warp's own, and not behind)
#pragma unroll 8
            for (int j = 0; j < w0; ++j) above += score[j] >= mine;
#pragma unroll 8
            for (int j = w0; j < w1; ++j) above += score[j] > mine || (score[j] == mine && j < t);
#pragma unroll 8
            for (int j = w1; j < n; ++j) above += score[j] > mine;
            if (above < K) put(above, t / K, in_lists[t], mine);
        }
        if (t >= count && t < K) none(t);
        return;
    }
    // the largest of the lists' heads, n_out times: list l in lane l of the first warp
    if (t < K) s_pairs[t] = 0xffff;
    __syncthreads();
    if (warp == 0) {
        int at = lane * K, end = lane < lists ? at + K : at;
        uint64_t mine = at < end ? score[at] : 0;
        for (int k = 0; k < K; ++k) {
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
            const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
            const uint64_t best = ((uint64_t)hi << 32) | lo;
            if (best == 0) break;
            if (lane == __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1) {
                s_pairs[k] = (uint16_t)at;
                ++at;
                mine = at < end ? score[at] : 0;
            }
        }
    }
    __syncthreads();
    if (t < K) {
        const int i = s_pairs[t];
        if (i == 0xffff) none(t);
        else put(t, i / K, in_lists[i], score[i]);
    }
}

template <typename T, bool TWO, int TH>
cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
    const int smem = Layout(p).bytes;
    if (smem > 32 * 1024) {
        const cudaError_t e = rc_host::ensure_smem<beam_select_kernel<T, TWO, TH>>(64 * 1024);
        if (e != cudaSuccess) return e;
    }
    if (p.cluster > kMaxCluster) {
        const cudaError_t e = cudaFuncSetAttribute(beam_select_kernel<T, TWO, TH>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.batch * p.cluster));
    cfg.blockDim = dim3(TH);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, beam_select_kernel<T, TWO, TH>, p);
}

template <typename T, bool TWO>
cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
    return p.threads == 128 ? launch_select<T, TWO, 128>(p, st) : launch_select<T, TWO, 256>(p, st);
}

struct ReorderParams {
    const int32_t* from;
    int32_t* to;
    int64_t table_len;
    const int32_t* start;   // [batch][beams]
    const int32_t* first;   // [batch]
    const int32_t* last;
    const int32_t* parents; // [batch][beams]
    int32_t beams, max_cols;
    int32_t* err;
};

// A thread owns COLS columns of all of a request's rows: it reads every new row's entry
// before it writes the first, so the rows may be reordered in place.
template <int W, int COLS>
__global__ void __launch_bounds__(128) beam_reorder_kernel(const ReorderParams p) {
    const int b = blockIdx.y, n = p.beams;
    const int64_t first = __ldg(p.first + b), last = __ldg(p.last + b);
    __shared__ int32_t s_start[W], s_from[W];
    bool bad = first < 0 || last - first > p.max_cols;
    if (threadIdx.x < n) {
        const int64_t at = __ldg(p.start + (int64_t)b * n + threadIdx.x);
        const int par = __ldg(p.parents + (int64_t)b * n + threadIdx.x);
        s_start[threadIdx.x] = (int32_t)at;
        const bool off = par < 0 || par >= n || (last > first && (at < 0 || at + last > p.table_len));
        bad = bad || off;
        s_from[threadIdx.x] = off ? 0 : __ldg(p.start + (int64_t)b * n + par);
    }
    if (__syncthreads_or(bad)) {  // the request's rows stay as they are
        if (blockIdx.x == 0 && threadIdx.x == 0) rc::flag_error(p.err, rc::kErrBadSlot);
        return;
    }
    const int64_t c0 = first + (int64_t)blockIdx.x * (128 * COLS) + threadIdx.x;
    int32_t v[COLS][W];
#pragma unroll
    for (int i = 0; i < COLS; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = j < n && c0 + 128 * i < last ? p.from[(int64_t)s_from[j] + c0 + 128 * i] : 0;
#pragma unroll
    for (int i = 0; i < COLS; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (j < n && c0 + 128 * i < last) p.to[(int64_t)s_start[j] + c0 + 128 * i] = v[i][j];
}

template <int W, int COLS>
void launch_reorder(const ReorderParams& p, int batch, cudaStream_t st) {
    const dim3 grid((unsigned)(((int64_t)p.max_cols + 128 * COLS - 1) / (128 * COLS)), (unsigned)batch);
    beam_reorder_kernel<W, COLS><<<grid, 128, 0, st>>>(p);
}

}  // namespace

extern "C" rc_status beam_select(const void* logits, int32_t logits_f32, int64_t stride, int32_t batch, int32_t beams,
                                 int32_t vocab, const float* scores, const uint8_t* done, int32_t end_token, int32_t n_out,
                                 float* out_scores, int32_t* out_tokens, int32_t* out_parents, uint8_t* out_done,
                                 int32_t* err, rc_stream_t stream) {
    if (batch < 0 || beams <= 0 || vocab <= 0 || n_out <= 0 || stride < vocab || end_token < -1 || end_token >= vocab ||
        (done && end_token < 0))
        return RC_ERR_ARG;
    if (beams > kMaxBeams || n_out > kMaxOut || vocab > (1 << 30)) return RC_ERR_UNSUPPORTED;
    if (batch == 0) return RC_OK;
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return RC_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & (logits_f32 ? 3 : 1)) return RC_ERR_ARG;
    const int64_t in = (int64_t)batch * beams, size = logits_f32 ? 4 : 2;
    const void* const outs[4] = {out_scores, out_tokens, out_parents, out_done};
    for (int i = 0; i < 4; ++i) {  // CTAs of this request and of others may still read
        const int64_t bytes = (int64_t)batch * n_out * (i < 3 ? 4 : 1);
        if (rc_host::overlap(outs[i], bytes, logits, in, stride * size, vocab * size) ||
            rc_host::overlap(outs[i], bytes, scores, in, 4, 4) || rc_host::overlap(outs[i], bytes, done, in, 1, 1))
            return RC_ERR_ARG;
    }
    SelectParams p{};
    p.logits = logits;
    p.stride = stride;
    p.batch = batch;
    p.beams = beams;
    p.vocab = vocab;
    p.n_out = n_out;
    p.scores = scores;
    p.done = done;
    p.end_token = end_token;
    p.out_scores = out_scores;
    p.out_tokens = out_tokens;
    p.out_parents = out_parents;
    p.out_done = out_done;
    p.err = err;
    // a CTA a beam (more beams than CTAs: every cluster-th), and several while they are
    // few and a piece is still long enough to pay for them
    const int words = (vocab - 1) / (logits_f32 ? 4 : 8) + 1;
    p.pieces = 1;
    p.cluster = beams < kMaxCluster ? beams : kMaxCluster;
    if (beams > kMaxCluster) {
        // up to 16 CTAs a request, while they all run at once (more than 8 have to find room in one part of
        // the chip): 16 and 8 CTAs, 1 x 16 x 32,000 bf16, n_out 32, 14.7 and 20.1 us, 8 x 10 x 50,257 fp32,
        // n_out 20, 24.5 and 43.4; beyond, 50 x 32 x 32,000 bf16, n_out 32 66.1 and 58.6, n_out 64 169 and 113
        const int most = beams < kWideCluster ? beams : kWideCluster;
        if ((int64_t)batch * most <= 4 * (int64_t)rc_host::sm_count()) p.cluster = most;
    }
    // 256 threads a row while all rows run at once, half of them beyond: the next rows then fill the gaps
    // that a row's stages leave (a single CTA does from the start, a cluster waits for room for all of it).
    // 256 and 128 threads: 200 x 4 x 32,003 bf16 28.1 and 21.9 us, 155 x 4 23.7 and 20.6, 1,000 x 4 85 and 66.5;
    // 700 x 1 x 50,257 fp32 33.0 and 43.6, 820 x 1 48.1 and 45.2
    const int64_t ctas = (int64_t)batch * p.cluster, slots = 4 * (int64_t)rc_host::sm_count();
    p.threads = ctas > (p.cluster > 1 ? slots : slots * 4 / 3) ? 128 : 256;
    const int group = p.threads * UN;  // words
    while (p.cluster + beams <= kMaxCluster && (int64_t)batch * (p.cluster + beams) <= 2 * (int64_t)rc_host::sm_count() &&
           words / (p.pieces + 1) >= group) {
        ++p.pieces;
        p.cluster += beams;
    }
    if ((int64_t)batch * p.cluster > 0x7fffffff) return RC_ERR_ARG;
    p.words = words;
    p.each = (words - 1) / p.pieces + 1;
    const int groups = (p.each - 1) / group + 1;
    p.per = (groups - 1) / kBlocks + 1;
    p.blocks = (groups - 1) / p.per + 1;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (logits_f32) e = n_out > 32 ? launch_select<float, true>(p, st) : launch_select<float, false>(p, st);
    else e = n_out > 32 ? launch_select<__nv_bfloat16, true>(p, st) : launch_select<__nv_bfloat16, false>(p, st);
    return rc_host::launch_status(e);
}

extern "C" rc_status beam_reorder(const int32_t* table, int32_t* out, int64_t table_len, const int32_t* start,
                                  const int32_t* first, const int32_t* last, const int32_t* parents, int32_t batch,
                                  int32_t beams, int32_t max_cols, int32_t* err, rc_stream_t stream) {
    if (batch < 0 || beams <= 0 || max_cols < 0 || table_len < 0) return RC_ERR_ARG;
    if (beams > kMaxBeams || batch > 65535) return RC_ERR_UNSUPPORTED;
    if (batch == 0 || max_cols == 0) return RC_OK;
    if (!table || !out || !start || !first || !last || !parents) return RC_ERR_ARG;
    const int64_t apart = reinterpret_cast<const char*>(out) - reinterpret_cast<const char*>(table);
    if (apart != 0 && apart < table_len * 4 && apart > -table_len * 4) return RC_ERR_ARG;  // neither in place nor apart
    // No row that lies in the table has more columns than it has entries ("no bound" launches no blocks for nothing).
    const int64_t most = table_len > 1 ? table_len : 1;
    const ReorderParams p{table, out,     table_len, start, first, last, parents, beams,
                          (int32_t)(max_cols < most ? max_cols : most), err};
    cudaStream_t st = (cudaStream_t)stream;
    if (beams <= 4) launch_reorder<4, 4>(p, batch, st);
    else if (beams <= 8) launch_reorder<8, 2>(p, batch, st);
    else if (beams <= 16) launch_reorder<16, 1>(p, batch, st);
    else launch_reorder<32, 1>(p, batch, st);
    return rc_host::launch_status(cudaGetLastError());
}
