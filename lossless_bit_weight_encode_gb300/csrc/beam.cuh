// Best continuations of every request over its beams and the vocabulary (w12_beam_select
// in include/w12.h).
//
// Mathematics.  Row (a beam) with logits x_v, M = max x_v: the candidate (beam, v) has
// the score s + ((x_v - M) - ln sum_v exp(x_v - M)).  Within a row the order of scores is
// that of the logits, so a part of a row needs to hand on no more than its `keep` largest
// logits and its share of the sum; what scores they have shows when the rows' sums are
// there.
//
// One launch.  A CTA takes one part of a row into registers (16-byte loads) and passes
// over it three times there: maximum, sum, selection.  The parts' sums are relative to a
// power of two 2^r, r = ceil(max log2(e)), with the exponent x log2(e) - r from two fused
// multiply-adds (the constant in two pieces), and are added in 64-bit fixed point: the
// joined sum does not depend on the parts' order and only the exponentials themselves
// (2^-22, independent from element to element) are rounded, so that scores of different
// beams compare right down to about 1e-8.  The selection's threshold is the smallest of
// as many thread groups' maxima as elements are kept: at least that many elements reach
// it and, in random order, a few times that many; they are sorted by counting.  Where too many reach
// it (a mask that leaves whole groups empty, equal logits), the exact one is found by
// bisection over the bits.  The CTA that arrives last at a request joins its parts the
// same way, in 64 bits.
//
// What bounds it: the logits are read once, from HBM or L2.
#pragma once

#include <cstdint>

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kBeamThreads = 256, kBeamKeep = 64, kBeamMost = 32;
constexpr int kBeamPool = 512;     // elements of a part that may reach the threshold
constexpr int kBeamJoin = 1024;    // and of a request
constexpr int kBeamVocab = 1 << 22;
constexpr int kBeamFixed = 40;     // bits of the sums' fraction

struct BeamStat {
    float top;      // largest logit of the part (-infinity: none)
    uint32_t pad;
    uint64_t sum;   // of 2^(x log2(e) - beam_ref(top)), times 2^kBeamFixed
};
struct BeamEntry {
    float x;
    int32_t token;  // -1: none
};

struct BeamParams {
    const void *logits;
    int64_t stride;
    const uint32_t *allowed;
    int64_t allowed_stride;
    const float *scores_in;
    float *scores;
    int32_t *tokens, *parents;
    int32_t *cand_tokens, *cand_parents;
    float *cand_scores;
    BeamStat *stats;      // [rows][parts]
    BeamEntry *entries;   // [rows][parts][keep], sorted
    uint32_t *counters;   // [requests]
    int32_t requests, beams, vocab, take, keep, eos;
    int32_t parts, part;  // parts of a row, their tokens
};

// Exponent that a part's sum is relative to, in powers of two.  Where the integer nearest
// to the largest logit is no exact float any more, that logit itself.
__device__ __forceinline__ bool beam_plain(float top) { return fabsf(top) <= 1048576.0f; }
constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.92596303e-8f;  // log2(e) - kLog2E
__device__ __forceinline__ double beam_ref(float top) {
    return beam_plain(top) ? (double)ceilf(top * kLog2E) : (double)top * 1.4426950408889634;
}

// Larger value, larger number (no NaN, no -0).
__device__ __forceinline__ uint32_t beam_order(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float beam_value(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t beam_order(double x) {
    const int64_t b = __double_as_longlong(x);
    return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double beam_value(uint64_t o) {
    return __longlong_as_double((int64_t)(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}
__device__ __forceinline__ float beam_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A thread's elements: E of them in pieces of 16 bytes, kBeamThreads pieces apart.  NaN
// and what is not there or not allowed are -infinity, -0 is 0.
template <bool BF16, int E>
struct BeamElems {
    static constexpr int VEC = BF16 ? 8 : 4, N = E / VEC;
    uint32_t w[BF16 ? E / 2 : E];

    __device__ __forceinline__ float get(int e) const {
        if constexpr (BF16) return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
        return __uint_as_float(w[e]);
    }
    __device__ __forceinline__ static uint32_t none() { return BF16 ? 0xFF80FF80u : 0xFF800000u; }

    // Tokens t0 + (j kBeamThreads + tid) VEC + e, of which those before t1 count; row: the
    // row's token 0, which may lie at any element: a thread has the same tokens of every row
    // (equal rows then have equal sums), from one 16-byte piece of memory or out of two.
    __device__ __forceinline__ void load(const uint8_t *row, int32_t t0, int32_t t1, int32_t vocab,
                                         const uint32_t *allowed) {
        constexpr int ELEM = BF16 ? 2 : 4, WORDS = 4;
        const int tid = threadIdx.x;
        const int32_t mis = (int32_t)((reinterpret_cast<uintptr_t>(row + (int64_t)t0 * ELEM) & 15u) / ELEM);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int32_t t = t0 + (j * kBeamThreads + tid) * VEC;
            uint32_t *to = w + j * WORDS;
            const uint8_t *at = row + (int64_t)t * ELEM;
            if (mis == 0 && t + VEC <= t1) {
                const uint4 u = *reinterpret_cast<const uint4 *>(at);
                to[0] = u.x, to[1] = u.y, to[2] = u.z, to[3] = u.w;
            } else if (mis != 0 && t + VEC <= t1 && t >= mis && t - mis + 2 * VEC <= vocab) {
                const uint4 u = reinterpret_cast<const uint4 *>(at - mis * ELEM)[0];
                const uint4 v = reinterpret_cast<const uint4 *>(at - mis * ELEM)[1];
                uint32_t y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                const int words = mis * ELEM / 4;
                if (words & 2) {
#pragma unroll
                    for (int i = 0; i < 6; ++i) y[i] = y[i + 2];
                }
                if (words & 1) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) y[i] = y[i + 1];
                }
                const int bits = BF16 ? (mis & 1) * 16 : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = __funnelshift_r(y[i], y[i + 1], bits);
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) to[i] = none();
                if (t < t1) {  // where a piece would reach out of the row
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if (t + e >= t1) continue;
                        if constexpr (BF16) {
                            const uint32_t x = reinterpret_cast<const uint16_t *>(at)[e];
                            to[e / 2] = e & 1 ? (to[e / 2] & 0xFFFFu) | x << 16 : (to[e / 2] & 0xFFFF0000u) | x;
                        } else {
                            to[e] = reinterpret_cast<const uint32_t *>(at)[e];
                        }
                    }
                }
            }
        }
        if (allowed) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int32_t t = t0 + (j * kBeamThreads + tid) * VEC;  // a multiple of VEC: one word has the bits
                const uint32_t bits = t < t1 ? allowed[t >> 5] >> (t & 31) : 0u;
                uint32_t *to = w + j * WORDS;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if ((bits >> e) & 1u) continue;
                    if constexpr (BF16)
                        to[e / 2] = e & 1 ? (to[e / 2] & 0xFFFFu) | 0xFF800000u : (to[e / 2] & 0xFFFF0000u) | 0xFF80u;
                    else
                        to[e] = 0xFF800000u;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? E / 2 : E); ++i) {
            if constexpr (BF16) {
                asm("{\n\t.reg .b32 t;\n\tadd.rn.bf16x2 t, %0, %1;\n\tmax.bf16x2 %0, t, %2;\n\t}"
                    : "+r"(w[i])
                    : "r"(0u), "r"(0xFF80FF80u));
            } else {
                w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]) + 0.0f, -INFINITY));
            }
        }
    }
    __device__ __forceinline__ float top() const {
        if constexpr (BF16) {
            uint32_t m = w[0];
#pragma unroll
            for (int i = 1; i < E / 2; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
            return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        } else {
            float m = get(0);
#pragma unroll
            for (int e = 1; e < E; ++e) m = fmaxf(m, get(e));
            return m;
        }
    }
    // Place of element e in the part's line of pieces (lower token, lower place).
    __device__ __forceinline__ static int32_t place(int e) {
        return (e / VEC * kBeamThreads + (int)threadIdx.x) * VEC + e % VEC;
    }
};

__device__ __forceinline__ uint64_t beam_shfl(uint64_t v, int d) {
    const uint32_t lo = __shfl_xor_sync(~0u, (uint32_t)v, d), hi = __shfl_xor_sync(~0u, (uint32_t)(v >> 32), d);
    return (uint64_t)hi << 32 | lo;
}

// Sum over the CTA, for all threads.
__device__ __forceinline__ int32_t beam_count(int32_t n, int32_t *s_warp) {
    n = __reduce_add_sync(~0u, n);
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = n;
    __syncthreads();
    int32_t all = 0;
#pragma unroll
    for (int i = 0; i < kBeamThreads / 32; ++i) all += s_warp[i];
    __syncthreads();
    return all;
}

// A candidate of a request: its score's order and its place beam * vocab + token.
struct BeamCand {
    uint64_t order, place;
};
__device__ __forceinline__ bool beam_before(const BeamCand &a, const BeamCand &b) {
    return a.order > b.order || (a.order == b.order && a.place < b.place);
}

struct BeamShared {
    int32_t warp[kBeamThreads / 32];
    alignas(16) uint32_t low[kBeamThreads / 2];
    uint32_t high[kBeamThreads / 32], limit;
    uint64_t sum[kBeamThreads / 32];
    int32_t n, last;
    union {
        struct {
            uint32_t order[kBeamPool];
            int32_t place[kBeamPool];
        } part;
        struct {
            BeamCand pool[kBeamJoin];
            BeamCand best[kBeamKeep];
            double add[kBeamMost];      // score - ln(sum of the row), relative to its largest logit
            float add32[kBeamMost], top[kBeamMost];
            uint64_t sum[kBeamMost];
            BeamCand warp[kBeamThreads / 32];
        } join;
    };
    uint8_t at[1];  // [beams * parts] behind it: how far the slow merge is in each list
};

template <bool BF16, int E>
__device__ __forceinline__ void beam_part(const BeamParams &p, BeamShared &s, int64_t row, int32_t part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    BeamElems<BF16, E> x;
    const int32_t t0 = part * p.part, t1 = min(t0 + p.part, p.vocab);
    x.load(static_cast<const uint8_t *>(p.logits) + row * p.stride * (BF16 ? 2 : 4), t0, t1, p.vocab,
           p.allowed ? p.allowed + row * p.allowed_stride : nullptr);
    const float own = x.top();
    // the largest of each group of threads, 32 groups at least and twice as many as elements are kept
    const int width = p.keep <= 16 ? 8 : p.keep <= 32 ? 4 : 2;
    const uint32_t mine = beam_order(own);
    uint32_t g = mine;
    for (int d = width / 2; d > 0; d >>= 1) g = max(g, __shfl_xor_sync(~0u, g, d));
    if (tid % width == 0) s.low[tid / width] = g;
    const uint32_t hi = __reduce_max_sync(~0u, g);
    if (lane == 0) s.high[warp] = hi;
    if (tid == 0) s.n = 0;
    __syncthreads();
    if (tid < kBeamThreads / width) {
        // their keep-th largest: as many elements reach it, and in random order few more
        const int groups = kBeamThreads / width;
        const uint32_t v = s.low[tid];
        int above = 0, equal = 0;
        for (int i = 0; i < groups; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&s.low[i]);
            above += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
            equal += (o.x == v) + (o.y == v) + (o.z == v) + (o.w == v);
        }
        if (above < p.keep && above + equal >= p.keep) s.limit = v;  // (the same value where several do)
    }
    uint32_t high = 0;
#pragma unroll
    for (int i = 0; i < kBeamThreads / 32; ++i) high = max(high, s.high[i]);
    const float top = beam_value(high);

    // the part's sum
    float sum = 0.0f;
    if (top == INFINITY) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum += x.get(e) == INFINITY ? 1.0f : 0.0f;
    } else if (beam_plain(top)) {
        const float r = -ceilf(top * kLog2E);
        const f2 ref = make_f2(r, r), big = make_f2(kLog2E, kLog2E), low = make_f2(kLog2ELow, kLog2ELow);
        f2 s0 = make_f2(0.0f, 0.0f), s1 = s0;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const f2 a = make_f2(x.get(e), x.get(e + 1)), b = make_f2(x.get(e + 2), x.get(e + 3));
            const f2 c = fma2(a, low, fma2(a, big, ref)), d = fma2(b, low, fma2(b, big, ref));
            s0 = s0 + make_f2(beam_ex2(f2_lo(c)), beam_ex2(f2_hi(c)));
            s1 = s1 + make_f2(beam_ex2(f2_lo(d)), beam_ex2(f2_hi(d)));
        }
        s0 = s0 + s1;
        sum = f2_lo(s0) + f2_hi(s0);
    } else if (top > -INFINITY) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum += beam_ex2((x.get(e) - top) * kLog2E);
    }
    uint64_t fixed = __float2ull_rn(sum * (float)(1ull << kBeamFixed));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) fixed += beam_shfl(fixed, d);
    if (lane == 0) s.sum[warp] = fixed;
    __syncthreads();
    // (no candidate is -infinity)
    const uint32_t limit_order = max(s.limit, beam_order(-INFINITY) + 1);
    const float limit = beam_value(limit_order);

    // the elements that reach the limit
    const auto push = [&](int e) {
        const int32_t at = atomicAdd(&s.n, 1);
        if (at < kBeamPool) s.part.order[at] = beam_order(x.get(e)), s.part.place[at] = x.place(e);
    };
    if (own >= limit) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (x.get(e) >= limit) push(e);
    }
    __syncthreads();
    int32_t n = s.n;
    if (n > kBeamPool) {
        // the keep-th largest value, then the places that its equals may have
        uint32_t at = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t c = at | 1u << bit;
            int32_t m = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) m += beam_order(x.get(e)) >= c;
            if (beam_count(m, s.warp) >= p.keep) at = c;
        }
        int32_t above = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) above += beam_order(x.get(e)) > at;
        const int32_t left = p.keep - beam_count(above, s.warp);
        int32_t upto = 0;  // fewer than `left` of them have places below it
        for (int bit = 14; bit >= 0; --bit) {
            int32_t m = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) m += beam_order(x.get(e)) == at && x.place(e) < upto + (1 << bit);
            if (beam_count(m, s.warp) < left) upto += 1 << bit;
        }
        if (tid == 0) s.n = 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t o = beam_order(x.get(e));
            if (o > at || (o == at && x.place(e) <= upto)) push(e);
        }
        __syncthreads();
        n = s.n;
    }
    // sorted by counting, four threads for each
    BeamEntry *to = p.entries + (row * p.parts + part) * p.keep;
    for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
        const int i = min(i0 + tid / 4, n - 1);
        const uint32_t o = s.part.order[i];
        const int32_t at = s.part.place[i];
        int32_t rank = 0;
        for (int j = tid % 4; j < n; j += 4) {
            const uint32_t other = s.part.order[j];
            rank += other > o || (other == o && s.part.place[j] < at);
        }
        rank += __shfl_xor_sync(~0u, rank, 1);
        rank += __shfl_xor_sync(~0u, rank, 2);
        if (tid % 4 == 0 && i0 + tid / 4 < n && rank < p.keep) to[rank] = BeamEntry{beam_value(o), t0 + at};
    }
    if (tid < p.keep && tid >= n) to[tid] = BeamEntry{-INFINITY, -1};
    if (tid == 0) {
        uint64_t all = 0;
#pragma unroll
        for (int i = 0; i < kBeamThreads / 32; ++i) all += s.sum[i];
        p.stats[row * p.parts + part] = BeamStat{top, 0, all};
    }
}

// The last CTA of a request: rows' sums, the best `keep` candidates, the outputs.
__device__ __forceinline__ void beam_join(const BeamParams &p, BeamShared &s, int32_t request) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)request * p.beams;
    for (int b = warp; b < p.beams; b += kBeamThreads / 32) {
        const BeamStat *st = p.stats + (row0 + b) * p.parts;
        float top = -INFINITY;
        for (int c = lane; c < p.parts; c += 32) top = fmaxf(top, __ldcg(&st[c].top));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const double ref = beam_ref(top);
        uint64_t sum = 0;
        for (int c = lane; c < p.parts; c += 32) {
            const float t = __ldcg(&st[c].top);
            uint64_t y = __ldcg(reinterpret_cast<const unsigned long long *>(&st[c].sum));
            if (t == -INFINITY || (top == INFINITY && t < top)) continue;
            if (t != top) {
                const double d = ref - beam_ref(t);  // whole, but for logits beyond 2^20
                if (d >= 64.0) y = 0;
                else if (d == rint(d)) y >>= (int)d;
                else y = (uint64_t)((double)y * exp2(-d));
            }
            sum += y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += beam_shfl(sum, d);
        if (lane == 0) s.join.top[b] = top, s.join.sum[b] = sum;
    }
    __syncthreads();
    if (tid < p.beams) {
        const float top = s.join.top[tid], score = p.scores_in[row0 + tid];
        const uint64_t sum = s.join.sum[tid];
        double add = -INFINITY;
        if (sum > 0 && isfinite(score)) {
            // ln of the sum relative to the largest logit
            const double shift = beam_plain(top) ? beam_ref(top) - (double)top * 1.4426950408889634 : 0.0;
            add = (double)score - (log2((double)sum) - kBeamFixed + shift) * 0.69314718055994530942;
        }
        s.join.add[tid] = add;
        s.join.add32[tid] = (float)add;
    }
    if (tid == 0) s.n = 0;
    __syncthreads();
    const int32_t lists = p.beams * p.parts;
    const BeamEntry *entries = p.entries + row0 * p.parts * p.keep;
    const auto load = [&](int32_t list, int32_t i) {
        const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(entries + (int64_t)list * p.keep + i));
        return BeamEntry{__uint_as_float(u.x), (int32_t)u.y};
    };
    const auto relative = [&](const BeamEntry &e, int b) { return e.x == s.join.top[b] ? 0.0f : e.x - s.join.top[b]; };
    const auto cand = [&](const BeamEntry &e, int b) {
        const double d = e.x == s.join.top[b] ? 0.0 : (double)e.x - (double)s.join.top[b];
        return BeamCand{beam_order(s.join.add[b] + d), (uint64_t)b * (uint64_t)p.vocab + (uint64_t)e.token};
    };
    // 32-bit scores differ from the true ones by less than this
    const auto slack = [&](float v, int b) { return 9.5e-7f * (fabsf(v) + fabsf(s.join.add32[b])); };
    const int width = p.keep <= 8 ? 32 : p.keep <= 16 ? 16 : p.keep <= 32 ? 8 : 4;
    float best = -INFINITY;
    // the lists go round the groups, so that few of them leave none empty
    const int32_t l0 = tid / width + kBeamThreads / width * (tid % width);
    for (int32_t l = l0; l < lists; l += kBeamThreads) {
        const int b = l / p.parts;
        if (s.join.add[b] == -INFINITY) continue;
        const BeamEntry e = load(l, 0);
        if (e.token < 0) continue;
        const float v = relative(e, b) + s.join.add32[b];
        best = fmaxf(best, v - slack(v, b));
    }
    uint32_t g = beam_order(best + 0.0f);
    for (int d = width / 2; d > 0; d >>= 1) g = max(g, __shfl_xor_sync(~0u, g, d));
    g = __reduce_min_sync(~0u, g);
    if (lane == 0) s.low[warp] = g;
    __syncthreads();
    uint32_t low = ~0u;
#pragma unroll
    for (int i = 0; i < kBeamThreads / 32; ++i) low = min(low, s.low[i]);
    const float limit = beam_value(low);
    for (int32_t l = tid; l < lists; l += kBeamThreads) {
        const int b = l / p.parts;
        if (s.join.add[b] == -INFINITY) continue;
        for (int32_t i = 0; i < p.keep; ++i) {
            const BeamEntry e = load(l, i);
            if (e.token < 0) break;
            const float v = relative(e, b) + s.join.add32[b];
            if (v + slack(v, b) < limit) break;  // (not so where v is -infinity and the slack infinite)
            const BeamCand c = cand(e, b);
            if (c.order <= beam_order(-(double)INFINITY)) break;
            const int32_t at = atomicAdd(&s.n, 1);
            if (at < kBeamJoin) s.join.pool[at] = c;
        }
    }
    __syncthreads();
    int32_t n = s.n;
    if (n <= kBeamJoin) {
        for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
            const int i = min(i0 + tid / 4, n - 1);
            const BeamCand c = s.join.pool[i];
            int32_t rank = 0;
            for (int j = tid % 4; j < n; j += 4) rank += beam_before(s.join.pool[j], c);
            rank += __shfl_xor_sync(~0u, rank, 1);
            rank += __shfl_xor_sync(~0u, rank, 2);
            if (tid % 4 == 0 && i0 + tid / 4 < n && rank < p.keep) s.join.best[rank] = c;
        }
        n = min(n, p.keep);
    } else {
        // too many (equal logits, say): the lists are merged, one candidate at a time
        for (int32_t l = tid; l < lists; l += kBeamThreads) s.at[l] = 0;
        for (n = 0; n < p.keep; ++n) {
            BeamCand c = {0, ~0ull};
            int32_t from = -1;
            for (int32_t l = tid; l < lists; l += kBeamThreads) {
                const int b = l / p.parts, i = s.at[l];
                if (i >= p.keep || s.join.add[b] == -INFINITY) continue;
                const BeamEntry e = load(l, i);
                if (e.token < 0) continue;
                const BeamCand other = cand(e, b);
                if (other.order > beam_order(-(double)INFINITY) && beam_before(other, c)) c = other, from = l;
            }
            BeamCand w = c;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const BeamCand other = {beam_shfl(w.order, d), beam_shfl(w.place, d)};
                if (beam_before(other, w)) w = other;
            }
            if (lane == 0) s.join.warp[warp] = w;
            __syncthreads();
            w = s.join.warp[0];
#pragma unroll
            for (int i = 1; i < kBeamThreads / 32; ++i)
                if (beam_before(s.join.warp[i], w)) w = s.join.warp[i];
            if (w.order == 0) break;  // no more
            if (from >= 0 && c.place == w.place) s.at[from] += 1;
            if (tid == 0) s.join.best[n] = w;
            __syncthreads();
        }
    }
    __syncthreads();
    // the candidates, and the beams that go on: those that do not end here
    if (warp == 0) {
        int32_t on = 0;
        for (int i0 = 0; i0 < p.keep; i0 += 32) {
            const int i = i0 + lane;
            int32_t token = -1, parent = -1;
            float score = -INFINITY;
            if (i < n) {
                const BeamCand c = s.join.best[i];
                const int b = (int)(c.place / (uint64_t)p.vocab);
                token = (int32_t)(c.place - (uint64_t)b * (uint64_t)p.vocab);
                parent = (int32_t)(row0 + b);
                score = (float)beam_value(c.order);
            }
            if (i < p.take) {
                const int64_t at = (int64_t)request * p.take + i;
                p.cand_tokens[at] = token, p.cand_parents[at] = parent, p.cand_scores[at] = score;
            }
            const uint32_t go = __ballot_sync(~0u, i < n && token != p.eos);
            const int32_t to = on + __popc(go & ((1u << lane) - 1u));
            if ((go >> lane & 1u) && to < p.beams) p.tokens[row0 + to] = token, p.parents[row0 + to] = parent, p.scores[row0 + to] = score;
            on += __popc(go);
        }
        for (int i = on + lane; i < p.beams; i += 32) p.tokens[row0 + i] = -1, p.parents[row0 + i] = -1, p.scores[row0 + i] = -INFINITY;
    }
}

template <bool BF16, int E>
__global__ void __launch_bounds__(kBeamThreads, E == 32 && !BF16 ? 4 : 6) w12_beam_select_kernel(const BeamParams p) {
    extern __shared__ uint4 beam_dyn[];
    BeamShared &s = *reinterpret_cast<BeamShared *>(beam_dyn);
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / p.parts;
    const int32_t part = (int32_t)(blockIdx.x - row * p.parts), request = (int32_t)(row / p.beams);
    pdl_launch_dependents();
    pdl_wait();
    if (isfinite(p.scores_in[row])) {
        beam_part<BF16, E>(p, s, row, part);
    } else {  // a beam that does not go on
        BeamEntry *to = p.entries + (row * p.parts + part) * p.keep;
        if (tid < p.keep) to[tid] = BeamEntry{-INFINITY, -1};
        if (tid == 0) p.stats[row * p.parts + part] = BeamStat{-INFINITY, 0, 0};
    }
    __syncthreads();
    if (tid == 0) {
        const uint32_t all = (uint32_t)p.beams * (uint32_t)p.parts;
        s.last = arrive_acq_rel(&p.counters[request]) == all - 1;
        if (s.last) p.counters[request] = 0;
    }
    __syncthreads();
    if (s.last) beam_join(p, s, request);
}

}  // namespace dev
}  // namespace w12
