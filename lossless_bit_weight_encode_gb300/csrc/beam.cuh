// Best continuations of every request over its beams and the vocabulary (w12_beam_select
// in include/w12.h).
//
// Mathematics.  Row (a beam) with logits x_v, M = max x_v: the candidate (beam, v) has
// the score s + ((x_v - M) - ln sum_v exp(x_v - M)).  Within a row the order of scores is
// that of the logits, so a part of a row needs to hand on no more than its `keep` largest
// logits and its share of the sum; what scores they have shows when the rows' sums are
// there.
//
// One launch.  A CTA takes one part of a row, tile by tile into registers (16-byte loads, the
// next tile's in flight), for the maximum and the sum; the selection reads the few threads'
// elements that may be among the best once more.  The threads' sums are relative to the warp's
// largest logit so far, are added in 64-bit fixed point relative to the part's and the row's
// largest one and do not depend on the parts' order.  The largest logit's own term is exactly
// 1, and what is summed depends on differences from it alone: a token that alone counts has
// the beam's score, and rows that differ by a constant compare as equal.  Every other term
// carries 2^-22 of the exponential, a thread's sum its fp32 roundings (2^-24 of it for each of
// some 20 additions) and a new maximum 2^-23: a score is within 4e-6 of the definition's if all
// went the same way, and mostly within 2e-7.  The selection's threshold is the smallest of
// as many thread groups' maxima as elements are kept: at least that many elements reach
// it and, in random order, a few times that many; they are sorted by counting.  Where too many reach
// it (a mask that leaves whole groups empty, equal logits), the exact one is found by
// bisection over the bits.  The CTA that arrives last at a request joins its parts the
// same way, in 64 bits.
//
// What bounds it: few rows the chain load, maximum, sum, selection, join (4 beams of 151936
// BF16 logits 10.0 us, where the bytes take 0.2); many rows, next to that chain, 15 instructions
// per 32 logits on SMs with uneven work (128 rows 21.1 us, 1.8 TB/s, 56 % of all issue slots:
// the instructions alone are 7.5 us, the bytes 5.8; parts are a whole number per row, here
// four of 4.6 tiles, so that an SM has three or four CTAs, up to 18.6 tiles where 15.6 are its
// share).  35 rows of 50257 fp32 logits under a mask 13.2 us: four CTAs per SM begin at once,
// and what follows the loads is as long as they are.
#pragma once

#include <cstdint>

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kBeamThreads = 256, kBeamCtas = 4, kBeamTiles = 16, kBeamKeep = 64, kBeamMost = 32;
constexpr int kBeamPool = 512;     // elements of a part that may reach the threshold
constexpr int kBeamJoin = 1024;    // and of a request
constexpr int kBeamVocab = 1 << 22;
constexpr int kBeamFixed = 40;     // bits of the sums' fraction

struct BeamStat {
    float top;      // largest logit of the part (-infinity: none)
    uint32_t pad;
    uint64_t sum;   // of exp(x - top), times 2^kBeamFixed
};
struct BeamEntry {
    float x;
    int32_t token;  // -1: none
};

// log2 of a positive whole number, to 3e-9.  x = 2^k f with 1 <= f < 2; of f's first six bits
// c is about 1 / f, in eight bits (1 for the first ones: a power of two's is exact), so that
// t = f c - 1 is small (2^-6) and exact, and
// log2(f) = log2(1 / c) + log2(1 + t), the first from a table and the second from its series,
// in 32 bits (2^-24 of 2^-6).
// exp(-d) for d > 0, to 1e-9 (in what beam_scaled does with it): -d log2(e) = n / 64 + t with n
// whole and t within 1 / 128, 2^(n mod 64 / 64) from a table, 2^t - 1 from its series in 32 bits.
struct BeamLog {
    double log[64];
    uint32_t power[64];    // 2^(i / 64) times 2^31
    uint16_t inverse[64];  // c times 256
    constexpr BeamLog() : log(), power(), inverse() {
        for (int i = 0; i < 64; ++i) {
            double term = 1, whole = 0;  // exp(i ln(2) / 64)
            for (int n = 1; n < 30; ++n) whole += term, term *= i / 64.0 * 0.69314718055994530942 / n;
            power[i] = (uint32_t)(whole * 2147483648.0 + 0.5);
            // 256 / (1 + (i + 0.5) / 64)
            inverse[i] = i == 0 ? 256 : (uint16_t)((2 * 256 * 64 * 2 + (2 * i + 1 + 128)) / (2 * (2 * i + 1 + 128)));
            // ln(256 / c) = 2 atanh(z)
            const double x = 256.0 / inverse[i], z = (x - 1) / (x + 1);
            double power = z, sum = 0;
            for (int n = 1; n < 60; n += 2) sum += power / n, power *= z * z;
            log[i] = 2 * sum * 1.4426950408889634;
        }
    }
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
    uint32_t per_row_inv;  // ceil(2^32 / (parts keep)): divides what is below 2^32 / (parts keep)
    BeamLog logs;         // (parameters are near; one lane's loads of a table in memory are not)
};

constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.92596303e-8f;  // log2(e) - kLog2E

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
    // Word i (not known when compiled: chosen bit by bit of i).
    __device__ __forceinline__ uint32_t word(int i) const {
        constexpr int WORDS = BF16 ? E / 2 : E;
        uint32_t y[WORDS];
#pragma unroll
        for (int k = 0; k < WORDS; ++k) y[k] = w[k];
#pragma unroll
        for (int half = WORDS / 2; half > 0; half /= 2) {
#pragma unroll
            for (int k = 0; k < half; ++k) y[k] = i & half ? y[k + half] : y[k];
        }
        return y[0];
    }
    __device__ __forceinline__ float element(int e) const {
        if constexpr (BF16) {
            const uint32_t u = word(e / 2);
            return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
        }
        return __uint_as_float(word(e));
    }
    __device__ __forceinline__ static uint32_t none() { return BF16 ? 0xFF80FF80u : 0xFF800000u; }

    // Tokens t0 + (j kBeamThreads + tid) VEC + e, of which those before t1 count; row: the
    // row's token 0, which may lie at any element: a thread has the same tokens of every row
    // (equal rows then have equal sums), from one 16-byte piece of memory or out of two.
    __device__ __forceinline__ void load(const uint8_t *row, int32_t t0, int32_t t1, int32_t vocab) {
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
    }
    // What does not count becomes -infinity.
    __device__ __forceinline__ void settle(int32_t t0, int32_t t1, const uint32_t *allowed) {
        constexpr int WORDS = 4;
        const int tid = threadIdx.x;
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

// A candidate of a request: its score's order and its place, beam and token.
struct BeamCand {
    uint64_t order, place;
};
__device__ __forceinline__ bool beam_before(const BeamCand &a, const BeamCand &b) {
    return a.order > b.order || (a.order == b.order && a.place < b.place);
}

// An element of a part: larger value, larger key; of equal ones the lower place in the part.
__device__ __forceinline__ uint64_t beam_key(uint32_t order, int32_t place) {
    return (uint64_t)order << 32 | (uint32_t)~place;
}

struct BeamShared {
    alignas(16) uint32_t low[kBeamThreads];
    uint32_t high[kBeamThreads / 32], limit;
    uint64_t sum[kBeamThreads / 32];
    int32_t bins[kBeamThreads];
    int32_t n, last;
    union {
        struct {
            float tops[kBeamTiles * kBeamThreads];  // the threads' largest logits of each tile
            uint64_t pool[kBeamPool];               // elements that may be among the part's best
        };
        struct {
            BeamEntry pool[kBeamJoin];
            int32_t row[kBeamJoin];
            uint64_t order[kBeamJoin];
            BeamEntry best[kBeamKeep];
            int32_t best_row[kBeamKeep];
            uint64_t best_order[kBeamKeep];
            double add[kBeamMost];  // score - ln(sum of the row), relative to its largest logit
            float add32[kBeamMost], top[kBeamMost];
            uint64_t sum[kBeamMost];
            BeamCand warp[kBeamThreads / 32];
        } join;
    };
    uint8_t at[1];  // [beams * parts] behind it: how far the slow merge is in each list
};

// The keep-th largest of the groups' maxima in s.low, to s.limit: as many elements reach it
// and, in random order, few more.
__device__ __forceinline__ void beam_limit(BeamShared &s, int32_t keep, int width) {
    const int groups = kBeamThreads / width;
    if ((int)threadIdx.x < groups) {
        const uint32_t v = s.low[threadIdx.x];
        int above = 0, equal = 0;
        for (int i = 0; i < groups; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&s.low[i]);
            above += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
            equal += (o.x == v) + (o.y == v) + (o.z == v) + (o.w == v);
        }
        if (above < keep && above + equal >= keep) s.limit = v;  // (the same value where several do)
    }
}

// exp(from - to) = 2^(n / 64) (1 + p) for from < to; false where that is below 2^-62.
__device__ __forceinline__ bool beam_power(float from, float to, int32_t &n, float &p) {
    const float d = from - to;
    if (!(d > -43.0f)) return false;
    const float part = d - from, low = (from - (d - part)) - (to + part);  // d and low are the difference
    const float whole = rintf(d * (64.0f * kLog2E));
    float t = fmaf(d, kLog2E, whole * -0.015625f);
    t = fmaf(low, kLog2E, fmaf(d, kLog2ELow, t));
    p = t * (0.69314718f + t * (0.24022651f + t * 0.05550411f));
    n = (int32_t)whole;
    return true;
}
// A sum relative to the logit `from` as one relative to `to`, at least as large.
__device__ __forceinline__ uint64_t beam_scaled(const BeamLog &table, uint64_t v, float from, float to) {
    int32_t n;
    float p;
    if (from == to) return v;
    if (!beam_power(from, to, n, p)) return 0;
    const uint64_t y = __umul64hi(v, (uint64_t)table.power[n & 63] << 32);  // v 2^(n mod 64 / 64) / 2
    return (y + (uint64_t)__float2ll_rn((float)y * p)) << 1 >> -(n >> 6);
}
__device__ __forceinline__ float beam_scaled(const BeamLog &table, float v, float from, float to) {
    int32_t n;
    float p;
    if (!beam_power(from, to, n, p)) return 0.0f;
    const float y = v * ((float)table.power[n & 63] * 4.656612873077393e-10f);  // 2^-31
    return fmaf(y, p, y) * __int_as_float(((n >> 6) + 127) << 23);
}

// Adds a part's sum (largest logit t) to that of others (largest logit top).
__device__ __forceinline__ void beam_add(const BeamLog &table, float &top, uint64_t &sum, float t, uint64_t y) {
    const float m = fmaxf(top, t);
    sum = beam_scaled(table, sum, top, m) + beam_scaled(table, y, t, m);
    top = m;
}

// The lanes' sums together, for all of them.
__device__ __forceinline__ void beam_total(const BeamLog &table, float &top, uint64_t &sum) {
    const float most = beam_value(__reduce_max_sync(~0u, beam_order(top)));
    sum = beam_scaled(table, sum, top, most);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += beam_shfl(sum, x);
    top = most;
}

__device__ __forceinline__ double beam_log2(const BeamLog &table, uint64_t x) {
    const int k = 63 - __clzll((long long)x);
    const uint64_t f = x << (63 - k);                      // times 2^63
    const int i = (int)(f >> 57) & 63;
    // f c - 1, times 2^63: the product's bits from 2^8 up
    const int64_t t = (int64_t)((__umul64hi(f, (uint64_t)table.inverse[i] << 48) << 8) - (1ull << 63));
    const float y = (float)t * 1.0842021724855044e-19f;    // 2^-63
    const float poly = y * (1.0f + y * (-0.5f + y * (0.33333333f + y * (-0.25f + y * (0.2f + y * -0.16666667f)))));
    return (double)k + table.log[i] + (double)poly * 1.4426950408889634;
}

// The tiles of one part of a row.
template <bool BF16, int E>
struct BeamTiles {
    static constexpr int32_t TILE = kBeamThreads * E;
    const uint8_t *base;
    const uint32_t *allowed;
    int32_t t0, t1, vocab;

    // One token's logit: the load, and what becomes of it.
    __device__ __forceinline__ uint32_t raw(int32_t token) const {
        const int32_t t = min(token, t1 - 1);
        if constexpr (BF16) return reinterpret_cast<const uint16_t *>(base)[t];
        return reinterpret_cast<const uint32_t *>(base)[t];
    }
    __device__ __forceinline__ float settled(uint32_t raw, int32_t token) const {
        if (token >= t1 || (allowed && !(allowed[token >> 5] >> (token & 31) & 1u))) return -INFINITY;
        return fmaxf(__uint_as_float(BF16 ? raw << 16 : raw) + 0.0f, -INFINITY);  // no NaN, no -0
    }
    // f(tile, its place in the part) for the thread's elements of each tile, the next one's
    // loads in flight while one is worked on; `next`: the first one's.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        BeamElems<BF16, E> next;
        next.load(base, t0, t1, vocab);
        each(next, f);
    }
    template <class F>
    __device__ __forceinline__ void each(BeamElems<BF16, E> &next, F f) const {
        for (int32_t a = t0; a < t1; a += TILE) {
            BeamElems<BF16, E> x = next;
            if (a + TILE < t1) next.load(base, a + TILE, t1, vocab);
            x.settle(a, t1, allowed);
            f(x, a - t0);
        }
    }
};

// Where too many elements reach the threshold (equal logits, say): the keep-th largest value
// and the place that the last of its equals may have, a byte of both at a time from the
// number of elements for each of its values.  All threads; the part has `keep` candidates or more.
template <bool BF16, int E>
__device__ __noinline__ void beam_exact(const BeamTiles<BF16, E> &tiles, BeamShared &s, int32_t keep, uint32_t least,
                                        uint32_t &limit, int32_t &upto) {
    const int tid = threadIdx.x;
    int32_t left = keep;
    limit = 0;
    upto = 0;
    for (int pass = 0; pass < 7; ++pass) {
        // bytes 3 to 0 of the order, from above; then bytes 2 to 0 of the place, from below
        const bool places = pass > 3;
        const int shift = places ? 8 * (6 - pass) : 8 * (3 - pass);
        s.bins[tid] = 0;
        __syncthreads();
        tiles.each([&](const BeamElems<BF16, E> &x, int32_t at) {
#pragma unroll 1
            for (int e = 0; e < E; ++e) {
                const uint32_t o = beam_order(x.element(e)), place = (uint32_t)(at + x.place(e));
                const bool in = places ? o == limit && (pass == 4 ||
                                                        place >> (shift + 8) == (uint32_t)upto >> (shift + 8))
                                       : o >= least && (pass == 0 || o >> (shift + 8) == limit >> (shift + 8));
                if (in) atomicAdd(&s.bins[((places ? place : o) >> shift) & 255u], 1);
            }
        });
        __syncthreads();
        int32_t seen = 0, bin = places ? 0 : 255;
        for (; bin != (places ? 255 : 0); bin += places ? 1 : -1) {
            if (seen + s.bins[bin] >= left) break;
            seen += s.bins[bin];
        }
        left -= seen;
        if (places) upto |= bin << shift;
        else limit |= (uint32_t)bin << shift;
        __syncthreads();
    }
}

// One part of a row.
template <bool BF16, int E>
__device__ __forceinline__ void beam_part(const BeamParams &p, BeamShared &s, int64_t row, int32_t part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t t0 = part * p.part;
    const BeamTiles<BF16, E> tiles = {static_cast<const uint8_t *>(p.logits) + row * p.stride * (BF16 ? 2 : 4),
                                      p.allowed ? p.allowed + row * p.allowed_stride : nullptr, t0,
                                      min(t0 + p.part, p.vocab), p.vocab};
    BeamElems<BF16, E> first;
    first.load(tiles.base, t0, tiles.t1, p.vocab);
    if (!isfinite(p.scores_in[row])) {  // a beam that does not go on
        if (tid < p.keep) p.entries[(row * p.parts + part) * p.keep + tid] = BeamEntry{-INFINITY, -1};
        if (tid == 0) p.stats[row * p.parts + part] = BeamStat{-INFINITY, 0, 0};
        return;
    }
    // the warp's largest logit so far, the thread's sum relative to it, the thread's largest
    float top = -INFINITY, sum = 0.0f, mine = -INFINITY;
    tiles.each(first, [&](const BeamElems<BF16, E> &x, int32_t at) {
        const float own = x.top();
        mine = fmaxf(mine, own);
        s.tops[at / E + tid] = own;
        const float most = fmaxf(top, beam_value(__reduce_max_sync(~0u, beam_order(own))));
        if (most != top) {  // the same for the warp
            if (sum > 0.0f) sum = beam_scaled(p.logs, sum, top, most);
            top = most;
        }
        if (top == INFINITY) {
#pragma unroll
            for (int e = 0; e < E; ++e) sum += x.get(e) == INFINITY ? 1.0f : 0.0f;
        } else if (top > -INFINITY) {
            const f2 minus = make_f2(-top, -top), by = make_f2(kLog2E, kLog2E);
            f2 s0 = make_f2(0.0f, 0.0f), s1 = s0;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const f2 c = (make_f2(x.get(e), x.get(e + 1)) + minus) * by;
                const f2 d = (make_f2(x.get(e + 2), x.get(e + 3)) + minus) * by;
                s0 = s0 + make_f2(beam_ex2(f2_lo(c)), beam_ex2(f2_hi(c)));
                s1 = s1 + make_f2(beam_ex2(f2_lo(d)), beam_ex2(f2_hi(d)));
            }
            s0 = s0 + s1;
            sum += f2_lo(s0) + f2_hi(s0);
        }
    });
    // the selection's threshold, from the largest of groups of threads; meanwhile the part's sum
    const int width = p.keep <= 16 ? 8 : p.keep <= 32 ? 4 : 2;
    uint32_t g = beam_order(mine);
    for (int d = width / 2; d > 0; d >>= 1) g = max(g, __shfl_xor_sync(~0u, g, d));
    if (tid % width == 0) s.low[tid / width] = g;
    if (tid == 0) s.n = 0;
    __syncthreads();
    beam_limit(s, p.keep, width);
    uint64_t fixed = __float2ull_rn(sum * (float)(1ull << kBeamFixed));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) fixed += beam_shfl(fixed, d);
    if (lane == 0) s.sum[warp] = fixed, s.high[warp] = __float_as_uint(top);
    __syncthreads();
    // no candidate is -infinity
    const uint32_t least = beam_order(__uint_as_float(BF16 ? 0xFF7F0000u : 0xFF7FFFFFu));
    uint32_t limit = max(s.limit, least);
    int32_t upto = 0x7FFFFFFF;
    const int32_t all_tiles = (tiles.t1 - t0 + tiles.TILE - 1) / tiles.TILE;
    for (int round = 0; round < 2; ++round) {
        // The elements that reach it: of the lanes and tiles whose largest one does (hits), a
        // lane for each element, read once more; several hits' loads are in flight.
        const float floor = beam_value(limit);
        constexpr int VEC = BeamElems<BF16, E>::VEC, B = 4;
        int32_t j = -1;
        uint32_t left = 0;
        while (true) {
            float v[B];
            uint32_t raw[B];
            int32_t place[B];
            int n = 0;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                while (left == 0 && ++j < all_tiles) left = __ballot_sync(~0u, s.tops[j * kBeamThreads + tid] >= floor);
                const int l = left ? __ffs((int)left) - 1 : 0, e = lane % E;
                place[k] = min(j, all_tiles - 1) * tiles.TILE + (e / VEC * kBeamThreads + warp * 32 + l) * VEC +
                           e % VEC;
                if (left) n = k + 1;
                left &= left - 1;
            }
#pragma unroll
            for (int k = 0; k < B; ++k) raw[k] = tiles.raw(t0 + place[k]);
#pragma unroll
            for (int k = 0; k < B; ++k) v[k] = k < n && lane < E ? tiles.settled(raw[k], t0 + place[k]) : -INFINITY;
            if (n == 0) break;
            uint32_t in[B];
            int32_t count = 0, base = 0;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                in[k] = __ballot_sync(~0u, v[k] > floor || (v[k] == floor && place[k] <= upto));
                count += __popc(in[k]);
            }
            if (lane == 0 && count) base = atomicAdd(&s.n, count);
            base = __shfl_sync(~0u, base, 0);
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int32_t to = base + __popc(in[k] & ((1u << lane) - 1u));
                if ((in[k] >> lane & 1u) && to < kBeamPool) s.pool[to] = beam_key(beam_order(v[k]), place[k]);
                base += __popc(in[k]);
            }
            if (n < B) break;
        }
        __syncthreads();
        if (s.n <= kBeamPool) break;
        beam_exact(tiles, s, p.keep, least, limit, upto);
        if (tid == 0) s.n = 0;
        __syncthreads();
    }
    // sorted by counting, four threads for each
    const int32_t n = s.n;
    BeamEntry *to = p.entries + (row * p.parts + part) * p.keep;
    for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
        const int i = min(i0 + tid / 4, n - 1);
        const uint64_t key = s.pool[i];
        int32_t rank = 0;
#pragma unroll 4
        for (int k = tid % 4; k < n; k += 4) rank += s.pool[k] > key;
        rank += __shfl_xor_sync(~0u, rank, 1);
        rank += __shfl_xor_sync(~0u, rank, 2);
        if (tid % 4 == 0 && i0 + tid / 4 < n && rank < p.keep)
            to[rank] = BeamEntry{beam_value((uint32_t)(key >> 32)), t0 + ~(int32_t)(uint32_t)key};
    }
    if (tid < p.keep && tid >= n) to[tid] = BeamEntry{-INFINITY, -1};
    if (warp == kBeamThreads / 32 - 1) {
        float most = lane < kBeamThreads / 32 ? __uint_as_float(s.high[lane]) : -INFINITY;
        uint64_t all = lane < kBeamThreads / 32 ? s.sum[lane] : 0;
        beam_total(p.logs, most, all);
        if (lane == 0) p.stats[row * p.parts + part] = BeamStat{most, 0, all};
    }
}

// The last CTA of a request: rows' sums, the best `keep` candidates, the outputs.
__device__ __forceinline__ void beam_join(const BeamParams &p, BeamShared &s, int32_t request) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)request * p.beams;
    const int32_t lists = p.beams * p.parts;
    const BeamEntry *entries = p.entries + row0 * p.parts * p.keep;
    const auto load = [&](int32_t list, int32_t i) {
        const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(entries + (int64_t)list * p.keep + i));
        return BeamEntry{__uint_as_float(u.x), (int32_t)u.y};
    };
    // A thread has every 256th entry of all lists.  The first kAhead of them are asked for
    // while the rows' sums are made.
    const int64_t total = (int64_t)lists * p.keep;
    constexpr int kAhead = 8;
    BeamEntry ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        ahead[k] = BeamEntry{-INFINITY, -1};
        if (tid + k * kBeamThreads < total) ahead[k] = load(0, tid + k * kBeamThreads);
    }
    for (int b = warp; b < p.beams; b += kBeamThreads / 32) {
        const BeamStat *st = p.stats + (row0 + b) * p.parts;
        float top = -INFINITY;
        uint64_t sum = 0;  // relative to `top`
        for (int c0 = 0; c0 < p.parts; c0 += 32) {
            uint4 u = make_uint4(0xFF800000u, 0, 0, 0);
            if (c0 + lane < p.parts) u = __ldcg(reinterpret_cast<const uint4 *>(st + c0 + lane));
            if (c0 == 0) top = __uint_as_float(u.x), sum = (uint64_t)u.w << 32 | u.z;
            else beam_add(p.logs, top, sum, __uint_as_float(u.x), (uint64_t)u.w << 32 | u.z);
        }
        beam_total(p.logs, top, sum);
        if (lane == 0) {
            const float score = p.scores_in[row0 + b];
            double add = -INFINITY;
            if (sum > 0 && isfinite(score))
                add = (double)score - (beam_log2(p.logs, sum) - kBeamFixed) * 0.69314718055994530942;
            s.join.top[b] = top;
            s.join.add[b] = add;
            s.join.add32[b] = (float)add;
        }
    }
    if (tid == 0) s.n = 0;
    __syncthreads();
    const auto relative = [&](float x, float top) { return x == top ? 0.0f : x - top; };
    const auto order_of = [&](float x, int b) {
        const float top = s.join.top[b];
        return beam_order(s.join.add[b] + (x == top ? 0.0 : (double)x - (double)top));
    };
    // 32-bit scores differ from the true ones by less than this
    const auto slack = [&](float v, float add) { return 9.5e-7f * (fabsf(v) + fabsf(add)); };
    // f(entry, its beam) for all of the thread's entries
    const int32_t per_row = p.parts * p.keep;
    const auto each = [&](auto f) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k * kBeamThreads < total)  // (entries that are not there have no token)
                f(ahead[k], (int)__umulhi((uint32_t)(tid + k * kBeamThreads), p.per_row_inv));
        for (int64_t i = tid + kAhead * kBeamThreads; i < total; i += kBeamThreads) {
            const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(entries + i));
            f(BeamEntry{__uint_as_float(u.x), (int32_t)u.y}, (int)(i / per_row));
        }
    };
    // the threshold: the keep-th largest of the best scores of groups of threads
    float best = -INFINITY;
    each([&](const BeamEntry &e, int b) {
        if (e.token < 0) return;
        const float add = s.join.add32[b];
        if (add == -INFINITY) return;
        const float v = relative(e.x, s.join.top[b]) + add;
        best = fmaxf(best, v - slack(v, add));
    });
    const int width = p.keep <= 16 ? 4 : p.keep <= 32 ? 2 : 1;
    uint32_t g = beam_order(best + 0.0f);
    for (int d = width / 2; d > 0; d >>= 1) g = max(g, __shfl_xor_sync(~0u, g, d));
    if (tid % width == 0) s.low[tid / width] = g;
    __syncthreads();
    beam_limit(s, p.keep, width);
    __syncthreads();
    const float limit = beam_value(s.limit);
    each([&](const BeamEntry &e, int b) {
        if (e.token < 0) return;
        const float add = s.join.add32[b];
        if (add == -INFINITY) return;
        const float v = relative(e.x, s.join.top[b]) + add;
        if (v + slack(v, add) < limit) return;  // (not so where v is -infinity and the slack infinite)
        const int32_t at = atomicAdd(&s.n, 1);
        if (at < kBeamJoin) s.join.pool[at] = e, s.join.row[at] = b;
    });
    __syncthreads();
    int32_t n = s.n;
    const uint64_t none = beam_order(-(double)INFINITY);
    if (n <= kBeamJoin) {
        for (int i = tid; i < n; i += kBeamThreads) s.join.order[i] = order_of(s.join.pool[i].x, s.join.row[i]);
        __syncthreads();
        int32_t real = 0;
        for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
            const int i = min(i0 + tid / 4, n - 1);
            const uint64_t order = s.join.order[i];
            const BeamEntry e = s.join.pool[i];
            const int32_t b = s.join.row[i];
            int32_t rank = 0;
#pragma unroll 4
            for (int k = tid % 4; k < n; k += 4) {
                const uint64_t other = s.join.order[k];
                rank += other > order;
                if (other == order) {  // the lower beam, then token
                    const int32_t c = s.join.row[k];
                    rank += c < b || (c == b && s.join.pool[k].token < e.token);
                }
            }
            rank += __shfl_xor_sync(~0u, rank, 1);
            rank += __shfl_xor_sync(~0u, rank, 2);
            if (tid % 4 == 0 && i0 + tid / 4 < n && order > none) {
                ++real;
                if (rank < p.keep) s.join.best[rank] = e, s.join.best_row[rank] = b, s.join.best_order[rank] = order;
            }
        }
        real = __reduce_add_sync(~0u, real);
        if (lane == 0) s.low[warp] = (uint32_t)real;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int i = 0; i < kBeamThreads / 32; ++i) n += (int32_t)s.low[i];
        n = min(n, p.keep);
    } else {
        // too many (equal logits, say): the lists are merged, one candidate at a time
        for (int32_t l = tid; l < lists; l += kBeamThreads) s.at[l] = 0;
        for (n = 0; n < p.keep; ++n) {
            BeamCand c = {0, ~0ull};
            BeamEntry mine = {0.0f, -1};
            int32_t from = -1;
            for (int32_t l = tid; l < lists; l += kBeamThreads) {
                const int b = l / p.parts, i = s.at[l];
                if (i >= p.keep || s.join.add32[b] == -INFINITY) continue;
                const BeamEntry e = load(l, i);
                if (e.token < 0) continue;
                const BeamCand other = {order_of(e.x, b), (uint64_t)b << 32 | (uint32_t)e.token};
                if (other.order > none && beam_before(other, c)) c = other, from = l, mine = e;
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
            if (from >= 0 && c.place == w.place) {
                s.at[from] += 1;
                s.join.best[n] = mine, s.join.best_row[n] = (int32_t)(w.place >> 32), s.join.best_order[n] = w.order;
            }
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
                token = s.join.best[i].token;
                parent = (int32_t)(row0 + s.join.best_row[i]);
                score = (float)beam_value(s.join.best_order[i]);
            }
            if (i < p.take) {
                const int64_t at = (int64_t)request * p.take + i;
                p.cand_tokens[at] = token, p.cand_parents[at] = parent, p.cand_scores[at] = score;
            }
            const uint32_t go = __ballot_sync(~0u, i < n && token != p.eos);
            const int32_t to = on + __popc(go & ((1u << lane) - 1u));
            if ((go >> lane & 1u) && to < p.beams)
                p.tokens[row0 + to] = token, p.parents[row0 + to] = parent, p.scores[row0 + to] = score;
            on += __popc(go);
        }
        for (int i = on + lane; i < p.beams; i += 32)
            p.tokens[row0 + i] = -1, p.parents[row0 + i] = -1, p.scores[row0 + i] = -INFINITY;
    }
}

template <bool BF16, int E>
__global__ void __launch_bounds__(kBeamThreads, kBeamCtas) w12_beam_select_kernel(const __grid_constant__ BeamParams p) {
    extern __shared__ uint4 beam_dyn[];
    BeamShared &s = *reinterpret_cast<BeamShared *>(beam_dyn);
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / p.parts;
    const int32_t part = (int32_t)(blockIdx.x - row * p.parts), request = (int32_t)(row / p.beams);
    pdl_launch_dependents();
    pdl_wait();
    beam_part<BF16, E>(p, s, row, part);
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
