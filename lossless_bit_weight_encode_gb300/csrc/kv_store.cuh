// Head norm, position rotation and the cache write of new tokens, and cached
// rows back (w12_kv_store and w12_kv_read in include/w12.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w             per head of q and k
//   (a, b) -> (a cos - b sin, b cos + a sin)       for the rotated pairs
//
// head_dim / 8 neighbouring lanes hold one head, eight elements (16 bytes) each:
// the mean is a butterfly over them, a rotation partner half a rotation apart is
// a shuffle (rot / 16 lanes away), one next door is in the lane itself.  All of
// it is fp32 on the BF16 inputs with one rounding at the store.
//
// Every element is read and written once and nothing is shared between heads, so a
// large call is bounded by HBM: 8192 tokens of 24 + 2 x 4 heads of 256 take 49.6 us,
// 5.6 TB/s (the norm, rotation and address instructions keep issue 65 % busy, which is
// why the arithmetic is packed in pairs); 30000 cached tokens of 4 heads of 256 read
// back take 38.3 us, 6.4 TB/s.  One token is a launch: 2.2 us.  The same chunk stored into
// an 8-bit cache and read back takes 77 us (46 at the HBM rate), in two launches.
#pragma once

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kStoreThreads = 64, kReadThreads = 128;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight BF16 as four pairs, and back.
__device__ __forceinline__ void unpack8(const uint4 &u, f2 (&x)[4]) {
    x[0] = make_f2(bf16_lo(u.x), bf16_hi(u.x)), x[1] = make_f2(bf16_lo(u.y), bf16_hi(u.y));
    x[2] = make_f2(bf16_lo(u.z), bf16_hi(u.z)), x[3] = make_f2(bf16_lo(u.w), bf16_hi(u.w));
}
__device__ __forceinline__ uint4 pack8(const f2 (&x)[4]) {
    return make_uint4(pack_bf16(f2_lo(x[0]), f2_hi(x[0])), pack_bf16(f2_lo(x[1]), f2_hi(x[1])),
                      pack_bf16(f2_lo(x[2]), f2_hi(x[2])), pack_bf16(f2_lo(x[3]), f2_hi(x[3])));
}

// slot / page_size without a 64-bit division: with page_inv = floor((2^64 - 1) /
// page_size) the high product is the quotient or one less (slot < 2^63).
struct KvSlot {
    int64_t page, off;
};
__device__ __forceinline__ KvSlot split_slot(const KvGeom &c, int64_t slot) {
    KvSlot r;
    r.page = (int64_t)__umul64hi((uint64_t)slot, c.page_inv);
    r.off = slot - r.page * c.page_size;
    if (r.off >= c.page_size) ++r.page, r.off -= c.page_size;
    return r;
}

// The lane's cosines and sines: of the columns 8 sub .. 8 sub + 7 (halves), or
// of its four pairs, each twice (cosines) or as -sin, sin (interleaved).
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_row(const float *row, int rot, int sub, f2 (&cs)[4], f2 (&sn)[4]) {
    const int h2 = rot / 2;
    if (INTERLEAVED) {
        const int c = 4 * sub;
        float a[4] = {1.0f, 1.0f, 1.0f, 1.0f}, b[4] = {};  // a pair that is not rotated
        if (h2 % 4 == 0) {                                  // 16-byte aligned rows
            if (c < h2) {
                const float4 x = *reinterpret_cast<const float4 *>(row + c);
                const float4 y = *reinterpret_cast<const float4 *>(row + h2 + c);
                a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
                b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < h2) a[i] = row[c + i], b[i] = row[h2 + c + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = make_f2(a[i], a[i]), sn[i] = make_f2(-b[i], b[i]);
    } else if (8 * sub < rot) {
        // the first half gets x cos - partner sin, the second x cos + partner sin
        const bool low = 8 * sub < h2;
        const int c = low ? 8 * sub : 8 * sub - h2;
        const float4 *x = reinterpret_cast<const float4 *>(row + c);
        const float4 *y = reinterpret_cast<const float4 *>(row + h2 + c);
        const float sg = low ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = x[i], b = y[i];
            cs[2 * i] = make_f2(a.x, a.y), cs[2 * i + 1] = make_f2(a.z, a.w);
            sn[2 * i] = make_f2(sg * b.x, sg * b.y), sn[2 * i + 1] = make_f2(sg * b.z, sg * b.w);
        }
    }
}

// Norm (norm set) and rotation (rot > 0) of the lane's eight elements of one
// head; norm and rot are the same for the whole warp.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void norm_rotate(f2 (&x)[4], bool norm, const uint4 &weight, float eps, int rot,
                                            const f2 (&cs)[4], const f2 (&sn)[4], int sub) {
    constexpr int LANES = D / 8;
    if (norm) {
        f2 q = x[0] * x[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) q = fma2(x[i], x[i], q);
        float s = f2_lo(q) + f2_hi(q);
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const float r = rsqrtf(s * (1.0f / (float)D) + eps);
        const f2 r2 = make_f2(r, r);
        f2 w[4];
        unpack8(weight, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = x[i] * r2 * w[i];
    }
    if (rot == 0) return;
    if (INTERLEAVED) {
        // (a, b) (cos, cos) + (b, a) (-sin, sin)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fma2(make_f2(f2_hi(x[i]), f2_lo(x[i])), sn[i], x[i] * cs[i]);
    } else {
        const int half = rot / 16;  // lanes of half the rotated columns
        const bool mine = sub < 2 * half, low = sub < half;
        const int lane = threadIdx.x & 31;
        const int partner = mine ? (low ? lane + half : lane - half) : lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 o =
                make_f2(__shfl_sync(~0u, f2_lo(x[i]), partner), __shfl_sync(~0u, f2_hi(x[i]), partner));
            if (mine) x[i] = fma2(o, sn[i], x[i] * cs[i]);
        }
    }
}

// One CTA handles the heads of one token, or a share of them where the tokens
// are few.  A warp takes D / 8 lanes per head, so 256 / D heads of one kind (q, k
// or v) at a time, four times in a row: their loads are all in flight before the
// first is used, and the token's cosines and sines are read once.  What bounds
// the large calls is HBM and, close behind it, the instructions per element:
// hence the packed arithmetic and the warp-uniform kinds.
template <int D, bool Q8, bool INTERLEAVED>
__global__ void __launch_bounds__(kStoreThreads, 16) w12_kv_store_kernel(KvStoreParams p) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES, WARPS = kStoreThreads / 32, U = 4;
    const int lane = threadIdx.x & 31, sub = lane % LANES, mine = lane / LANES;
    const int hk = p.c.kv_heads;
    const int nq = (p.heads + HEADS - 1) / HEADS, nk = (hk + HEADS - 1) / HEADS, all = nq + 2 * nk;
    // the warp's number by a shuffle: the compiler then knows that what follows
    // from it is the same for the whole warp
    const int first = blockIdx.x * WARPS + __shfl_sync(~0u, (int)threadIdx.x / 32, 0), stride = gridDim.x * WARPS;
    const int col = mine * D + 8 * sub;
    pdl_launch_dependents();
    pdl_wait();
    uint32_t flags = 0;
    for (int t = blockIdx.y; (uint32_t)t < (uint32_t)p.tokens; t = (int)((uint32_t)t + gridDim.y)) {
        const int64_t slot = p.slots[t];
        int64_t pos = p.rot > 0 ? p.positions[t] : 0;
        const uint16_t *const qt = p.q + t * p.q_stride, *const kt = p.k + t * p.k_stride,
                              *const vt = p.v + t * p.v_stride;
        f2 cs[4] = {}, sn[4] = {};
        for (int j0 = first; j0 < all; j0 += U * stride) {
            uint4 u[U];
#pragma unroll
            for (int r = 0; r < U; ++r) {
                const int j = j0 + r * stride;
                u[r] = make_uint4(0, 0, 0, 0);
                const int h = (j < nq ? j : j < nq + nk ? j - nq : j - nq - nk) * HEADS;  // of lane group 0
                const uint16_t *src = j < nq ? qt : j < nq + nk ? kt : vt;
                if (j < all && h + mine < (j < nq ? p.heads : hk))
                    u[r] = *reinterpret_cast<const uint4 *>(src + h * D + col);
            }
            if (j0 == first && p.rot > 0 && first < nq + nk) {
                if (pos < 0 || pos >= p.rope_rows) {
                    flags |= kStatusKvIndex;
                    pos = pos < 0 ? 0 : p.rope_rows - 1;
                }
                rope_row<INTERLEAVED>(p.rope + pos * p.rot, p.rot, sub, cs, sn);
            }
            const KvSlot at = split_slot(p.c, slot < 0 ? 0 : slot);
            const bool kept = slot >= 0 && at.page < p.c.num_pages;
            if (slot >= 0 && !kept) flags |= kStatusKvIndex;
            const int64_t row = at.page * p.c.page_stride + at.off * p.c.row_stride;
#pragma unroll
            for (int r = 0; r < U; ++r) {
                const int j = j0 + r * stride;
                if (j >= all) break;
                const bool is_q = j < nq, is_v = j >= nq + nk;
                const int h0 = (is_q ? j : is_v ? j - nq - nk : j - nq) * HEADS, h = h0 + mine;
                f2 x[4];
                unpack8(u[r], x);
                if (!is_v) {
                    const uint16_t *wp = is_q ? p.q_norm : p.k_norm;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (wp) w = reinterpret_cast<const uint4 *>(wp)[sub];
                    norm_rotate<D, INTERLEAVED>(x, wp != nullptr, w, p.eps, p.rot, cs, sn, sub);
                }
                if (is_q) {
                    if (h < p.heads)
                        *reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + h0 * D + col) = pack8(x);
                    continue;
                }
                const bool write = h < hk && kept;
                const int64_t e = row + h * p.c.head_stride + 8 * sub;
                if (!Q8) {
                    if (write) reinterpret_cast<uint4 *>(is_v ? p.c.v : p.c.k)[e / 8] = is_v ? u[r] : pack8(x);
                    continue;
                }
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) a = max_nan(max_nan(a, fabsf(f2_lo(x[i]))), fabsf(f2_hi(x[i])));
#pragma unroll
                for (int d = LANES / 2; d > 0; d >>= 1) a = max_nan(a, __shfl_xor_sync(~0u, a, d));
                const float s = a / 127.0f;
                if (write) {
                    // a scale that is NaN or infinite keeps q = 0: the row reads
                    // back as NaN
                    const bool usual = s > 0.0f && s < INFINITY;
                    uint32_t b[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float v = (i & 1) ? f2_hi(x[i / 2]) : f2_lo(x[i / 2]);
                        const float q = usual ? fminf(fmaxf(rintf(v / s), -127.0f), 127.0f) : 0.0f;
                        b[i / 4] |= ((uint32_t)(int)q & 0xFFu) << (8 * (i % 4));
                    }
                    reinterpret_cast<uint2 *>(is_v ? p.c.v : p.c.k)[e / 8] = make_uint2(b[0], b[1]);
                    if (sub == 0)
                        p.c.scales[((at.page * hk + h) * p.c.page_size + at.off) * 2 + (is_v ? 1 : 0)] = s;
                }
            }
        }
    }
    if (flags && lane == 0) atomicOr(p.status, flags);
}

// Rows of k and v by slot.  A warp takes the same 256 / D heads of a token's k and
// v, for four (token, heads) items at a time, so that eight loads per lane are in
// flight.
template <int D, bool Q8>
__global__ void __launch_bounds__(kReadThreads) w12_kv_read_kernel(KvReadParams p) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES, U = 4;
    const int lane = threadIdx.x & 31, sub = lane % LANES, mine = lane / LANES;
    const int hk = p.c.kv_heads, rounds = (hk + HEADS - 1) / HEADS;
    const int64_t items = (int64_t)p.tokens * rounds;
    const int64_t stride = (int64_t)gridDim.x * (kReadThreads / 32);
    pdl_launch_dependents();
    pdl_wait();
    uint32_t flags = 0;
    for (int64_t i0 = (int64_t)blockIdx.x * (kReadThreads / 32) + threadIdx.x / 32; i0 < items; i0 += U * stride) {
        int64_t slot[U], to[U];
        int h[U];
#pragma unroll
        for (int r = 0; r < U; ++r) {
            const int64_t i = i0 + r * stride;
            int64_t t = (int64_t)__umul64hi((uint64_t)i, p.rounds_inv);  // i / rounds
            int j = (int)(i - t * rounds);
            if (j >= rounds) ++t, j -= rounds;
            h[r] = j * HEADS + mine;
            const bool live = i < items && h[r] < hk;
            slot[r] = i < items ? p.slots[t] : -1;
            to[r] = live ? ((t * hk + h[r]) * D) / 8 + sub : -1;
        }
        uint4 k[U], v[U];
        float2 s[U];
#pragma unroll
        for (int r = 0; r < U; ++r) {
            const KvSlot at = split_slot(p.c, slot[r] < 0 ? 0 : slot[r]);
            const bool kept = slot[r] >= 0 && at.page < p.c.num_pages;
            if (slot[r] >= 0 && !kept) flags |= kStatusKvIndex;
            k[r] = v[r] = make_uint4(0, 0, 0, 0);
            s[r] = make_float2(0.0f, 0.0f);
            if (kept && to[r] >= 0) {
                const int64_t e =
                    at.page * p.c.page_stride + h[r] * p.c.head_stride + at.off * p.c.row_stride + 8 * sub;
                if (!Q8) {
                    k[r] = reinterpret_cast<const uint4 *>(p.c.k)[e / 8];
                    v[r] = reinterpret_cast<const uint4 *>(p.c.v)[e / 8];
                } else {
                    const uint2 a = reinterpret_cast<const uint2 *>(p.c.k)[e / 8];
                    const uint2 b = reinterpret_cast<const uint2 *>(p.c.v)[e / 8];
                    k[r].x = a.x, k[r].y = a.y, v[r].x = b.x, v[r].y = b.y;
                    s[r] = reinterpret_cast<const float2 *>(
                        p.c.scales)[(at.page * hk + h[r]) * p.c.page_size + at.off];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < U; ++r) {
            if (to[r] < 0) continue;
            if (Q8) {
                f2 x[4], y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t i = (c < 2 ? k[r].x : k[r].y) >> (16 * (c % 2));
                    const uint32_t j = (c < 2 ? v[r].x : v[r].y) >> (16 * (c % 2));
                    x[c] = make_f2((float)(int8_t)i * s[r].x, (float)(int8_t)(i >> 8) * s[r].x);
                    y[c] = make_f2((float)(int8_t)j * s[r].y, (float)(int8_t)(j >> 8) * s[r].y);
                }
                k[r] = pack8(x);
                v[r] = pack8(y);
            }
            reinterpret_cast<uint4 *>(p.k_out)[to[r]] = k[r];
            reinterpret_cast<uint4 *>(p.v_out)[to[r]] = v[r];
        }
    }
    if (flags && lane == 0) atomicOr(p.status, flags);
}

}  // namespace dev
}  // namespace w12
