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
#pragma once

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kStoreThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 to packed BF16, round to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Norm and rotation of the lane's eight elements (columns 8 * sub ..) of one
// head.  `any` and `rot` are the same for the whole warp (the shuffles need every
// lane); `norm` says whether this lane's head takes the norm.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool any, bool norm, const float (&w)[8], float eps,
                                            int rot, const float (&cs)[8], const float (&sn)[8], int sub) {
    constexpr int LANES = D / 8;
    if (any) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const float r = rsqrtf(s / (float)D + eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = norm ? x[i] * r * w[i] : x[i];
    }
    if (rot == 0) return;
    if (INTERLEAVED) {
        // cs, sn: entries 0..3 for the lane's four pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (8 * sub + 2 * i < rot) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cs[i] - b * sn[i];
                x[2 * i + 1] = b * cs[i] + a * sn[i];
            }
        }
    } else {
        const int half = rot / 16;  // lanes of half the rotated columns
        const bool mine = sub < 2 * half, low = sub < half;
        const int lane = threadIdx.x & 31;
        const int partner = mine ? (low ? lane + half : lane - half) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(~0u, x[i], partner);
            if (mine) x[i] = low ? x[i] * cs[i] - o * sn[i] : x[i] * cs[i] + o * sn[i];
        }
    }
}

// Cosines and sines of the lane's columns (pairs, when interleaved: four of each).
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_row(const float *row, int rot, int sub, float (&cs)[8], float (&sn)[8]) {
    const int h2 = rot / 2;
    if (INTERLEAVED) {
        const int c = 4 * sub;
        if (h2 % 4 == 0) {  // 16-byte aligned rows
            if (c < h2) {
                const float4 a = *reinterpret_cast<const float4 *>(row + c);
                const float4 b = *reinterpret_cast<const float4 *>(row + h2 + c);
                cs[0] = a.x, cs[1] = a.y, cs[2] = a.z, cs[3] = a.w;
                sn[0] = b.x, sn[1] = b.y, sn[2] = b.z, sn[3] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c + i < h2) cs[i] = row[c + i], sn[i] = row[h2 + c + i];
            }
        }
    } else if (8 * sub < rot) {
        const int c = 8 * sub >= h2 ? 8 * sub - h2 : 8 * sub;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(row + c + i);
            const float4 b = *reinterpret_cast<const float4 *>(row + h2 + c + i);
            cs[i] = a.x, cs[i + 1] = a.y, cs[i + 2] = a.z, cs[i + 3] = a.w;
            sn[i] = b.x, sn[i + 1] = b.y, sn[i + 2] = b.z, sn[i + 3] = b.w;
        }
    }
}

// One CTA handles the heads (q, then k, then v) of one token, or a share of
// them where the tokens are few.  A lane group takes every GROUPS-th head, four
// at a time: their loads are all in flight before the first is used, and the
// token's cosines and sines are read once per group and not once per head.
template <int D, bool Q8, bool INTERLEAVED>
__global__ void __launch_bounds__(kStoreThreads, 3) w12_kv_store_kernel(KvStoreParams p) {
    constexpr int LANES = D / 8, GROUPS = kStoreThreads / LANES, U = 4;
    const int sub = threadIdx.x % LANES, group = blockIdx.x * GROUPS + threadIdx.x / LANES;
    const int stride = gridDim.x * GROUPS;
    const int heads = p.heads, hk = p.c.kv_heads, all = heads + 2 * hk;
    pdl_launch_dependents();
    pdl_wait();
    const bool norm_q = p.q_norm != nullptr, norm_k = p.k_norm != nullptr;
    uint32_t flags = 0;
    for (int64_t t = blockIdx.y; t < p.tokens; t += gridDim.y) {
        const int64_t slot = p.slots[t];
        int64_t pos = p.rot > 0 ? p.positions[t] : 0;
        float cs[8] = {}, sn[8] = {};
        // the shuffles want whole warps: every group of the CTA runs the same rounds
        for (int j0 = blockIdx.x * GROUPS; j0 < all; j0 += U * stride) {
            const int jg = j0 - blockIdx.x * GROUPS + group;
            uint4 u[U];
#pragma unroll
            for (int r = 0; r < U; ++r) {
                const int j = jg + r * stride;
                u[r] = make_uint4(0, 0, 0, 0);
                if (j < all) {
                    const uint16_t *src = j < heads        ? p.q + t * p.q_stride + (int64_t)j * D
                                          : j < heads + hk ? p.k + t * p.k_stride + (int64_t)(j - heads) * D
                                                           : p.v + t * p.v_stride + (int64_t)(j - heads - hk) * D;
                    u[r] = reinterpret_cast<const uint4 *>(src)[sub];
                }
            }
            if (j0 == blockIdx.x * GROUPS && p.rot > 0) {
                if (pos < 0 || pos >= p.rope_rows) {
                    flags |= kStatusKvIndex;
                    pos = pos < 0 ? 0 : p.rope_rows - 1;
                }
                rope_row<INTERLEAVED>(p.rope + pos * p.rot, p.rot, sub, cs, sn);
            }
            const int64_t page = slot / p.c.page_size, off = slot - page * p.c.page_size;
            const bool kept = slot >= 0 && page < p.c.num_pages;
            if (slot >= 0 && !kept) flags |= kStatusKvIndex;
#pragma unroll
            for (int r = 0; r < U; ++r) {
                const int j = jg + r * stride;
                if (j0 + r * stride >= all) break;  // the same for the whole CTA
                const bool is_q = j < heads, is_v = j >= heads + hk;
                const bool is_k = !is_q && !is_v;
                const int h = is_q ? j : is_k ? j - heads : j - heads - hk;
                float x[8];
                unpack8(u[r], x);
                // a warp of values alone has nothing to norm or rotate
                if (__any_sync(~0u, !is_v)) {
                    float y[8], w[8] = {};
                    if (is_q ? norm_q : norm_k && is_k)
                        unpack8(reinterpret_cast<const uint4 *>(is_q ? p.q_norm : p.k_norm)[sub], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i];
                    norm_rotate<D, INTERLEAVED>(y, norm_q || norm_k, is_q ? norm_q : norm_k, w, p.eps, p.rot, cs, sn,
                                                sub);
                    if (!is_v) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = y[i];
                    }
                }
                if (is_q) {
                    reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + (int64_t)h * D)[sub] = pack8(x);
                }
                const bool write = j < all && !is_q && kept;
                const int64_t e = page * p.c.page_stride + h * p.c.head_stride + off * p.c.row_stride + 8 * sub;
                if (!Q8) {
                    if (write) reinterpret_cast<uint4 *>(is_k ? p.c.k : p.c.v)[e / 8] = is_k ? pack8(x) : u[r];
                } else if (__any_sync(~0u, !is_q)) {
                    float a = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(x[i]));
#pragma unroll
                    for (int d = LANES / 2; d > 0; d >>= 1) a = max_nan(a, __shfl_xor_sync(~0u, a, d));
                    const float s = a / 127.0f;
                    if (write) {
                        // a scale that is NaN or infinite keeps q = 0: the row
                        // reads back as NaN
                        const bool usual = s > 0.0f && s < INFINITY;
                        uint32_t b[2] = {0, 0};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float r8 = usual ? fminf(fmaxf(rintf(x[i] / s), -127.0f), 127.0f) : 0.0f;
                            b[i / 4] |= ((uint32_t)(int)r8 & 0xFFu) << (8 * (i % 4));
                        }
                        reinterpret_cast<uint2 *>(is_k ? p.c.k : p.c.v)[e / 8] = make_uint2(b[0], b[1]);
                        if (sub == 0)
                            p.c.scales[((page * hk + h) * p.c.page_size + off) * 2 + (is_k ? 0 : 1)] = s;
                    }
                }
            }
        }
    }
    if (flags && sub == 0) atomicOr(p.status, flags);
}

// Rows of k and v by slot, eight elements per thread.
template <int D, bool Q8>
__global__ void __launch_bounds__(kStoreThreads) w12_kv_read_kernel(KvReadParams p) {
    constexpr int LANES = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int hk = p.c.kv_heads;
    const int64_t total = (int64_t)p.tokens * hk * LANES;
    uint32_t flags = 0;
    for (int64_t i = (int64_t)blockIdx.x * kStoreThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kStoreThreads) {
        const int sub = (int)(i % LANES);
        const int64_t r = i / LANES;
        const int h = (int)(r % hk);
        const int64_t slot = p.slots[r / hk];
        const int64_t page = slot / p.c.page_size, off = slot - page * p.c.page_size;
        const bool kept = slot >= 0 && page < p.c.num_pages;
        if (slot >= 0 && !kept) flags |= kStatusKvIndex;
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (kept) {
            const int64_t e = page * p.c.page_stride + h * p.c.head_stride + off * p.c.row_stride + 8 * sub;
            if (!Q8) {
                k = reinterpret_cast<const uint4 *>(p.c.k)[e / 8];
                v = reinterpret_cast<const uint4 *>(p.c.v)[e / 8];
            } else {
                const float2 s =
                    reinterpret_cast<const float2 *>(p.c.scales)[(page * hk + h) * p.c.page_size + off];
                const uint2 a = reinterpret_cast<const uint2 *>(p.c.k)[e / 8];
                const uint2 b = reinterpret_cast<const uint2 *>(p.c.v)[e / 8];
                float x[8], y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    x[c] = (float)(int8_t)((c < 4 ? a.x : a.y) >> (8 * (c % 4))) * s.x;
                    y[c] = (float)(int8_t)((c < 4 ? b.x : b.y) >> (8 * (c % 4))) * s.y;
                }
                k = pack8(x);
                v = pack8(y);
            }
        }
        reinterpret_cast<uint4 *>(p.k_out)[i] = k;
        reinterpret_cast<uint4 *>(p.v_out)[i] = v;
    }
    if (flags) atomicOr(p.status, flags);
}

}  // namespace dev
}  // namespace w12
