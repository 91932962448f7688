// Pages copied inside caches (w12_kv_copy in include/w12.h): keys, values and an 8-bit
// cache's scales, bit by bit.
//
// Two bytes move per byte copied, so HBM bounds a large call and the launch a small one.
// A warp takes 16 tokens of one head's keys or values (4 KB for 128 BF16 columns): the
// lanes' 16-byte loads, up to eight each, are all in flight before the first store, and
// a call of a few pages spreads over all SMs.  All layers' copies are one launch: after a
// step of beam search a model has one such call, not one per layer.
//
// Measured: partly filled pages of 32 beams (32 tokens, 8 heads of 128) in 8 layers at once
// 5.0 us, where an empty launch takes 2; 2500 whole pages of 64 tokens 190 us, 6.9 TB/s, 103 %
// of a plain copy's rate.
#pragma once

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kCopyThreads = 256, kCopyCaches = 64, kCopySlice = 16;

struct KvCopyParams {
    uint8_t *k[kCopyCaches], *v[kCopyCaches];
    float *scales[kCopyCaches];
    const int32_t *src, *dst, *rows;
    int64_t num_pages;
    int64_t page_bytes, head_bytes, row_bytes;  // strides
    int64_t items;
    uint64_t slices_inv, heads_inv, pairs_inv;  // floor((2^64 - 1) / n)
    int32_t pairs, page_size, kv_heads;
    uint32_t *status;
};

// x = q n + r with inv = floor((2^64 - 1) / n): the high product is the quotient or one less.
__device__ __forceinline__ int64_t copy_div(int64_t x, int32_t n, uint64_t inv, int32_t &r) {
    int64_t q = (int64_t)__umul64hi((uint64_t)x, inv);
    int64_t left = x - q * n;
    if (left >= n) ++q, left -= n;
    r = (int32_t)left;
    return q;
}

// ROW: bytes of a token's row of one head.
template <int ROW, bool Q8>
__global__ void __launch_bounds__(kCopyThreads) w12_kv_copy_kernel(const __grid_constant__ KvCopyParams p) {
    constexpr int CH = ROW / 16, N = kCopySlice * CH / 32;  // 16-byte chunks of a row, of a lane
    constexpr int G = N < 8 ? N : 8;
    const int lane = threadIdx.x & 31;
    const int32_t slices = p.page_size / kCopySlice;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t item = (int64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32; item < p.items;
         item += (int64_t)gridDim.x * (kCopyThreads / 32)) {
        int32_t slice, head, pair;
        const int64_t a = copy_div(item >> 1, slices, p.slices_inv, slice);
        const int64_t b = copy_div(a, p.kv_heads, p.heads_inv, head);
        const int32_t layer = (int32_t)copy_div(b, p.pairs, p.pairs_inv, pair);
        const bool values = item & 1;
        const int32_t from = p.src[pair], to = p.dst[pair];
        int32_t rows = p.rows ? p.rows[pair] : p.page_size;
        if (from < 0 || to < 0) continue;  // none
        if (from >= p.num_pages || to >= p.num_pages) {
            if (lane == 0) atomicOr(p.status, kStatusKvIndex);
            continue;
        }
        rows = min(rows, p.page_size) - slice * kCopySlice;  // of this slice, if positive
        if (rows <= 0 || from == to) continue;
        uint8_t *base = values ? p.v[layer] : p.k[layer];
        const int64_t at = head * p.head_bytes + (int64_t)slice * kCopySlice * p.row_bytes;
        const uint8_t *s = base + from * p.page_bytes + at;
        uint8_t *d = base + to * p.page_bytes + at;
        float4 sc;
        int64_t sat = 0;
        const bool scaled = Q8 && !values && lane < kCopySlice / 2 && 2 * lane < rows;
        if (Q8 && scaled) {  // two tokens' (key, value) scales
            sat = ((int64_t)head * p.page_size + slice * kCopySlice) * 2 + 4 * lane;
            sc = *reinterpret_cast<const float4 *>(p.scales[layer] + (int64_t)from * p.kv_heads * p.page_size * 2 + sat);
        }
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += G) {
            uint4 u[G];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int x = (i0 + i) * 32 + lane, row = x / CH;
                if (row < rows) u[i] = *reinterpret_cast<const uint4 *>(s + row * p.row_bytes + x % CH * 16);
            }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int x = (i0 + i) * 32 + lane, row = x / CH;
                if (row < rows) *reinterpret_cast<uint4 *>(d + row * p.row_bytes + x % CH * 16) = u[i];
            }
        }
        if (Q8 && scaled) {
            float *to_s = p.scales[layer] + (int64_t)to * p.kv_heads * p.page_size * 2 + sat;
            if (2 * lane + 1 < rows) *reinterpret_cast<float4 *>(to_s) = sc;
            else *reinterpret_cast<float2 *>(to_s) = make_float2(sc.x, sc.y);
        }
    }
}

}  // namespace dev
}  // namespace w12
