// The joining kernel of attention behind shared prefixes (w12_kv_attend_shared in
// include/w12.h).
//
// Mathematics.  Softmax sums over disjoint sets of keys join as in kv_attend.cuh, whatever
// rows were computed together: the kernels of kv_attend.cuh and kv_attend_tc.cuh run over the
// groups' prefixes, where the rows of all of a group's requests meet the prefix's keys at
// once (32 beams of six query heads: 192 rows, on the tensor cores), and over what each
// request has of its own, and leave the sums of every row's parts; this kernel joins them.
//
// Groups and requests are one line of units and one launch where that serves both: the
// tcgen05 kernel takes a BF16 tile of 64 keys in 0.6 us on each SM, faster than HBM brings it,
// however few of its 128 rows are used.  Else (8-bit caches, very many requests; the rule is
// in kv.cu) the own tokens are a second launch with tiles of their own rows, which takes the
// SMs as the first one's CTAs end.
//
// What bounds the call: a prefix's bytes are read once per group instead of once per request,
// so with a long prefix of few rows it is HBM (16 samples behind 100000 tokens 88 us, 5.2
// TB/s), with many rows the softmax of a tile, and with short own contexts what a piece
// costs beside its tiles (kv_attend_tc.cuh).  Prompts gain nothing: their row blocks are full
// without the other requests' rows, and their own blocks are more than the line counts for them
// (kv_common.cuh); 4 x 300 new tokens behind 4000 384 us, without a prefix 210.
#pragma once

#include "kv_attend.cuh"

namespace w12 {
namespace dev {

struct KvSharedJoin {
    uint16_t *out;
    float *lse;
    int64_t out_stride;
    const int32_t *cu_new;
    const int32_t *prefix_cu;
    int32_t tokens, heads, requests, groups;
    const float *row_part;
    const float2 *row_ml;
    const int4 *row_info;
    uint32_t *status;
    struct Line {
        const float *part;
        const float2 *part_ml;
        int32_t rows, ctas;  // of a row block, of the launch
    } line[2];  // of the prefixes, of the own tokens
};

// A warp per output row (token and head, heads fastest) takes its parts, first the prefix's in
// range order, then the own ones; eight loads in flight (four: twenty trees over 256 columns,
// eight parts a row, 50.5 us in all against 47.7).  2 us behind the last part.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) w12_kv_join_shared_kernel(const __grid_constant__ KvSharedJoin p) {
    constexpr int W = kJoinThreads / 32, V = D / 32;  // columns of a lane
    constexpr int U = 8;                              // parts whose loads are in flight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * W + warp, own_rows = (int64_t)p.tokens * p.heads;
    const int32_t tok = (int32_t)(row / p.heads), h = (int32_t)(row - (int64_t)tok * p.heads);
    pdl_launch_dependents();
    pdl_wait();
    if (row == 0 && lane == 0 && (p.prefix_cu[0] != 0 || p.prefix_cu[p.groups] != p.requests))
        atomicOr(p.status, kStatusKvSizes);
    if (row >= own_rows) return;
    int4 prefix = __ldcg(&p.row_info[row]), own = __ldcg(&p.row_info[own_rows + row]);
    // rows of no request have no note
    if (tok >= __ldcg(&p.cu_new[p.requests]) || tok < __ldcg(&p.cu_new[0])) return;
    // a group whose requests share different numbers of tokens, or a row that no group or
    // request has (a cu that is no prefix sum): its note may be anything
    const auto fits = [&](const int4 &i, const KvSharedJoin::Line &l) {
        return i.y == 1 || ((uint32_t)(i.y - 1) < (uint32_t)l.ctas &&
                            (uint32_t)i.x <= (uint32_t)((2 * (l.ctas - i.y) + 1) * l.rows));
    };
    if (own.z <= 0) prefix.y = 0;
    else if (prefix.z != own.z || !fits(prefix, p.line[0])) own.x = -1;
    if (own.x < 0 || !fits(own, p.line[1])) {
        prefix.y = own.y = 0;
        if (lane == 0) atomicOr(p.status, kStatusKvSizes);
    }
    const int32_t n0 = prefix.y, n = n0 + own.y;
    float acc[V] = {}, mm = -INFINITY, sum = 0.0f;
    for (int32_t k0 = 0; k0 < n; k0 += U) {
        float y[U][V];
        float2 s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t kk = min(k0 + u, n - 1);
            const bool mine = kk >= n0;
            const int32_t k = mine ? kk - n0 : kk;
            const int4 info = mine ? own : prefix;
            const KvSharedJoin::Line &l = p.line[mine];
            const bool whole = info.y == 1;
            // the first CTA's part is in its second slot, every other one's in its first
            const int64_t at = whole ? row + (mine ? own_rows : 0) : info.x + (int64_t)(2 * k + (k == 0)) * l.rows;
            s[u] = __ldcg((whole ? p.row_ml : l.part_ml) + at);
            const float *src = (whole ? p.row_part : l.part) + at * D;
            if constexpr (V == 2) {
                const float2 a = __ldcg(reinterpret_cast<const float2 *>(src) + lane);
                y[u][0] = a.x, y[u][1] = a.y;
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 a = __ldcg(reinterpret_cast<const float4 *>(src) + lane * (V / 4) + e / 4);
                    y[u][e] = a.x, y[u][e + 1] = a.y, y[u][e + 2] = a.z, y[u][e + 3] = a.w;
                }
            }
        }
        float mn = mm;
#pragma unroll
        for (int u = 0; u < U; ++u) mn = fmaxf(mn, s[u].x);
        const float base = kv_part_base(mn), f0 = ex2(mm - base);
        mm = mn;
        sum *= f0;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= f0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u < n) {
                const float g = ex2(s[u].x - base);
                sum = fmaf(g, s[u].y, sum);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(g, y[u][e], acc[e]);
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + tok * p.out_stride + (int64_t)h * D) + lane * (V / 2);
#pragma unroll
    for (int e = 0; e < V; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[row] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
}

}  // namespace dev
}  // namespace w12
