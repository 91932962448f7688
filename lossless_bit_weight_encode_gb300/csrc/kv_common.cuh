// Pieces shared by the paged key-value cache kernels.
#pragma once

#include <cstdint>

#include "kv_tiles.hpp"

namespace w12 {
namespace dev {

// Status word bits of the paged-cache calls (w12_check_status).
constexpr uint32_t kStatusKvPages = 64u;   // the ring of free pages ran out, or was full
constexpr uint32_t kStatusKvSizes = 128u;  // a length or the token count had to be clamped
constexpr uint32_t kStatusKvIndex = 256u;  // a slot or position outside its table

// Cache geometry as the kernels take it (w12_kv_cache in include/w12.h).
struct KvGeom {
    uint8_t *k, *v;
    float *scales;
    int64_t num_pages;
    int64_t page_stride, head_stride, row_stride;  // elements
    uint64_t page_inv;                             // floor((2^64 - 1) / page_size)
    int32_t page_size, kv_heads;
};

struct KvPlanParams {
    const int32_t *lens, *new_lens;
    const int32_t *owned_in;
    int32_t *owned_out;
    int32_t *tables;
    int64_t table_stride;
    int32_t *ring;
    const int64_t *state_in;
    int64_t *state_out;
    int32_t *cu_new;
    int32_t *positions;
    int64_t *slots;
    uint64_t ring_inv;  // floor((2^64 - 1) / ring_size)
    int32_t requests, max_blocks, page_size, ring_size, tokens, trim;
    uint32_t *status;
};

struct KvStoreParams {
    KvGeom c;
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const uint16_t *q_norm, *k_norm;
    const float *rope;
    const int32_t *positions;
    const int64_t *slots;
    int64_t rope_rows;
    int32_t tokens, heads, rot;
    float eps;
    uint32_t *status;
};

struct KvReadParams {
    KvGeom c;
    const int64_t *slots;
    uint16_t *k_out, *v_out;
    uint64_t rounds_inv;  // floor((2^64 - 1) / warp rounds per token)
    int32_t tokens;
    uint32_t *status;
};

struct KvAttendParams {
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t q_stride, out_stride;
    const int32_t *tables;
    int64_t table_stride;
    const int32_t *lens, *cu_new;
    const uint32_t *tree;
    const int32_t *positions;  // of a windowed tree's tokens; null: their numbers place them
    const uint16_t *v;  // a BF16 cache's values, and their strides in elements
    int64_t v_page_stride, v_head_stride, v_row_stride;
    const float *scales;
    int64_t num_pages;
    int32_t requests, max_keys, tokens, kv_heads, group, window, page_size;
    float scale_log2;  // softmax scale times log2(e)
    float *part;       // partial outputs [2 * CTAs][rows][head_dim]
    float2 *part_ml;   // their maxima and sums [2 * CTAs][rows]
    uint32_t *counters;
    uint32_t n_counters;
    int32_t join_later;  // warps per row of w12_kv_join_kernel, which joins the parts; 0: no such launch
    uint32_t *status;
    uint64_t timeout_ns;
};

// n / d of 0 <= n < 2^31 as a product: with 2^(s - 1) < d <= 2^s and mul = ceil(2^(31 + s) / d),
// mul d is less than d above 2^(31 + s), which moves the quotient by less than
// n / 2^(31 + s) < 1 / d.
struct KvDivisor {
    uint32_t mul, shift;
};
inline KvDivisor kv_divisor(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return {(uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d), 31 + s};
}
__device__ __forceinline__ int32_t kv_over(int32_t n, const KvDivisor &d) {
    return (int32_t)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

// A call with shared prefixes (w12_kv_attend_shared): its spans are the groups' prefixes and
// then what each request has of its own; a row block in one range leaves its rows' sums in
// row_part and row_ml, and row_info says of every row {row of its first part, parts (1: whole),
// tokens of the prefix, of the own ones: that the request shares}.  All three have the prefixes'
// rows first, then the own ones'.
struct KvSharedParams : KvAttendParams {
    const int32_t *prefix_cu, *prefix_lens;
    int32_t groups;
    KvDivisor by_group, by_page;
    float *row_part;  // [2][tokens * heads][head_dim]
    float2 *row_ml;   // [2][tokens * heads]
    int4 *row_info;   // [2][tokens * heads]
};
// Row over query heads per key head, token over page size.
__device__ __forceinline__ int32_t kv_over_group(const KvAttendParams &p, int32_t n) { return n / p.group; }
__device__ __forceinline__ int32_t kv_over_group(const KvSharedParams &p, int32_t n) { return kv_over(n, p.by_group); }
__device__ __forceinline__ int32_t kv_over_page(const KvAttendParams &p, int32_t n) { return n / p.page_size; }
__device__ __forceinline__ int32_t kv_over_page(const KvSharedParams &p, int32_t n) { return kv_over(n, p.by_page); }

template <KvSpans KIND>
struct KvSpanParams : KvSharedParams {
    // the first of the launch's spans among all
    __device__ __forceinline__ int32_t first_span() const { return KIND == kKvOwnSpans ? groups : 0; }
};
// What a row block costs beside its tiles (its q, the pipeline's start and end), in tiles:
// the line counts that many units more for each, so that CTAs with many short blocks have
// fewer of them.  64 requests of 225 tokens behind a prompt of 4000: 2 units 39.6 us, 3 36.6,
// 4 38.3, 6 41.2; twenty trees behind four prompts of 10000: 49.5, 48.5, 47.1, 46.3.  A full
// block of a prompt's own tokens costs much more, 12 us with five tiles that all need masks, and
// these blocks stand together at the line's end: with hundreds of new tokens per request the
// CTAs that get them take twice as long as the others.
constexpr int32_t kKvBlockUnits = 3;

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

// Pairs of fp32 in one 64-bit register and the packed arithmetic on them (each
// half rounds as the scalar operation does).
struct f2 {
    uint64_t v;
};
__device__ __forceinline__ f2 make_f2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float f2_lo(f2 a) { return __uint_as_float((uint32_t)a.v); }
__device__ __forceinline__ float f2_hi(f2 a) { return __uint_as_float((uint32_t)(a.v >> 32)); }
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 operator+(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

}  // namespace dev
}  // namespace w12
