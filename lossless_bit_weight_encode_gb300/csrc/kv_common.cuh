// Pieces shared by the paged key-value cache kernels.
#pragma once

#include <cstdint>

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
