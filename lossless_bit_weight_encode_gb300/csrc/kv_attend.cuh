// Attention of a step's new tokens over the paged cache (w12_kv_attend in
// include/w12.h).
//
// Mathematics.  Per request, key head and row (a row is one new token and one
// query head of the key head's group): x_j = scale * log2(e) * q . k_j, one pass
// over the keys with the running maximum m, sum l = sum 2^(x_j - m) and output
// o = sum 2^(x_j - m) v_j.  Two partial results join as
//   m = max(m1, m2), l = l1 2^(m1-m) + l2 2^(m2-m), o likewise,
// and out = o / l, lse = m ln 2 + ln l.  The running maximum is only raised when
// a score passes it by more than 8 (2^8 is harmless in fp32), so that most tiles
// need neither the cross-lane maximum nor a rescaling of o.
//
// What bounds it: the keys and values are read once, from HBM; per byte of a
// BF16 cache there are 2 * rows flops.  Layout for that: a producer warp keeps a
// ring of tiles (64 or 128 keys, see AttendTile) full by TMA (one 5-D box of 16 tokens x head_dim per k and
// v: 16 tokens are the page granularity, so any page size that is a multiple of
// 16 works and a box never crosses a page), and four consumer warps multiply on
// the tensor cores straight from shared memory.  The rows are few, so they are
// the 8-wide N of mma.m16n8k16 and the keys (for k q^T) or the head's columns
// (for v^T p^T) its M: nothing is padded from 6 rows to 128.  The probabilities
// go from accumulator to operand layout with one movmatrix per 8 x 8.  Warps
// split a tile's keys (WK) and, where a warp's registers do not hold the sums of all
// rows, the rows (WR).
//
// Work split.  The unit is one tile of one (request, key head, row block);
// all units form one line that the CTAs cut into equal ranges, whatever the
// lengths.  A request's row blocks all have its tiles, from the first key that its first
// token sees to its last key: a block of a long prompt also walks the tiles that none of
// its own rows sees.  A range that covers a row block's keys only in part leaves its
// partial result in the workspace, and the CTA that arrives last at the block's
// counter joins the parts in range order (the same result in every run).  Where
// that would be a long chain for one CTA (kv_launch.cuh has the rule), a second
// kernel joins every row with a CTA of its own.
//
// Q8 cache: int8 elements become BF16 exactly in registers; a key's scale
// multiplies its score, a value's scale its probability.
//
// Measured: 64 requests of 8000 tokens, 48 heads over 8 of 128: BF16 311 us, 6.8 TB/s
// (a copy of that many bytes takes as long); Q8 190 us, 5.7 TB/s, where issue (the
// conversion) is close behind HBM.  Two of 100001, 24 heads over 4 of 256: 116 us,
// 6.6 TB/s.  128 windows of 1024 keys: 55 us, 5.0 TB/s; calls this short spend some
// 14 us before the ring is full and after it has run dry.  One request of 777 tokens:
// 7.2 us, all of it latency (two launches, TMA, the join).
#pragma once

#include <cuda.h>

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kAttendTile = 64;       // keys of a tile of the tcgen05 kernel
constexpr int kAttendSlice = 16;      // keys of one TMA box and of one mma
constexpr int kAttendThreads = 160;   // four consumer warps and the producer
constexpr float kAttendLazy = 8.0f;   // how far a score may pass the running maximum (log2)
constexpr float kLn2 = 0.69314718055994530942f;

// CTAs per SM that a variant is made for, by bytes of a stage and registers.
template <int D, bool Q8, int NT>
constexpr int attend_ctas() {
    return D == 256 && !Q8 ? 1 : D == 64 && Q8 && NT == 1 ? 3 : 2;
}

// Keys of a pipeline stage: 128 where they fit 32 KB, so that a warp has two slices
// for each wait and works on both at once; else 64.
template <int D, bool Q8>
struct AttendTile {
    static constexpr int kKeys = D * (Q8 ? 1 : 2) <= 128 ? 128 : 64;
};

template <int D, bool Q8, int WK, int WR, int NT>
struct AttendCfg {
    static_assert(WK * WR == 4, "four consumer warps");
    static constexpr int kRows = WR * NT * 8;
    static constexpr int kElem = Q8 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem < 128 ? D * kElem : 128;  // swizzled box rows
    static constexpr int kHalves = D * kElem / kRowBytes;
    static constexpr int kSliceBytes = kAttendSlice * D * kElem;
    static constexpr int kTile = AttendTile<D, Q8>::kKeys;
    static constexpr int kSlices = kTile / kAttendSlice;
    static constexpr int kPair = kSlices / WK >= 2 ? 2 : 1;  // slices a warp works on at once
    static constexpr int kTileBytes = kSlices * kSliceBytes;  // k (or v) of a stage
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kCtas = attend_ctas<D, Q8, NT>();
    static constexpr int kRing = (kCtas == 1 ? 192 : kCtas == 2 ? 96 : 60) * 1024;
    static constexpr int kStages = kRing / kStageBytes > 8 ? 8 : kRing / kStageBytes;
    static_assert(kStages >= 2, "a ring");
    static constexpr int kScaleBytes = Q8 ? kTile * 8 : 0;  // per stage: (k, v) of each key
    static constexpr int kMergeStride = 68;           // floats: 64 columns and 4 of skew
    static constexpr int kOffScales = kStages * kStageBytes;
    static constexpr int kOffMerge = kOffScales + kStages * kScaleBytes;
    static constexpr int kOffMl = kOffMerge + WK * kRows * kMergeStride * 4;
    static constexpr int kOffBars = kOffMl + WK * kRows * 8;
    static constexpr int kSmemBytes = kOffBars + 2 * 8 * kStages + 4 * kStages + 16 + 1024;  // 1024: alignment
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// c += a (16 x 16) * b (16 x 8), BF16 operands, fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (a & mask) ^ bits as one instruction (left to itself the compiler makes two, each
// with a constant of its own).
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

// Four int8 to BF16, exactly: bytes 0 and 2 to lo, bytes 1 and 3 to hi.  With
// b = byte: 128 + (b & 127) is BF16 0x4300 | (b & 127); adding -128 (b >= 0) or
// -256 (b < 0), which is BF16 0xC300 | (b & 128), gives b, which BF16 holds.
__device__ __forceinline__ void q8_to_bf16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t h = w >> 8;
    const uint32_t a0 = and_xor(w, 0x007F007Fu, 0x43004300u), b0 = and_xor(w, 0x00800080u, 0xC300C300u);
    const uint32_t a1 = and_xor(h, 0x007F007Fu, 0x43004300u), b1 = and_xor(h, 0x00800080u, 0xC300C300u);
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a0), "r"(b0));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(a1), "r"(b1));
}

// 5-D tiled copy global -> shared.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int32_t c1, int32_t c3, int32_t c4,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7];" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(c1), "r"(0), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// One request as the kernel sees it.
struct KvRequest {
    int32_t past, q0, qlen, kv, first, tile0, ntiles, rblocks;
    int64_t units;
};

template <int ROWS, int TILE>
__device__ __forceinline__ KvRequest kv_request(const KvAttendParams &p, int b) {
    KvRequest r;
    r.q0 = min(max(p.cu_new[b], 0), p.tokens);
    r.qlen = min(max(p.cu_new[b + 1], r.q0), p.tokens) - r.q0;
    r.past = min(max(p.lens[b], 0), p.max_keys);
    r.kv = (int32_t)min((int64_t)r.past + r.qlen, (int64_t)p.max_keys);
    // first key that any of the request's new tokens sees
    r.first = p.window > 0 ? (int32_t)max((int64_t)r.past + 1 - p.window, (int64_t)0) : 0;
    r.tile0 = min(r.first, r.kv) / TILE;
    r.ntiles = r.kv > 0 ? max((r.kv - 1) / TILE + 1 - r.tile0, 1) : 1;
    r.rblocks = (int32_t)(((int64_t)r.qlen * p.group + ROWS - 1) / ROWS);
    r.units = (int64_t)p.kv_heads * r.rblocks * r.ntiles;
    return r;
}

// A CTA's range of units and its place in it; every warp keeps its own copy.
struct KvWalk {
    int64_t total, u, end;  // all units, the next one, the range's end
    int64_t start;          // first unit of request b
    int32_t b, ctas;
};

// Units of all requests, and of those before each lane's: a lane sums a block of
// consecutive requests (their loads overlap), one warp scan joins the blocks.
struct KvSums {
    int64_t total, before;  // all units; those before the lane's block
    int32_t per;            // requests of a block
};

template <int ROWS, int TILE>
__device__ __forceinline__ KvSums kv_sum_units(const KvAttendParams &p) {
    const int lane = threadIdx.x & 31;
    KvSums s;
    s.per = (int32_t)(((uint32_t)p.requests + 31u) / 32u);
    int64_t sum = 0;
#pragma unroll 4
    for (int i = 0; i < s.per; ++i) {
        const int b = lane * s.per + i;
        if (b < p.requests) sum += kv_request<ROWS, TILE>(p, b).units;
    }
    int64_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += x;
    }
    s.total = __shfl_sync(~0u, inc, 31);
    s.before = inc - sum;
    return s;
}

template <int ROWS, int TILE>
__device__ __forceinline__ bool kv_walk_init(const KvAttendParams &p, KvWalk &w, KvRequest &r) {
    const KvSums s = kv_sum_units<ROWS, TILE>(p);
    w.total = s.total;
    w.ctas = (int32_t)min((int64_t)gridDim.x, w.total);
    if ((int)blockIdx.x >= w.ctas) return false;
    w.u = w.total * blockIdx.x / w.ctas;
    w.end = w.total * (blockIdx.x + 1) / w.ctas;
    // the last block that starts at or before u, then the request in it
    const int src = 31 - __clz(__ballot_sync(~0u, s.before <= w.u));
    w.start = __shfl_sync(~0u, s.before, src);
    w.b = src * s.per;
    r = kv_request<ROWS, TILE>(p, w.b);
    while (w.u >= w.start + r.units) {
        w.start += r.units;
        r = kv_request<ROWS, TILE>(p, ++w.b);
    }
    return true;
}

// Table entries that the request's keys take.
__device__ __forceinline__ int32_t kv_entries(const KvAttendParams &p, const KvRequest &r) {
    return r.kv > 0 ? (r.kv - 1) / p.page_size + 1 : 0;
}

// The piece at w.u: its (key head, row block) and its tiles [ja, jb).
struct KvPiece {
    int32_t head, rb, ja, jb;
};

__device__ __forceinline__ KvPiece kv_piece(const KvWalk &w, const KvRequest &r) {
    const int64_t off = w.u - w.start;
    const int32_t item = (int32_t)(off / r.ntiles);
    KvPiece c;
    c.head = item / r.rblocks;
    c.rb = item - c.head * r.rblocks;
    c.ja = (int32_t)(off - (int64_t)item * r.ntiles);
    c.jb = (int32_t)min((int64_t)r.ntiles, w.end - w.u + c.ja);
    return c;
}

// Moves on by n units within the request, to the next request where it ends.
template <int ROWS, int TILE>
__device__ __forceinline__ void kv_advance(const KvAttendParams &p, KvWalk &w, KvRequest &r, int32_t n) {
    w.u += n;
    while (w.u < w.end && w.u >= w.start + r.units) {
        w.start += r.units;
        r = kv_request<ROWS, TILE>(p, ++w.b);
    }
}

// Which keys of a slice one row sees.
struct KvRowView {
    int32_t index;  // of the row's token in the request: past + i; in a windowed tree its position
    uint32_t tree;
};

__device__ __forceinline__ int32_t kv_index(const KvRequest &r, int32_t i) {
    return (int32_t)min((int64_t)r.past + i, (int64_t)0x7FFFFFFF);
}

// The view of new token i.  PLACED: a windowed tree with positions.  There a token's
// position lies between past and its number past + i, so that what bounds the tiles for
// numbers bounds them too.  New tokens that the window leaves out by position are taken
// out of the mask; those that stay have numbers at or above their positions, so they pass
// the comparison of key numbers that the cached keys need.
template <bool PLACED>
__device__ __forceinline__ KvRowView kv_row_view(const KvAttendParams &p, const KvRequest &r, int32_t i) {
    KvRowView v;
    v.index = kv_index(r, i);
    v.tree = p.tree ? p.tree[r.q0 + i] : 0u;
    if (PLACED) {
        const int32_t *at = p.positions + r.q0;
        v.index = min(max(at[i], r.past), v.index);
        if (v.index - r.past >= p.window) {  // deeper than the window is long
            for (uint32_t left = v.tree; left; left &= left - 1) {
                const int32_t j = __ffs((int)left) - 1;
                if (j >= r.qlen) break;  // no such token: never seen
                if (min(max(at[j], r.past), kv_index(r, j)) <= v.index - p.window) v.tree &= ~(1u << j);
            }
        }
    }
    return v;
}

__device__ __forceinline__ bool kv_sees(const KvAttendParams &p, const KvRequest &r, const KvRowView &v, int32_t key) {
    bool s = key < r.kv;
    if (p.tree) {
        const int32_t j = key - r.past;
        s = s && (j < 0 || (j < 32 && ((v.tree >> j) & 1u)));
    } else {
        s = s && key <= v.index;
    }
    return s && (p.window <= 0 || key > v.index - p.window);
}

// What parts are scaled to when the largest of their maxima is m: a part with maximum
// m_i counts 2^(m_i - base), 0 where m_i = -infinity.  Such a part saw nothing and has
// sum and output 0, or its scores are all NaN and so are they (the maximum passes over
// NaN): it is multiplied and added like any other, so that the NaN stays (0 * NaN).
__device__ __forceinline__ float kv_part_base(float m) { return m == -INFINITY ? 0.0f : m; }

// Row lr of a piece: out = acc / sum (four columns from col on) and, with the
// first of them, lse.
template <int ROWS, int D>
__device__ __forceinline__ void kv_emit(const KvAttendParams &p, const KvRequest &r, const KvPiece &c, int lr, int col,
                                        float mm, float sum, const float4 &acc) {
    const int32_t rr = c.rb * ROWS + lr, i = rr / p.group, tok = r.q0 + i, h = c.head * p.group + rr - i * p.group;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint2 b;
    b.x = pack_bf16(acc.x * inv, acc.y * inv);
    b.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(p.out + tok * p.out_stride + (int64_t)h * D + col) = b;
    if (p.lse && col == 0)
        p.lse[(int64_t)tok * (p.group * p.kv_heads) + h] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
}

// A row block whose keys several CTAs shared: where its parts are and its counter.
struct KvParts {
    int64_t first;  // row of the first CTA's first slot
    int64_t counter;
    int32_t n;  // parts, one per CTA in range order
};

template <int ROWS>
__device__ __forceinline__ KvParts kv_parts(const KvAttendParams &p, const KvWalk &w, const KvRequest &r,
                                            const KvPiece &c) {
    const int64_t s0 = w.u - c.ja;  // the row block's first unit
    const int32_t c0 = (int32_t)(((s0 + 1) * w.ctas - 1) / w.total);
    const int32_t c1 = (int32_t)(((s0 + r.ntiles) * w.ctas - 1) / w.total);
    KvParts q;
    q.first = 2 * (int64_t)c0 * ROWS;
    q.counter = c.head + (int64_t)p.kv_heads * (w.b + (int64_t)r.q0 * p.group / ROWS + c.rb);
    q.n = c1 - c0 + 1;
    return q;
}

// Called by the 128 consumer threads when they have written the CTA's part to its
// slot: true (for all of them) in the CTA that arrives last.
__device__ __forceinline__ bool kv_arrive(const KvAttendParams &p, const KvParts &q, volatile uint32_t *last_flag) {
    const bool counted = q.counter < p.n_counters;  // false only for a cu_new that is not a prefix sum
    __threadfence();
    consumers_sync();
    if (threadIdx.x == 0) {
        uint32_t is_last = 0;
        if (counted) is_last = atomicAdd(&p.counters[q.counter], 1u) == (uint32_t)(q.n - 1);
        else atomicOr(p.status, kStatusKvSizes);
        if (is_last) p.counters[q.counter] = 0;
        *last_flag = is_last;
    }
    consumers_sync();
    if (!*last_flag) return false;
    __threadfence();
    return true;
}

// The parts' joining in range order by `threads` threads, P parts at a time: a
// thread has the loads of 2 P parts in flight (P: what the kernel has registers
// for) and raises its maximum once per P.
template <int ROWS, int D, int P>
__device__ __forceinline__ void kv_join(const KvAttendParams &p, const KvParts &q, const KvRequest &r, const KvPiece &c,
                                        int32_t nrows, int tid, int threads) {
    constexpr int U = 2;
    const int items = nrows * (D / 4);
    for (int i0 = tid; i0 < items; i0 += U * threads) {
        float4 acc[U];
        float mm[U], sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f), mm[u] = -INFINITY, sum[u] = 0.0f;
        for (int32_t k0 = 0; k0 < q.n; k0 += P) {
            float4 y[U][P];
            float2 s[U][P];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = min(i0 + u * threads, items - 1), lr = i / (D / 4), v4 = i % (D / 4);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    // the first CTA's part is in its second slot, every other one's
                    // in its first
                    const int32_t kk = min(k0 + k, q.n - 1);
                    const int64_t at = q.first + (2 * kk + (kk == 0)) * ROWS + lr;
                    s[u][k] = __ldcg(&p.part_ml[at]);
                    y[u][k] = __ldcg(reinterpret_cast<const float4 *>(p.part + at * D) + v4);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float mn = mm[u];
#pragma unroll
                for (int k = 0; k < P; ++k) mn = fmaxf(mn, s[u][k].x);
                const float base = kv_part_base(mn), f0 = ex2(mm[u] - base);
                mm[u] = mn;
                sum[u] *= f0;
                acc[u].x *= f0, acc[u].y *= f0, acc[u].z *= f0, acc[u].w *= f0;
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    if (k0 + k >= q.n) continue;
                    const float g = ex2(s[u][k].x - base);
                    const float4 v = y[u][k];
                    sum[u] = fmaf(g, s[u][k].y, sum[u]);
                    acc[u].x = fmaf(g, v.x, acc[u].x), acc[u].y = fmaf(g, v.y, acc[u].y);
                    acc[u].z = fmaf(g, v.z, acc[u].z), acc[u].w = fmaf(g, v.w, acc[u].w);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * threads;
            if (i < items) kv_emit<ROWS, D>(p, r, c, i / (D / 4), (i % (D / 4)) * 4, mm[u], sum[u], acc[u]);
        }
    }
}

// A request's page numbers from one of its entries on, 64 of them in a warp's
// registers (entry base + lane, base + 32 + lane): the load of a tile's pages is
// then far behind its use.  Every lane takes part in every call.
struct KvPageWindow {
    const int32_t *row;
    int32_t base, last, cur, next;

    __device__ __forceinline__ int32_t load(int32_t e) const { return e <= last ? row[e] : -1; }
    // entries `first` to `end` - 1 will be asked for, in order
    __device__ __forceinline__ void start(const int32_t *table_row, int32_t first, int32_t end) {
        row = table_row;
        base = first;
        last = end - 1;
        cur = load(base + (int)(threadIdx.x & 31));
        next = load(base + 32 + (int)(threadIdx.x & 31));
    }
    // page of entry e (of each lane's own; all within 32 entries from `low`, the
    // smallest, which never falls)
    __device__ __forceinline__ int32_t get(int32_t low, int32_t e) {
        while (low >= base + 32) {
            base += 32;
            cur = next;
            next = load(base + 32 + (int)(threadIdx.x & 31));
        }
        const int32_t at = e - base;
        const int32_t a = __shfl_sync(~0u, cur, at & 31), b = __shfl_sync(~0u, next, at & 31);
        return at < 32 ? a : b;
    }
};

template <int D, bool Q8, int WK, int WR, int NT>
__global__ void __launch_bounds__(kAttendThreads, attend_ctas<D, Q8, NT>()) w12_kv_attend_kernel(const KvAttendParams p,
                                                                       const __grid_constant__ CUtensorMap tm_k,
                                                                       const __grid_constant__ CUtensorMap tm_v) {
    using C = AttendCfg<D, Q8, WK, WR, NT>;
    constexpr int ROWS = C::kRows, KS = D / 16, TILE = C::kTile, PAIR = C::kPair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *merge = reinterpret_cast<float *>(smem + C::kOffMerge);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBars);
    uint64_t *empty = full + C::kStages;
    uint32_t *present = reinterpret_cast<uint32_t *>(empty + C::kStages);
    volatile uint32_t *last_flag = present + C::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 128) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();  // after the wait: w12_kv_join_kernel relies on it
    const uint64_t deadline = globaltimer_ns() + p.timeout_ns;

    KvWalk w;
    KvRequest r;
    if (!kv_walk_init<ROWS, TILE>(p, w, r)) return;  // the same for the whole CTA

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        uint32_t it = 0;
        bool ok = true;
        while (ok && w.u < w.end) {
            const KvPiece c = kv_piece(w, r);
            KvPageWindow pages;
            pages.start(p.tables + (int64_t)w.b * p.table_stride, (r.tile0 + c.ja) * TILE / p.page_size,
                        kv_entries(p, r));
            for (int j = c.ja; ok && j < c.jb; ++j, ++it) {
                const uint32_t stage = it % C::kStages, round = it / C::kStages;
                // lane s deals with slice s
                const int32_t t0 = (r.tile0 + j) * TILE, kb = t0 + (lane % C::kSlices) * kAttendSlice;
                const bool want = lane < C::kSlices && kb < r.kv && kb + kAttendSlice > r.first;
                const int32_t e = kb / p.page_size, off = kb - e * p.page_size;
                const int32_t found = pages.get(t0 / p.page_size, e), page = want ? found : -1;
                if (round > 0) ok = mbar_wait(&empty[stage], (round - 1) & 1, deadline);
                ok = __shfl_sync(~0u, ok, 0);
                if (!ok) break;
                const bool here = page >= 0 && page < p.num_pages;
                const uint32_t mask = __ballot_sync(~0u, here);
                if (lane == 0) {
                    present[stage] = mask;
                    mbar_arrive_expect_tx(&full[stage],
                                          (uint32_t)__popc(mask) * (2 * C::kSliceBytes + (Q8 ? 128 : 0)));
                }
                __syncwarp();
                if (here) {
                    const uint32_t dst = smem_u32(smem + stage * C::kStageBytes + lane * C::kSliceBytes);
                    const uint32_t bar = smem_u32(&full[stage]);
                    tma_load_5d(dst, &tm_k, off, c.head, page, bar);
                    tma_load_5d(dst + C::kTileBytes, &tm_v, off, c.head, page, bar);
                    if (Q8)
                        bulk_g2s(smem + C::kOffScales + stage * C::kScaleBytes + lane * 128,
                                 p.scales + (((int64_t)page * p.kv_heads + c.head) * p.page_size + off) * 2, 128,
                                 &full[stage]);
                }
            }
            if (ok) kv_advance<ROWS, TILE>(p, w, r, c.jb - c.ja);
        }
        if (!ok) {
            // no copy may still be in flight when the CTA ends
            if (lane == 0) {
                atomicOr(p.status, 8u);
                const uint64_t late = globaltimer_ns() + p.timeout_ns;
                for (uint32_t k = it > C::kStages ? it - C::kStages : 0; k < it; ++k)
                    if (!mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1, late)) break;
            }
            __syncwarp();
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int wk = warp % WK, wr = warp / WK;
    const int g = lane >> 2, t = lane & 3;
    uint32_t it = 0;
    bool ok = true;
    while (w.u < w.end) {
        const KvPiece c = kv_piece(w, r);
        const int32_t nrows = min((int64_t)ROWS, (int64_t)r.qlen * p.group - (int64_t)c.rb * ROWS);
        const int32_t row0 = c.rb * ROWS;
        // every row sees the keys from low on and before lim
        const int32_t lim = min(r.kv, p.tree ? r.past : r.past + 1);
        const int32_t low = p.window > 0 ? (int32_t)max((int64_t)r.past + r.qlen - p.window, (int64_t)0) : 0;

        // q as the mma's B operand: row (n) g of each 8-row tile, columns (k) of
        // step ks in the order the A operand's layout wants
        uint32_t qf[NT][KS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int lr = (wr * NT + nt) * 8 + g;
            const int32_t rr = row0 + lr;
            const int32_t i = rr / p.group;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                p.q + (int64_t)(r.q0 + (lr < nrows ? i : 0)) * p.q_stride +
                (int64_t)(c.head * p.group + (lr < nrows ? rr - i * p.group : 0)) * D);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a = 0, b = 0;
                if (lr < nrows) {
                    if (Q8) {
                        // columns 4t..4t+3 of the step; pairs (0, 2) and (1, 3), as q8_to_bf16 gives them
                        const uint32_t x = src[ks * 8 + 2 * t], y = src[ks * 8 + 2 * t + 1];
                        a = prmt(x, y, 0x5410u);
                        b = prmt(x, y, 0x7632u);
                    } else {
                        a = src[ks * 8 + t];
                        b = src[ks * 8 + 4 + t];
                    }
                }
                qf[nt][ks][0] = a;
                qf[nt][ks][1] = b;
            }
        }
        float o[KS][NT][4] = {};
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.0f;

        for (int j = c.ja; j < c.jb; ++j, ++it) {
            const uint32_t stage = it % C::kStages, round = it / C::kStages;
            // after a timeout the walk goes on without waiting (its reads stay
            // inside shared memory) so that every barrier below is reached
            if (ok && !mbar_wait(&full[stage], round & 1, deadline)) {
                ok = false;
                if (lane == 0) atomicOr(p.status, 8u);
            }
            __syncwarp();
            const uint32_t mask = present[stage];
            const int32_t tb = (r.tile0 + j) * TILE;
            const uint32_t kbase = smem_u32(smem + stage * C::kStageBytes), vbase = kbase + C::kTileBytes;
#pragma unroll 1
            for (int s0 = wk; s0 < C::kSlices; s0 += PAIR * WK) {
                // slices s0 (and s0 + WK)
                const uint32_t both = PAIR == 2 ? (mask >> s0 & 1u) | (mask >> (s0 + WK) & 1u) << 1 : mask >> s0 & 1u;
                if (both == 0) continue;
                // scores of 16 keys (rows g, g + 8) and NT * 8 rows (columns 2t, 2t + 1)
                float x[PAIR][NT][4] = {};
                float vs[PAIR][2];
                {
                    const int krow = ((lane >> 3) & 1) * 8 + (lane & 7);
                    constexpr int CH = C::kRowBytes / 16;  // 16-byte chunks of a box row
                    const int sw = CH == 8 ? krow & 7 : (krow >> 1) & 3;
                    const uint32_t row = kbase + s0 * C::kSliceBytes + krow * C::kRowBytes;
                    constexpr int STEP = Q8 ? 2 : 1;
#pragma unroll
                    for (int ks = 0; ks < KS; ks += STEP) {
                        const int chunk = Q8 ? ks + (lane >> 4) : 2 * ks + (lane >> 4);
                        const uint32_t at = (chunk / CH) * (16 * C::kRowBytes) + (((chunk % CH) ^ sw) << 4);
#pragma unroll
                        for (int u = 0; u < PAIR; ++u) {
                            uint32_t w4[4];
                            ldsm4(row + u * WK * C::kSliceBytes + at, w4);
                            if (!Q8) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_bf16(x[u][nt], w4, qf[nt][ks][0], qf[nt][ks][1]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    uint32_t a[4];
                                    q8_to_bf16(w4[2 * e], a[0], a[2]);
                                    q8_to_bf16(w4[2 * e + 1], a[1], a[3]);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        mma_bf16(x[u][nt], a, qf[nt][ks + e][0], qf[nt][ks + e][1]);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < PAIR; ++u) {
                    float sc0 = p.scale_log2, sc1 = p.scale_log2;
                    vs[u][0] = vs[u][1] = 1.0f;
                    if (Q8) {
                        const float2 *sc =
                            reinterpret_cast<const float2 *>(smem + C::kOffScales + stage * C::kScaleBytes) +
                            (s0 + u * WK) * 16;
                        const float2 a = sc[g], b = sc[g + 8];
                        sc0 *= a.x, sc1 *= b.x, vs[u][0] = a.y, vs[u][1] = b.y;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        x[u][nt][0] *= sc0, x[u][nt][1] *= sc0, x[u][nt][2] *= sc1, x[u][nt][3] *= sc1;
                }

                // keys that some row does not see, or that are not there
                const int32_t kb = tb + s0 * kAttendSlice;
                constexpr int SPAN = ((PAIR - 1) * WK + 1) * kAttendSlice;
                const bool edge = kb > lim - SPAN || kb < low || both != (1u << PAIR) - 1u;
                uint32_t seen = ~0u;  // bit 4 (u NT + nt) + c: score c of tile nt of slice u
                if (edge) {
                    seen = 0;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int32_t lr = (wr * NT + nt) * 8 + 2 * t + e;
                            const int32_t i = (row0 + min(lr, nrows - 1)) / p.group;
                            const KvRowView v = p.positions ? kv_row_view<true>(p, r, i) : kv_row_view<false>(p, r, i);
#pragma unroll
                            for (int u = 0; u < PAIR; ++u) {
                                const int32_t key = kb + u * WK * kAttendSlice + g;
                                if (!((both >> u) & 1u)) continue;
                                if (kv_sees(p, r, v, key)) seen |= 1u << (4 * (u * NT + nt) + e);
                                if (kv_sees(p, r, v, key + 8)) seen |= 1u << (4 * (u * NT + nt) + e + 2);
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < PAIR; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!((seen >> (4 * (u * NT + nt) + e)) & 1u)) x[u][nt][e] = -INFINITY;
                }

                // running maximum
                bool raise = false;
                float top[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[nt][e] = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
                        if (PAIR == 2)
                            top[nt][e] = fmaxf(fmaxf(top[nt][e], x[PAIR - 1][nt][e]), x[PAIR - 1][nt][e + 2]);
                        raise |= top[nt][e] > m[nt][e] + kAttendLazy;
                    }
                if (__any_sync(~0u, raise)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = top[nt][e];
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
                            v = fmaxf(v, m[nt][e]);
                            al[e] = v == -INFINITY ? 1.0f : ex2(m[nt][e] - v);
                            m[nt][e] = v;
                            l[nt][e] *= al[e];
                        }
#pragma unroll
                        for (int mt = 0; mt < KS; ++mt)
                            o[mt][nt][0] *= al[0], o[mt][nt][1] *= al[1], o[mt][nt][2] *= al[0], o[mt][nt][3] *= al[1];
                    }
                }
                // probabilities; l sums them in fp32, the tensor cores get them (with
                // Q8 times the value's scale) rounded to BF16: at most 2^-8 of each
                // weight, as the rounding of the output
                uint32_t pb[PAIR][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
                    const float m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
                    for (int u = 0; u < PAIR; ++u) {
                        float p0 = ex2(x[u][nt][0] - m0), p1 = ex2(x[u][nt][1] - m1);
                        float p2 = ex2(x[u][nt][2] - m0), p3 = ex2(x[u][nt][3] - m1);
                        l[nt][0] += p0 + p2;
                        l[nt][1] += p1 + p3;
                        if (Q8) {
                            p0 *= vs[u][0], p1 *= vs[u][0], p2 *= vs[u][1], p3 *= vs[u][1];
                            if (edge) {  // an unseen key's scale may be anything
                                const uint32_t sn = seen >> (4 * (u * NT + nt));
                                p0 = sn & 1u ? p0 : 0.0f, p1 = sn & 2u ? p1 : 0.0f;
                                p2 = sn & 4u ? p2 : 0.0f, p3 = sn & 8u ? p3 : 0.0f;
                            }
                        }
                        pb[u][nt][0] = movmatrix(pack_bf16(p0, p1));
                        pb[u][nt][1] = movmatrix(pack_bf16(p2, p3));
                    }
                }

                // o (columns of the head x rows) += v^T p^T
                const uint32_t vs0 = vbase + s0 * C::kSliceBytes;
                if (!Q8) {
                    const int vrow = (lane >> 4) * 8 + (lane & 7);
                    constexpr int CH = C::kRowBytes / 16;
                    auto v_at = [&](int u, int mt) {
                        const int chunk = 2 * mt + ((lane >> 3) & 1);
                        return vs0 + u * WK * C::kSliceBytes + (chunk / CH) * (16 * C::kRowBytes) +
                               vrow * C::kRowBytes + (((chunk % CH) ^ (vrow & 7)) << 4);
                    };
                    bool odd = false;  // a value that is not finite behind a key that some row does not see
                    uint32_t keep[PAIR][2];
#pragma unroll
                    for (int u = 0; u < PAIR; ++u) keep[u][0] = keep[u][1] = ~0u;
                    if (edge) {
#pragma unroll
                        for (int u = 0; u < PAIR; ++u) {
                            // keys behind the request's last one, and missing slices, hold
                            // anything: zero
                            const int32_t nv = (both >> u) & 1u ? r.kv - (kb + u * WK * kAttendSlice) : 0;
                            keep[u][0] = (2 * t < nv ? 0xFFFFu : 0u) | (2 * t + 1 < nv ? 0xFFFF0000u : 0u);
                            keep[u][1] = (2 * t + 8 < nv ? 0xFFFFu : 0u) | (2 * t + 9 < nv ? 0xFFFF0000u : 0u);
#pragma unroll 4
                            for (int mt = 0; mt < KS; ++mt) {
                                uint32_t a[4];
                                ldsm4_trans(v_at(u, mt), a);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    a[e] &= keep[u][e / 2];
                                    odd |= (a[e] & 0x7F80u) == 0x7F80u || (a[e] & 0x7F800000u) == 0x7F800000u;
                                }
                            }
                        }
                        odd = __any_sync(~0u, odd);
                    }
                    if (!odd) {
#pragma unroll
                        for (int mt = 0; mt < KS; ++mt) {
#pragma unroll
                            for (int u = 0; u < PAIR; ++u) {
                                uint32_t a[4];
                                ldsm4_trans(v_at(u, mt), a);
                                a[0] &= keep[u][0], a[1] &= keep[u][0], a[2] &= keep[u][1], a[3] &= keep[u][1];
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[mt][nt], a, pb[u][nt][0], pb[u][nt][1]);
                            }
                        }
                    } else {
                        // 0 * NaN must not reach a row that does not see the key: one
                        // row at a time, with the values of its unseen keys zeroed
#pragma unroll
                        for (int u = 0; u < PAIR; ++u) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t bal[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    bal[e] = __ballot_sync(~0u, (seen >> (4 * (u * NT + nt) + e)) & 1u);
#pragma unroll 1
                                for (int n = 0; n < 8; ++n) {
                                    // ballot bit 4 g + t holds key g (or g + 8) of row 2t + e
                                    const uint32_t lo = (n & 1 ? bal[1] : bal[0]) >> (n >> 1);
                                    const uint32_t hi = (n & 1 ? bal[3] : bal[2]) >> (n >> 1);
                                    uint32_t z0 = 0, z1 = 0;
                                    if ((lo >> (8 * t)) & 1u) z0 |= 0xFFFFu;
                                    if ((lo >> (8 * t + 4)) & 1u) z0 |= 0xFFFF0000u;
                                    if ((hi >> (8 * t)) & 1u) z1 |= 0xFFFFu;
                                    if ((hi >> (8 * t + 4)) & 1u) z1 |= 0xFFFF0000u;
                                    const uint32_t b0 = g == n ? pb[u][nt][0] : 0u, b1 = g == n ? pb[u][nt][1] : 0u;
#pragma unroll
                                    for (int mt = 0; mt < KS; ++mt) {
                                        uint32_t a[4];
                                        ldsm4_trans(v_at(u, mt), a);
                                        a[0] &= z0, a[1] &= z0, a[2] &= z1, a[3] &= z1;
                                        float y[4] = {};
                                        mma_bf16(y, a, b0, b1);
                                        // the other rows' sums are 0 * value here: only
                                        // row n's count
                                        if (2 * t == (n & ~1)) {
                                            if (n & 1) o[mt][nt][1] += y[1], o[mt][nt][3] += y[3];
                                            else o[mt][nt][0] += y[0], o[mt][nt][2] += y[2];
                                        }
                                    }
                                }
                            }
                        }
                    }
                } else {
                    constexpr int CH = C::kRowBytes / 16;
                    const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7);
                    const int sw = CH == 8 ? vrow & 7 : (vrow >> 1) & 3;
#pragma unroll
                    for (int m2 = 0; m2 < KS; m2 += 2) {
                        const int chunk = m2 + (lane >> 4);
                        const uint32_t at = vs0 + (chunk / CH) * (16 * C::kRowBytes) + vrow * C::kRowBytes +
                                            (((chunk % CH) ^ sw) << 4);
#pragma unroll
                        for (int u = 0; u < PAIR; ++u) {
                            uint32_t w4[4];
                            ldsm4_trans(at + u * WK * C::kSliceBytes, w4);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                // rows g of the tile are the even columns 2g, rows g + 8 the odd ones
                                uint32_t a[4];
                                q8_to_bf16(w4[2 * e], a[0], a[1]);
                                q8_to_bf16(w4[2 * e + 1], a[2], a[3]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[m2 + e][nt], a, pb[u][nt][0], pb[u][nt][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
        }

        // ------------------------------------------------------------ join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(~0u, v, 4);
                v += __shfl_xor_sync(~0u, v, 8);
                v += __shfl_xor_sync(~0u, v, 16);
                if (g == 0) ml[wk * ROWS + (wr * NT + nt) * 8 + 2 * t + e] = make_float2(m[nt][e], v);
            }
        const bool whole = c.ja == 0 && c.jb == r.ntiles;
        const int32_t slot = 2 * (int32_t)blockIdx.x + (c.ja > 0 ? 0 : 1);
#pragma unroll
        for (int dc = 0; dc < D / 64; ++dc) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float *dst = merge + (wk * ROWS + (wr * NT + nt) * 8 + 2 * t) * C::kMergeStride + mt * 16;
                    const int d0 = Q8 ? 2 * g : g, d1 = Q8 ? 2 * g + 1 : g + 8;
                    dst[d0] = o[dc * 4 + mt][nt][0];
                    dst[d0 + C::kMergeStride] = o[dc * 4 + mt][nt][1];
                    dst[d1] = o[dc * 4 + mt][nt][2];
                    dst[d1 + C::kMergeStride] = o[dc * 4 + mt][nt][3];
                }
            }
            consumers_sync();
            for (int i = threadIdx.x; i < nrows * 16; i += 128) {
                const int lr = i >> 4, v4 = i & 15;
                float mm = -INFINITY;
#pragma unroll
                for (int k = 0; k < WK; ++k) mm = fmaxf(mm, ml[k * ROWS + lr].x);
                const float base = kv_part_base(mm);
                float sum = 0.0f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float2 s = ml[k * ROWS + lr];
                    const float f = ex2(s.x - base);
                    const float4 y =
                        *reinterpret_cast<const float4 *>(merge + (k * ROWS + lr) * C::kMergeStride + v4 * 4);
                    sum += f * s.y;
                    acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
                }
                if (whole) {
                    kv_emit<ROWS, D>(p, r, c, lr, dc * 64 + v4 * 4, mm, sum, acc);
                } else {
                    *reinterpret_cast<float4 *>(p.part + ((int64_t)slot * ROWS + lr) * D + dc * 64 + v4 * 4) = acc;
                    if (dc == 0 && v4 == 0) p.part_ml[(int64_t)slot * ROWS + lr] = make_float2(mm, sum);
                }
            }
            consumers_sync();
        }

        if (!whole && !p.join_later) {
            const KvParts q = kv_parts<ROWS>(p, w, r, c);
            if (kv_arrive(p, q, last_flag))
                kv_join<ROWS, D, C::kCtas < 3 ? 8 : 4>(p, q, r, c, nrows, (int)threadIdx.x, 128);
        }
        kv_advance<ROWS, TILE>(p, w, r, c.jb - c.ja);
    }
    if (!ok && warp == 0 && lane == 0) {
        // a wait ran out: no copy may still be in flight when the CTA ends
        const uint64_t late = globaltimer_ns() + p.timeout_ns;
        for (uint32_t k = it > C::kStages ? it - C::kStages : 0; k < it; ++k)
            if (!mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1, late)) break;
    }
}

// Joins the parts of the output rows (token and head, heads fastest) of a launch with
// ROWS-row blocks and `grid` CTAs; a row that one CTA had whole is finished already.
// WPR warps share a row: they take its parts in turn and meet in shared memory,
// both in a fixed order.
constexpr int kJoinThreads = 256;

template <int D, int ROWS, int TILE, int WPR>
__global__ void __launch_bounds__(kJoinThreads) w12_kv_join_kernel(const KvAttendParams p, int grid) {
    constexpr int W = kJoinThreads / 32, V = D / 32;  // columns of a lane
    __shared__ float s_acc[WPR > 1 ? W : 1][D];
    __shared__ float2 s_ml[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = p.group * p.kv_heads;
    const int64_t out_row = (int64_t)blockIdx.x * (W / WPR) + warp / WPR;
    const int32_t tok = (int32_t)(out_row / heads), h = (int32_t)(out_row - (int64_t)tok * heads);
    // Lengths and offsets come from before the attention kernel, which lets this one
    // start only when it has itself seen all that is before it.  This kernel has not
    // waited yet, though: the fence keeps its loads from lines that the SM's L1 has had
    // since before they were written.  (With loads from L2 instead, the sum over 128
    // requests in every row's warp took 117 us to 199, three tokens on windows.)
    __threadfence();
    const KvSums sums = kv_sum_units<ROWS, TILE>(p);
    const int64_t total = sums.total;
    // the token's request: the block that has it, then the request in it
    int64_t start = -1;
    KvRequest r;
    int32_t b = 0;
    {
        const int first = lane * sums.per, end = (int)min((int64_t)first + sums.per, (int64_t)p.requests);
        const bool mine = first < p.requests && tok >= min(max(p.cu_new[first], 0), p.tokens) &&
                          tok < min(max(p.cu_new[end], 0), p.tokens);
        const uint32_t hit = __ballot_sync(~0u, mine);
        if (hit) {
            const int src = __ffs(hit) - 1;
            int64_t at = __shfl_sync(~0u, sums.before, src);
            const int32_t last = (int32_t)min((int64_t)(src + 1) * sums.per, (int64_t)p.requests);
            for (b = src * sums.per; b < last; ++b) {
                r = kv_request<ROWS, TILE>(p, b);
                if (tok >= r.q0 && tok < r.q0 + r.qlen) {
                    start = at;
                    break;
                }
                at += r.units;
            }
        }
    }
    KvParts q;
    q.n = 0;
    int32_t lr = 0;
    if (start >= 0) {  // the same for the whole warp, and for all warps of a row
        const int32_t rr = (tok - r.q0) * p.group + h % p.group;
        KvPiece c;
        KvWalk w;
        c.head = h / p.group;
        c.rb = rr / ROWS;
        c.ja = 0;
        w.total = total;
        w.ctas = (int32_t)min((int64_t)grid, total);
        w.b = b;
        w.u = start + ((int64_t)c.head * r.rblocks + c.rb) * r.ntiles;
        q = kv_parts<ROWS>(p, w, r, c);
        lr = rr - c.rb * ROWS;
    }
    pdl_launch_dependents();
    pdl_wait();
    if (WPR == 1 && q.n <= 1) return;
    float acc[V] = {}, mm = -INFINITY, sum = 0.0f;
    constexpr int U = V == 8 || WPR > 1 ? 4 : 8;  // parts whose loads are in flight
    for (int32_t k0 = warp % WPR; q.n > 1 && k0 < q.n; k0 += U * WPR) {
        float y[U][V];
        float2 s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t k = min(k0 + u * WPR, q.n - 1);
            const int64_t at = q.first + (2 * k + (k == 0)) * ROWS + lr;
            s[u] = __ldcg(&p.part_ml[at]);
            const float *src = p.part + at * D;
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
            if (k0 + u * WPR < q.n) {
                const float g = ex2(s[u].x - base);
                sum = fmaf(g, s[u].y, sum);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(g, y[u][e], acc[e]);
            }
        }
    }
    if constexpr (WPR > 1) {
        static_assert(WPR == W, "one row per CTA");
        if (lane == 0) s_ml[warp] = make_float2(mm, sum);
#pragma unroll
        for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
        __syncthreads();
        if (warp > 0 || q.n <= 1) return;
        mm = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) mm = fmaxf(mm, s_ml[k].x);
        const float base = kv_part_base(mm);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float f = ex2(s_ml[k].x - base);
            sum += f * s_ml[k].y;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += f * s_acc[k][lane * V + e];
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + tok * p.out_stride + (int64_t)h * D) + lane * (V / 2);
#pragma unroll
    for (int e = 0; e < V; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[(int64_t)tok * heads + h] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
}

}  // namespace dev
}  // namespace w12
