// Paged-cache attention for many rows per key head, on tcgen05 (the mathematics,
// the work split and the joining are those of kv_attend.cuh).
//
// Where several drafted tokens meet a wide group (rows = new tokens x query heads
// per key head), the warp-level products of kv_attend.cuh become the bound: every
// warp reads (and, of an 8-bit cache, converts) the same keys for its own few rows.
// Here 128 rows are the M of one tcgen05.mma: a tile's keys are read from shared
// memory once for all rows.  Per 64-key tile
//   S [128 x 64]  = Q (TMEM or shared)   x K^T (shared, K-major)
//   P             = 2^(S - m), 16 rows of a warp at a time, BF16, over S
//   O [128 x D] += P (TMEM)              x V (shared, MN-major)
// S has two or four buffers, so the tensor cores make the next tiles' scores while
// the softmax warps work on this one's.  O stays in TMEM for a whole piece; it is
// rescaled only when a row's maximum rises by more than 2^8.
//
// Two warps fill the K and V rings by TMA.  A Q8 cache's rows arrive as bytes in
// rings of their own and four or eight warps turn them into BF16 operands;
// the order of the columns within every four (0, 2, 1, 3) is what comes out of the
// byte pairs cheapest, and Q's columns and O's follow it.
//
// What a CTA has of a row block that others share goes to the workspace and is
// joined by w12_kv_join_kernel: 128 rows of parts are too much for one CTA.
//
// For head_dim 64, and 128 with a Q8 cache, a CTA takes half of TMEM and less than half
// of the shared memory, so two share an SM and fill each other's waits.
//
// Measured, 16-token trees over eight requests of 16000 tokens, 48 heads over 8 of
// 128 (96 rows): BF16 96 us, 5.6 TB/s; Q8 117 us.  HBM would take 81 and 42 us, the
// products 22.  Taking the softmax's or the conversion's instructions out shortens the
// Q8 call by 7 % each, both by 26 %: it is bounded by the chain of bytes, operand,
// scores, weights and product, of which two CTAs per SM overlap two.  30 rows of 64
// requests of 8000: BF16 320 us, 6.6 TB/s, Q8 332.  72 rows of 256 columns, two of
// 100001: BF16 128 us, Q8 107.
#pragma once

#include "kv_attend.cuh"

namespace w12 {
namespace dev {

constexpr int kTcRows = 128;
constexpr int kTcInfo = 16;  // ring of per-tile facts (present slices, scales)

// A softmax warp's place: kept in shared memory, so that the loop over a piece's
// tiles has the registers.
struct TcPlace {
    KvWalk w;
    KvRequest r;
    KvPiece c;
};

template <int D, bool Q8>
struct AttendTcCfg {
    // Q is the scores' A operand: from TMEM, written there once per piece, where there
    // are columns for it beside O and the scores; else from shared memory, where every
    // tile's products read it again (128 columns, BF16: 96 us from TMEM, 102 from shared
    // memory, for the trees above) and where it takes the room of ring slots.  Only the
    // 8-bit cache of 128 columns has no columns left: its two CTAs per SM are worth more
    // (117 us; one CTA with Q in TMEM 116, but 404 against 365 at 64000 tokens).
    static constexpr bool kQTmem = !Q8 || D != 128;
    // One CTA per SM or two (with half of TMEM each).
    static constexpr bool kOne = D == 256 || (D == 128 && kQTmem);
    // Score buffers, and how many tiles the scores are made ahead of the products.
    static constexpr int kS = D == 128 && kQTmem ? 4 : 2, kAheadS = kS / 2;
    // Softmax warps, then two loaders, the MMA warp (and one that idles), the converters
    // in groups of four.  Where one CTA has the SM, eight softmax warps (16 rows each)
    // shorten the way from scores to weights; where two share it, four (32 rows each, 16
    // at a time) fill it as well and leave the registers.  72 rows of 256 columns, two
    // requests of 100001: 127 us with eight, 133 with four; 96 rows of 128, the 8-bit
    // trees: 122 and 116.  Keys and values have a group of converters each where there
    // are threads for it (256 columns, 8-bit: 107 us, 140 with one group and one operand
    // buffer; 128: 376 against 365 with one, at 64000 tokens).
    static constexpr int kSoft = kOne ? 8 : 4;
    static constexpr int kGroups = !Q8 ? 0 : kOne ? 2 : 1;
    static constexpr int kThreads = 32 * (kSoft + (Q8 ? 4 + 4 * kGroups : kOne ? 4 : 3));
    // Registers per thread at launch, then of the softmax warps and of the others: the
    // softmax warps take what the others give up (0: no exchange).
    static constexpr int kRegs = !Q8 ? 0 : kOne ? 96 : 80;
    static constexpr int kSoftRegs = kOne ? 144 : 128;
    static constexpr int kRestRegs = kOne ? 64 : 56;
    static_assert(kRegs == 0 || 32 * kSoft * kSoftRegs + (kThreads - 32 * kSoft) * kRestRegs == kThreads * kRegs,
                  "a split with more than the launch has would wait for ever");
    static constexpr int kQBytes = kQTmem ? 0 : kTcRows * D * 2;
    static constexpr int kTileBytes = kAttendTile * D * 2;  // K or V of a tile as BF16 operand
    static constexpr int kRawBytes = kAttendTile * D;       // K or V of a tile as bytes (Q8)
    static constexpr int kBlocks = D / 64;                  // 128-byte column blocks of an operand row
    // operand rings (filled by TMA, or by the converting warps) and byte rings
    static constexpr int kOps = Q8 ? (D == 256 ? 2 : 1) : D == 64 ? 5 : D == 128 ? 6 : 3;
    static constexpr int kRaws = Q8 ? (D == 64 ? 6 : 2) : 0;
    // A slot of the ring of facts is written again after the softmax of its tile: the
    // loader is at most the byte ring, the operand ring and the score buffers ahead.
    static_assert(kRaws + kOps + kS <= kTcInfo, "the ring of facts");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQBytes;
    static constexpr int kOffV = kOffK + kOps * kTileBytes;
    static constexpr int kOffRaw = kOffV + kOps * kTileBytes;  // K, V of stage 0, K, V of stage 1, ...
    static constexpr int kOffRawScale = kOffRaw + kRaws * 2 * kRawBytes;
    static constexpr int kInfoBytes = 528;  // 64 key scales, 64 value scales, the largest key scale
    static constexpr int kOffScale = kOffRawScale + kRaws * 512;  // [kTcInfo][kInfoBytes] (Q8)
    static constexpr int kOffBars = kOffScale + (Q8 ? kTcInfo * kInfoBytes : 0);
    static constexpr int kBars = 4 * kOps + 4 * kRaws + 3 * kS + 3;
    static constexpr int kOffInfo = kOffBars + 8 * kBars;
    static constexpr int kOffStats = kOffInfo + 4 * kTcInfo + 32;  // (max, sum) of the 128 rows
    static constexpr int kOffPlaces = kOffStats + 8 * kTcRows;
    static constexpr int kSmemBytes = kOffPlaces + kSoft * (int)sizeof(TcPlace) + 1024;  // 1024: alignment
    // O from column 0, kS score buffers of 64 columns, Q
    static constexpr int kTmemCols = kOne ? 512 : 256, kSCol = D, kQCol = kSCol + 64 * kS;
    static_assert(kQCol + (kQTmem ? D / 2 : 0) <= kTmemCols, "TMEM");
};

// Warp-collective 32-column TMEM load (lane i <- TMEM lane base + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// 4-D tiled copy global -> shared: column, token in page, head, page.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint64_t low_bits(int64_t n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Bit k: the row sees key kb + k of the tile (kv_sees and the present slices).
__device__ __forceinline__ uint64_t kv_seen64(const KvAttendParams &p, int32_t kv, int32_t past, const KvRowView &v,
                                              int32_t kb, uint32_t present) {
    uint64_t m = low_bits((int64_t)kv - kb);
    if (p.tree) {
        const int64_t sh = (int64_t)past - kb;
        const uint64_t drawn =
            sh >= 64 ? 0 : sh >= 0 ? (uint64_t)v.tree << sh : sh > -32 ? (uint64_t)(v.tree >> -sh) : 0;
        m &= low_bits(sh) | drawn;
    } else {
        m &= low_bits((int64_t)v.index + 1 - kb);
    }
    if (p.window > 0) m &= ~low_bits((int64_t)v.index - p.window + 1 - kb);
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (!((present >> s) & 1u)) m &= ~(0xFFFFull << (16 * s));
    return m;
}

// True in one lane of the warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}

// One pipeline barrier's phase by use count.  The parity tells a phase only from
// its neighbours: who waits for use n knows that use n - 1 is over, and use n + 1
// cannot be over.  So what is waited for every tile (scores, probabilities,
// products) has a barrier per score buffer: the scores of tile g are made after the
// product of tile g - kS.
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t use, uint64_t deadline) {
    return mbar_wait(bar, use & 1u, deadline);
}

// 16 TMEM lanes (rows) at a time, spread as a product's accumulator is: lane 4 g + t
// has rows g and g + 8, of every eight 32-bit columns 2 t and 2 t + 1 (of row g first).
__device__ __forceinline__ void tmem_ld16x64(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
                 "}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
                   "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
                   "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
                   "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
                 "}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
                   "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16x32(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {"
                 "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
                 "};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
// The same rows, of every four columns t (of row g first): pairs of BF16 columns.
__device__ __forceinline__ void tmem_st16x32p(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {"
                 "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
                 "};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// The softmax of 16 rows' 64 scores x, which become BF16 weights at ts, over them.
// A thread has 16 keys of two rows (see tmem_ld16x64), so it needs the scales of 16
// keys and not of 64: with a row per thread their broadcast reads from shared memory
// alone took a fifth of its bandwidth.  sc (Q8): the tile's 64 key scales with the
// softmax scale in them, its 64 value scales and the largest key scale, from the
// thread's first key on; scale: the softmax scale, not negative (BF16).  m, l: the
// rows' running maximum (the same in the four threads of a row) and the thread's share
// of their sum.  EDGE: only the keys of `seen`, shifted so that bit 8 j + e is the
// thread's key 2 j + e.  rescale(a0, a1) multiplies the rows' output so far.
template <bool Q8, bool EDGE, class Rescale>
__device__ __forceinline__ void tc_softmax(uint32_t ts, const uint32_t (&x)[32], const float *sc, float scale,
                                           float (&m)[2], float (&l)[2], uint64_t seen0, uint64_t seen1,
                                           Rescale rescale) {
    const auto pair = [&](int j, int row) {
        return make_f2(__uint_as_float(x[4 * j + 2 * row]), __uint_as_float(x[4 * j + 2 * row + 1]));
    };
    const auto scale_of = [&](int j) {  // of the thread's keys 2 j and 2 j + 1, the softmax scale in it
        if (!Q8) return make_f2(scale, scale);
        const float2 s = *reinterpret_cast<const float2 *>(sc + 8 * j);
        return make_f2(s.x, s.y);
    };
    const auto sees = [&](int j, int row, int e) { return (((row ? seen1 : seen0) >> (8 * j + e)) & 1ull) != 0; };
    float top[2] = {-INFINITY, -INFINITY};
    bool exact = EDGE || !Q8;
    if (!exact) {
        // the largest product times the tile's largest scale bounds the scores and
        // mostly shows that the running maximum can stay
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
                top[r] = fmaxf(fmaxf(top[r], fabsf(__uint_as_float(x[4 * j + 2 * r]))),
                               fabsf(__uint_as_float(x[4 * j + 2 * r + 1])));
        }
        // (not <=, so that a NaN scale takes the exact way too)
        const float largest = sc[128 - 2 * (int)(threadIdx.x & 3)];
        exact = __any_sync(~0u, !(top[0] * largest <= m[0] + kAttendLazy) || !(top[1] * largest <= m[1] + kAttendLazy));
    }
    if (exact) {
        top[0] = top[1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const f2 ks = scale_of(j);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const f2 y = Q8 ? pair(j, r) * ks : pair(j, r);
                const float y0 = !EDGE || sees(j, r, 0) ? f2_lo(y) : -INFINITY;
                const float y1 = !EDGE || sees(j, r, 1) ? f2_hi(y) : -INFINITY;
                top[r] = fmaxf(fmaxf(top[r], y0), y1);
            }
        }
        if (!Q8) top[0] *= scale, top[1] *= scale;
        if (__any_sync(~0u, top[0] > m[0] + kAttendLazy || top[1] > m[1] + kAttendLazy)) {
            float al[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
                v = fmaxf(fmaxf(v, __shfl_xor_sync(~0u, v, 2)), m[r]);
                al[r] = v == -INFINITY ? 1.0f : ex2(m[r] - v);
                m[r] = v;
                l[r] *= al[r];
            }
            rescale(al[0], al[1]);
        }
    }
    uint32_t pk[16];
    f2 minus[2], sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float m0 = m[r] == -INFINITY ? 0.0f : -m[r];
        minus[r] = make_f2(m0, m0);
        sum[r] = make_f2(0.0f, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const f2 ks = scale_of(j);
        float2 vs = make_float2(1.0f, 1.0f);
        if (Q8) vs = *reinterpret_cast<const float2 *>(sc + 64 + 8 * j);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const f2 y = fma2(pair(j, r), ks, minus[r]);
            float a = ex2(f2_lo(y)), b = ex2(f2_hi(y));
            if (EDGE) {
                if (!sees(j, r, 0)) a = 0.0f;
                if (!sees(j, r, 1)) b = 0.0f;
            }
            f2 e = make_f2(a, b);
            sum[r] = sum[r] + e;
            if (Q8) {
                e = e * make_f2(vs.x, vs.y);
                if (EDGE)  // an unseen key's scale may be anything
                    e = make_f2(sees(j, r, 0) ? f2_lo(e) : 0.0f, sees(j, r, 1) ? f2_hi(e) : 0.0f);
            }
            pk[2 * j + r] = pack_bf16(f2_lo(e), f2_hi(e));
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) l[r] += f2_lo(sum[r]) + f2_hi(sum[r]);
    tmem_st16x32p(ts, pk);
}

// Fills a ring with the keys or the values of the CTA's tiles, one tile per step().
// Keys and values have a loader (and a warp) each: a ring's next tile is then asked
// for as soon as its own slot is free, up to a ring (kOps or kRaws tiles) ahead of its use.
template <int D, bool Q8>
struct TcLoader {
    using C = AttendTcCfg<D, Q8>;
    static constexpr uint32_t N = Q8 ? C::kRaws : C::kOps;
    const void *map;
    uint8_t *ring;            // slot 0
    uint64_t *full, *empty;   // [N] each
    uint32_t slot_bytes;
    uint8_t *scales;          // with Q8 keys: slot 0 of the scales
    uint32_t *present;        // with the keys: kTcInfo tiles' slices
    KvWalk w;
    KvRequest r;
    KvPiece c;
    KvPageWindow pages;
    int32_t j;
    uint32_t it;

    __device__ __forceinline__ void open(const KvAttendParams &p) {
        c = kv_piece(w, r);
        j = c.ja;
        pages.start(p.tables + (int64_t)w.b * p.table_stride, (r.tile0 + c.ja) * kAttendTile / p.page_size,
                    kv_entries(p, r));
    }
    __device__ __forceinline__ void start(const KvAttendParams &p, const KvWalk &walk, const KvRequest &req) {
        w = walk;
        r = req;
        it = 0;
        if (w.u < w.end) open(p);
    }
    // False when a wait ran out.  Nothing happens behind the last tile.
    __device__ __forceinline__ bool step(const KvAttendParams &p, uint64_t deadline) {
        const int lane = threadIdx.x & 31;
        if (w.u >= w.end) return true;
        // lane 4 b + s deals with slice s (and with column block b)
        const int s = lane & 3, blk = lane >> 2;
        const int32_t t0 = (r.tile0 + j) * kAttendTile, kb = t0 + s * kAttendSlice;
        const bool want = lane < (Q8 ? 4 : 4 * C::kBlocks) && kb < r.kv && kb + kAttendSlice > r.first;
        const int32_t e = kb / p.page_size, off = kb - e * p.page_size;
        const int32_t found = pages.get(t0 / p.page_size, e), page = want ? found : -1;
        const bool here = page >= 0 && page < p.num_pages;
        const uint32_t mask = __ballot_sync(~0u, here) & 15u;
        constexpr uint32_t bytes = kAttendSlice * D * (Q8 ? 1 : 2);  // of a slice
        const uint32_t stage = it % N, use = it / N;
        if (use > 0 && !__all_sync(~0u, tc_wait(&empty[stage], use - 1, deadline))) return false;
        if (lane == 0) {
            if (present) present[it % kTcInfo] = mask;
            mbar_arrive_expect_tx(&full[stage], (uint32_t)__popc(mask) * (bytes + (scales ? 128u : 0u)));
        }
        __syncwarp();
        if (here) {
            const uint32_t bar = smem_u32(&full[stage]);
            const uint32_t at = stage * slot_bytes +
                                (Q8 ? s * bytes : blk * (kAttendTile * 128) + s * (kAttendSlice * 128));
            tma_load_4d(smem_u32(ring) + at, map, Q8 ? 0 : 64 * blk, off, c.head, page, bar);
            if (scales)
                bulk_g2s(scales + stage * 512 + s * 128,
                         p.scales + (((int64_t)page * p.kv_heads + c.head) * p.page_size + off) * 2, 128, &full[stage]);
        }
        ++it;
        if (++j == c.jb) {
            kv_advance<kTcRows, kAttendTile>(p, w, r, c.jb - c.ja);
            if (w.u < w.end) open(p);
        }
        return true;
    }
    // After a timeout: no copy may still be in flight when the CTA ends.
    __device__ __forceinline__ void drain(uint64_t deadline) {
        for (uint32_t k = it > N ? it - N : 0; k < it; ++k)
            if (!tc_wait(&full[k % N], k / N, deadline)) break;
    }
};

// PLACED (a windowed tree with positions) is a kernel of its own: with the choice at run
// time the tile loop's registers went another way (trees over an 8-bit cache 116 us, 144
// with the positions looked up in the loop, 118 with nothing but their load there).
template <int D, bool Q8, bool PLACED>
__global__ void __launch_bounds__(AttendTcCfg<D, Q8>::kThreads, AttendTcCfg<D, Q8>::kOne ? 1 : 2)
    w12_kv_attend_tc_kernel(const KvAttendParams p, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v) {
    using C = AttendTcCfg<D, Q8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *kfull = reinterpret_cast<uint64_t *>(smem + C::kOffBars), *kempty = kfull + C::kOps;
    uint64_t *vfull = kempty + C::kOps, *vempty = vfull + C::kOps;
    uint64_t *rkfull = vempty + C::kOps, *rkempty = rkfull + C::kRaws;
    uint64_t *rvfull = rkempty + C::kRaws, *rvempty = rvfull + C::kRaws;
    uint64_t *sfull = rvempty + C::kRaws, *pfull = sfull + C::kS;
    uint64_t *pvdone = pfull + C::kS, *qfull = pvdone + C::kS, *ofree = qfull + 1, *drain = ofree + 1;
    uint32_t *present = reinterpret_cast<uint32_t *>(smem + C::kOffInfo);
    volatile uint32_t *poison = present + kTcInfo;
    uint32_t *tmem_slot = present + kTcInfo + 3;
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    constexpr int kLoadK = C::kSoft, kMma = kLoadK + 1, kLoadV = kLoadK + 2, kConvert = kLoadK + 4;  // warps

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(&kfull[i], Q8 ? 4 : 1);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], Q8 ? 4 : 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < C::kRaws; ++i) {
            mbar_init(&rkfull[i], 1);
            mbar_init(&rkempty[i], 4);
            mbar_init(&rvfull[i], 1);
            mbar_init(&rvempty[i], 4);
        }
        for (int i = 0; i < C::kS; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], C::kSoft);
            mbar_init(&pvdone[i], 1);
        }
        mbar_init(qfull, C::kSoft);
        mbar_init(ofree, C::kSoft);
        mbar_init(drain, 1);
        fence_mbar_init();
        poison[0] = poison[1] = poison[2] = 0;
    }
    if (threadIdx.x == 32 * kMma) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    pdl_wait();
    const uint64_t deadline = globaltimer_ns() + p.timeout_ns;
    KvWalk w;
    KvRequest r;
    if (!kv_walk_init<kTcRows, kAttendTile>(p, w, r)) return;  // the same for the whole CTA
    // TMEM only after the kernel before has finished, and the kernel behind only
    // when every CTA here has its TMEM: neither can then hold columns that the
    // other waits for
    if (warp == kMma) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp < C::kSoft) {
        if constexpr (C::kRegs > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        // ------------------------------------------------------------ softmax and output
        // Warps w and w + 4 can reach the TMEM lanes 32 w ..: with eight warps each makes
        // the softmax of 16 of those rows and puts out half of the columns of all 32.
        // (What is written for HALVES == 2 is the same numbers in the form that the
        // compiler makes the shortest loop of: 116 us against 123 for an 8-bit tree.)
        constexpr int HALVES = 8 / C::kSoft;  // 16-row halves of a warp
        const int quarter = HALVES == 2 ? warp : warp & 3, half = HALVES == 2 ? 0 : warp >> 2;
        const int lr = HALVES == 2 ? threadIdx.x : 32 * quarter + lane;  // output: the thread's row
        const int base = 32 * quarter + 16 * half;                       // softmax: the warp's first row
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        float2 *stats = reinterpret_cast<float2 *>(smem + C::kOffStats);
        const int g8 = lane >> 2, t4 = lane & 3;
        // of a BF16 cache the softmax scale's sign is in Q, so that the largest product
        // is the largest score
        const float scale = fabsf(p.scale_log2);
        uint32_t it = 0, piece = 0;
        TcPlace &place = reinterpret_cast<TcPlace *>(smem + C::kOffPlaces)[warp];
        if (lane == 0) place = TcPlace{w, r, kv_piece(w, r)};
        __syncwarp();
        // Q rows of a piece to TMEM or shared memory, rows behind the last one zero; for a
        // Q8 cache in the column order of the converted keys
        auto load_q = [&](const KvRequest &rq, const KvPiece &pc) {
            constexpr int CH = D / 8, STEPS = HALVES * CH / 2, G = STEPS < 8 ? STEPS : 8;  // 16-byte chunks; 32 a step
            if constexpr (C::kQTmem) {
                // the lane's row; where a quarter has two warps, half of its columns each
                const int64_t rows = min((int64_t)kTcRows, (int64_t)rq.qlen * p.group - (int64_t)pc.rb * kTcRows);
                const int32_t rr = pc.rb * kTcRows + lr, tok = rr / p.group;
                const uint16_t *src = p.q + (int64_t)(rq.q0 + tok) * p.q_stride +
                                      (int64_t)(pc.head * p.group + rr - tok * p.group) * D;
#pragma unroll
                for (int c0 = 0; c0 < HALVES * D / 4; c0 += 32) {
                    const int col = half * (D / 4) + c0;
                    uint32_t x[32];
                    uint4 u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = make_uint4(0, 0, 0, 0);
                    if (lr < rows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = reinterpret_cast<const uint4 *>(src + 2 * col)[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint4 v = u[i];
                        if (!Q8 && p.scale_log2 < 0.0f)  // the softmax scale's sign
                            v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
                        if (Q8)
                            v = make_uint4(prmt(v.x, v.y, 0x5410u), prmt(v.x, v.y, 0x7632u), prmt(v.z, v.w, 0x5410u),
                                           prmt(v.z, v.w, 0x7632u));
                        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                    }
                    tmem_st32(tl + C::kQCol + col, x);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
                return;
            }
            // where each lane's row is (of 16 or 32); the steps then ask the lanes
            const int64_t rows = min((int64_t)kTcRows, (int64_t)rq.qlen * p.group - (int64_t)pc.rb * kTcRows);
            const int mine = HALVES == 2 ? lr : base + lane % 16;
            const int32_t rr = pc.rb * kTcRows + mine, tok = rr / p.group;
            const int64_t src = mine < rows ? (int64_t)(rq.q0 + tok) * p.q_stride +
                                                  (int64_t)(pc.head * p.group + rr - tok * p.group) * D
                                            : -1;
#pragma unroll
            for (int s0 = 0; s0 < STEPS; s0 += G) {
                uint4 u[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int i = (s0 + g) * 32 + lane;
                    const int64_t at = __shfl_sync(~0u, src, i / CH);
                    u[g] = make_uint4(0, 0, 0, 0);
                    if (at >= 0) u[g] = reinterpret_cast<const uint4 *>(p.q + at)[i % CH];
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int i = (s0 + g) * 32 + lane, row = base + i / CH, ch = i % CH;
                    uint4 v = u[g];
                    if (!Q8 && p.scale_log2 < 0.0f)  // the softmax scale's sign
                        v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
                    if (Q8)
                        v = make_uint4(prmt(v.x, v.y, 0x5410u), prmt(v.x, v.y, 0x7632u), prmt(v.z, v.w, 0x5410u),
                                       prmt(v.z, v.w, 0x7632u));
                    *reinterpret_cast<uint4 *>(smem + C::kOffQ + (ch / 8) * (kTcRows * 128) + row * 128 +
                                               (((ch % 8) ^ (row & 7)) << 4)) = v;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
        };
        load_q(place.r, place.c);
        while (true) {
            int32_t nrows, i, row0, kb, tiles, keys, past, lim, low;
            {
                const KvRequest &r = place.r;
                const KvPiece &c = place.c;
                nrows = (int32_t)min((int64_t)kTcRows, (int64_t)r.qlen * p.group - (int64_t)c.rb * kTcRows);
                row0 = c.rb * kTcRows;
                i = (row0 + min(lr, nrows - 1)) / p.group;  // new token of TMEM lane lr's row
                kb = (r.tile0 + c.ja) * kAttendTile;
                tiles = c.jb - c.ja;
                keys = r.kv;
                past = r.past;
                // every row sees the keys from low on and before lim
                lim = min(r.kv, p.tree ? r.past : r.past + 1);
                low = p.window > 0 ? (int32_t)max((int64_t)r.past + r.qlen - p.window, (int64_t)0) : 0;
            }
            // the keys of the tile at kb that row `row` of the block sees
            const auto seen_by = [&](int row, uint32_t here) -> uint64_t {
                const int32_t tok = (row0 + min(row, nrows - 1)) / p.group;
                return kv_seen64(p, keys, past, kv_row_view<PLACED>(p, place.r, tok), kb, here) >> (2 * t4);
            };
            const bool busy = base < nrows;  // a warp without rows only keeps step
            // rows g and g + 8 of each half, as tc_softmax has them
            float mr[HALVES][2], sr[HALVES][2];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) mr[h][0] = mr[h][1] = -INFINITY, sr[h][0] = sr[h][1] = 0.0f;
            for (int j = 0; j < tiles; ++j, ++it, kb += kAttendTile) {
                // after a timeout the walk goes on without waiting, so that every
                // barrier below is reached
                if (ok) ok = tc_wait(&sfull[it % C::kS], it / C::kS, deadline);
                ok = __all_sync(~0u, ok);
                tc_fence_after();
                const uint32_t here = present[it % kTcInfo];
                // a tile whose keys not all rows see, or of which a slice is missing
                const bool edge = here != 15u || kb > lim - kAttendTile || kb < low;
                if (busy) {
                    const float *sc =
                        reinterpret_cast<const float *>(smem + C::kOffScale + (it % kTcInfo) * C::kInfoBytes) + 2 * t4;
                    uint32_t x[HALVES][32];
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const int row = base + 16 * h;
                        if (row >= nrows) break;  // the same for the warp
                        const uint32_t to = tl + ((uint32_t)(16 * (h + half)) << 16);
                        const uint32_t ts = to + C::kSCol + 64 * (it % C::kS);
                        tmem_ld16x64(ts, x[h]);
                        tmem_wait_ld();
                        const auto rescale = [&](float a0, float a1) {
                            if (j == 0) return;  // nothing there yet
                            if (ok) ok = tc_wait(&pvdone[(it - 1) % C::kS], (it - 1) / C::kS, deadline);
                            ok = __all_sync(~0u, ok);
                            tc_fence_after();
#pragma unroll 1
                            for (int d0 = 0; d0 < D; d0 += 32) {
                                uint32_t o[16];
                                tmem_ld16x32(to + d0, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * ((k & 2) ? a1 : a0));
                                tmem_st16x32(to + d0, o);
                            }
                            tmem_wait_st();
                        };
                        if (edge)
                            tc_softmax<Q8, true>(ts, x[h], sc, scale, mr[h], sr[h], seen_by(row + g8, here),
                                                 seen_by(row + g8 + 8, here), rescale);
                        else
                            tc_softmax<Q8, false>(ts, x[h], sc, scale, mr[h], sr[h], 0, 0, rescale);
                    }
                    tmem_wait_st();
                }
                if (!Q8 && edge) {
                    // values behind the request's last token or of missing slices
                    // become zero, and so do (noted, for the rows that see them)
                    // values that are not finite: the product must not meet 0 * NaN
                    const uint32_t stage = it % C::kOps;
                    if (ok) ok = tc_wait(&vfull[stage], it / C::kOps, deadline);
                    ok = __all_sync(~0u, ok);
                    constexpr int CH = D / 8;
                    for (int q = threadIdx.x; q < kAttendTile * CH; q += 32 * C::kSoft) {
                        const int key = q / CH, ch = q % CH;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + C::kOffV + stage * C::kTileBytes +
                                                              (ch / 8) * (kAttendTile * 128) + key * 128 +
                                                              (((ch % 8) ^ (key & 7)) << 4));
                        uint4 u = *at;
                        if (kb + key >= keys || !((here >> (key / 16)) & 1u)) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            uint32_t e[4] = {u.x, u.y, u.z, u.w};
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((e[k] & 0x7F80u) == 0x7F80u) e[k] &= 0xFFFF0000u, hit = true;
                                if ((e[k] & 0x7F800000u) == 0x7F800000u) e[k] &= 0xFFFFu, hit = true;
                            }
                            if (hit) {
                                *at = make_uint4(e[0], e[1], e[2], e[3]);
                                poison[piece % 3] = 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[it % C::kS]);
            }
            // the next piece's Q while the last products of this one run (all
            // scores of this piece are there, so nothing reads Q any more)
            const KvWalk w1 = place.w;
            const KvRequest r1 = place.r;
            const KvPiece c1 = place.c;
            bool more;
            {
                KvWalk w2 = w1;
                KvRequest r2 = r1;
                kv_advance<kTcRows, kAttendTile>(p, w2, r2, tiles);
                more = w2.u < w2.end;
                if (more) {
                    const KvPiece c2 = kv_piece(w2, r2);
                    load_q(r2, c2);
                    if (lane == 0) place = TcPlace{w2, r2, c2};
                    __syncwarp();
                }
            }
            if (ok) ok = tc_wait(&pvdone[(it - 1) % C::kS], (it - 1) / C::kS, deadline);
            ok = __all_sync(~0u, ok);
            tc_fence_after();
            // the rows' statistics, summed over a row's four threads, for who puts the
            // rows out; and every thread's note of values that are not finite.  One sync
            // covers both: the notes take turns, and the next piece's is cleared while
            // no thread can be reading or setting it
            float m = 0.0f, l = 0.0f;
#pragma unroll
            for (int k = 0; k < 2 * HALVES; ++k) {
                float s = sr[k / 2][k % 2];
                s += __shfl_xor_sync(~0u, s, 1);
                s += __shfl_xor_sync(~0u, s, 2);
                if constexpr (HALVES == 1) {
                    if (t4 == 0) stats[base + 8 * k + g8] = make_float2(mr[0][k], s);
                } else {  // the warp has all of its rows: row 8 k + g from lane 4 g
                    const float a = __shfl_sync(~0u, mr[k / 2][k % 2], (lane & 7) * 4);
                    const float b = __shfl_sync(~0u, s, (lane & 7) * 4);
                    if (lane >> 3 == k) m = a, l = b;
                }
            }
            bool bad = false;
            if constexpr (!Q8 || HALVES == 1) {
                if (threadIdx.x == 0) poison[(piece + 1) % 3] = 0;
                asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kSoft) : "memory");
                if (HALVES == 1) m = stats[lr].x, l = stats[lr].y;
                bad = !Q8 && poison[piece % 3] != 0;
            }
            ++piece;
            const bool whole = c1.ja == 0 && c1.jb == r1.ntiles;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (c1.ja > 0 ? 0 : 1);
            if (32 * quarter < nrows) {
                const int32_t head = c1.head * p.group + c1.rb * kTcRows + lr - i * p.group;
                uint16_t *dst = p.out + (r1.q0 + i) * p.out_stride + (int64_t)head * D;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
                for (int d0 = half * (D / 2); d0 < (half + HALVES) * (D / 2); d0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tl + d0, o);
                    tmem_wait_ld();
                    if (bad && lr < nrows) {
                        // values that are not finite count, as they are, for the
                        // rows that see their keys (a weight is positive; what went
                        // through the product already stays what it is)
                        for (int j = c1.ja; j < c1.jb; ++j) {
                            const int32_t kb = (r1.tile0 + j) * kAttendTile;
                            uint64_t seen =
                                kv_seen64(p, r1.kv, r1.past, kv_row_view<PLACED>(p, r1, i), kb, 15u);
                            for (; seen; seen &= seen - 1) {
                                const int32_t key = kb + __ffsll((long long)seen) - 1, e = key / p.page_size;
                                const int32_t page = p.tables[(int64_t)w1.b * p.table_stride + e];
                                if (page < 0 || page >= p.num_pages) continue;
                                const uint16_t *v = p.v + page * p.v_page_stride + c1.head * p.v_head_stride +
                                                    (int64_t)(key - e * p.page_size) * p.v_row_stride + d0;
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if ((v[k] & 0x7F80u) == 0x7F80u)
                                        o[k] = __float_as_uint(__uint_as_float(o[k]) +
                                                               __uint_as_float((uint32_t)v[k] << 16));
                            }
                        }
                    }
                    if (lr < nrows) {
                        float y[32];  // Q8: columns (0, 2, 1, 3) of every four
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            y[k] = __uint_as_float(o[!Q8 || k % 4 == 0 || k % 4 == 3 ? k : k % 4 == 1 ? k + 1 : k - 1]);
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < 32; k += 8)
                                *reinterpret_cast<uint4 *>(dst + d0 + k) = make_uint4(
                                    pack_bf16(y[k] * inv, y[k + 1] * inv), pack_bf16(y[k + 2] * inv, y[k + 3] * inv),
                                    pack_bf16(y[k + 4] * inv, y[k + 5] * inv),
                                    pack_bf16(y[k + 6] * inv, y[k + 7] * inv));
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<float4 *>(p.part + (slot * kTcRows + lr) * D + d0 + k) =
                                    make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                        }
                    }
                }
                if (half == 0 && lr < nrows) {
                    if (!whole) p.part_ml[slot * kTcRows + lr] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[(int64_t)(r1.q0 + i) * (p.group * p.kv_heads) + head] =
                            l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ofree);
            if (!more) break;
        }
        if (!ok && lane == 0) atomicOr(p.status, 8u);
    } else {
        if constexpr (C::kRegs > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRestRegs));
        if (warp == kLoadK || warp == kLoadV) {
            // ------------------------------------------------------------ loaders
            TcLoader<D, Q8> load;
            const bool keys = warp == kLoadK;
            load.map = keys ? &tm_k : &tm_v;
            load.ring = smem + (Q8 ? C::kOffRaw + (keys ? 0 : C::kRawBytes) : keys ? C::kOffK : C::kOffV);
            load.full = Q8 ? (keys ? rkfull : rvfull) : keys ? kfull : vfull;
            load.empty = Q8 ? (keys ? rkempty : rvempty) : keys ? kempty : vempty;
            load.slot_bytes = Q8 ? 2 * C::kRawBytes : C::kTileBytes;
            load.scales = Q8 && keys ? smem + C::kOffRawScale : nullptr;
            load.present = keys ? present : nullptr;
            load.start(p, w, r);
            while (ok && load.w.u < load.w.end) ok = load.step(p, deadline);
            if (!ok && lane == 0) {
                atomicOr(p.status, 8u);
                load.drain(globaltimer_ns() + p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == kMma) {
            // ------------------------------------------------------------ MMA
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kAttendTile);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D) | (1u << 16);  // B is MN-major
            // The whole warp walks; one elected lane issues.  What the products' operands
            // are computed from comes out of shuffles and votes, so that the compiler
            // knows it to be the same for the warp: an operand that could differ between
            // lanes costs each product a move to a uniform register, and issuing then
            // took longer than the products (700 cycles for a tile's eight).
            const uint32_t tm = __shfl_sync(~0u, tmem, 0);
            const bool leader = elect_one();
            uint32_t it = 0, done = 0, piece = 0;  // tiles whose scores, whose products have been issued; pieces
            // scores of tile `it` into their buffer, when the product of the tile that had
            // it before is over
            auto scores = [&]() -> bool {
                const uint32_t stage = it % C::kOps, buf = it % C::kS;
                bool good = it < C::kS || tc_wait(&pvdone[buf], it / C::kS - 1, deadline);
                good = good && tc_wait(&kfull[stage], it / C::kOps, deadline);
                if (!__all_sync(~0u, good)) return false;
                tc_fence_after();
                if (leader) {
                    const uint64_t b = smem_desc(smem_u32(smem + C::kOffK + stage * C::kTileBytes), 16u, 1024u, 2u);
                    const uint32_t d = tm + C::kSCol + 64 * buf;
                    if constexpr (C::kQTmem) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_tmem_a(d, tm + C::kQCol + 8 * k,
                                       b + (uint64_t)((k >> 2) * (kAttendTile * 128 / 16) + (k & 3) * 2), idesc_qk,
                                       k > 0);
                    } else {
                        const uint64_t a = smem_desc(smem_u32(smem + C::kOffQ), 16u, 1024u, 2u);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_smem_a(d, a + (uint64_t)((k >> 2) * (kTcRows * 128 / 16) + (k & 3) * 2),
                                       b + (uint64_t)((k >> 2) * (kAttendTile * 128 / 16) + (k & 3) * 2), idesc_qk,
                                       k > 0);
                    }
                    mma_commit(&kempty[stage]);
                    mma_commit(&sfull[buf]);
                }
                __syncwarp();
                ++it;
                return true;
            };
            while (ok) {
                int n = w.u < w.end ? (int)min((int64_t)r.ntiles - (w.u - w.start) % r.ntiles, w.end - w.u) : 0;
                n = __shfl_sync(~0u, n, 0);
                if (n == 0) break;
                ok = __all_sync(~0u, tc_wait(qfull, piece, deadline));
                // (a loop of its own: with one that catches up at every tile 337 us became 344)
                for (int j = 0; ok && j < min(n, C::kAheadS); ++j) ok = scores();
                for (int j = 0; ok && j < n; ++j) {
                    if (j + C::kAheadS < n && !(ok = scores())) break;
                    const uint32_t g = done, stage = g % C::kOps, buf = g % C::kS;  // the tile to multiply
                    bool good = tc_wait(&pfull[buf], g / C::kS, deadline) &&
                                tc_wait(&vfull[stage], g / C::kOps, deadline);
                    if (good && j == 0 && piece > 0) good = tc_wait(ofree, piece - 1, deadline);
                    if (!(ok = __all_sync(~0u, good))) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t a = tm + C::kSCol + 64 * buf;
                        const uint64_t b =
                            smem_desc(smem_u32(smem + C::kOffV + stage * C::kTileBytes), kAttendTile * 128, 1024u, 2u);
#pragma unroll
                        for (int k = 0; k < kAttendTile / 16; ++k)
                            mma_tmem_a(tm, a + 8 * k, b + (uint64_t)(k * (16 * 128 / 16)), idesc_pv, j > 0 || k > 0);
                        mma_commit(&vempty[stage]);
                        mma_commit(&pvdone[buf]);
                    }
                    __syncwarp();
                    ++done;
                }
                ++piece;
                if (ok) kv_advance<kTcRows, kAttendTile>(p, w, r, n);
            }
            if (leader) {
                if (!ok) atomicOr(p.status, 8u);
                mma_commit(drain);  // nothing issued may still run when TMEM is given back
                tc_wait(drain, 0, globaltimer_ns() + p.timeout_ns);
            }
            __syncwarp();
        } else if (Q8 && warp >= kConvert) {
            // ------------------------------------------------------------ converters of a Q8 cache
            const int cw = (warp - kConvert) & 3, ct = cw * 32 + lane;
            constexpr uint32_t N = C::kRaws + !Q8;
            constexpr int CH = D / 16;  // 16-byte chunks of a row
            // the thread's first chunk and where its two operand chunks go; odd column
            // blocks in the other order, so that eight lanes write eight different
            // 16-byte bank groups
            const int ckey = ct / CH, cc = ct % CH;
            const bool turn = (cc / 4) & 1;
            const uint32_t base = (cc / 4) * (kAttendTile * 128) + ckey * 128;
            const uint32_t at0 = base + (((2 * (cc % 4) + (turn ? 1 : 0)) ^ (ckey & 7)) << 4);
            const uint32_t at1 = base + (((2 * (cc % 4) + (turn ? 0 : 1)) ^ (ckey & 7)) << 4);
            const uint32_t total = (uint32_t)(w.end - w.u);
            // K or V of tile x to its operand buffer, which the tile before it there must have left
            auto convert = [&](bool values, uint32_t x) -> bool {
                const uint32_t stage = x % N;
                bool good = tc_wait(values ? &rvfull[stage] : &rkfull[stage], x / N, deadline);
                const uint32_t op = x % C::kOps;
                if (good && x >= C::kOps)
                    good = tc_wait(values ? &vempty[op] : &kempty[op], x / C::kOps - 1, deadline);
                if (!__all_sync(~0u, good)) return false;
                if (!values && cw < 2) {
                    // scales of the tile's keys, the softmax scale in the keys' ones, and
                    // the largest of those
                    const float2 *src = reinterpret_cast<const float2 *>(smem + C::kOffRawScale + stage * 512);
                    float *dst = reinterpret_cast<float *>(smem + C::kOffScale + (x % kTcInfo) * C::kInfoBytes);
                    if (cw == 0) {
                        const float a = src[lane].x * p.scale_log2, b = src[lane + 32].x * p.scale_log2;
                        dst[lane] = a;
                        dst[lane + 32] = b;
                        float top = max_nan(fabsf(a), fabsf(b));
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, d));
                        if (lane == 0) dst[128] = top;
                    } else {
                        dst[64 + lane] = src[lane].y;
                        dst[96 + lane] = src[lane + 32].y;
                    }
                }
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(smem + C::kOffRaw + (stage * 2 + values) * C::kRawBytes) + ct;
                uint8_t *dst = smem + (values ? C::kOffV : C::kOffK) + op * C::kTileBytes;
                constexpr int N4 = kAttendTile * CH / 128;  // 16-byte chunks of a thread, 128 / CH keys apart
                constexpr int G = N4 < 4 ? N4 : 4;
#pragma unroll
                for (int i0 = 0; i0 < N4; i0 += G) {
                    uint4 u[G];
#pragma unroll
                    for (int i = 0; i < G; ++i) u[i] = src[(i0 + i) * 128];
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        uint4 a, b;
                        q8_to_bf16(turn ? u[i].z : u[i].x, a.x, a.y);
                        q8_to_bf16(turn ? u[i].w : u[i].y, a.z, a.w);
                        q8_to_bf16(turn ? u[i].x : u[i].z, b.x, b.y);
                        q8_to_bf16(turn ? u[i].y : u[i].w, b.z, b.w);
                        // 128 / CH keys further: a multiple of 8, the same swizzle
                        uint8_t *row = dst + (i0 + i) * (128 / CH) * 128;
                        *reinterpret_cast<uint4 *>(row + at0) = a;
                        *reinterpret_cast<uint4 *>(row + at1) = b;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(values ? &vfull[op] : &kfull[op]);
                    mbar_arrive(values ? &rvempty[stage] : &rkempty[stage]);
                }
                return true;
            };
            if constexpr (C::kGroups == 2) {
                const bool values = warp >= kConvert + 4;
                for (uint32_t x = 0; ok && x < total; ++x) ok = convert(values, x);
            } else {
                // the keys run one tile ahead: their buffer is free as soon as the scores
                // are made, the values' only after the softmax
                ok = convert(false, 0);
                for (uint32_t x = 0; ok && x < total; ++x) {
                    if (x + 1 < total) ok = convert(false, x + 1);
                    ok = ok && convert(true, x);
                }
            }
            if (!ok && lane == 0) atomicOr(p.status, 8u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace dev
}  // namespace w12
