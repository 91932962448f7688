// Page tables of requests that go on from others (w12_kv_fork in include/w12.h).
//
// Per page P, with shares[P] its holders less one:
//   h(P) = shares[P] - (rows that held P) + (rows that want P as a full page)
// is what it is without the rows that want it as their last, partly filled page; such a
// row may keep it only where h(P) = -1 (no one else), and the first of them does.  The
// others get pages from the ring and a copy each; a page with h(P) = -1 that no row keeps
// goes back to the ring.
//
// A page stands at one entry c of every table that holds it, so a CTA that has some
// columns of all rows has all that happens to their pages.  It counts with atomics on shares
// (none where a row wants the page that it had, as in most of a shared prefix) and finds the
// first row of a page by an atomic minimum on the same word, which until its end holds,
// below -1, the smallest row so far: rows that keep in [-1 - 2 R, -2 - R], rows that free
// in [-1 - R, -2], so that one that keeps wins.  The columns go through shared memory, so
// that the tables are permuted in place.
//
// Places in the ring need what all CTAs count: small tables are one CTA's and one launch,
// larger ones have up to eight columns (a 32-byte sector of a row) per CTA and two launches, the
// first of which counts.  Pages go back in the order of their entries, then rows, and
// come in the order of rows: nothing depends on timing.
//
// What bounds it: latency, of the loads that wait for one another (lengths, table entries,
// holders, marks, the ring) and of the launches; it reads and writes a few bytes per table entry.
// Measured: 4 rows of 128 entries 7.3 us; 32 to 128 rows of 256 entries 12 to 13 us; 1024 rows of
// 256 entries 25 us, with eight columns per CTA instead of two (32 CTAs instead of 128) 44.5.
#pragma once

#include "kv_plan.cuh"

namespace w12 {
namespace dev {

constexpr int kForkRows = 4096, kForkCols = 8;
// Table entries that one CTA takes: 512 are 8.0 us in one launch and 10.6 in two, 2048 13.4 and
// 12.3, 8192 24 and 12.
constexpr int kForkOne = 1024;
// With fewer columns per CTA than kForkCols: at most one per SM (a constant, for the workspace's
// size is asked for without a device).
constexpr int kForkCtas = 152;

struct KvForkParams {
    const int32_t *parents, *lens;
    int32_t *lens_out, *owned, *tables;
    int64_t table_stride;
    int32_t *ring;
    int64_t *state;
    int32_t *shares;
    int32_t *src, *dst, *rows;
    const int32_t *prefix_cu;
    int32_t *prefix_lens;
    int64_t num_pages;
    uint64_t ring_inv;
    // from the first launch to the second: pages wanted (top bit: the last partly filled),
    // pages held, parents and whether a copy is needed of each row, the ring's state, the
    // pages that each CTA frees; and (zero before and after a call) of each group's first
    // live row max_blocks less the first entry at which the group differs
    int32_t *need, *held, *parent, *copies, *counts, *differ;
    int64_t *old_state;
    uint32_t rows_inv;  // ceil(2^32 / requests)
    int32_t requests, max_blocks, page_size, ring_size, groups, cols, ctas;
    uint32_t *status;
};

// Rows of a column in shared memory: a sector's eight entries of four rows lie in 32 banks.
__host__ __device__ constexpr int fork_pitch(int rows) { return rows < 32 ? rows | 1 : (rows + 31) / 32 * 32 + 4; }
__host__ __device__ constexpr int fork_smem(int rows, int cols) {
    return (cols * fork_pitch(rows) + rows * 4) * 4 + rows * 6;
}

// Sum over the CTA's warps of those before `warp`, and of all; s_warp: their numbers.
__device__ __forceinline__ void fork_sums(const int32_t *s_warp, int warp, int32_t &before, int32_t &all) {
    before = all = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) {
        before += i < warp ? s_warp[i] : 0;
        all += s_warp[i];
    }
}

// STEP 1: the first launch, 2: the second; 0: both in one CTA.
template <int STEP>
__global__ void __launch_bounds__(1024, 1) w12_kv_fork_kernel(const __grid_constant__ KvForkParams p) {
    extern __shared__ int32_t fork_dyn[];
    __shared__ int32_t s_warp[32];
    __shared__ int32_t s_freed;
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int R = p.requests, pitch = fork_pitch(R), cols = p.cols, c0 = blockIdx.x * cols;
    int32_t *s_e = fork_dyn;               // [cols][pitch]: the rows' old pages, -1: none
    int32_t *s_need = s_e + cols * pitch;  // pages wanted; the top bit: the last one is partly filled
    int32_t *s_owned = s_need + R;         // pages held so far
    int32_t *s_lead = s_owned + R;         // at a group's first row: its first live row (and bit 30: two live)
    int32_t *s_differ = s_lead + R;        // as p.differ
    int16_t *s_parent = reinterpret_cast<int16_t *>(s_differ + R);
    uint16_t *s_start = reinterpret_cast<uint16_t *>(s_parent + R);  // the row's group's first row
    uint8_t *s_copy = reinterpret_cast<uint8_t *>(s_start + R);
    constexpr int32_t kTwo = 1 << 30;
    const bool prefix = p.prefix_lens != nullptr;
    // the second launch has one CTA more for the prefixes
    const bool last = STEP == 2 && (int)blockIdx.x == p.ctas, groups = prefix && (STEP != 2 || last);
    const int32_t *cu = s_differ;  // at first the groups' first rows, where every row looks for its own
    pdl_launch_dependents();
    pdl_wait();
    uint32_t flags = 0;
    if (tid == 0) s_freed = 0;
    int64_t head, tail;
    if (STEP == 2) head = __ldcg(&p.old_state[0]), tail = __ldcg(&p.old_state[1]);
    else head = __ldcg(&p.state[0]), tail = __ldcg(&p.state[1]);
    const int32_t cu_end = groups ? p.prefix_cu[p.groups] : 0;
    // parents and lengths wait in the places of what comes of them
    for (int i = tid; i < R; i += T) {
        const int32_t o = STEP == 2 ? p.held[i] : p.owned[i];
        const int32_t par = STEP == 2 ? p.parent[i] : p.parents[i], n = STEP == 2 ? p.need[i] : p.lens[i];
        const int32_t copy = STEP == 2 ? p.copies[i] : 0, start = groups && i < p.groups ? p.prefix_cu[i] : 0;
        s_owned[i] = min(max(o, 0), p.max_blocks);
        s_lead[i] = kTwo - 1;
        s_differ[i] = start;
        s_copy[i] = copy != 0;
        s_need[i] = n;
        s_parent[i] = (int16_t)(par >= 0 && par < R ? par : -1);
        if (o != s_owned[i] || (STEP != 2 && (par < -1 || par >= R))) flags |= kStatusKvSizes;
    }
    __syncthreads();
    // the columns' old entries
    if (!last)
#pragma unroll 4
        for (int i = tid; i < cols * R; i += T) {
            const int r = STEP == 0 ? i / cols : i >> (__ffs(cols) - 1), k = i - r * cols;
            int32_t e = -1;
            if (c0 + k < s_owned[r]) e = __ldcg(p.tables + r * p.table_stride + c0 + k);
            s_e[k * pitch + r] = e >= 0 && e < p.num_pages ? e : -1;
        }
    for (int i = tid; i < R; i += T) {
        if (STEP != 2) {
            const int32_t par = s_parent[i], l = s_need[i];
            const int64_t most = par >= 0 ? (int64_t)s_owned[par] * p.page_size : 0;
            const int32_t keep = clamp_i32(l, 0, most);
            if (par >= 0 && keep != l) flags |= kStatusKvSizes;
            const int32_t need = (int32_t)(((int64_t)keep + p.page_size - 1) / p.page_size);
            const bool part = need * (int64_t)p.page_size != keep;
            s_need[i] = need | (part ? (int32_t)0x80000000 : 0);
            if (STEP == 1 && blockIdx.x == 0) {
                p.need[i] = s_need[i];
                p.held[i] = s_owned[i];
                p.parent[i] = par;
            }
        }
        if (groups) {
            int lo = 0, hi = p.groups;  // the last group that starts at or before i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= i) lo = mid;
                else hi = mid;
            }
            const int32_t a = cu[lo], b = lo + 1 < p.groups ? cu[lo + 1] : cu_end;
            const int start = i >= a && i < b ? max(a, 0) : i;  // in no group: one of its own
            s_start[i] = (uint16_t)start;
            if ((s_need[i] & 0x7FFFFFFF) > 0) atomicMin(&s_lead[start], i);
        }
    }
    if (STEP == 1 && blockIdx.x == 0 && tid == 0) p.old_state[0] = head, p.old_state[1] = tail;
    __syncthreads();
    if (STEP != 1 && groups) {
        for (int i = tid; i < R; i += T) s_differ[i] = 0;
        __syncthreads();
    }

    // the page that row r wants at column k as a full one (-1: none)
    const auto wants = [&](int r, int k) {
        const int32_t n = s_need[r], full = (n & 0x7FFFFFFF) - (n < 0 ? 1 : 0);
        return c0 + k < full ? s_e[k * pitch + s_parent[r]] : -1;
    };
    // whether row r ends in these columns, and at which
    const auto ends = [&](int r, int &k) {
        k = (s_need[r] & 0x7FFFFFFF) - 1 - c0;
        return k >= 0 && k < cols;
    };
    const auto keep_mark = [&](int r) { return -1 - 2 * R + r; };
    const auto free_mark = [&](int r) { return -1 - R + r; };
    // f(row, column) over the (entry, row) line
    const auto column = [&](int x) { return R == 1 ? x : (int)__umulhi((uint32_t)x, p.rows_inv); };
    const auto each = [&](auto f) {
#pragma unroll 4
        for (int x = tid; x < cols * R; x += T) {
            const int k = column(x);
            f(x - k * R, k);
        }
    };

    const auto prefixes = [&]() {
        for (int r = tid; r < R; r += T) {
            const int lead = s_lead[s_start[r]] & (kTwo - 1);
            if ((s_need[r] & 0x7FFFFFFF) == 0) continue;
            if (lead != r) atomicOr(&s_lead[s_start[r]], kTwo);
            if (STEP == 2 && lead == r) s_differ[r] = __ldcg(&p.differ[r]), p.differ[r] = 0;
        }
        __syncthreads();
        for (int r = tid; r < R; r += T) {
            int32_t tokens = 0;
            if ((s_need[r] & 0x7FFFFFFF) > 0) {
                const int32_t l = s_lead[s_start[r]], lead = l & (kTwo - 1), m = s_need[lead];
                const int32_t full = (m & 0x7FFFFFFF) - (m < 0 ? 1 : 0), d = s_differ[lead];
                if (l & kTwo) tokens = min(full, d > 0 ? p.max_blocks - d : full) * p.page_size;
            }
            p.prefix_lens[r] = tokens;
        }
    };
    if (last) {
        prefixes();
        return;
    }

    // ------------------------------------------------------------ counting
    bool any = false;
    {
        int at = -1, best = 0;  // a group's first live row and the largest number for it so far
        const auto flush = [&]() {
            if (at >= 0) atomicMax(STEP == 0 ? &s_differ[at] : &p.differ[at], best);
        };
        each([&](int r, int k) {
            const int32_t b = wants(r, k);
            any |= s_e[k * pitch + r] != b;
            if (STEP != 2 && prefix && (s_need[r] & 0x7FFFFFFF) > 0) {
                const int lead = s_lead[s_start[r]] & (kTwo - 1);
                const int32_t m = s_need[lead], full = (m & 0x7FFFFFFF) - (m < 0 ? 1 : 0);
                if (c0 + k < full) {
                    const int32_t l = wants(lead, k), v = p.max_blocks - c0 - k;
                    if ((b != l || l < 0) && (lead != at || v > best)) {
                        if (lead != at) flush(), best = 0;
                        at = lead, best = max(best, v);
                    }
                }
            }
        });
        if (STEP != 2) flush();
    }
    for (int r = tid; r < R; r += T) {
        int k;
        any |= ends(r, k) && s_need[r] < 0;
    }
    any = __syncthreads_or(any);
    if (STEP != 2 && any) {
        each([&](int r, int k) {
            const int32_t a = s_e[k * pitch + r], b = wants(r, k);
            if (a == b) return;
            if (a >= 0) atomicAdd(&p.shares[a], -1);
            if (b >= 0) atomicAdd(&p.shares[b], 1);
        });
        __syncthreads();
        for (int r = tid; r < R; r += T) {
            int k;
            if (!ends(r, k) || s_need[r] >= 0) continue;
            const int32_t b = s_e[k * pitch + s_parent[r]];
            if (b >= 0 && __ldcg(&p.shares[b]) < 0) atomicMin(&p.shares[b], keep_mark(r));
        }
        each([&](int r, int k) {
            const int32_t a = s_e[k * pitch + r];
            if (a >= 0 && a != wants(r, k) && __ldcg(&p.shares[a]) < 0) atomicMin(&p.shares[a], free_mark(r));
        });
        __syncthreads();
    }
    // rows that end here and have to copy: those whose page has another one's mark
    for (int r = tid; STEP != 2 && r < R; r += T) {
        int k;
        if (!ends(r, k)) continue;
        const int32_t b = s_need[r] < 0 ? s_e[k * pitch + s_parent[r]] : -1;
        const bool copy = b >= 0 && __ldcg(&p.shares[b]) != keep_mark(r);
        s_copy[r] = copy;
        if (STEP == 1) p.copies[r] = copy;
    }
    if (STEP == 1 && blockIdx.x == 0)
        for (int r = tid; r < R; r += T)
            if ((s_need[r] & 0x7FFFFFFF) == 0) p.copies[r] = 0;
    const auto frees = [&](int r, int k) {
        const int32_t a = s_e[k * pitch + r];
        return a >= 0 && a != wants(r, k) && __ldcg(&p.shares[a]) == free_mark(r);
    };
    if (STEP == 1) {
        int32_t n = 0;
        if (any) each([&](int r, int k) { n += frees(r, k); });
        n = (int32_t)__reduce_add_sync(~0u, (unsigned)n);
        if (lane == 0 && n) atomicAdd(&s_freed, n);
        __syncthreads();
        if (tid == 0) p.counts[blockIdx.x] = s_freed;
        if (flags && blockIdx.x == 0) atomicOr(p.status, flags);
        return;
    }

    // ------------------------------------------------------------ places in the ring
    const int32_t avail = clamp_i32(tail - head, 0, p.ring_size), room = p.ring_size - avail;
    const int32_t head_at = ring_base(head, p.ring_size, p.ring_inv);
    const int32_t tail_at = ring_base(tail, p.ring_size, p.ring_inv);
    if (tail - head != avail) flags |= kStatusKvPages;
    int32_t before = 0, all = 0, here = 1;  // pages freed before these columns, in all, and here (0: none)
    if (STEP == 2) {
        int32_t a = 0, b = 0;
        for (int i = tid; i < p.ctas; i += T) {
            const int32_t n = p.counts[i];
            a += i < (int)blockIdx.x ? n : 0;
            b += n;
        }
        a = (int32_t)__reduce_add_sync(~0u, (unsigned)a), b = (int32_t)__reduce_add_sync(~0u, (unsigned)b);
        if (lane == 0) s_warp[warp] = a;
        __syncthreads();
        int32_t unused;
        fork_sums(s_warp, 0, unused, before);
        __syncthreads();
        if (lane == 0) s_warp[warp] = b;
        __syncthreads();
        fork_sums(s_warp, 0, unused, all);
        __syncthreads();
        here = p.counts[blockIdx.x];
    }
    if (any && here > 0) {
        // a warp has a run of the (entry, row) line
        const int32_t line = cols * R, run = (line + T - 1) / T * 32, from = warp * run, end = min(line, from + run);
        const auto walk = [&](auto f) {
            for (int32_t x0 = from; x0 < end; x0 += 32) {
                const int32_t x = x0 + lane, k = column(x), r = x - k * R;
                const bool is = x < end && frees(r, k);
                f(__ballot_sync(~0u, is), is, r, k);
            }
        };
        int32_t mine = 0, ahead, sum;
        walk([&](uint32_t hit, bool, int, int) { mine += __popc(hit); });
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        fork_sums(s_warp, warp, ahead, sum);
        int32_t at = before + ahead;
        if (mine)
            walk([&](uint32_t hit, bool is, int r, int k) {
                const int32_t to = at + __popc(hit & ((1u << lane) - 1u));
                if (is && to < room) p.ring[ring_at(tail_at, to, p.ring_size)] = s_e[k * pitch + r];
                at += __popc(hit);
            });
        if (STEP == 0) all = sum;
    }
    __syncthreads();  // the marks have been read
    if (any)
        each([&](int r, int k) {
            const int c = c0 + k;
            const int32_t a = s_e[k * pitch + r], n = s_need[r], need = n & 0x7FFFFFFF;
            int32_t b = wants(r, k);
            // the marks go: a freed page is held by no one, a kept one by its row
            if (a >= 0 && a != b && __ldcg(&p.shares[a]) == free_mark(r)) p.shares[a] = 0;
            if (c >= need) return;
            if (n < 0 && c == need - 1) {
                if (s_copy[r]) return;  // a fresh page, below
                b = s_e[k * pitch + s_parent[r]];
                if (b >= 0) p.shares[b] = 0;
            }
            if (b != a || b < 0 || c >= s_owned[r]) p.tables[r * p.table_stride + c] = b;
        });
    // fresh pages in row order, and what is one per row, by the CTA that has the row's end
    const bool first = blockIdx.x == 0;
    bool mine = false;
    for (int r = tid; r < R; r += T) {
        int k;
        mine |= ends(r, k) && s_copy[r];
    }
    if (!__syncthreads_or(mine || first)) mine = false;
    else mine = true;
    int32_t given = 0;  // copies of the rows before
    for (int r0 = 0; r0 < R; r0 += T) {
        const int r = r0 + tid;
        const bool want = mine && r < R && s_copy[r];
        const uint32_t hit = __ballot_sync(~0u, want);
        int32_t at = given;
        if (mine) {
            if (lane == 0) s_warp[warp] = __popc(hit);
            __syncthreads();
            int32_t ahead, sum;
            fork_sums(s_warp, warp, ahead, sum);
            __syncthreads();
            at += ahead + __popc(hit & ((1u << lane) - 1u));
            given += sum;
        }
        int k;
        if (r >= R || !(ends(r, k) || (first && (s_need[r] & 0x7FFFFFFF) == 0))) continue;
        const int32_t n = s_need[r], need = n & 0x7FFFFFFF;
        int32_t len = need * p.page_size, rows = 0, page = -1, from = -1;
        if (n < 0) {
            len = p.lens[r];  // not clamped: a clamped length has whole pages
            rows = len - (need - 1) * p.page_size;
        }
        if (want) {
            page = at < avail ? p.ring[ring_at(head_at, at, p.ring_size)] : -1;
            if (page < 0 || page >= p.num_pages) page = -1, flags |= kStatusKvPages;
            if (page >= 0) from = s_e[k * pitch + s_parent[r]];
            p.tables[r * p.table_stride + need - 1] = page;
        }
        p.src[r] = from;
        p.dst[r] = page;
        p.rows[r] = page < 0 ? 0 : rows;
        p.owned[r] = need;
        if (p.lens_out) p.lens_out[r] = len;
    }
    if (first) {
        if (tid == 0) {
            if (given > avail || all > room) flags |= kStatusKvPages;
            p.state[0] = head + min(given, avail);
            p.state[1] = tail + min(all, room);
        }
    }
    if (STEP == 0 && prefix) prefixes();
    if (flags && (STEP == 0 || first || (flags & kStatusKvPages))) atomicOr(p.status, flags);
}

}  // namespace dev
}  // namespace w12
