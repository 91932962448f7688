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
// columns of all rows has all that happens to their pages: it counts with atomics on
// shares and finds the first row of a page by an atomic minimum on the same word, which
// until its end holds, below -1, the smallest row so far (rows that keep in
// [-1 - R, -2], rows that free below).  The columns of eight entries (a 32-byte sector of
// each row) go round in shared memory, so that the tables are permuted in place.
//
// One cluster of up to 16 CTAs, one launch: its barriers are between the counting, what
// needs all counts (places in the ring, fresh pages), and the entries of fresh pages.
// Pages go back in the order of their entries, then rows, and come in the order of rows:
// nothing depends on timing.
#pragma once

#include "kv_plan.cuh"

namespace w12 {
namespace dev {

constexpr int kForkThreads = 512, kForkRows = 4096, kForkCols = 8;

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
    int32_t requests, max_blocks, page_size, ring_size, groups;
    uint32_t *status;
};

// Rows of a column in shared memory: a sector's eight entries of four rows lie in 32 banks.
__host__ __device__ constexpr int fork_pitch(int rows) { return (rows + 31) / 32 * 32 + 4; }
__host__ __device__ constexpr int fork_smem(int rows) { return kForkCols * fork_pitch(rows) * 4 + rows * 16; }

__device__ __forceinline__ int32_t dsmem_load(const int32_t *mine, uint32_t rank) {
    uint32_t at;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__global__ void __launch_bounds__(kForkThreads, 1) w12_kv_fork_kernel(const KvForkParams p) {
    extern __shared__ int32_t fork_dyn[];
    constexpr int W = kForkThreads / 32;
    __shared__ int32_t s_freed, s_cols;  // pages that the CTA frees; entries in use
    __shared__ int32_t s_warp[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = p.requests, pitch = fork_pitch(R);
    int32_t *s_e = fork_dyn;                                  // [kForkCols][pitch]: the rows' old pages, -1: none
    int32_t *s_need = s_e + kForkCols * pitch;                // pages wanted; the top bit: the last one is partly filled
    int32_t *s_owned = s_need + R;                            // pages held so far
    int32_t *s_lead = s_owned + R;                            // at a group's first row: its first live row (and bit 30: two live)
    int16_t *s_parent = reinterpret_cast<int16_t *>(s_lead + R);
    uint16_t *s_start = reinterpret_cast<uint16_t *>(s_parent + R);  // the row's group's first row
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    constexpr int32_t kTwo = 1 << 30;
    const bool prefix = p.prefix_lens != nullptr;
    pdl_launch_dependents();
    pdl_wait();
    uint32_t flags = 0;
    if (tid == 0) s_freed = 0, s_cols = 0;
    for (int i = tid; i < R; i += kForkThreads) {
        const int32_t o = p.owned[i];
        s_owned[i] = min(max(o, 0), p.max_blocks);
        s_lead[i] = kTwo - 1;
        if (o != s_owned[i]) flags |= kStatusKvSizes;
    }
    __syncthreads();
    {
        int32_t cols = 0;
        for (int i = tid; i < R; i += kForkThreads) {
            const int32_t par = p.parents[i], l = p.lens[i];
            const bool real = par >= 0 && par < R;
            const int64_t most = real ? (int64_t)s_owned[par] * p.page_size : 0;
            const int32_t keep = clamp_i32(l, 0, most);
            if ((real && keep != l) || par < -1 || par >= R) flags |= kStatusKvSizes;
            const int32_t need = (int32_t)(((int64_t)keep + p.page_size - 1) / p.page_size);
            const bool part = need * (int64_t)p.page_size != keep;
            s_parent[i] = real ? (int16_t)par : (int16_t)-1;
            s_need[i] = need | (part ? (int32_t)0x80000000 : 0);
            cols = max(cols, max(need, s_owned[i]));
            if (prefix) {
                int lo = 0, hi = p.groups;  // the last group that starts at or before i
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (p.prefix_cu[mid] <= i) lo = mid;
                    else hi = mid;
                }
                const int32_t a = p.prefix_cu[lo], b = p.prefix_cu[lo + 1];
                const int start = i >= a && i < b ? max(a, 0) : i;  // in no group: one of its own
                s_start[i] = (uint16_t)start;
                if (keep > 0) atomicMin(&s_lead[start], i);
            }
            if (rank == 0) {
                if (need == 0) p.src[i] = -1, p.dst[i] = -1;
                if (prefix) p.prefix_lens[i] = (need - part) * p.page_size;  // of a group's first live row: what it can be
            }
        }
        atomicMax(&s_cols, cols);
    }
    __syncthreads();
    if (prefix)
        for (int i = tid; i < R; i += kForkThreads)
            if ((s_need[i] & 0x7FFFFFFF) > 0 && (s_lead[s_start[i]] & (kTwo - 1)) != i) atomicOr(&s_lead[s_start[i]], kTwo);
    const int chunks = (s_cols + kForkCols - 1) / kForkCols, per = (chunks + ranks - 1) / ranks;
    const int first = min(rank * per, chunks), last = min(first + per, chunks);

    const auto load = [&](int chunk) {  // the chunk's old entries
        for (int i = tid; i < kForkCols * R; i += kForkThreads) {
            const int r = i / kForkCols, k = i % kForkCols, c = chunk * kForkCols + k;
            int32_t e = -1;
            if (c < s_owned[r]) e = __ldcg(p.tables + r * p.table_stride + c);
            s_e[k * pitch + r] = e >= 0 && e < p.num_pages ? e : -1;
        }
        __syncthreads();
    };
    // the page that row r wants at entry c as a full one (-1: none)
    const auto wants = [&](int r, int c, int k) {
        const int32_t n = s_need[r], full = (n & 0x7FFFFFFF) - (n < 0 ? 1 : 0);
        return c < full ? s_e[k * pitch + s_parent[r]] : -1;
    };
    const int32_t keeps = -1 - R, frees = -1 - 2 * R;  // + row + ...: marks of the row that keeps, that frees
    // row r's mark: the smaller the row, the smaller the mark, all of one kind below the other's
    const auto keep_mark = [&](int r) { return keeps + r; };   // [-1 - R, -2]
    const auto free_mark = [&](int r) { return frees + r; };   // [-1 - 2 R, -2 - R]

    // f(row, column of the chunk) over the chunk's (entry, row) line
    const auto each = [&](auto f) {
#pragma unroll 4
        for (int x = tid; x < kForkCols * R; x += kForkThreads) {
            const int k = x / R;
            f(x - k * R, k);
        }
    };

    // ------------------------------------------------------------ counting
    for (int chunk = first; chunk < last; ++chunk) {
        load(chunk);
        const int c0 = chunk * kForkCols;
        each([&](int r, int k) {
            const int32_t a = s_e[k * pitch + r], b = wants(r, c0 + k, k);
            if (a == b) return;  // most of a shared prefix
            if (a >= 0) atomicAdd(&p.shares[a], -1);
            if (b >= 0) atomicAdd(&p.shares[b], 1);
        });
        __syncthreads();
        // rows whose last, partly filled page is in this chunk
        const auto partial = [&](int r, int &k) {
            const int32_t n = s_need[r];
            k = (n & 0x7FFFFFFF) - 1 - c0;
            return n < 0 && k >= 0 && k < kForkCols;
        };
        for (int r = tid; r < R; r += kForkThreads) {
            int k;
            if (!partial(r, k)) continue;
            const int32_t b = s_e[k * pitch + s_parent[r]];
            if (b >= 0 && __ldcg(&p.shares[b]) < 0) atomicMin(&p.shares[b], keep_mark(r));
        }
        __syncthreads();
        for (int r = tid; r < R; r += kForkThreads) {
            int k;
            const bool part = partial(r, k);
            if (!part && !(k >= 0 && k < kForkCols)) continue;  // another chunk's
            const int32_t b = part ? s_e[k * pitch + s_parent[r]] : -1;
            const bool copy = b >= 0 && __ldcg(&p.shares[b]) != keep_mark(r);
            p.src[r] = copy ? b : -1;
            p.dst[r] = copy ? -2 : -1;
        }
        each([&](int r, int k) {
            const int32_t a = s_e[k * pitch + r];
            if (a < 0 || a == wants(r, c0 + k, k)) return;
            const int32_t v = __ldcg(&p.shares[a]);
            if (v == -1 || v < keeps) atomicMin(&p.shares[a], free_mark(r));
        });
        __syncthreads();
        int32_t n = 0;
        each([&](int r, int k) {
            const int32_t a = s_e[k * pitch + r];
            if (a >= 0 && a != wants(r, c0 + k, k) && __ldcg(&p.shares[a]) == free_mark(r)) ++n;
        });
        n = (int32_t)__reduce_add_sync(~0u, (unsigned)n);
        if (lane == 0 && n) atomicAdd(&s_freed, n);
        __syncthreads();
    }
    cluster_sync();

    // ------------------------------------------------------------ places in the ring
    const int64_t head = p.state[0], tail = p.state[1];
    const int32_t avail = clamp_i32(tail - head, 0, p.ring_size), room = p.ring_size - avail;
    const int32_t head_at = ring_base(head, p.ring_size, p.ring_inv), tail_at = ring_base(tail, p.ring_size, p.ring_inv);
    if (tail - head != avail) flags |= kStatusKvPages;
    int32_t before = 0, all = 0;
    for (int i = 0; i < ranks; ++i) {
        const int32_t n = dsmem_load(&s_freed, (uint32_t)i);
        if (i < rank) before += n;
        all += n;
    }
    for (int chunk = first; chunk < last; ++chunk) {
        if (last - first > 1) load(chunk);
        const int c0 = chunk * kForkCols;
        // a warp has a run of the chunk's (entry, row) line
        const int32_t line = kForkCols * R, run = (line + W * 32 - 1) / (W * 32) * 32;
        const int32_t end = min(line, (warp + 1) * run);
        int32_t mine = 0;
        for (int pass = 0; pass < 2; ++pass) {
            int32_t at = before;
            if (pass == 1) {
                int32_t sum = 0;
                for (int i = 0; i < W; ++i) {
                    if (i == warp) at += sum;
                    sum += s_warp[i];
                }
                before += sum;
                if (sum == 0) break;
            }
            for (int32_t x0 = warp * run; x0 < end; x0 += 32) {
                const int32_t x = x0 + lane, k = x / R, r = x - k * R;
                bool is = false;
                int32_t a = -1;
                if (x < end) {
                    a = s_e[k * pitch + r];
                    is = a >= 0 && a != wants(r, c0 + k, k) && __ldcg(&p.shares[a]) == free_mark(r);
                }
                const uint32_t hit = __ballot_sync(~0u, is);
                if (pass == 0) {
                    mine += __popc(hit);
                } else if (is) {
                    const int32_t to = at + __popc(hit & ((1u << lane) - 1u));
                    if (to < room) p.ring[ring_at(tail_at, to, p.ring_size)] = a;
                }
                if (pass == 1) at += __popc(hit);
            }
            if (pass == 0) {
                if (lane == 0) s_warp[warp] = mine;
                __syncthreads();
            }
        }
        __syncthreads();  // the marks have been read
        each([&](int r, int k) {
            const int c = c0 + k;
            const int32_t a = s_e[k * pitch + r], n = s_need[r], need = n & 0x7FFFFFFF;
            int32_t b = wants(r, c, k);
            // the marks go: a freed page is held by no one, a kept one by its row
            if (a >= 0 && a != b && __ldcg(&p.shares[a]) == free_mark(r)) p.shares[a] = 0;
            if (prefix && need > 0) {
                const int lead = s_lead[s_start[r]] & (kTwo - 1);
                const int32_t m = s_need[lead], full = (m & 0x7FFFFFFF) - (m < 0 ? 1 : 0);
                if (c < full) {
                    const int32_t l = wants(lead, c, k);
                    if ((b != l || l < 0) && c * p.page_size < __ldcg(&p.prefix_lens[lead]))
                        atomicMin(&p.prefix_lens[lead], c * p.page_size);
                }
            }
            if (c >= need) return;
            if (n < 0 && c == need - 1) {
                b = s_e[k * pitch + s_parent[r]];
                if (b >= 0) {
                    if (__ldcg(&p.shares[b]) == keep_mark(r)) p.shares[b] = 0;
                    else b = -1;  // a fresh page comes here at the end
                }
            }
            if (b != a || b < 0 || c >= s_owned[r]) p.tables[r * p.table_stride + c] = b;
        });
        __syncthreads();
    }
    if (rank == ranks - 1) {
        // fresh pages in row order, and what is one per row
        int32_t given = 0;
        for (int r0 = 0; r0 < R; r0 += kForkThreads) {
            const int r = r0 + tid;
            const bool want = r < R && __ldcg(&p.dst[r]) == -2;
            const uint32_t hit = __ballot_sync(~0u, want);
            if (lane == 0) s_warp[warp] = __popc(hit);
            __syncthreads();
            int32_t at = given;
            for (int i = 0; i < W; ++i) {
                if (i < warp) at += s_warp[i];
                given += s_warp[i];
            }
            __syncthreads();
            if (r < R) {
                const int32_t n = s_need[r], need = n & 0x7FFFFFFF;
                int32_t len = need * p.page_size, rows = 0;
                if (n < 0) {
                    const int32_t l = p.lens[r];  // not clamped: a clamped length has whole pages
                    rows = l - (need - 1) * p.page_size;
                    len = l;
                }
                if (want) {
                    at += __popc(hit & ((1u << lane) - 1u));
                    const bool has = at < avail;
                    int32_t page = has ? p.ring[ring_at(head_at, at, p.ring_size)] : -1;
                    if (page < 0 || page >= p.num_pages) page = -1, flags |= kStatusKvPages;
                    p.dst[r] = page;
                    if (page < 0) p.src[r] = -1;
                    p.rows[r] = page < 0 ? 0 : rows;
                } else {
                    p.rows[r] = 0;
                }
                p.owned[r] = need;
                if (p.lens_out) p.lens_out[r] = len;
            }
        }
        __syncthreads();
        if (tid == 0) {
            if (given > avail || all > room) flags |= kStatusKvPages;
            p.state[0] = head + min(given, avail);
            p.state[1] = tail + min(all, room);
        }
    }
    cluster_sync();
    // nobody reads the old entries any more
    for (int r = rank * kForkThreads + tid; r < R; r += ranks * kForkThreads) {
        const int32_t n = s_need[r], need = n & 0x7FFFFFFF;
        if (n < 0) {
            const int32_t page = __ldcg(&p.dst[r]);
            if (page >= 0) p.tables[r * p.table_stride + need - 1] = page;
        }
        if (prefix) {
            const int32_t l = s_lead[s_start[r]], lead = l & (kTwo - 1);
            p.prefix_lens[r] = need > 0 && (l & kTwo) ? __ldcg(&p.prefix_lens[lead]) : 0;
        }
    }
    if (flags) atomicOr(p.status, flags);
}

}  // namespace dev
}  // namespace w12
