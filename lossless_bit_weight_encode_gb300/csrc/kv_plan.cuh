// Page tables, positions and slots of one step (w12_kv_plan in include/w12.h).
//
// Per request: need = ceil((len + new) / page), grow = max(need - owned, 0),
// drop = max(owned - need, 0) with trim.  Three prefix sums over the requests
// (new tokens, grow, drop) place every token, every page taken and every page
// given back; each of the three lists is then walked flat, one element per
// thread, its request found by a binary search in the prefix sums, so that one
// long prompt among short ones costs no more than the same tokens spread out.
//
// The call is latency: it moves 20 bytes per request and 12 per token (at the HBM
// rate 0.06 us of the 7.0 us that 1024 requests with 32768 new tokens take; one request
// with one token takes 3.2, an empty kernel 2).  What is left is the chain: lengths,
// prefix sums, search, ring or table entry, store.  One cluster of CTAs (one CTA
// where its threads have at most two tokens each) computes the sums redundantly and
// shares the lists, so that there is one launch and nothing in memory between; its
// barrier is what allows owned and the ring state to be updated in place.  No
// CTA reads what another writes: a taken page is read from the ring, never from
// the table entry it goes to, and the ring positions given back are not those
// taken (only as many go back as entries of the ring were not free at the start; the
// pages without room stay where they are, the last of each request going back first).
#pragma once

#include "kv_common.cuh"
#include "w12_device.cuh"

namespace w12 {
namespace dev {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int32_t clamp_i32(int64_t v, int64_t lo, int64_t hi) {
    return (int32_t)(v < lo ? lo : v > hi ? hi : v);
}

// Largest i in [0, n) with start[i] <= v (start[0] <= v holds).  Requests with
// nothing share their successor's start, so the largest one is the owner.
__device__ __forceinline__ int find_start(const int32_t *start, int n, int32_t v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Entry (base + i) of the ring, base < size (more than size entries on: only for an
// inconsistent ring state).
__device__ __forceinline__ int32_t ring_at(int32_t base, int32_t i, int32_t size) {
    uint32_t x = (uint32_t)base + (uint32_t)i;
    if (x >= (uint32_t)size) x -= (uint32_t)size;
    if (x >= (uint32_t)size) x %= (uint32_t)size;
    return (int32_t)x;
}

// v mod size for v >= 0, with inv = floor((2^64 - 1) / size): the high product is the
// quotient or one less.
__device__ __forceinline__ int32_t ring_base(int64_t v, int32_t size, uint64_t inv) {
    const uint64_t u = v < 0 ? 0 : (uint64_t)v;
    const int64_t r = (int64_t)(u - __umul64hi(u, inv) * (uint64_t)size);
    return (int32_t)(r >= size ? r - size : r);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanThreads, 1) w12_kv_plan_kernel(KvPlanParams p) {
    // prefix sums of the chunk's requests: all fit 32 bits (the tables have fewer than
    // 2^31 entries), but for the tokens, which are cut there
    __shared__ int32_t s_tok[kPlanThreads], s_grow[kPlanThreads], s_drop[kPlanThreads];
    __shared__ int32_t s_len[kPlanThreads], s_owned[kPlanThreads], s_need[kPlanThreads];
    __shared__ int64_t s_wtok[32];
    __shared__ int32_t s_wgrow[32], s_wdrop[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int32_t first = (int32_t)rank * kPlanThreads + tid, step = (int32_t)ranks * kPlanThreads;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t head = p.state_in[0], tail = p.state_in[1];
    const int32_t avail = clamp_i32(tail - head, 0, p.ring_size), room = p.ring_size - avail;
    const int32_t head_at = ring_base(head, p.ring_size, p.ring_inv);
    const int32_t tail_at = ring_base(tail, p.ring_size, p.ring_inv);
    const int32_t cap = p.max_blocks * p.page_size;
    int64_t tok0 = 0;
    int32_t grow0 = 0, drop0 = 0;  // totals of the chunks before
    uint32_t flags = tail - head != avail ? kStatusKvPages : 0;
    for (int64_t base = 0; base < p.requests; base += kPlanThreads) {
        const int n = (int)min((int64_t)kPlanThreads, p.requests - base);
        int32_t len = 0, add = 0, owned = 0, need = 0;
        if (tid < n) {
            const int32_t l = p.lens[base + tid], a = p.new_lens[base + tid], o = p.owned_in[base + tid];
            len = min(max(l, 0), cap);
            add = min(max(a, 0), cap - len);
            owned = min(max(o, 0), p.max_blocks);
            if (len != l || add != max(a, 0) || owned != o) flags |= kStatusKvSizes;
            need = (int32_t)(((int64_t)len + add + p.page_size - 1) / p.page_size);
        }
        const int32_t grow = max(need - owned, 0), drop = p.trim ? max(owned - need, 0) : 0;
        int64_t a = add;  // inclusive sums
        int32_t b = grow, c = drop;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(~0u, a, d);
            const int32_t y = __shfl_up_sync(~0u, b, d), z = __shfl_up_sync(~0u, c, d);
            if (lane >= d) a += x, b += y, c += z;
        }
        if (lane == 31) s_wtok[warp] = a, s_wgrow[warp] = b, s_wdrop[warp] = c;
        __syncthreads();
        if (warp == 0) {
            int64_t x = s_wtok[lane];
            int32_t y = s_wgrow[lane], z = s_wdrop[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t u = __shfl_up_sync(~0u, x, d);
                const int32_t v = __shfl_up_sync(~0u, y, d), w = __shfl_up_sync(~0u, z, d);
                if (lane >= d) x += u, y += v, z += w;
            }
            s_wtok[lane] = x, s_wgrow[lane] = y, s_wdrop[lane] = z;
        }
        __syncthreads();
        if (warp > 0) a += s_wtok[warp - 1], b += s_wgrow[warp - 1], c += s_wdrop[warp - 1];
        const int64_t tok_n = s_wtok[31];
        const int32_t grow_n = s_wgrow[31], drop_n = s_wdrop[31];
        s_tok[tid] = (int32_t)min(tok0 + a - add, (int64_t)0x7FFFFFFF);
        s_grow[tid] = grow0 + b - grow;
        s_drop[tid] = drop0 + c - drop;
        s_len[tid] = len;
        s_owned[tid] = owned;
        s_need[tid] = need;
        const int32_t given = min(grow, max(avail - (grow0 + b - grow), 0));
        const int32_t back = min(drop, max(room - (drop0 + c - drop), 0));
        if (given < grow || back < drop) flags |= kStatusKvPages;
        // every CTA has read its inputs of this chunk before any output of it
        // is written (owned_out may be owned_in)
        if (ranks > 1) cluster_sync();
        else __syncthreads();
        if (rank == 0 && tid < n) {
            p.owned_out[base + tid] = owned + given - back;
            if (base + tid == 0) p.cu_new[0] = 0;
            p.cu_new[base + tid + 1] = (int32_t)min(tok0 + a, (int64_t)0x7FFFFFFF);
        }
        // tokens
        const int32_t tok_end = (int32_t)min(tok0 + tok_n, (int64_t)p.tokens);
        for (int64_t t = tok0 + first; t < tok_end; t += step) {
            const int r = find_start(s_tok, n, (int32_t)t);
            const int32_t pos = s_len[r] + (int32_t)t - s_tok[r], j = pos / p.page_size;
            int32_t page = -1;
            if (j < s_owned[r]) {
                page = p.tables[(base + r) * p.table_stride + j];
            } else {
                const int32_t at = s_grow[r] + j - s_owned[r];
                if (at < avail) page = p.ring[ring_at(head_at, at, p.ring_size)];
            }
            p.positions[t] = pos;
            p.slots[t] = page < 0 ? -1 : (int64_t)page * p.page_size + (pos - j * p.page_size);
        }
        // pages taken (or missing) and pages given back (counted without a sign: a step
        // past close to 2^31 of them must not wrap)
        for (uint32_t i = first; i < (uint32_t)grow_n; i += step) {
            const int32_t g = grow0 + (int32_t)i;
            const int r = find_start(s_grow, n, g);
            const int32_t j = s_owned[r] + g - s_grow[r];
            p.tables[(base + r) * p.table_stride + j] =
                g < avail ? p.ring[ring_at(head_at, g, p.ring_size)] : -1;
        }
        const int32_t back_n = min(drop_n, max(room - drop0, 0));
        for (uint32_t i = first; i < (uint32_t)back_n; i += step) {
            const int32_t g = drop0 + (int32_t)i;
            const int r = find_start(s_drop, n, g);
            // the last min(drop, room left) of the request's pages, in table order
            const int32_t left = room - s_drop[r], j = max(s_need[r], s_owned[r] - left) + g - s_drop[r];
            p.ring[ring_at(tail_at, g, p.ring_size)] = p.tables[(base + r) * p.table_stride + j];
        }
        tok0 += tok_n;
        grow0 += grow_n;
        drop0 += drop_n;
        __syncthreads();  // the shared arrays are free for the next chunk
    }
    for (int64_t t = tok0 + first; t < p.tokens; t += step) {
        p.positions[t] = 0;
        p.slots[t] = -1;
    }
    if (tok0 > p.tokens) flags |= kStatusKvSizes;
    if (rank == 0 && tid == 0) {
        // (at least one request:) every CTA has passed a chunk's cluster barrier,
        // so it has read the state
        p.state_out[0] = head + min(grow0, avail);
        p.state_out[1] = tail + min(drop0, room);
    }
    if (flags && rank == 0) atomicOr(p.status, flags);
}

}  // namespace dev
}  // namespace w12
