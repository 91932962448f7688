// Host launchers of the paged key-value cache calls (checks are in capi.cpp).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "kv_launch.cuh"
#include "kv_plan.cuh"
#include "kv_store.cuh"

namespace w12 {
namespace launch {

template <>
int attend_dim<64>(const DeviceView &, bool, int, int *, const dev::KvAttendParams *, const CUtensorMap *,
                   const CUtensorMap *, int, void *, std::string *);
template <>
int attend_dim<128>(const DeviceView &, bool, int, int *, const dev::KvAttendParams *, const CUtensorMap *,
                    const CUtensorMap *, int, void *, std::string *);
template <>
int attend_dim<256>(const DeviceView &, bool, int, int *, const dev::KvAttendParams *, const CUtensorMap *,
                    const CUtensorMap *, int, void *, std::string *);

namespace {

dev::KvGeom geometry(const w12_kv_cache &c) {
    dev::KvGeom g;
    g.k = static_cast<uint8_t *>(c.k_dev);
    g.v = static_cast<uint8_t *>(c.v_dev);
    g.scales = c.scales_dev;
    g.num_pages = c.num_pages;
    g.page_stride = c.page_stride;
    g.head_stride = c.head_stride;
    g.row_stride = c.row_stride;
    g.page_inv = ~uint64_t(0) / (uint64_t)c.page_size;
    g.page_size = c.page_size;
    g.kv_heads = c.kv_heads;
    return g;
}

template <int D>
cudaError_t store_dim(const DeviceView &d, bool q8, bool inter, dim3 grid, const dev::KvStoreParams &p, void *st) {
    const auto kernel = q8      ? inter ? &dev::w12_kv_store_kernel<D, true, true>
                                        : &dev::w12_kv_store_kernel<D, true, false>
                        : inter ? &dev::w12_kv_store_kernel<D, false, true>
                                : &dev::w12_kv_store_kernel<D, false, false>;
    return kv_launch(d, kernel, grid, dev::kStoreThreads, 0, 1, st, p);
}

template <int D>
cudaError_t read_dim(const DeviceView &d, bool q8, int grid, const dev::KvReadParams &p, void *st) {
    const auto kernel = q8 ? &dev::w12_kv_read_kernel<D, true> : &dev::w12_kv_read_kernel<D, false>;
    return kv_launch(d, kernel, dim3((unsigned)grid), dev::kReadThreads, 0, 1, st, p);
}

// Held over the launches of an attend call: the joining kernel reads what the attention
// kernel before it left in the workspace, so nothing of another host thread's call with
// the same workspace may come between the two.  One lock for a few workspaces (by
// address), so that threads with workspaces of their own seldom meet.
std::mutex &workspace_lock(const void *workspace) {
    static std::mutex locks[64];
    const uint64_t at = reinterpret_cast<uintptr_t>(workspace) >> 8;
    return locks[(at ^ at >> 6 ^ at >> 12) % 64];
}

int attend_call(const DeviceView &d, const w12_kv_cache &c, int rows, int *resident, const dev::KvAttendParams *p,
                const CUtensorMap *tm_k, const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    const bool q8 = c.dtype == W12_KV_Q8;
    switch (c.head_dim) {
    case 64: return attend_dim<64>(d, q8, rows, resident, p, tm_k, tm_v, ctas, stream, err);
    case 128: return attend_dim<128>(d, q8, rows, resident, p, tm_k, tm_v, ctas, stream, err);
    default: return attend_dim<256>(d, q8, rows, resident, p, tm_k, tm_v, ctas, stream, err);
    }
}

// How long an attend kernel's waits may go on, counted from its start: the option's
// limit, which is far above any decoding step, and the time that the call's operations
// would take at 4 TFLOP/s (blocks of eight rows over heads of 64, among the slowest, do
// 55), for a long prompt in one call may rightly take many seconds.  The keys are bounded by the
// tables' width.  (A limit from each wait's own start costs the loops registers: three
// tokens on windows of an 8-bit cache 173 us, 186.)
uint64_t attend_timeout_ns(const DeviceView &d, const w12_kv_cache &c, const w12_kv_attend_args &a) {
    const double flops = 4.0 * a.heads * c.head_dim * a.tokens * ((double)a.max_blocks * c.page_size);
    return d.timeout_ns + (uint64_t)std::min(flops / 4e3, 600e9);  // 4e3 per ns; ten minutes at most
}

int attend_plan(const DeviceView &d, const w12_kv_cache &c, const w12_kv_attend_args &a, AttendPlan *plan,
                std::string *err) {
    const int group = a.heads / c.kv_heads;
    plan->rows = attend_rows(a.max_new, group, c.kv_heads, a.requests, c.dtype == W12_KV_Q8, d.sm_count);
    int resident = 0;
    const int rc = attend_call(d, c, plan->rows, &resident, nullptr, nullptr, nullptr, 0, nullptr, err);
    if (rc != W12_OK) return rc;
    // no more CTAs than units can exist: row blocks times tiles of the longest request
    const int64_t blocks = a.requests + (int64_t)a.tokens * group / plan->rows;
    const int64_t tiles = ((int64_t)a.max_blocks * c.page_size + dev::kAttendTile - 1) / dev::kAttendTile;
    plan->ctas = (int)std::min<int64_t>(resident, std::max<int64_t>(1, blocks * c.kv_heads * tiles));
    const int64_t counters = (blocks + 1) * c.kv_heads;
    if (counters > 0x7FFFFFFF) {
        *err = "too many row blocks";
        return W12_ERR_SHAPE;
    }
    plan->n_counters = (uint32_t)counters;
    // kPartElems per SM and two pieces per CTA; (max, sum) pairs: per row, so at
    // most kPartElems / 64 per SM
    plan->off_ml = (size_t)2 * d.sm_count * kPartElems * sizeof(float);
    plan->off_counters = plan->off_ml + (size_t)2 * d.sm_count * (kPartElems / 64) * sizeof(float2);
    plan->bytes = plan->off_counters + (size_t)counters * sizeof(uint32_t);
    return W12_OK;
}

// [pages][kv_heads][page_size][head_dim] as (16-byte-chunked row, token, 128-byte
// block of the row, head, page): a box is 16 tokens of one head, its 128-byte
// blocks one after the other, each swizzled for ldmatrix.
// The tcgen05 kernel (`tc`) takes its boxes as [pages][kv_heads][page_size][head_dim]:
// 16 tokens x 64 BF16 columns, swizzled as its operands are, or 16 tokens x all
// columns in bytes.
int cache_map(const w12_kv_cache &c, bool tc, const void *base, CUtensorMap *tm, std::string *err) {
    auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode(err));
    if (!encode) return W12_ERR_CUDA;
    const bool q8 = c.dtype == W12_KV_Q8;
    const cuuint64_t elem = q8 ? 1 : 2;
    if (tc) {
        const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                                    (cuuint64_t)c.num_pages};
        const cuuint64_t strides[3] = {(cuuint64_t)c.row_stride * elem, (cuuint64_t)c.head_stride * elem,
                                       (cuuint64_t)c.page_stride * elem};
        const cuuint32_t box[4] = {q8 ? (cuuint32_t)c.head_dim : 64u, (cuuint32_t)dev::kAttendSlice, 1, 1};
        const cuuint32_t unit[4] = {1, 1, 1, 1};
        const CUresult r = encode(tm, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                                  const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r == CUDA_SUCCESS) return W12_OK;
        *err = "cuTensorMapEncodeTiled failed for the cache (code " + std::to_string((int)r) + ")";
        return W12_ERR_CUDA;
    }
    const cuuint64_t row = std::min<cuuint64_t>(128, c.head_dim * elem);
    const cuuint64_t dims[5] = {row / elem, (cuuint64_t)c.page_size, (cuuint64_t)c.head_dim * elem / row,
                                (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)c.row_stride * elem, row, (cuuint64_t)c.head_stride * elem,
                                   (cuuint64_t)c.page_stride * elem};
    const cuuint32_t box[5] = {(cuuint32_t)(row / elem), (cuuint32_t)dev::kAttendSlice, (cuuint32_t)dims[2], 1, 1};
    const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(tm, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                              const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = "cuTensorMapEncodeTiled failed for the cache (code " + std::to_string((int)r) + ")";
        return W12_ERR_CUDA;
    }
    return W12_OK;
}

}  // namespace

int kv_plan(const w12_kv_plan_args &a, void *stream, std::string *err) {
    DeviceView d;
    const int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    dev::KvPlanParams p;
    p.lens = a.lens;
    p.new_lens = a.new_lens;
    p.owned_in = a.owned_in;
    p.owned_out = a.owned_out;
    p.tables = a.tables;
    p.table_stride = a.table_stride;
    p.ring = a.ring;
    p.state_in = a.ring_state_in;
    p.state_out = a.ring_state_out;
    p.cu_new = a.cu_new;
    p.positions = a.positions;
    p.slots = a.slots;
    p.requests = a.requests;
    p.max_blocks = a.max_blocks;
    p.page_size = a.page_size;
    p.ring_size = a.ring_size;
    p.ring_inv = ~uint64_t(0) / (uint64_t)a.ring_size;
    p.tokens = a.tokens;
    p.trim = a.trim != 0;
    p.status = d.status;
    // One CTA while it has at most two tokens per thread; else a cluster of 16 (more
    // than the portable 8: the call is bound by its instructions on the few SMs it
    // has: 1024 requests with 32768 token slots 6.8 us, 8.9 with 8; one request on
    // one CTA 3.2 us).
    const int cluster = a.tokens > 2 * dev::kPlanThreads || a.requests > dev::kPlanThreads ? 16 : 1;
    static std::mutex mu;
    static bool set[kKvMaxDevices] = {};
    cudaError_t e = cudaSuccess;
    if (cluster > 8 && d.device >= 0 && d.device < kKvMaxDevices) {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[d.device])
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&dev::w12_kv_plan_kernel),
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_plan set-up", err);
        set[d.device] = true;
    }
    e = kv_launch(d, &dev::w12_kv_plan_kernel, dim3((unsigned)cluster), dev::kPlanThreads, 0, cluster, stream, p);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_plan launch", err);
    return W12_OK;
}

int kv_store(const w12_kv_cache &c, const w12_kv_store_args &a, void *stream, std::string *err) {
    DeviceView d;
    const int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    if (a.tokens == 0) return W12_OK;
    dev::KvStoreParams p;
    p.c = geometry(c);
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.q_out = a.q_out;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_out_stride = a.q_out_stride;
    p.q_norm = a.q_norm;
    p.k_norm = a.k_norm;
    p.rope = a.rope;
    p.positions = a.positions;
    p.slots = a.slots;
    p.rope_rows = a.rope_rows;
    p.tokens = a.tokens;
    p.heads = a.heads;
    p.rot = a.rot;
    p.eps = a.eps;
    p.status = d.status;
    const int per = 256 / c.head_dim, groups = dev::kStoreThreads / 32;  // heads of a warp's round, warps
    const int all = (a.heads + per - 1) / per + 2 * ((c.kv_heads + per - 1) / per);
    // few tokens: a warp per round; many: as few CTAs per token as fill the device
    const int want = (all + groups - 1) / groups;
    const int64_t fill = (int64_t)d.sm_count * 16;
    const int gx = (int)std::max<int64_t>(1, std::min<int64_t>(want, fill / a.tokens));
    const dim3 grid((unsigned)gx, (unsigned)std::min<int64_t>(a.tokens, 65535));
    const bool q8 = c.dtype == W12_KV_Q8, inter = a.interleaved != 0;
    const cudaError_t e = c.head_dim == 64    ? store_dim<64>(d, q8, inter, grid, p, stream)
                          : c.head_dim == 128 ? store_dim<128>(d, q8, inter, grid, p, stream)
                                              : store_dim<256>(d, q8, inter, grid, p, stream);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_store launch", err);
    return W12_OK;
}

int kv_read(const w12_kv_cache &c, const int64_t *slots, int32_t tokens, uint16_t *k_out, uint16_t *v_out,
            void *stream, std::string *err) {
    DeviceView d;
    const int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    if (tokens == 0) return W12_OK;
    dev::KvReadParams p;
    p.c = geometry(c);
    p.slots = slots;
    p.k_out = k_out;
    p.v_out = v_out;
    p.tokens = tokens;
    p.status = d.status;
    const int per = 256 / c.head_dim, rounds = (c.kv_heads + per - 1) / per, warps = dev::kReadThreads / 32;
    p.rounds_inv = ~uint64_t(0) / (uint64_t)rounds;
    const int64_t items = (int64_t)tokens * rounds;
    const int grid = (int)std::min<int64_t>((items + warps - 1) / warps, (int64_t)d.sm_count * 32);
    const bool q8 = c.dtype == W12_KV_Q8;
    const cudaError_t e = c.head_dim == 64    ? read_dim<64>(d, q8, grid, p, stream)
                          : c.head_dim == 128 ? read_dim<128>(d, q8, grid, p, stream)
                                              : read_dim<256>(d, q8, grid, p, stream);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_read launch", err);
    return W12_OK;
}

int kv_attend_workspace_size(const w12_kv_cache &c, const w12_kv_attend_args &a, size_t *bytes, std::string *err) {
    DeviceView d;
    int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    AttendPlan plan;
    rc = attend_plan(d, c, a, &plan, err);
    if (rc == W12_OK) *bytes = plan.bytes;
    return rc;
}

int kv_attend(const w12_kv_cache &c, const w12_kv_attend_args &a, void *workspace, size_t ws_bytes, void *stream,
              std::string *err) {
    DeviceView d;
    int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    AttendPlan plan;
    rc = attend_plan(d, c, a, &plan, err);
    if (rc != W12_OK) return rc;
    if (ws_bytes < plan.bytes) {
        *err = "workspace smaller than w12_kv_attend_workspace_size";
        return W12_ERR_BUFFER_TOO_SMALL;
    }
    CUtensorMap tm_k, tm_v;
    const bool tc = plan.rows == dev::kTcRows;
    rc = cache_map(c, tc, c.k_dev, &tm_k, err);
    if (rc == W12_OK) rc = cache_map(c, tc, c.v_dev, &tm_v, err);
    if (rc != W12_OK) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    dev::KvAttendParams p;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.tables = a.tables;
    p.table_stride = a.table_stride;
    p.lens = a.lens;
    p.cu_new = a.cu_new;
    p.tree = a.tree;
    p.positions = a.tree && a.window > 0 ? a.positions : nullptr;
    p.v = static_cast<const uint16_t *>(c.v_dev);
    p.v_page_stride = c.page_stride;
    p.v_head_stride = c.head_stride;
    p.v_row_stride = c.row_stride;
    p.scales = c.scales_dev;
    p.num_pages = c.num_pages;
    p.requests = a.requests;
    p.max_keys = a.max_blocks * c.page_size;
    p.tokens = a.tokens;
    p.kv_heads = c.kv_heads;
    p.group = a.heads / c.kv_heads;
    p.window = a.window;
    p.page_size = c.page_size;
    p.scale_log2 = a.scale * 1.44269504088896340736f;
    p.counters = reinterpret_cast<uint32_t *>(ws + plan.off_counters);
    p.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
    p.part = reinterpret_cast<float *>(ws);
    p.n_counters = plan.n_counters;
    p.join_later = join_warps(plan.rows, p.group, c.kv_heads, a.max_new, a.requests, plan.ctas);
    p.status = d.status;
    p.timeout_ns = attend_timeout_ns(d, c, a);
    int resident = 0;
    const std::lock_guard<std::mutex> lock(workspace_lock(workspace));
    return attend_call(d, c, plan.rows, &resident, &p, &tm_k, &tm_v, plan.ctas, stream, err);
}

}  // namespace launch
}  // namespace w12
