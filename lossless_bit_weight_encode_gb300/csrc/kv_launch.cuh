// Launch helpers of the paged-cache kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <string>
#include <utility>

#include "kv_attend.cuh"
#include "kv_attend_tc.cuh"
#include "kv_tiles.hpp"
#include "w12.h"
#include "w12_launch.hpp"

namespace w12 {
namespace launch {

inline int kv_cuda_fail(cudaError_t e, const char *what, std::string *err) {
    *err = std::string(what) + ": " + cudaGetErrorString(e);
    return W12_ERR_CUDA;
}

// Launch that may start while the kernel before it finishes (the kernels wait
// with griddepcontrol.wait before they touch memory); cluster > 1: a cluster of
// that many CTAs.
template <class... KArgs, class... Args>
cudaError_t kv_launch(const DeviceView &d, void (*kernel)(KArgs...), dim3 grid, int threads, int smem, int cluster,
                      void *stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (d.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

constexpr int kKvMaxDevices = 64;

// Workspace: the partial outputs, their maxima and sums, the counters.  The
// first two have the same size in every plan of a device (kPartElems bounds rows x
// head_dim x CTAs per SM), so that the counters lie at one place and calls of
// different shapes can share a workspace: what one leaves zero is what another
// finds.
constexpr int kPartElems = 128 * 256;
struct AttendPlan {
    int rows = 8, ctas = 1;
    size_t off_ml = 0, off_counters = 0, bytes = 0;
    uint32_t n_counters = 0;
};

// Whether the parts of a row block that several CTAs share are joined by a second
// kernel (a CTA per output row) or by the CTA that arrives last.  With two parts
// per row block or more (few requests, as far as the host knows) the chain through
// the last CTA is the longer way: one request of 777 tokens 7.4 against 10.4 us, two
// of 100001 116 against 121; with fewer, most rows have one part and the second
// kernel only costs: 128 requests of 1024 visible tokens 74 against 56 us.
// Returns the warps per row of the second kernel, 0: none.
inline int join_warps(int rows, int group, int kv_heads, int max_new, int requests, int ctas) {
    const int64_t blocks = ((int64_t)(max_new < 1 ? 1 : max_new) * group + rows - 1) / rows * kv_heads * requests;
    return ctas >= 16 * blocks ? 8 : ctas >= 2 * blocks || rows == dev::kTcRows ? 1 : 0;
}

// The second kernel, for launches of `rows`-row blocks.  A warp per row where a row
// has up to 16 parts or so (16-token trees, 5 parts: 5 us against 19 with eight
// warps, a CTA per row); eight where it has more.
template <int D, int TILE, int WPR>
int join_launch(const DeviceView &d, int rows, const dev::KvAttendParams &p, int ctas, void *stream, std::string *err) {
    const auto kernel = rows == 8    ? &dev::w12_kv_join_kernel<D, 8, TILE, WPR>
                        : rows == 16 ? &dev::w12_kv_join_kernel<D, 16, TILE, WPR>
                                     : &dev::w12_kv_join_kernel<D, dev::kTcRows, dev::kAttendTile, WPR>;
    const int64_t out_rows = (int64_t)p.tokens * p.group * p.kv_heads, per = dev::kJoinThreads / 32 / WPR;
    const cudaError_t e = kv_launch(d, kernel, dim3((unsigned)((out_rows + per - 1) / per)), dev::kJoinThreads, 0, 1,
                                    stream, p, ctas);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_attend join launch", err);
    return W12_OK;
}

template <int D, bool Q8>
int join_parts(const DeviceView &d, int rows, const dev::KvAttendParams &p, int ctas, void *stream, std::string *err) {
    constexpr int TILE = dev::AttendTile<D, Q8>::kKeys;
    return p.join_later > 1 ? join_launch<D, TILE, 8>(d, rows, p, ctas, stream, err)
                            : join_launch<D, TILE, 1>(d, rows, p, ctas, stream, err);
}

// One head_dim's kernels (kv_attend_*.cu): CTAs resident on the whole device
// (with `p` null), or the launch.
template <int D>
int attend_dim(const DeviceView &d, bool q8, int rows, int *resident, const dev::KvAttendParams *p,
               const CUtensorMap *tm_k, const CUtensorMap *tm_v, int ctas, void *stream, std::string *err);

// Occupancy of one kernel on first use (at most `most` CTAs per SM), then (with `p`)
// its launch.  regs > 0: the registers per thread it has to have been compiled to.
template <class P>
int attend_kernel(const DeviceView &d, void (*kernel)(P, CUtensorMap, CUtensorMap), int most, int threads, int regs,
                  int smem, std::mutex &mu, int *per_sm, int *resident, const P *p, const CUtensorMap *tm_k,
                  const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    if (d.device < 0 || d.device >= kKvMaxDevices) {
        *err = "device ordinal out of range";
        return W12_ERR_CUDA;
    }
    {
        std::lock_guard<std::mutex> lock(mu);
        if (per_sm[d.device] == 0) {
            void *k = reinterpret_cast<void *>(kernel);
            cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_attend set-up", err);
            int occ = 0;
            const int rc = resident_ctas(k, threads, smem, d.device, err, &occ);
            if (rc != W12_OK) return rc;
            // a kernel whose warps exchange registers was made for so many of them; with
            // fewer, who takes some on would wait for ever
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, k);
            if (e != cudaSuccess) return kv_cuda_fail(e, "cudaFuncGetAttributes", err);
            if (regs > 0 && fa.numRegs != regs) {
                *err = "w12_kv_attend was compiled to another register count than it is made for";
                return W12_ERR_CUDA;
            }
            per_sm[d.device] = occ < most ? occ : most;
        }
        *resident = per_sm[d.device] * d.sm_count;
    }
    if (!p) return W12_OK;
    const cudaError_t e =
        kv_launch(d, kernel, dim3((unsigned)ctas), threads, smem, 1, stream, *p, *tm_k, *tm_v);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_kv_attend launch", err);
    return W12_OK;
}

template <int D, bool Q8, int WK, int WR, int NT, class P>
int attend_variant(const DeviceView &d, int *resident, const P *p, const CUtensorMap *tm_k,
                   const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    using C = dev::AttendCfg<D, Q8, WK, WR, NT>;
    static std::mutex mu;
    static int per_sm[kKvMaxDevices] = {};
    return attend_kernel(d, &dev::w12_kv_attend_kernel<D, Q8, WK, WR, NT, P>, kPartElems / (C::kRows * D),
                         dev::kAttendThreads, 0, C::kSmemBytes, mu, per_sm, resident, p, tm_k, tm_v, ctas, stream, err);
}

template <int D, bool Q8, bool PLACED, class P>
int attend_tc_variant(const DeviceView &d, int *resident, const P *p, const CUtensorMap *tm_k,
                      const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    using C = dev::AttendTcCfg<D, Q8, dev::kKvShared<P>>;
    static std::mutex mu;
    static int per_sm[kKvMaxDevices] = {};
    return attend_kernel(d, &dev::w12_kv_attend_tc_kernel<D, Q8, PLACED, P>,
                         std::min(kPartElems / (dev::kTcRows * D), 512 / C::kTmemCols), C::kThreads, C::kRegs,
                         C::kSmemBytes, mu, per_sm, resident, p, tm_k, tm_v, ctas, stream, err);
}

// The variants of one head_dim.  With 8 rows the warps split a tile's keys; so they
// do with 16, but for 256 columns, whose sums for 16 rows do not fit a warp: there
// they split the rows too.
template <int D, bool Q8, class P>
int attend_rows_variant(const DeviceView &d, int rows, int *resident, const P *p, const CUtensorMap *tm_k,
                        const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    switch (rows) {
    case 8: return attend_variant<D, Q8, 4, 1, 1>(d, resident, p, tm_k, tm_v, ctas, stream, err);
    case 16:
        return attend_variant<D, Q8, D == 256 ? 2 : 4, D == 256 ? 2 : 1, D == 256 ? 1 : 2>(d, resident, p, tm_k, tm_v,
                                                                                          ctas, stream, err);
    default:
        if constexpr (dev::kKvShared<P>)
            return attend_tc_variant<D, Q8, false>(d, resident, p, tm_k, tm_v, ctas, stream, err);
        else
            return p && p->positions
                       ? attend_tc_variant<D, Q8, true>(d, resident, p, tm_k, tm_v, ctas, stream, err)
                       : attend_tc_variant<D, Q8, false>(d, resident, p, tm_k, tm_v, ctas, stream, err);
    }
}

// The same for calls with shared prefixes (kv_shared_*.cu), over one kind of spans.
template <int D>
int shared_dim(const DeviceView &d, bool q8, int rows, dev::KvSpans kind, int *resident, const dev::KvSharedParams *p,
               const CUtensorMap *tm_k, const CUtensorMap *tm_v, int ctas, void *stream, std::string *err);

template <int D, bool Q8, dev::KvSpans KIND>
int shared_kind(const DeviceView &d, int rows, int *resident, const dev::KvSharedParams *p, const CUtensorMap *tm_k,
                const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    dev::KvSpanParams<KIND> spans;
    if (p) static_cast<dev::KvSharedParams &>(spans) = *p;
    const auto *q = p ? &spans : nullptr;
    if (shared_kernel_rows(KIND, Q8, rows) != rows) {
        *err = "w12_kv_attend_shared has no kernel for a launch of " + std::to_string(rows) + "-row tiles";
        return W12_ERR_CUDA;
    }
    if constexpr (KIND == dev::kKvAllSpans) {
        return attend_rows_variant<D, Q8>(d, rows, resident, q, tm_k, tm_v, ctas, stream, err);
    } else {
        if constexpr (shared_kernel_rows(KIND, Q8, dev::kTcRows) != 0)
            if (rows == dev::kTcRows)
                return attend_tc_variant<D, Q8, false>(d, resident, q, tm_k, tm_v, ctas, stream, err);
        if constexpr (shared_kernel_rows(KIND, Q8, 8) != 0)
            if (rows == 8) return attend_variant<D, Q8, 4, 1, 1>(d, resident, q, tm_k, tm_v, ctas, stream, err);
        if constexpr (shared_kernel_rows(KIND, Q8, 16) != 0)
            if (rows == 16)
                return attend_variant<D, Q8, D == 256 ? 2 : 4, D == 256 ? 2 : 1, D == 256 ? 1 : 2>(
                    d, resident, q, tm_k, tm_v, ctas, stream, err);
        return W12_ERR_CUDA;  // (not reached)
    }
}

}  // namespace launch
}  // namespace w12
