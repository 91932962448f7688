// Host launcher of w12_beam_select (checks are in capi.cpp).
#include <algorithm>

#include "beam.cuh"
#include "kv_launch.cuh"

namespace w12 {
namespace launch {

namespace {

struct BeamPlan {
    int32_t parts = 1, part = 0, keep = 0;
    size_t off_stats = 0, off_entries = 0, bytes = 0;
};

BeamPlan beam_plan(const DeviceView &d, const w12_beam_args &a) {
    BeamPlan plan;
    const int64_t rows = (int64_t)a.requests * a.beams;
    // As many parts as fill the device once, of a tile (16 KB) or more: one threshold serves all
    // tiles of a part, and a CTA's start costs more than another tile.  Half tiles, twice the
    // CTAs: 16 x 8 rows of 151936 BF16 logits 22.3 us against 21.3, 4 rows 10.3 against 10.0.
    const int64_t fill = (int64_t)d.sm_count * dev::kBeamCtas;
    const int32_t tile = dev::kBeamThreads * (a.dtype == W12_BEAM_BF16 ? 32 : 16);
    const int32_t most = (a.vocab + tile - 1) / tile;
    const int32_t parts = (int32_t)std::max<int64_t>((most + dev::kBeamTiles - 1) / dev::kBeamTiles,
                                                     std::min<int64_t>(most, fill / rows));
    plan.part = ((a.vocab + parts - 1) / parts + 31) / 32 * 32;
    plan.parts = (a.vocab + plan.part - 1) / plan.part;
    // as many as may end, and the beams behind them
    plan.keep = std::max(a.take, a.eos >= 0 ? 2 * a.beams : a.beams);
    const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    plan.off_stats = up((size_t)a.requests * sizeof(uint32_t));
    plan.off_entries = plan.off_stats + up((size_t)rows * plan.parts * sizeof(dev::BeamStat));
    plan.bytes = plan.off_entries + up((size_t)rows * plan.parts * plan.keep * sizeof(dev::BeamEntry));
    return plan;
}

}  // namespace

int beam_workspace_size(const w12_beam_args &a, size_t *bytes, std::string *err) {
    DeviceView d;
    const int rc = device_view(&d, err);
    if (rc == W12_OK) *bytes = beam_plan(d, a).bytes;
    return rc;
}

int beam_select(const w12_beam_args &a, void *workspace, size_t ws_bytes, void *stream, std::string *err) {
    DeviceView d;
    const int rc = device_view(&d, err);
    if (rc != W12_OK) return rc;
    const BeamPlan plan = beam_plan(d, a);
    if (ws_bytes < plan.bytes) {
        *err = "workspace smaller than w12_beam_workspace_size";
        return W12_ERR_BUFFER_TOO_SMALL;
    }
    const int64_t ctas = (int64_t)a.requests * a.beams * plan.parts;
    if (ctas > 0x7FFFFFFF) {
        *err = "too many rows";
        return W12_ERR_SHAPE;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    static constexpr dev::BeamLog logs;
    dev::BeamParams p;
    p.logs = logs;
    p.logits = a.logits;
    p.stride = a.logits_stride;
    p.allowed = a.allowed;
    p.allowed_stride = a.allowed_stride;
    p.scores_in = a.scores_in;
    p.scores = a.scores;
    p.tokens = a.tokens;
    p.parents = a.parents;
    p.cand_tokens = a.cand_tokens;
    p.cand_parents = a.cand_parents;
    p.cand_scores = a.cand_scores;
    p.counters = reinterpret_cast<uint32_t *>(ws);
    p.stats = reinterpret_cast<dev::BeamStat *>(ws + plan.off_stats);
    p.entries = reinterpret_cast<dev::BeamEntry *>(ws + plan.off_entries);
    p.requests = a.requests;
    p.beams = a.beams;
    p.vocab = a.vocab;
    p.take = a.take;
    p.keep = plan.keep;
    p.eos = a.eos;
    p.parts = plan.parts;
    p.part = plan.part;
    const uint64_t per_row = (uint64_t)plan.parts * plan.keep;
    p.per_row_inv = (uint32_t)(((uint64_t(1) << 32) + per_row - 1) / per_row);
    const int smem = (int)sizeof(dev::BeamShared) + a.beams * plan.parts;
    const auto kernel = a.dtype == W12_BEAM_BF16 ? &dev::w12_beam_select_kernel<true, 32>
                                                 : &dev::w12_beam_select_kernel<false, 16>;
    const cudaError_t e = kv_launch(d, kernel, dim3((unsigned)ctas), dev::kBeamThreads, smem, 1, stream, p);
    if (e != cudaSuccess) return kv_cuda_fail(e, "w12_beam_select launch", err);
    return W12_OK;
}

}  // namespace launch
}  // namespace w12
