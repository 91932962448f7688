// Paged-cache attention behind shared prefixes: the kernels for heads of 64 columns.
#include "kv_launch.cuh"

namespace w12 {
namespace launch {

template <>
int shared_dim<64>(const DeviceView &d, bool q8, int rows, dev::KvSpans kind, int *resident,
                    const dev::KvSharedParams *p, const CUtensorMap *tm_k, const CUtensorMap *tm_v, int ctas,
                    void *stream, std::string *err) {
    const auto run = kind == dev::kKvAllSpans ? q8 ? &shared_kind<64, true, dev::kKvAllSpans>
                                                   : &shared_kind<64, false, dev::kKvAllSpans>
                     : kind == dev::kKvPrefixes ? q8 ? &shared_kind<64, true, dev::kKvPrefixes>
                                                     : &shared_kind<64, false, dev::kKvPrefixes>
                     : q8                       ? &shared_kind<64, true, dev::kKvOwnSpans>
                                                : &shared_kind<64, false, dev::kKvOwnSpans>;
    return run(d, rows, resident, p, tm_k, tm_v, ctas, stream, err);
}

}  // namespace launch
}  // namespace w12
