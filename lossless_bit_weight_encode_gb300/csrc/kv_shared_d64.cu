// Paged-cache attention behind shared prefixes: the kernels for heads of 64 columns.
#include "kv_launch.cuh"

namespace w12 {
namespace launch {

template <>
int shared_dim<64>(const DeviceView &d, bool q8, int rows, int *resident, const dev::KvPrefixParams *p, const CUtensorMap *tm_k,
                   const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    return q8 ? attend_rows_variant<64, true>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err)
              : attend_rows_variant<64, false>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err);
}

template <>
int shared_dim<64>(const DeviceView &d, bool q8, int rows, int *resident, const dev::KvOwnParams *p, const CUtensorMap *tm_k,
                   const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    return q8 ? attend_rows_variant<64, true>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err)
              : attend_rows_variant<64, false>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err);
}

}  // namespace launch
}  // namespace w12
