// Paged-cache attention kernels for heads of 64 columns.
#include "kv_launch.cuh"

namespace w12 {
namespace launch {

template <>
int attend_dim<64>(const DeviceView &d, bool q8, int rows, int *resident, const dev::KvAttendParams *p,
                   const CUtensorMap *tm_k, const CUtensorMap *tm_v, int ctas, void *stream, std::string *err) {
    const int rc = q8 ? attend_rows_variant<64, true>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err)
                      : attend_rows_variant<64, false>(d, rows, resident, p, tm_k, tm_v, ctas, stream, err);
    if (rc != W12_OK || !p || !p->join_later) return rc;
    return q8 ? join_parts<64, true>(d, rows, *p, ctas, stream, err)
              : join_parts<64, false>(d, rows, *p, ctas, stream, err);
}

}  // namespace launch
}  // namespace w12
