// Attention over INT4 records for few query rows per key head.
#include "attend_rows.h"

namespace hkv {

hipError_t launch_rows_int4(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                            hipStream_t stream) {
  return launch_rows_format<kINT4>(p, hp, nt, grid, bytes, stream);
}

}  // namespace hkv
