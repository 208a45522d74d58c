// Attention over FP8 records for few query rows per key head.
#include "attend_rows.h"

namespace hkv {

hipError_t launch_rows_fp8(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                            hipStream_t stream) {
  return launch_rows_format<kFP8>(p, hp, nt, grid, bytes, stream);
}

}  // namespace hkv
