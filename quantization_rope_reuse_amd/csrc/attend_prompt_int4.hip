// Attention over INT4 records for many query rows per key head.
#include "attend_prompt.h"

namespace hkv {

hipError_t launch_prompt_int4(const AttendParams& p, dim3 grid, hipStream_t stream) {
  return launch_prompt_format<kINT4>(p, grid, stream);
}

}  // namespace hkv
