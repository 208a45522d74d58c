// Attention over FP8 records for many query rows per key head.
#include "attend_prompt.h"

namespace hkv {

hipError_t launch_prompt_fp8(const AttendParams& p, dim3 grid, hipStream_t stream) {
  return launch_prompt_format<kFP8>(p, grid, stream);
}

}  // namespace hkv
