// The rows kernel of attention over pages in bf16.
#include "attend_pages_rows.h"

namespace hkv {

hipError_t launch_page_rows_bf16(const PageAttendParams& p, dim3 grid, hipStream_t stream) {
  return launch_page_rows<kBF16>(p, grid, stream);
}

}  // namespace hkv
