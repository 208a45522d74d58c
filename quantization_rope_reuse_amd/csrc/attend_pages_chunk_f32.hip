// The chunk kernel of attention over pages in f32.
#include "attend_pages_chunk.h"

namespace hkv {

hipError_t launch_page_chunk_f32(const PageAttendParams& p, dim3 grid, hipStream_t stream) {
  return launch_page_chunk<kF32>(p, grid, stream);
}

}  // namespace hkv
