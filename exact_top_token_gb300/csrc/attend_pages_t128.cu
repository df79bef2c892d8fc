// attend_pages_t128.cu -- the instance of the attention of single rows over pages for d = 128.
#include "attend_pages_tokens.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_tokens_d128(const AttendArgs& a, int ctas, bool join, cudaStream_t st) {
  return launch_attend_tokens<TCfg<128>>(a, ctas, join, st);
}

}  // namespace pages
}  // namespace hytopk
