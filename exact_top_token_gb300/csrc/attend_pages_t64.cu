// attend_pages_t64.cu -- the instance of the attention of single rows over pages for d = 64.
#include "attend_pages_tokens.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_tokens_d64(const AttendArgs& a, int ctas, bool join, cudaStream_t st) {
  return launch_attend_tokens<TCfg<64>>(a, ctas, join, st);
}

}  // namespace pages
}  // namespace hytopk
