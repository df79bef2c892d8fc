// attend_pages_t64.cu -- the instances of the attention of single rows over pages for d = 64.
#include "attend_pages_tokens.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_tokens_d64(const AttendArgs& a, int ctas, cudaStream_t st) {
  return a.G <= 16 ? launch_attend_tokens<TCfg<64, 16>>(a, ctas, st)
                   : launch_attend_tokens<TCfg<64, 64>>(a, ctas, st);
}

}  // namespace pages
}  // namespace hytopk
