// attend_pages_t128.cu -- the instances of the attention of single rows over pages for d = 128.
#include "attend_pages_tokens.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_tokens_d128(const AttendArgs& a, int ctas, cudaStream_t st) {
  return a.G <= 16 ? launch_attend_tokens<TCfg<128, 16>>(a, ctas, st)
                   : launch_attend_tokens<TCfg<128, 64>>(a, ctas, st);
}

}  // namespace pages
}  // namespace hytopk
