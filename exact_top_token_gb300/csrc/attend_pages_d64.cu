// attend_pages_d64.cu -- the instance of the attention over pages for d = 64.
#include "attend_pages_engine.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_pages_d64(const AttendArgs& a, int ctas, cudaStream_t st) {
  return a.several ? launch_attend_pages<PCfg<64>, true>(a, ctas, st)
                   : launch_attend_pages<PCfg<64>, false>(a, ctas, st);
}

}  // namespace pages
}  // namespace hytopk
