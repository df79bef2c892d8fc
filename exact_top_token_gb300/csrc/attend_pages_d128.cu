// attend_pages_d128.cu -- the instance of the attention over pages for d = 128.
#include "attend_pages_engine.cuh"

namespace hytopk {
namespace pages {

cudaError_t launch_attend_pages_d128(const AttendArgs& a, int ctas, cudaStream_t st) {
  return a.several ? launch_attend_pages<PCfg<128>, true>(a, ctas, st)
                   : launch_attend_pages<PCfg<128>, false>(a, ctas, st);
}

}  // namespace pages
}  // namespace hytopk
