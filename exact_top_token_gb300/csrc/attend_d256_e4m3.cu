// attend_d256_e4m3.cu -- instantiations of the attention engine for d = 256, e4m3 rows.
#include "attend_engine.cuh"

namespace hytopk {

cudaError_t launch_attend_d256_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st) {
  (void)f32;  // fp32 results: d <= 128
  if (a.G <= 16) return att::launch_attend<att::Cfg<256, 16, true, false>>(a, sms, st);
  return att::launch_attend<att::Cfg<256, 64, true, false>>(a, sms, st);
}

}  // namespace hytopk
