// attend_d128_e4m3.cu -- instantiations of the attention engine for d = 128, e4m3 rows.
#include "attend_engine.cuh"

namespace hytopk {

cudaError_t launch_attend_d128_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st) {
  if (f32) {
    if (a.G <= 16) return att::launch_attend<att::Cfg<128, 16, true, true>>(a, sms, st);
    return att::launch_attend<att::Cfg<128, 64, true, true>>(a, sms, st);
  }
  if (a.G <= 16) return att::launch_attend<att::Cfg<128, 16, true, false>>(a, sms, st);
  if (a.G > 64) return att::launch_attend<att::Cfg<128, 128, true, false>>(a, sms, st);
  return att::launch_attend<att::Cfg<128, 64, true, false>>(a, sms, st);
}

}  // namespace hytopk
