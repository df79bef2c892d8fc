// attend_d64_e4m3.cu -- instantiations of the attention engine for d = 64, e4m3 rows.
#include "attend_engine.cuh"

namespace hytopk {

cudaError_t launch_attend_d64_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st) {
  if (f32) {
    if (a.G <= 16) return att::launch_attend<att::Cfg<64, 16, true, true>>(a, sms, st);
    return att::launch_attend<att::Cfg<64, 64, true, true>>(a, sms, st);
  }
  if (a.G <= 16) {
    if ((int64_t)a.n * a.Hkv > sms)
      return att::launch_attend<att::Cfg<64, 16, true, false, 2>>(a, sms, st);
    return att::launch_attend<att::Cfg<64, 16, true, false>>(a, sms, st);
  }
  if (a.G <= 64) return att::launch_attend<att::Cfg<64, 64, true, false>>(a, sms, st);
  return att::launch_attend<att::Cfg<64, 128, true, false>>(a, sms, st);
}

}  // namespace hytopk
