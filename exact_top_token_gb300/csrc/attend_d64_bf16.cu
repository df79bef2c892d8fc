// attend_d64_bf16.cu -- instantiations of the attention engine for d = 64, bf16 rows.
#include "attend_engine.cuh"

namespace hytopk {

cudaError_t launch_attend_d64_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st) {
  if (f32) {
    if (a.G <= 16) return att::launch_attend<att::Cfg<64, 16, false, true>>(a, sms, st);
    return att::launch_attend<att::Cfg<64, 64, false, true>>(a, sms, st);
  }
  if (a.G <= 16) {
    if ((int64_t)a.n * a.Hkv > sms)
      return att::launch_attend<att::Cfg<64, 16, false, false, 2>>(a, sms, st);
    return att::launch_attend<att::Cfg<64, 16, false, false>>(a, sms, st);
  }
  if (a.G <= 64) return att::launch_attend<att::Cfg<64, 64, false, false>>(a, sms, st);
  return att::launch_attend<att::Cfg<64, 128, false, false>>(a, sms, st);
}

}  // namespace hytopk
