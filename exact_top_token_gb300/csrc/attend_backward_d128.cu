// attend_backward_d128.cu -- instantiations of the attention's backward engine for d = 128.
#include "attend_backward_engine.cuh"

namespace hytopk {

cudaError_t launch_attend_backward_d128(const att::Args& a, bool out_f32, int sms, cudaStream_t st) {
  if (a.G <= 16)
    return out_f32 ? att::launch_backward<att::BCfg<128, 16>, true>(a, sms, st)
                   : att::launch_backward<att::BCfg<128, 16>, false>(a, sms, st);
  return out_f32 ? att::launch_backward<att::BCfg<128, 64>, true>(a, sms, st)
                 : att::launch_backward<att::BCfg<128, 64>, false>(a, sms, st);
}

}  // namespace hytopk
