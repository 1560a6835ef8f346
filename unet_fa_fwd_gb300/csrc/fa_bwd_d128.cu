// fa_bwd_d128.cu — the attention gradient's kernels for head dimension 128.
#include "fa_bwd_impl.cuh"

namespace fa {

int launch_bwd_d128(const BwdParams& prm, int mask, int device, cudaStream_t s) {
  return launch_bwd<128>(prm, mask, device, s);
}

}  // namespace fa
