// fa_bwd_d64.cu — the attention gradient's kernels for head dimension 64.
#include "fa_bwd_impl.cuh"

namespace fa {

int launch_bwd_d64(const BwdParams& prm, int mask, int device, cudaStream_t s) {
  return launch_bwd<64>(prm, mask, device, s);
}

}  // namespace fa
