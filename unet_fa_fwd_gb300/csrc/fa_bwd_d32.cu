// fa_bwd_d32.cu — the attention gradient's kernels for head dimension 32.
#include "fa_bwd_impl.cuh"

namespace fa {

int launch_bwd_d32(const BwdParams& prm, int mask, int device, cudaStream_t s) {
  return launch_bwd<32>(prm, mask, device, s);
}

}  // namespace fa
