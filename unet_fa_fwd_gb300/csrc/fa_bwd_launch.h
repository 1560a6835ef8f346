// fa_bwd_launch.h — host launchers of the attention gradient's kernels, one per
// head dimension, each in a translation unit of its own
// (fa_bwd_d32.cu / fa_bwd_d64.cu / fa_bwd_d128.cu, built in parallel).
#pragma once

#include <cuda_runtime.h>

#include "fa_bwd_kernel.cuh"

namespace fa {

// -L, -delta and the bits of a mask's tiles; before it, a boolean mask's bits.
int launch_bwd_prep(BwdPrepParams& p, long long heads, int D, cudaStream_t s);
int launch_bwd_bits(const BwdBitsParams& p, long long heads, cudaStream_t s);

// dQ, dK and dV of prm.plan, with the join where units are cut.  mask: kBwdMask*.
// FA_OK, FA_ERR_UNSUPPORTED (a build whose register split does not fit) or
// FA_ERR_CUDA.
int launch_bwd_d32(const BwdParams& prm, int mask, int device, cudaStream_t s);
int launch_bwd_d64(const BwdParams& prm, int mask, int device, cudaStream_t s);
int launch_bwd_d128(const BwdParams& prm, int mask, int device, cudaStream_t s);

}  // namespace fa
