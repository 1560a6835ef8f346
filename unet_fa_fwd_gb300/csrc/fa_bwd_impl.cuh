// fa_bwd_impl.cuh — body of the launchers declared in fa_bwd_launch.h (included
// only by fa_bwd_d{32,64,128}.cu).
#pragma once

#include <cuda_runtime.h>

#include <mutex>

#include "fa.h"
#include "fa_bwd_launch.h"
#include "fa_log.h"

namespace fa {

constexpr int kBwdMaxDevices = 64;

// A launch whose kernel waits (griddepcontrol.wait) for the one before it itself.
template <typename K>
int launch_bwd_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const BwdParams& prm) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, prm) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, int MK>
int launch_bwd_one(const BwdParams& prm, int device, cudaStream_t s) {
  using C = BwdCfg<D, MK>;
  static std::mutex mu;
  static bool ready[kBwdMaxDevices] = {};
  if (device < 0 || device >= kBwdMaxDevices) return FA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[device]) {
      if (cudaFuncSetAttribute(fa_bwd_kernel<D, MK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
          cudaSuccess)
        return FA_ERR_CUDA;
      // The register split must fit in what the launch reserves, or the
      // increase would wait forever.
      cudaFuncAttributes attr;
      if (cudaFuncGetAttributes(&attr, fa_bwd_kernel<D, MK>) != cudaSuccess) return FA_ERR_CUDA;
      if (128 * kBwdGroups * C::REGS_ROWS + 128 * C::REGS_OTHER > attr.numRegs * kBwdThreads)
        return FA_ERR_UNSUPPORTED;
      ready[device] = true;
    }
  }
  static const char* kNames[] = {"none", "key", "additive", "bool"};
  const BwdPlan &k = prm.plan[0], &q = prm.plan[1];
  log_launch("fa_bwd_kernel<D=%d,mask %s> grid %d + %d x %d threads smem %d B, dK dV: %d units of %d x 128 rows (%d "
             "whole, %d cuts inside units), dQ: %d of %d (%d, %d), Hq %d Hk %d Nq %d Nk %d causal %d",
             D, kNames[MK], k.ctas, q.ctas, kBwdThreads, C::SMEM_BYTES, k.units.count(), k.units.tiles, k.whole,
             k.joins, q.units.count(), q.units.tiles, q.whole, q.joins, prm.Hq, prm.Hk, prm.Nq, prm.Nk, prm.causal);
  const unsigned ctas = (unsigned)(k.ctas + q.ctas);
  const int rc = launch_bwd_after(fa_bwd_kernel<D, MK>, dim3(ctas), kBwdThreads, C::SMEM_BYTES, s, prm);
  if (rc != FA_OK || k.joins + q.joins == 0) return rc;
  log_launch("fa_bwd_join_kernel<D=%d> grid %u x %d x 128 threads", D, ctas, 2 * D / 8);
  return launch_bwd_after(fa_bwd_join_kernel<D>, dim3(ctas, 2 * D / 8), 128, 0, s, prm);
}

template <int D>
int launch_bwd(const BwdParams& prm, int mask, int device, cudaStream_t s) {
  switch (mask) {
    case kBwdMaskNone: return launch_bwd_one<D, kBwdMaskNone>(prm, device, s);
    case kBwdMaskKey: return launch_bwd_one<D, kBwdMaskKey>(prm, device, s);
    case kBwdMaskAdd: return launch_bwd_one<D, kBwdMaskAdd>(prm, device, s);
    default: return launch_bwd_one<D, kBwdMaskBool>(prm, device, s);
  }
}

}  // namespace fa
