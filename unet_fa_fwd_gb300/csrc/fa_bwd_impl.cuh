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

template <int D, int MK, bool KV>
int launch_bwd_one(const BwdParams& prm, int device, cudaStream_t s) {
  using C = BwdCfg<D, KV>;
  static std::mutex mu;
  static bool ready[kBwdMaxDevices] = {};
  if (device < 0 || device >= kBwdMaxDevices) return FA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[device]) {
      if (cudaFuncSetAttribute(fa_bwd_kernel<D, MK, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM_BYTES) != cudaSuccess)
        return FA_ERR_CUDA;
      // The register split must fit in what the launch reserves, or the
      // increase would wait forever.
      cudaFuncAttributes attr;
      if (cudaFuncGetAttributes(&attr, fa_bwd_kernel<D, MK, KV>) != cudaSuccess) return FA_ERR_CUDA;
      if (2 * 128 * C::REGS_ROWS + 128 * C::REGS_OTHER > attr.numRegs * C::THREADS) return FA_ERR_UNSUPPORTED;
      ready[device] = true;
    }
  }
  static const char* kNames[] = {"none", "key", "additive", "bool"};
  log_launch("fa_bwd_kernel<D=%d,%s,mask %s> grid %d x %d threads smem %d B, %d units of %d x 128 rows (%d whole, %d "
             "cuts inside units) Hq %d Hk %d Nq %d Nk %d causal %d",
             D, KV ? "dK dV" : "dQ", kNames[MK], prm.plan.ctas, C::THREADS, C::SMEM_BYTES, prm.plan.units.count(),
             prm.plan.units.tiles, prm.plan.whole, prm.plan.joins, prm.Hq, prm.Hk, prm.Nq, prm.Nk, prm.causal);
  fa_bwd_kernel<D, MK, KV><<<prm.plan.ctas, C::THREADS, C::SMEM_BYTES, s>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (!prm.plan.joins) return FA_OK;
  constexpr int NC = KV ? D : D / 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (it waits for the kernel before it itself)
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)prm.plan.ctas, NC / 8, 2);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  log_launch("fa_bwd_join_kernel<D=%d,%s> grid %d x %d x 2 x 128 threads", D, KV ? "dK dV" : "dQ", prm.plan.ctas, NC / 8);
  return cudaLaunchKernelEx(&cfg, fa_bwd_join_kernel<D, KV>, prm) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool KV>
int launch_bwd_masked(const BwdParams& prm, int mask, int device, cudaStream_t s) {
  switch (mask) {
    case kBwdMaskNone: return launch_bwd_one<D, kBwdMaskNone, KV>(prm, device, s);
    case kBwdMaskKey: return launch_bwd_one<D, kBwdMaskKey, KV>(prm, device, s);
    case kBwdMaskAdd: return launch_bwd_one<D, kBwdMaskAdd, KV>(prm, device, s);
    default: return launch_bwd_one<D, kBwdMaskBool, KV>(prm, device, s);
  }
}

template <int D>
int launch_bwd(const BwdParams& prm, bool kv, int mask, int device, cudaStream_t s) {
  return kv ? launch_bwd_masked<D, true>(prm, mask, device, s) : launch_bwd_masked<D, false>(prm, mask, device, s);
}

}  // namespace fa
