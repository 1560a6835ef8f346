// fa_cache_chunk.cu — the cached attention's kernel for many rows: its
// instantiations and launcher (a translation unit of its own, built in
// parallel).
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "fa_cache_chunk.cuh"
#include "fa_cache_launch.h"
#include "fa_log.h"

namespace fa {
namespace {

template <int D, bool ONE, bool PAIR>
int launch_chunk(CacheAttnParams& p, const CachePlan& plan, const DeviceState& st, cudaStream_t s) {
  using C = ChunkCfg<D, PAIR>;
  static std::mutex mu;
  static bool ready[64] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[st.device]) {
      if (cudaFuncSetAttribute(fa_cache_chunk_kernel<D, ONE, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM_BYTES) != cudaSuccess)
        return FA_ERR_CUDA;
      ready[st.device] = true;
    }
  }
  int64_t grid = st.sm_count < kChunkMaxGrid ? st.sm_count : kChunkMaxGrid;
  if (grid > plan.tiles) grid = plan.tiles;
  p.ctas = (int)grid;
  log_launch("fa_cache_chunk_kernel<D=%d,%s%s> grid %d x %d threads smem %d B tmem 512 cols stages %d + %d, %lld units "
                 "a sequence, %lld tiles at most", D, ONE ? "a page a tile" : "pages in tiles", PAIR ? ",pairs" : "", p.ctas,
                 kChunkThreads, C::SMEM_BYTES, C::K_STAGES, C::V_STAGES, (long long)plan.units,
                 (long long)plan.tiles);
  fa_cache_chunk_kernel<D, ONE, PAIR><<<p.ctas, kChunkThreads, C::SMEM_BYTES, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (!plan.total) return FA_OK;  // no unit can be cut
  const unsigned blocks = (unsigned)p.ctas * (D / 16);
  log_launch("fa_cache_chunk_merge_kernel<D=%d> grid %u x %d threads", D, blocks, kChunkRows);
  return launch_after(fa_cache_chunk_merge_kernel<D>, blocks, kChunkRows, p, s);
}

template <int D>
int launch_chunk(CacheAttnParams& p, const CachePlan& plan, const DeviceState& st, cudaStream_t s) {
  const bool one = p.c.page == kCacheTile;
  if (plan.R <= 128)
    return one ? launch_chunk<D, true, true>(p, plan, st, s) : launch_chunk<D, false, true>(p, plan, st, s);
  return one ? launch_chunk<D, true, false>(p, plan, st, s) : launch_chunk<D, false, false>(p, plan, st, s);
}

}  // namespace

int launch_cache_chunk(CacheAttnParams& p, const CachePlan& plan, int D, const DeviceState& st, cudaStream_t s) {
  switch (D) {
    case 32: return launch_chunk<32>(p, plan, st, s);
    case 64: return launch_chunk<64>(p, plan, st, s);
    default: return launch_chunk<128>(p, plan, st, s);
  }
}

}  // namespace fa
