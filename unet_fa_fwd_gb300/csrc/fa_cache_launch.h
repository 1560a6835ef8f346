// fa_cache_launch.h — host side of the cached attention shared by its two
// translation units: the plan of a call, and the launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_cache_attn.cuh"
#include "fa_host.h"

namespace fa {

// Rows of a key head that share a pass over its tiles: 4, 8 or 16, the least
// that holds them all, in the kernel for few rows (fa_cache_attn.cuh, up to
// kCacheFewRows); kChunkRows in the one for many (fa_cache_chunk.cuh).  More rows
// in two passes of 16 instead: 16 sequences of up to 8192 tokens with 8 key
// heads, 24 rows 83 us for 58 at D = 64 and 80 for 52 at D = 32, 32 rows 97 for 83
// at D = 128; 8 of up to 4111 with 4 key heads, 20 rows at D = 64, 32 for 31.
// (Where a CTA gets a tile or two, two passes are ahead: 17 rows of one key head
// on those, 26 us for 34.)
constexpr int kCacheFewRows = 16;
constexpr int kChunkMaxGrid = 192;  // CTAs of the kernel for many rows (one per SM) that partial results are sized for

struct CachePlan {
  int R, rt, row_tiles;
  int64_t units;        // per batch entry
  int64_t tiles;        // at most, all units
  size_t part_o, cut, total;  // workspace: partial O; up to their maxima and sums; in all
};

// Launches a merge so that its blocks may start while the kernel before it on
// the stream finishes (it waits for that kernel itself).
inline int launch_after(void (*kernel)(const CacheAttnParams), unsigned blocks, unsigned threads,
                 const CacheAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The kernel for many rows and its merge (fa_cache_chunk.cu).
int launch_cache_chunk(CacheAttnParams& p, const CachePlan& plan, int D, const DeviceState& st, cudaStream_t s);

}  // namespace fa
