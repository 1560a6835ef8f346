// fa_cache.cu — C ABI of the operators around a cached attention (declared in
// include/fa.h): rotary positions, the paged e4m3 key/value cache, and the
// attention that reads it.  Arguments are validated before any CUDA call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "fa.h"
#include "fa_cache_attn.cuh"
#include "fa_cache_launch.h"
#include "fa_cache_quant.cuh"
#include "fa_host.h"
#include "fa_log.h"
#include "fa_rope.cuh"
#include "fa_strided.h"

namespace {

using fa::aligned16;
using fa::apart;
using fa::CachePlan;
using fa::extent;
using fa::fits_int;
using fa::head_dim_ok;
using fa::launch_after;
using fa::ranges_overlap;
using fa::rows16;
using fa::same;
using fa::writes_once;

// ---- rotary positions ----

template <typename T, int D, int E, bool HALVES>
int launch_rope(fa::RopeParams& p, int sm_count, cudaStream_t s) {
  constexpr int CHUNKS = HALVES ? D / 2 / E : D / E;
  const long long blocks = (p.tokens * CHUNKS + fa::kRopeThreads - 1) / fa::kRopeThreads;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARGUMENT;
  // Heads are dealt to several blocks a token until the blocks fill the SMs'
  // 8 x 256 threads twice over, but each block keeps 16 heads (its sines and
  // cosines cost about as much as 8) unless even half a filling is missing:
  // 4608 tokens x 48 heads of 128 take 21.3 us in groups of 8 heads, 19.6 of 16;
  // 16896 tokens in fp32 129 us in one group, 126 in two.
  const int batches = (p.heads + fa::kRopeBatch - 1) / fa::kRopeBatch;
  const long long fill = (16LL * sm_count + blocks - 1) / blocks;
  const long long quarter = (4LL * sm_count + blocks - 1) / blocks, wide = (batches + 3) / 4;
  long long groups = quarter > wide ? quarter : wide;
  if (groups > fill) groups = fill;
  if (groups > batches) groups = batches;
  const int per = (int)((batches + groups - 1) / groups);
  p.heads_per_block = per * fa::kRopeBatch;
  const int gy = (batches + per - 1) / per;
  fa::log_launch("fa_rope_kernel<D=%d,%d-byte elements,%d per access,%s> grid %lld x %d x %d threads, %lld tokens, "
                 "%d heads%s", D, (int)sizeof(T), E, HALVES ? "halves" : "adjacent", blocks, gy, fa::kRopeThreads,
                 p.tokens, p.heads, p.inverse ? ", inverse" : "");
  fa::fa_rope_kernel<T, D, E, HALVES><<<dim3((unsigned)blocks, gy), fa::kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <typename T, int D>
int dispatch_rope(fa::RopeParams& p, bool vec, bool halves, int sm_count, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  if (halves)
    return vec ? launch_rope<T, D, E, true>(p, sm_count, s) : launch_rope<T, D, 2, true>(p, sm_count, s);
  return vec ? launch_rope<T, D, E, false>(p, sm_count, s) : launch_rope<T, D, 2, false>(p, sm_count, s);
}

template <typename T>
int dispatch_rope(int D, fa::RopeParams& p, bool vec, bool halves, int sm_count, cudaStream_t s) {
  switch (D) {
    case 32: return dispatch_rope<T, 32>(p, vec, halves, sm_count, s);
    case 64: return dispatch_rope<T, 64>(p, vec, halves, sm_count, s);
    default: return dispatch_rope<T, 128>(p, vec, halves, sm_count, s);
  }
}

// ---- the cache ----

struct CacheBytes {
  size_t code, scale;
};

int validate_cache(const fa_cache* c, const int* table, int width, int B, CacheBytes* bytes) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !table) return FA_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 1 || c->H < 1 || width < 1 || B < 1) return FA_ERR_INVALID_ARGUMENT;
  if (!head_dim_ok(c->D)) return FA_ERR_UNSUPPORTED;
  if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return FA_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) || (reinterpret_cast<uintptr_t>(table) & 3u))
    return FA_ERR_INVALID_ARGUMENT;
  // (page, head) pairs are a coordinate of the tensor maps; positions are 32-bit
  if ((int64_t)c->num_pages * c->H > INT_MAX || (int64_t)width * c->page_tokens > INT_MAX)
    return FA_ERR_INVALID_ARGUMENT;
  const size_t heads = (size_t)c->num_pages * c->H;
  bytes->code = heads * c->page_tokens * c->D;
  bytes->scale = heads * sizeof(float);
  const void* p[4] = {c->k, c->v, c->k_scale, c->v_scale};
  const size_t n[4] = {bytes->code, bytes->code, bytes->scale, bytes->scale};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (ranges_overlap(p[i], n[i], p[j], n[j])) return FA_ERR_INVALID_ARGUMENT;
    if (ranges_overlap(p[i], n[i], table, (size_t)B * width * sizeof(int))) return FA_ERR_INVALID_ARGUMENT;
  }
  return FA_OK;
}

bool overlaps_cache(const fa_cache* c, const CacheBytes& n, const void* p, size_t bytes) {
  return ranges_overlap(p, bytes, c->k, n.code) || ranges_overlap(p, bytes, c->v, n.code) ||
         ranges_overlap(p, bytes, c->k_scale, n.scale) || ranges_overlap(p, bytes, c->v_scale, n.scale);
}

// A per-sequence array of ints (or NULL where it may be left out).
bool ints_ok(const int* a, bool optional) {
  return a ? (reinterpret_cast<uintptr_t>(a) & 3u) == 0 : optional;
}

fa::CacheView view(const fa_cache* c, const int* table, int width) {
  fa::CacheView v;
  v.code[0] = static_cast<uint8_t*>(c->k);
  v.code[1] = static_cast<uint8_t*>(c->v);
  v.scale[0] = c->k_scale;
  v.scale[1] = c->v_scale;
  v.table = table;
  v.width = width;
  v.num_pages = c->num_pages;
  v.H = c->H;
  v.page = c->page_tokens;
  return v;
}

template <int D, int PAGE>
void launch_write(const fa::CacheWriteParams& p, bool vec, unsigned blocks, cudaStream_t s) {
  if (vec)
    fa::fa_cache_write_kernel<D, PAGE, true><<<blocks, fa::kWriteThreads, 0, s>>>(p);
  else
    fa::fa_cache_write_kernel<D, PAGE, false><<<blocks, fa::kWriteThreads, 0, s>>>(p);
}

template <int D>
void launch_write(const fa::CacheWriteParams& p, bool vec, unsigned blocks, cudaStream_t s) {
  switch (p.c.page) {
    case 32: launch_write<D, 32>(p, vec, blocks, s); break;
    case 64: launch_write<D, 64>(p, vec, blocks, s); break;
    default: launch_write<D, 128>(p, vec, blocks, s); break;
  }
}

// The plan of a call.
CachePlan cache_plan(int B, int Hq, int Hk, int Nq, int D, int width, int page) {
  CachePlan l{};
  l.R = (int)((int64_t)Hq / Hk * Nq);
  l.rt = l.R > fa::kCacheFewRows ? fa::kChunkRows : (l.R <= 4 ? 4 : (l.R <= 8 ? 8 : 16));
  l.row_tiles = (l.R + l.rt - 1) / l.rt;
  l.units = (int64_t)Hk * l.row_tiles;
  const int64_t per = fa::cache_tiles(width * page);
  l.tiles = per * l.units * B;
  if (per > 1) {  // a unit of one tile is never cut
    const int64_t most = l.rt == fa::kChunkRows ? fa::kChunkMaxGrid : fa::kCacheMaxGrid;
    const size_t slots = 2 * (size_t)(l.tiles < most ? l.tiles : most);
    l.part_o = (slots * l.rt * D * sizeof(float) + 255) & ~size_t(255);
    l.cut = l.part_o + ((slots * l.rt * 2 * sizeof(float) + 255) & ~size_t(255));
    l.total = l.cut + slots / 2 * sizeof(int4);
  }
  return l;
}

// Tensor map over a cache's codes [num_pages * H][page][D] bytes: one box is a
// page of a head, swizzled over its D-byte rows as the MMA operands are.
int encode_cache_map(CUtensorMap* map, void* base, const fa_cache* c) {
  cuuint64_t dims[3] = {(cuuint64_t)c->D, (cuuint64_t)c->page_tokens, (cuuint64_t)c->num_pages * c->H};
  cuuint64_t strides[2] = {(cuuint64_t)c->D, (cuuint64_t)c->D * c->page_tokens};
  cuuint32_t box[3] = {(cuuint32_t)c->D, (cuuint32_t)c->page_tokens, 1u};
  cuuint32_t estride[3] = {1u, 1u, 1u};
  const CUtensorMapSwizzle sw = c->D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                            : (c->D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  const CUresult r = fa::tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box,
                                              estride, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

template <int D, int RT>
int launch_cache_attn(fa::CacheAttnParams& p, const CachePlan& plan, const fa::DeviceState& st, cudaStream_t s) {
  using C = fa::CacheCfg<D, RT>;
  static std::mutex mu;
  static int resident[64] = {};  // CTAs an SM holds, per device
  int per_sm = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    int& r = resident[st.device];
    if (!r) {
      // By shared memory, registers and tensor memory (the occupancy query
      // answers 1 for kernels that allocate tensor memory, whose columns it
      // does not see).
      int smem = 0, reserved = 0, regs = 0;
      cudaFuncAttributes attr;
      if (cudaFuncSetAttribute(fa::fa_cache_attn_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM_BYTES) != cudaSuccess ||
          cudaFuncSetAttribute(fa::fa_cache_attn_kernel<D, RT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
          cudaFuncGetAttributes(&attr, fa::fa_cache_attn_kernel<D, RT>) != cudaSuccess ||
          cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, st.device) != cudaSuccess ||
          cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, st.device) != cudaSuccess ||
          cudaDeviceGetAttribute(&regs, cudaDevAttrMaxRegistersPerMultiprocessor, st.device) != cudaSuccess)
        return FA_ERR_CUDA;
      int n = smem / (C::SMEM_BYTES + reserved);
      const int by_regs = regs / ((attr.numRegs + 7) / 8 * 8 * fa::kCacheThreads);
      n = n < by_regs ? n : by_regs;
      n = n < 512 / C::TMEM_COLS ? n : 512 / C::TMEM_COLS;
      r = n < 1 ? 1 : n;
    }
    per_sm = r;
  }
  int64_t grid = (int64_t)per_sm * st.sm_count;
  if (grid > fa::kCacheMaxGrid) grid = fa::kCacheMaxGrid;
  if (grid > plan.tiles) grid = plan.tiles;
  p.ctas = (int)grid;
  fa::log_launch("fa_cache_attn_kernel<D=%d,%d rows> grid %d x %d threads (%d per SM) smem %d B tmem %d cols "
                 "stages %d, %lld units a sequence, %lld tiles at most", D, RT, p.ctas, fa::kCacheThreads, per_sm,
                 C::SMEM_BYTES, C::TMEM_COLS, C::STAGES, (long long)plan.units, (long long)plan.tiles);
  fa::fa_cache_attn_kernel<D, RT><<<p.ctas, fa::kCacheThreads, C::SMEM_BYTES, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (!plan.total) return FA_OK;  // no unit can be cut
  const unsigned blocks = (unsigned)p.ctas * RT;
  fa::log_launch("fa_cache_merge_kernel<D=%d,%d rows> grid %u x 128 threads", D, RT, blocks);
  return launch_after(fa::fa_cache_merge_kernel<D, RT>, blocks, 128, p, s);
}

template <int D>
int launch_cache_attn(fa::CacheAttnParams& p, const CachePlan& plan, const fa::DeviceState& st, cudaStream_t s) {
  if (plan.rt == fa::kChunkRows) return fa::launch_cache_chunk(p, plan, D, st, s);
  switch (plan.rt) {
    case 4: return launch_cache_attn<D, 4>(p, plan, st, s);
    case 8: return launch_cache_attn<D, 8>(p, plan, st, s);
    default: return launch_cache_attn<D, 16>(p, plan, st, s);
  }
}

}  // namespace

extern "C" {

int fa_rope(const fa_rope_axes* axes, const int* pos, long long pos_stride_b, const fa_tensor* q,
            const fa_tensor* q_out, int Hq, const fa_tensor* k, const fa_tensor* k_out, int Hk, int B,
            int N, int D, int dtype, int pairing, int inverse, void* stream) {
  // ---- validation: no CUDA call before this block passes ----
  if (!axes || !pos || !q || !q_out || !q->data || !q_out->data) return FA_ERR_INVALID_ARGUMENT;
  if ((k == nullptr) != (k_out == nullptr) || (k && (!k->data || !k_out->data || Hk < 1)))
    return FA_ERR_INVALID_ARGUMENT;
  if (B < 1 || N < 1 || Hq < 1 || pos_stride_b < 0) return FA_ERR_INVALID_ARGUMENT;
  if (!head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_FP32) return FA_ERR_UNSUPPORTED;
  if (pairing != FA_ROPE_ADJACENT && pairing != FA_ROPE_HALVES) return FA_ERR_INVALID_ARGUMENT;
  fa::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  if (fa::rope_pairs(axes, D, p.freq, p.axis) != FA_OK) return FA_ERR_INVALID_ARGUMENT;
  const int size = dtype == FA_DTYPE_FP32 ? 4 : 2;
  const int nt = k ? 2 : 1;
  const fa_tensor in[2] = {*q, k ? *k : *q}, out[2] = {*q_out, k_out ? *k_out : *q_out};
  const int H[2] = {Hq, k ? Hk : 0};
  if ((int64_t)Hq + H[1] > INT_MAX - fa::kRopeBatch) return FA_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(pos) & 3u)) return FA_ERR_INVALID_ARGUMENT;
  const int64_t pos_n = fa::rope_positions(pos_stride_b, B, N, axes->count);
  if (pos_n < 0) return FA_ERR_INVALID_ARGUMENT;
  bool vec = true;
  for (int i = 0; i < nt; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(in[i].data) | reinterpret_cast<uintptr_t>(out[i].data);
    if (a % size) return FA_ERR_INVALID_ARGUMENT;
    const int64_t ei = extent(in[i], B, H[i], N, D), eo = extent(out[i], B, H[i], N, D);
    if (!ei || !eo || !writes_once(out[i], B, H[i], N, D)) return FA_ERR_INVALID_ARGUMENT;
    if (ranges_overlap(out[i].data, (size_t)eo * size, pos, (size_t)pos_n * sizeof(int)))
      return FA_ERR_INVALID_ARGUMENT;
    vec = vec && rows16(in[i], B, H[i], N, size) && rows16(out[i], B, H[i], N, size);
  }
  for (int i = 0; i < nt; ++i)
    for (int j = 0; j < nt; ++j) {
      if (!(i == j && same(out[i], in[j], B, H[i], N)) && !apart(out[i], H[i], in[j], H[j], B, N, D, size))
        return FA_ERR_INVALID_ARGUMENT;
      if (i < j && !apart(out[i], H[i], out[j], H[j], B, N, D, size)) return FA_ERR_INVALID_ARGUMENT;
    }

  for (int i = 0; i < nt; ++i)
    p.t[i] = fa::RopeTensor{in[i].data, out[i].data, in[i].stride_b, in[i].stride_h, in[i].stride_n,
                            out[i].stride_b, out[i].stride_h, out[i].stride_n, H[i]};
  p.pos = pos;
  p.pos_b = pos_stride_b;
  p.A = axes->count;
  p.N = N;
  p.heads = Hq + H[1];
  p.tokens = (long long)B * N;
  p.inverse = inverse ? 1 : 0;
  fa::DeviceState* st = nullptr;
  const int rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool halves = pairing == FA_ROPE_HALVES;
  switch (dtype) {
    case FA_DTYPE_BF16: return dispatch_rope<__nv_bfloat16>(D, p, vec, halves, st->sm_count, s);
    case FA_DTYPE_FP16: return dispatch_rope<__half>(D, p, vec, halves, st->sm_count, s);
    default: return dispatch_rope<float>(D, p, vec, halves, st->sm_count, s);
  }
}

int fa_cache_write(const fa_cache* cache, const fa_tensor* k, const fa_tensor* v, const int* table, int table_width,
                   const int* start, const int* count, int B, int N, void* stream) {
  CacheBytes bytes;
  int rc = validate_cache(cache, table, table_width, B, &bytes);
  if (rc != FA_OK) return rc;
  if (!k || !v || !k->data || !v->data || N < 1 || !ints_ok(start, false) || !ints_ok(count, true))
    return FA_ERR_INVALID_ARGUMENT;
  const int D = cache->D, H = cache->H, page = cache->page_tokens;
  if ((int64_t)table_width * page + N > INT_MAX) return FA_ERR_INVALID_ARGUMENT;
  bool vec = true;
  const fa_tensor* in[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    const int64_t e = extent(*in[i], B, H, N, D);
    if (!e || (reinterpret_cast<uintptr_t>(in[i]->data) & 1u)) return FA_ERR_INVALID_ARGUMENT;
    if (overlaps_cache(cache, bytes, in[i]->data, (size_t)e * 2)) return FA_ERR_INVALID_ARGUMENT;
    vec = vec && rows16(*in[i], B, H, N, 2);
  }
  if (overlaps_cache(cache, bytes, start, (size_t)B * sizeof(int)) ||
      (count && overlaps_cache(cache, bytes, count, (size_t)B * sizeof(int))))
    return FA_ERR_INVALID_ARGUMENT;
  fa::CacheWriteParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = view(cache, table, table_width);
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const __nv_bfloat16*>(in[i]->data);
    p.xb[i] = in[i]->stride_b;
    p.xh[i] = in[i]->stride_h;
    p.xn[i] = in[i]->stride_n;
  }
  p.start = start;
  p.count = count;
  p.B = B;
  p.N = N;
  p.slots = (N + page - 2) / page + 1;  // N tokens from anywhere in a page
  if (!fits_int(2LL * B, H, p.slots)) return FA_ERR_INVALID_ARGUMENT;
  const int64_t blocks = 2LL * B * H * p.slots;

  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  p.status = st->status;
  fa::log_launch("fa_cache_write_kernel<D=%d,page %d,%s> grid %lld x %d threads (%d pages a sequence and head at most)",
                 D, page, vec ? "16-byte loads" : "scalar loads", (long long)blocks, fa::kWriteThreads, p.slots);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (D) {
    case 32: launch_write<32>(p, vec, (unsigned)blocks, s); break;
    case 64: launch_write<64>(p, vec, (unsigned)blocks, s); break;
    default: launch_write<128>(p, vec, (unsigned)blocks, s); break;
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_cache_read(const fa_cache* cache, const int* table, int table_width, const int* lens, const int* first,
                  void* k_out, void* v_out, int B, int N, void* stream) {
  CacheBytes bytes;
  int rc = validate_cache(cache, table, table_width, B, &bytes);
  if (rc != FA_OK) return rc;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || N < 1 || !ints_ok(lens, false) ||
      !ints_ok(first, true))
    return FA_ERR_INVALID_ARGUMENT;
  const int D = cache->D, H = cache->H;
  const int64_t per = ((int64_t)N * (D / 16) + fa::kReadThreads - 1) / fa::kReadThreads;
  if (!fits_int(2LL * B, H, per)) return FA_ERR_INVALID_ARGUMENT;
  const size_t out = (size_t)B * H * N * D * 2, ints = (size_t)B * sizeof(int);
  void* outs[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i)
    if (overlaps_cache(cache, bytes, outs[i], out) || ranges_overlap(outs[i], out, lens, ints) ||
        ranges_overlap(outs[i], out, first, ints) ||
        ranges_overlap(outs[i], out, table, (size_t)B * table_width * sizeof(int)))
      return FA_ERR_INVALID_ARGUMENT;
  if (ranges_overlap(k_out, out, v_out, out)) return FA_ERR_INVALID_ARGUMENT;
  fa::CacheReadParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = view(cache, table, table_width);
  p.out[0] = static_cast<__nv_bfloat16*>(k_out);
  p.out[1] = static_cast<__nv_bfloat16*>(v_out);
  p.lens = lens;
  p.first = first;
  p.B = B;
  p.N = N;
  p.blocks = (int)per;

  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  p.status = st->status;
  const unsigned blocks = (unsigned)(per * B * H * 2);
  fa::log_launch("fa_cache_read_kernel<D=%d> grid %u x %d threads", D, blocks, fa::kReadThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (D) {
    case 32: fa::fa_cache_read_kernel<32><<<blocks, fa::kReadThreads, 0, s>>>(p); break;
    case 64: fa::fa_cache_read_kernel<64><<<blocks, fa::kReadThreads, 0, s>>>(p); break;
    default: fa::fa_cache_read_kernel<128><<<blocks, fa::kReadThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_cache_workspace_bytes(int B, int Hq, int Hk, int Nq, int D, int table_width, int page_tokens) {
  if (B < 1 || Hk < 1 || Hq < 1 || Hq % Hk || Nq < 1 || !head_dim_ok(D) || table_width < 1 || page_tokens < 1 ||
      !fits_int(B, Hq, Nq) || (int64_t)table_width * page_tokens > INT_MAX)
    return 0;
  return cache_plan(B, Hq, Hk, Nq, D, table_width, page_tokens).total;
}

int fa_fwd_cache(const void* q, const fa_cache* cache, const int* table, int table_width, const int* lens,
                 const int* q_start, int causal, void* out, float* lse, int B, int Hq, int Nq, float scale,
                 void* workspace, size_t workspace_bytes, void* stream) {
  CacheBytes bytes;
  int rc = validate_cache(cache, table, table_width, B, &bytes);
  if (rc != FA_OK) return rc;
  if (!q || !out || !lse || !aligned16(q) || !aligned16(out) || !aligned16(lse) || !ints_ok(lens, false) ||
      !ints_ok(q_start, true))
    return FA_ERR_INVALID_ARGUMENT;
  if (Nq < 1 || Hq < 1 || Hq % cache->H) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale)) return FA_ERR_INVALID_ARGUMENT;
  if (!fits_int(B, Hq, Nq)) return FA_ERR_INVALID_ARGUMENT;
  const int D = cache->D;
  const int64_t rows = (int64_t)B * Hq * Nq;
  const size_t qb = (size_t)rows * D * 2, lb = (size_t)rows * 4, ints = (size_t)B * sizeof(int);
  if (ranges_overlap(out, qb, q, qb) || ranges_overlap(out, qb, lse, lb) || ranges_overlap(lse, lb, q, qb) ||
      overlaps_cache(cache, bytes, out, qb) || overlaps_cache(cache, bytes, lse, lb) ||
      ranges_overlap(out, qb, table, (size_t)B * table_width * sizeof(int)) ||
      ranges_overlap(lse, lb, table, (size_t)B * table_width * sizeof(int)) || ranges_overlap(out, qb, lens, ints) ||
      ranges_overlap(lse, lb, lens, ints) || ranges_overlap(out, qb, q_start, ints) ||
      ranges_overlap(lse, lb, q_start, ints))
    return FA_ERR_INVALID_ARGUMENT;
  const CachePlan plan = cache_plan(B, Hq, cache->H, Nq, D, table_width, cache->page_tokens);
  if (plan.units * B > INT_MAX) return FA_ERR_INVALID_ARGUMENT;
  const size_t need = plan.total;
  if (need) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return FA_ERR_INVALID_ARGUMENT;
    if (ranges_overlap(workspace, need, q, qb) || ranges_overlap(workspace, need, out, qb) ||
        ranges_overlap(workspace, need, lse, lb) || overlaps_cache(cache, bytes, workspace, need) ||
        ranges_overlap(workspace, need, table, (size_t)B * table_width * sizeof(int)) ||
        ranges_overlap(workspace, need, lens, ints) || ranges_overlap(workspace, need, q_start, ints))
      return FA_ERR_INVALID_ARGUMENT;
  }

  fa::DeviceState* st = nullptr;
  rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  fa::CacheAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = view(cache, table, table_width);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.rows = fa::CacheRows{lens, q_start, B, cache->H, Hq / cache->H, Nq, plan.R, plan.rt, plan.row_tiles,
                         causal ? 1 : 0, table_width * cache->page_tokens,
                         fa::FastDiv::make((uint32_t)(Hq / cache->H))};
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.status = st->status;
  p.debug_record = st->debug_record;
  if (need) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_o);
    p.cut = reinterpret_cast<int4*>(static_cast<char*>(workspace) + plan.cut);
  }
  p.timeout_ns = fa::timeout_ns_from_env();
  const char* inject = std::getenv("FA_FAULT_INJECT");
  p.inject_stall = (inject && std::strcmp(inject, "stall") == 0) ? 1 : 0;
  if (encode_cache_map(&p.tm_k, cache->k, cache) != FA_OK || encode_cache_map(&p.tm_v, cache->v, cache) != FA_OK)
    return FA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (D) {
    case 32: return launch_cache_attn<32>(p, plan, *st, s);
    case 64: return launch_cache_attn<64>(p, plan, *st, s);
    default: return launch_cache_attn<128>(p, plan, *st, s);
  }
}

}  // extern "C"
