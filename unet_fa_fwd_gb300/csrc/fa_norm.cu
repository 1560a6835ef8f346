// fa_norm.cu — C ABI of the norm of queries and keys with the rotary positions
// and of its gradient (declared in include/fa.h).  Arguments are validated
// before any CUDA call.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "fa.h"
#include "fa_host.h"
#include "fa_log.h"
#include "fa_norm_rope.cuh"
#include "fa_strided.h"

namespace {

using fa::apart;
using fa::extent;
using fa::NormParams;
using fa::ranges_overlap;
using fa::rows16;
using fa::same;

size_t part_bytes(int D) { return (size_t)fa::kNormMaxBlocks * 2 * D * sizeof(float); }

template <typename T, int D, bool VEC, bool HALVES, bool BACK>
int launch(NormParams& p, int sm_count, float* dwq, float* dwk, cudaStream_t s) {
  using Shape = fa::NormShape<T, D, HALVES, BACK>;
  const long long blocks = p.blocks = (p.tokens + Shape::TOKENS - 1) / Shape::TOKENS;
  for (int i = 0; i < 2; ++i) p.batches[i] = (p.t[i].H + Shape::BATCH - 1) / Shape::BATCH;
  const int batches = p.batches[0] + p.batches[1];
  if (blocks > LLONG_MAX / batches / (2 * fa::kNormMaxBlocks)) return FA_ERR_INVALID_ARGUMENT;
  long long grid;
  if (BACK) {
    // The blocks that are resident share the batches of heads evenly, q's before
    // k's: each leaves a row of partial sums for either.
    p.items = blocks * batches;
    const long long most = (long long)fa::kNormBackPerSm * sm_count;
    grid = most < fa::kNormMaxBlocks ? most : fa::kNormMaxBlocks;
    grid = p.items < grid ? p.items : grid;
  } else {
    // Heads are dealt to several blocks a token until the SMs' 4 blocks are
    // filled; sines and weights are computed once for each of them.
    const int all = (p.heads + Shape::BATCH - 1) / Shape::BATCH;
    const long long fill = (4LL * sm_count + blocks - 1) / blocks;
    const int groups = (int)(fill < all ? fill : all), per = (all + groups - 1) / groups;
    p.heads_per_item = per * Shape::BATCH;
    p.groups = (all + per - 1) / per;
    p.items = blocks * p.groups;
    grid = p.items < INT_MAX ? p.items : INT_MAX;
  }
  fa::log_launch("fa_norm_rope_kernel<D=%d,%d-byte elements,%s,%s,%s> grid %lld x %d threads, %lld tokens, %d heads "
                 "(%d batches)", D, (int)sizeof(T), VEC ? "16-byte accesses" : "single elements",
                 HALVES ? "halves" : "adjacent", BACK ? "gradient" : "forward", grid, fa::kNormThreads, p.tokens,
                 p.heads, batches);
  fa::fa_norm_rope_kernel<T, D, VEC, HALVES, BACK><<<(unsigned)grid, fa::kNormThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (!BACK || !p.part) return FA_OK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(32 * fa::kNormReduceRows);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  fa::log_launch("fa_norm_weight_kernel grid %d x %d threads, %lld rows", 2 * D / 32, 32 * fa::kNormReduceRows, grid);
  const float* part = p.part;
  return cudaLaunchKernelEx(&cfg, fa::fa_norm_weight_kernel, part, (int)grid, D, dwq, dwk) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

struct Call {
  NormParams p;
  bool vec, halves, back;
  int D, dtype, sm_count;
  float *dwq, *dwk;
  cudaStream_t stream;
};

template <typename T, int D>
int dispatch(Call& c) {
  auto go = [&](auto vec, auto halves, auto back) {
    return launch<T, D, decltype(vec)::value, decltype(halves)::value, decltype(back)::value>(c.p, c.sm_count, c.dwq,
                                                                                             c.dwk, c.stream);
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (c.back) {
    if (c.vec) return c.halves ? go(Y{}, Y{}, Y{}) : go(Y{}, N{}, Y{});
    return c.halves ? go(N{}, Y{}, Y{}) : go(N{}, N{}, Y{});
  }
  if (c.vec) return c.halves ? go(Y{}, Y{}, N{}) : go(Y{}, N{}, N{});
  return c.halves ? go(N{}, Y{}, N{}) : go(N{}, N{}, N{});
}

template <typename T>
int dispatch(Call& c) {
  switch (c.D) {
    case 32: return dispatch<T, 32>(c);
    case 64: return dispatch<T, 64>(c);
    default: return dispatch<T, 128>(c);
  }
}

// Both directions: dy is nullptr in the forward.  Tensors in the order q, k.
int norm_call(const fa_rope_axes* axes, const fa_norm* norm, const int* pos, long long pos_b, const fa_tensor* const dy[2],
              const fa_tensor* const x[2], const fa_tensor* const out[2], int Hq, int Hk, float* dwq, float* dwk,
              bool back, int B, int N, int D, int dtype, int pairing, void* workspace, size_t workspace_bytes,
              void* stream) {
  // ---- validation: no CUDA call before this block passes ----
  if (!axes || !norm || !pos) return FA_ERR_INVALID_ARGUMENT;
  const int nt = x[1] || out[1] || (back && dy[1]) ? 2 : 1;
  const int H[2] = {Hq, nt == 2 ? Hk : 0};
  for (int i = 0; i < nt; ++i)
    if (!x[i] || !x[i]->data || !out[i] || !out[i]->data || (back && (!dy[i] || !dy[i]->data)) || H[i] < 1)
      return FA_ERR_INVALID_ARGUMENT;
  if (B < 1 || N < 1 || pos_b < 0) return FA_ERR_INVALID_ARGUMENT;
  if (!fa::head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_FP32) return FA_ERR_UNSUPPORTED;
  if (pairing != FA_ROPE_ADJACENT && pairing != FA_ROPE_HALVES) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(norm->eps) || norm->eps < 0.f) return FA_ERR_INVALID_ARGUMENT;
  const void* const w[2] = {norm->q_weight, norm->k_weight};
  if ((w[0] || w[1]) && norm->weight_dtype != dtype && norm->weight_dtype != FA_DTYPE_FP32) return FA_ERR_UNSUPPORTED;
  if (nt == 1 && w[1]) return FA_ERR_INVALID_ARGUMENT;
  float* const dw[2] = {dwq, dwk};
  Call c;
  std::memset(&c.p, 0, sizeof(c.p));
  if (fa::rope_pairs(axes, D, c.p.freq, c.p.axis) != FA_OK) return FA_ERR_INVALID_ARGUMENT;
  const int size = dtype == FA_DTYPE_FP32 ? 4 : 2;
  const size_t w_size = norm->weight_dtype == FA_DTYPE_FP32 ? 4 : 2, w_bytes = (size_t)D * w_size;
  if ((int64_t)Hq + H[1] > INT_MAX - fa::kRopeBatch) return FA_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return FA_ERR_INVALID_ARGUMENT;
  const int64_t pos_n = fa::rope_positions(pos_b, B, N, axes->count);
  if (pos_n < 0) return FA_ERR_INVALID_ARGUMENT;
  bool vec = true;
  for (int i = 0; i < nt; ++i) {
    const fa_tensor* all[3] = {x[i], out[i], back ? dy[i] : x[i]};
    for (const fa_tensor* t : all) {
      if (reinterpret_cast<uintptr_t>(t->data) % size || !extent(*t, B, H[i], N, D)) return FA_ERR_INVALID_ARGUMENT;
      vec = vec && rows16(*t, B, H[i], N, size);
    }
    const size_t out_bytes = (size_t)extent(*out[i], B, H[i], N, D) * size;
    if (!fa::writes_once(*out[i], B, H[i], N, D) ||
        ranges_overlap(out[i]->data, out_bytes, pos, (size_t)pos_n * sizeof(int)))
      return FA_ERR_INVALID_ARGUMENT;
    if (w[i] && reinterpret_cast<uintptr_t>(w[i]) % w_size) return FA_ERR_INVALID_ARGUMENT;
    if (back && (w[i] != nullptr) != (dw[i] != nullptr)) return FA_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < 2; ++j) {
      if (ranges_overlap(out[i]->data, out_bytes, w[j], w_bytes)) return FA_ERR_INVALID_ARGUMENT;
      if (ranges_overlap(out[i]->data, out_bytes, dw[j], (size_t)D * 4)) return FA_ERR_INVALID_ARGUMENT;
    }
  }
  if (back && nt == 1 && dwk) return FA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < nt; ++i)
    for (int j = 0; j < nt; ++j) {
      const fa_tensor* in[2] = {x[j], back ? dy[j] : x[j]};
      for (const fa_tensor* t : in)
        if (!(i == j && same(*out[i], *t, B, H[i], N)) && !apart(*out[i], H[i], *t, H[j], B, N, D, size))
          return FA_ERR_INVALID_ARGUMENT;
      if (i < j && !apart(*out[i], H[i], *out[j], H[j], B, N, D, size)) return FA_ERR_INVALID_ARGUMENT;
    }
  const size_t dw_bytes = (size_t)D * sizeof(float), need = dwq || dwk ? part_bytes(D) : 0;
  if (dwq || dwk) {
    if (!workspace || !fa::aligned16(workspace) || workspace_bytes < need) return FA_ERR_INVALID_ARGUMENT;
    if (dwq && dwk && ranges_overlap(dwq, dw_bytes, dwk, dw_bytes)) return FA_ERR_INVALID_ARGUMENT;
    const struct { const void* p; size_t n; } written[3] = {{dwq, dwq ? dw_bytes : 0}, {dwk, dwk ? dw_bytes : 0},
                                                             {workspace, need}};
    for (int a = 0; a < 3; ++a) {
      if (!written[a].n) continue;
      if (reinterpret_cast<uintptr_t>(written[a].p) & 3u) return FA_ERR_INVALID_ARGUMENT;
      if (a < 2 && ranges_overlap(written[a].p, written[a].n, workspace, need)) return FA_ERR_INVALID_ARGUMENT;
      if (ranges_overlap(written[a].p, written[a].n, pos, (size_t)pos_n * sizeof(int)))
        return FA_ERR_INVALID_ARGUMENT;
      for (int i = 0; i < nt; ++i) {
        if (ranges_overlap(written[a].p, written[a].n, w[i], w_bytes)) return FA_ERR_INVALID_ARGUMENT;
        const fa_tensor* all[3] = {x[i], out[i], dy[i]};
        for (const fa_tensor* t : all)
          if (ranges_overlap(written[a].p, written[a].n, t->data, (size_t)extent(*t, B, H[i], N, D) * size))
            return FA_ERR_INVALID_ARGUMENT;
      }
    }
  }

  for (int i = 0; i < nt; ++i) {
    const fa_tensor& g = back ? *dy[i] : *x[i];
    c.p.t[i] = fa::NormTensor{x[i]->data, g.data, out[i]->data, x[i]->stride_b, x[i]->stride_h, x[i]->stride_n,
                              g.stride_b, g.stride_h, g.stride_n, out[i]->stride_b, out[i]->stride_h,
                              out[i]->stride_n, w[i], H[i]};
  }
  c.p.pos = pos;
  c.p.pos_b = pos_b;
  c.p.A = axes->count;
  c.p.N = N;
  c.p.heads = Hq + H[1];
  c.p.w_f32 = norm->weight_dtype == FA_DTYPE_FP32 ? 1 : 0;
  c.p.eps = norm->eps;
  c.p.tokens = (long long)B * N;
  c.p.part = need ? static_cast<float*>(workspace) : nullptr;
  fa::DeviceState* st = nullptr;
  const int rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  c.vec = vec;
  c.halves = pairing == FA_ROPE_HALVES;
  c.back = back;
  c.D = D;
  c.sm_count = st->sm_count;
  c.dwq = dwq;
  c.dwk = dwk;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case FA_DTYPE_BF16: return dispatch<__nv_bfloat16>(c);
    case FA_DTYPE_FP16: return dispatch<__half>(c);
    default: return dispatch<float>(c);
  }
}

}  // namespace

extern "C" {

int fa_norm_rope(const fa_rope_axes* axes, const fa_norm* norm, const int* pos, long long pos_stride_b,
                 const fa_tensor* q, const fa_tensor* q_out, int Hq, const fa_tensor* k, const fa_tensor* k_out, int Hk,
                 int B, int N, int D, int dtype, int pairing, void* stream) {
  const fa_tensor *dy[2] = {nullptr, nullptr}, *x[2] = {q, k}, *out[2] = {q_out, k_out};
  return norm_call(axes, norm, pos, pos_stride_b, dy, x, out, Hq, Hk, nullptr, nullptr, false, B, N, D, dtype, pairing,
                   nullptr, 0, stream);
}

int fa_norm_rope_bwd(const fa_rope_axes* axes, const fa_norm* norm, const int* pos, long long pos_stride_b,
                     const fa_tensor* dq_out, const fa_tensor* q, const fa_tensor* dq, int Hq, const fa_tensor* dk_out,
                     const fa_tensor* k, const fa_tensor* dk, int Hk, float* dq_weight, float* dk_weight, int B, int N,
                     int D, int dtype, int pairing, void* workspace, size_t workspace_bytes, void* stream) {
  const fa_tensor *dy[2] = {dq_out, dk_out}, *x[2] = {q, k}, *out[2] = {dq, dk};
  return norm_call(axes, norm, pos, pos_stride_b, dy, x, out, Hq, Hk, dq_weight, dk_weight, true, B, N, D, dtype,
                   pairing, workspace, workspace_bytes, stream);
}

size_t fa_norm_rope_workspace_bytes(int D) { return fa::head_dim_ok(D) ? part_bytes(D) : 0; }

}  // extern "C"
