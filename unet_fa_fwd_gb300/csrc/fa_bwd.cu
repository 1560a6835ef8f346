// fa_bwd.cu — C ABI of the attention gradient (declared in include/fa.h):
// validation, tensor maps, the plan of both kinds of unit and the launches.  Arguments
// are validated before any CUDA call.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "fa.h"
#include "fa_bwd_launch.h"
#include "fa_host.h"
#include "fa_log.h"
#include "fa_strided.h"

namespace fa {

int launch_bwd_prep(BwdPrepParams& p, long long heads, int D, cudaStream_t s) {
  p.head_blocks = p.nqp / (D == 32 ? kBwdPrepRows<32> : D == 64 ? kBwdPrepRows<64> : kBwdPrepRows<128>);
  p.div_blocks = FastDiv::make((uint32_t)p.head_blocks);
  p.row_blocks = heads * p.head_blocks;
  const long long words = p.key_mask ? (long long)p.heads * p.tile_words_q
                          : p.some   ? (long long)p.heads * ((long long)p.tiles_of_q * p.tile_words_q +
                                                             (long long)p.tiles_of_k * p.tile_words_k)
                                     : 0;
  const long long blocks = p.row_blocks + (words + 7) / 8;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARGUMENT;
  log_launch("fa_bwd_prep_kernel<D=%d> grid %lld x 256 threads, %lld rows", D, blocks, heads * p.nqp);
  // Behind the kernel of a boolean mask's bits its blocks may start beside that one's
  // (the blocks that read its results wait themselves).
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = p.some ? 1 : 0;
  const BwdPrepParams& prm = p;
  auto go = [&](auto d) {
    constexpr int W = decltype(d)::value;
    return cudaLaunchKernelEx(&cfg,
                              p.mask   ? fa_bwd_prep_kernel<W, true, true>
                              : p.some ? fa_bwd_prep_kernel<W, true, false>
                                       : fa_bwd_prep_kernel<W, false, false>,
                              prm);
  };
  const cudaError_t e = D == 32   ? go(std::integral_constant<int, 32>{})
                        : D == 64 ? go(std::integral_constant<int, 64>{})
                                  : go(std::integral_constant<int, 128>{});
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int launch_bwd_bits(const BwdBitsParams& p, long long heads, cudaStream_t s) {
  const long long blocks = heads * p.tiles_q * p.tiles_k;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARGUMENT;
  log_launch("fa_bwd_bits_kernel grid %lld x 256 threads", blocks);
  fa_bwd_bits_kernel<<<(unsigned)blocks, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa

namespace {

using fa::aligned16;
using fa::apart;
using fa::extent;
using fa::ranges_overlap;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Iterations that a partial result and its join count for (fa_bwd_geom.h), so that no
// range is shorter than its join: the writing of 64 KB (32 KB of dQ) by a CTA and the
// join's launch take 4 to 5 us.  (A bound, not a setting: with 2 or 7 every case measured
// takes the same time within 1 %.)
constexpr int kJoinCost = 4;

// Sizes that the entry points take.
bool sizes_ok(int B, int Hq, int Hk, int Nq, int Nk, int D) {
  if (B < 1 || Hq < 1 || Hk < 1 || Hq % Hk || Nq < 1 || Nk < 1 || !fa::head_dim_ok(D)) return false;
  const int64_t qt = ((int64_t)Nq + 127) / 128, kt = ((int64_t)Nk + 127) / 128, most = 1 << 30;
  // units, a unit's iterations, and positions of whole tiles are 32-bit numbers
  return (__int128)B * Hq * qt <= most && (__int128)B * Hk * kt <= most && (int64_t)(Hq / Hk) * qt <= most &&
         qt * 128 <= most && kt * 128 <= most;
}

// Sizes of a full mask that the entry points take.
bool mask_ok(int B, int Hq, int Nq, int Nk, int heads) {
  return (heads == 1 || heads == Hq) && (__int128)B * heads * Nq * Nk <= ((__int128)1 << 58);
}

constexpr int kSlotCtas = 160;  // CTAs (one per SM) that partial sums are kept for

// The workspace, in order (each part 256-byte aligned).  Partial sums are for
// the most CTAs a plan has: it does not depend on the GPU.  bool_heads: heads of
// a boolean mask (0: no such mask), whose bits are kept by rows and by keys, with
// those of its tiles; without one, the key tiles' of a key-padding mask.  The
// total is at least kBwdMaxCtas' partial sums and two floats a row, in which flags
// and references fit up to 5900 tiles of queries (D = 32; 23800 for D = 128).
struct Layout {
  size_t stat, flags, ref, part_kv, part_q, bits_q, bits_k, some, tiles_q, tiles_k, total;
};

Layout layout(int B, int Hq, int Nq, int Nk, int D, int bool_heads) {
  const size_t qt = ((size_t)Nq + 127) / 128, kt = ((size_t)Nk + 127) / 128, tiles = (size_t)B * Hq * qt;
  const size_t slots = 2 * (size_t)kSlotCtas, tile = 128 * (size_t)D * sizeof(float);
  const size_t masks = (size_t)B * bool_heads;
  Layout l{};
  size_t off = 0;
  l.stat = off;     off += tiles * fa::kStatTile * sizeof(float);
  l.flags = off;    off += align256(tiles * fa::kFlagTile * sizeof(uint32_t));
  l.ref = off;      off += align256(tiles * 128 * sizeof(float));
  l.part_kv = off;  off += slots * 2 * tile;
  l.part_q = off;   off += slots * tile;
  const size_t least = tiles * fa::kStatTile * sizeof(float) + 2 * (size_t)fa::kBwdMaxCtas * 3 * tile;
  off = off < least ? least : off;
  l.bits_q = off;   off += align256(masks * Nq * kt * 16);
  l.bits_k = off;   off += align256(masks * Nk * qt * 16);
  l.some = off;     off += align256(masks * qt * kt * 4);
  l.tiles_q = off;  off += align256((bool_heads ? masks * qt : B) * ((kt + 31) / 32) * 4);
  l.tiles_k = off;  off += align256(masks * kt * ((qt + 31) / 32) * 4);
  l.total = off;
  return l;
}

// 4-D tensor map over a strided bf16 [B][H][N][D] tensor: one box is a chunk of
// 128 rows (inner extent = the swizzle span), swizzled as the MMA operands are.
// Rows past N read zeros.
int encode(CUtensorMap* map, const fa_tensor& t, int B, int H, int N, int D) {
  const int sw = D >= 64 ? 128 : 64;
  const cuuint64_t any = (cuuint64_t)D * 2;  // strides of axes of size 1 are not used
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  cuuint64_t strides[3] = {N > 1 ? (cuuint64_t)t.stride_n * 2 : any, H > 1 ? (cuuint64_t)t.stride_h * 2 : any,
                           B > 1 ? (cuuint64_t)t.stride_b * 2 : any};
  cuuint32_t box[4] = {(cuuint32_t)(sw / 2), 128u, 1u, 1u};
  cuuint32_t step[4] = {1u, 1u, 1u, 1u};
  const CUresult r = fa::tensor_map_encoder()(
      map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      sw == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// A tensor the kernels can take: whole 16-byte pieces of rows, strides that a
// tensor map holds, no broadcast axis.
bool tensor_ok(const fa_tensor* t, int B, int H, int N, int D) {
  if (!t || !t->data || !extent(*t, B, H, N, D) || !fa::rows16(*t, B, H, N, 2)) return false;
  const long long st[3] = {t->stride_b, t->stride_h, t->stride_n};
  const int size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1 && (st[i] < 8 || st[i] >= (1LL << 39))) return false;
  return true;
}

fa::BwdTensor view(const fa_tensor& t) {
  return fa::BwdTensor{static_cast<__nv_bfloat16*>(t.data), t.stride_b, t.stride_h, t.stride_n};
}

int launch(const fa::BwdParams& p, int D, int mask, int device, cudaStream_t s) {
  switch (D) {
    case 32: return fa::launch_bwd_d32(p, mask, device, s);
    case 64: return fa::launch_bwd_d64(p, mask, device, s);
    default: return fa::launch_bwd_d128(p, mask, device, s);
  }
}

}  // namespace

extern "C" {

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hk, int Nq, int Nk, int D, int bool_mask_heads) {
  if (!sizes_ok(B, Hq, Hk, Nq, Nk, D)) return 0;
  if (bool_mask_heads != 0 && !mask_ok(B, Hq, Nq, Nk, bool_mask_heads)) return 0;
  return layout(B, Hq, Nq, Nk, D, bool_mask_heads).total;
}

int fa_bwd(const fa_tensor* dout, const fa_tensor* q, const fa_tensor* k, const fa_tensor* v, const fa_tensor* out,
           const float* lse, const float* dlse, const fa_mask* mask, int causal, const fa_tensor* dq,
           const fa_tensor* dk, const fa_tensor* dv, int B, int Hq, int Hk, int Nq, int Nk, int D, float scale,
           void* workspace, size_t workspace_bytes, void* stream) {
  // ---- validation: no CUDA call before this block passes ----
  if (B < 1 || Hq < 1 || Hk < 1 || Nq < 1 || Nk < 1) return FA_ERR_INVALID_ARGUMENT;
  if (!fa::head_dim_ok(D)) return FA_ERR_UNSUPPORTED;
  if (!sizes_ok(B, Hq, Hk, Nq, Nk, D) || !std::isfinite(scale) || !lse) return FA_ERR_INVALID_ARGUMENT;
  struct Side {
    const fa_tensor* t;
    int H, N;
  };
  const Side in[5] = {{dout, Hq, Nq}, {q, Hq, Nq}, {out, Hq, Nq}, {k, Hk, Nk}, {v, Hk, Nk}};
  const Side res[3] = {{dq, Hq, Nq}, {dk, Hk, Nk}, {dv, Hk, Nk}};
  for (const Side& x : in)
    if (!tensor_ok(x.t, B, x.H, x.N, D)) return FA_ERR_INVALID_ARGUMENT;
  for (const Side& x : res)
    if (!tensor_ok(x.t, B, x.H, x.N, D) || !fa::writes_once(*x.t, B, x.H, x.N, D)) return FA_ERR_INVALID_ARGUMENT;
  const size_t row_bytes = (size_t)B * Hq * Nq * sizeof(float);
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(dlse) & 3u)) return FA_ERR_INVALID_ARGUMENT;
  int kind = FA_MASK_NONE, mask_heads = 1;
  const void* mask_data = nullptr;
  size_t mask_bytes = 0;
  if (mask && mask->kind != FA_MASK_NONE) {
    kind = mask->kind;
    mask_data = mask->data;
    if (!mask_data) return FA_ERR_INVALID_ARGUMENT;
    if (kind == FA_MASK_KEY_PADDING) {
      mask_bytes = (size_t)B * Nk * 4;
    } else if (kind == FA_MASK_ADDITIVE || kind == FA_MASK_BOOL) {
      mask_heads = mask->heads;
      if (!mask_ok(B, Hq, Nq, Nk, mask_heads)) return FA_ERR_INVALID_ARGUMENT;
      mask_bytes = (size_t)B * mask_heads * Nq * Nk * (kind == FA_MASK_ADDITIVE ? 4 : 1);
    } else {
      return FA_ERR_INVALID_ARGUMENT;
    }
    if (kind != FA_MASK_BOOL && (reinterpret_cast<uintptr_t>(mask_data) & 3u)) return FA_ERR_INVALID_ARGUMENT;
  }
  const Layout l = layout(B, Hq, Nq, Nk, D, kind == FA_MASK_BOOL ? mask_heads : 0);
  if (!workspace || !aligned16(workspace) || workspace_bytes < l.total) return FA_ERR_INVALID_ARGUMENT;
  // Results share no element with what is read or with each other, and nothing
  // of the call lies in the workspace.
  struct Flat {
    const void* p;
    size_t n;
  };
  const Flat flat[3] = {{lse, row_bytes}, {dlse, dlse ? row_bytes : 0}, {mask_data, mask_bytes}};
  auto bytes = [&](const Side& x) { return (size_t)extent(*x.t, B, x.H, x.N, D) * 2; };
  for (const Flat& f : flat)
    if (ranges_overlap(workspace, l.total, f.p, f.n)) return FA_ERR_INVALID_ARGUMENT;
  for (const Side& x : in)
    if (ranges_overlap(workspace, l.total, x.t->data, bytes(x))) return FA_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i) {
    if (ranges_overlap(workspace, l.total, res[i].t->data, bytes(res[i]))) return FA_ERR_INVALID_ARGUMENT;
    for (const Flat& f : flat)
      if (ranges_overlap(res[i].t->data, bytes(res[i]), f.p, f.n)) return FA_ERR_INVALID_ARGUMENT;
    // (`apart` takes one length; tensors of two lengths in one buffer are told
    // apart by their ranges)
    auto meet = [&](const Side& y) {
      return res[i].N == y.N ? !apart(*res[i].t, res[i].H, *y.t, y.H, B, y.N, D, 2)
                             : ranges_overlap(res[i].t->data, bytes(res[i]), y.t->data, bytes(y));
    };
    for (const Side& x : in)
      if (meet(x)) return FA_ERR_INVALID_ARGUMENT;
    for (int j = i + 1; j < 3; ++j)
      if (meet(res[j])) return FA_ERR_INVALID_ARGUMENT;
  }

  // ---- set-up ----
  fa::DeviceState* st = nullptr;
  int rc = fa::current_device(&st);
  if (rc != FA_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const int qt = (Nq + 127) / 128, kt = (Nk + 127) / 128, group = Hq / Hk;
  fa::BwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.Hq = Hq;
  p.Hk = Hk;
  p.group = group;
  p.Nq = Nq;
  p.Nk = Nk;
  p.nqp = qt * 128;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.stat = reinterpret_cast<float*>(ws + l.stat);
  p.flags = reinterpret_cast<uint32_t*>(ws + l.flags);
  p.ref = reinterpret_cast<float*>(ws + l.ref);
  p.mask = mask_data;
  p.mask_heads = mask_heads;
  p.div_group = fa::FastDiv::make((uint32_t)group);
  p.timeout_ns = fa::timeout_ns_from_env();
  p.status = st->status;
  p.debug_record = st->debug_record;
  const char* inject = std::getenv("FA_FAULT_INJECT");
  p.inject_stall = (inject && std::strcmp(inject, "stall") == 0) ? 1 : 0;
  const int mk = kind == FA_MASK_KEY_PADDING ? fa::kBwdMaskKey
                 : kind == FA_MASK_ADDITIVE  ? fa::kBwdMaskAdd
                 : kind == FA_MASK_BOOL      ? fa::kBwdMaskBool
                                             : fa::kBwdMaskNone;
  p.mask_vec = Nk % 4 == 0 && aligned16(mask_data);
  p.bits_q = reinterpret_cast<uint32_t*>(ws + l.bits_q);
  p.bits_k = reinterpret_cast<uint32_t*>(ws + l.bits_k);
  p.words_q = kt * 4;
  p.words_k = qt * 4;
  p.tiles_q = reinterpret_cast<uint32_t*>(ws + l.tiles_q);
  p.tiles_k = reinterpret_cast<uint32_t*>(ws + l.tiles_k);
  p.tile_words_q = (kt + 31) / 32;
  p.tile_words_k = (qt + 31) / 32;
  p.dq = view(*dq);
  p.dk = view(*dk);
  p.dv = view(*dv);
  p.part[0] = reinterpret_cast<float*>(ws + l.part_kv);
  p.part[1] = reinterpret_cast<float*>(ws + l.part_q);
  p.div_hq = fa::FastDiv::make((uint32_t)Hq);
  p.div_hk = fa::FastDiv::make((uint32_t)Hk);
  if (encode(&p.q, *q, B, Hq, Nq, D) != FA_OK || encode(&p.dout, *dout, B, Hq, Nq, D) != FA_OK ||
      encode(&p.k, *k, B, Hk, Nk, D) != FA_OK || encode(&p.v, *v, B, Hk, Nk, D) != FA_OK)
    return FA_ERR_CUDA;
  for (int kv = 1; kv >= 0; --kv) {
    fa::BwdUnits u{};
    u.heads = B * (kv ? Hk : Hq);
    u.tiles = kv ? kt : qt;
    u.other = kv ? qt : kt;
    u.group = kv ? group : 1;
    u.causal = p.causal;
    u.rows_q = !kv;
    // Units of equal weight together where they are causal, unless a head alone
    // fills the SMs (its tiles then stay in L2).
    u.spread = p.causal && u.tiles < st->sm_count ? 1 : 0;
    u.div_heads = fa::FastDiv::make((uint32_t)u.heads);
    u.div_tiles = fa::FastDiv::make((uint32_t)u.tiles);
    p.plan[kv ? 0 : 1] = fa::bwd_plan(u, st->sm_count < kSlotCtas ? st->sm_count : kSlotCtas, kJoinCost);
  }

  if (kind == FA_MASK_BOOL) {
    fa::BwdBitsParams bp;
    bp.mask = static_cast<const uint8_t*>(mask_data);
    bp.bits_q = reinterpret_cast<uint32_t*>(ws + l.bits_q);
    bp.bits_k = reinterpret_cast<uint32_t*>(ws + l.bits_k);
    bp.some = reinterpret_cast<uint32_t*>(ws + l.some);
    bp.Nq = Nq;
    bp.Nk = Nk;
    bp.tiles_q = qt;
    bp.tiles_k = kt;
    rc = fa::launch_bwd_bits(bp, (long long)B * mask_heads, s);
    if (rc != FA_OK) return rc;
  }
  fa::BwdPrepParams pp;
  std::memset(&pp, 0, sizeof(pp));
  pp.out = view(*out);
  pp.dout = view(*dout);
  pp.lse = lse;
  pp.dlse = dlse;
  pp.q = view(*q);
  pp.k = view(*k);
  pp.v = view(*v);
  pp.stat = reinterpret_cast<float*>(ws + l.stat);
  pp.flags = reinterpret_cast<uint8_t*>(ws + l.flags);
  pp.ref = reinterpret_cast<float*>(ws + l.ref);
  if (kind == FA_MASK_KEY_PADDING || kind == FA_MASK_ADDITIVE) pp.mask = static_cast<const float*>(mask_data);
  pp.mask_heads = mask_heads;
  pp.mask_rows = kind == FA_MASK_ADDITIVE;
  pp.causal = p.causal;
  pp.group = group;
  pp.scale_log2 = p.scale_log2;
  pp.Hq = Hq;
  pp.Nq = Nq;
  pp.nqp = p.nqp;
  pp.div_h = fa::FastDiv::make((uint32_t)Hq);
  if (kind == FA_MASK_BOOL) pp.some = reinterpret_cast<const uint32_t*>(ws + l.some);
  if (kind == FA_MASK_KEY_PADDING) pp.key_mask = static_cast<const float*>(mask_data);
  pp.tiles_q = reinterpret_cast<uint32_t*>(ws + l.tiles_q);
  pp.tiles_k = reinterpret_cast<uint32_t*>(ws + l.tiles_k);
  pp.heads = kind == FA_MASK_BOOL ? B * mask_heads : B;
  pp.tiles_of_q = qt;
  pp.tiles_of_k = kt;
  pp.Nk = Nk;
  pp.tile_words_q = p.tile_words_q;
  pp.tile_words_k = p.tile_words_k;
  rc = fa::launch_bwd_prep(pp, (long long)B * Hq, D, s);
  if (rc != FA_OK) return rc;
  return launch(p, D, mk, st->device, s);
}

}  // extern "C"
