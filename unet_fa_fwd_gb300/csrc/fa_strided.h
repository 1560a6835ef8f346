// fa_strided.h — host-side checks of strided [B][H][N][D] tensors (the last
// axis contiguous) and of the axes of rotary positions, shared by the
// translation units of the C ABI.  No CUDA calls.
#pragma once

#include <climits>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"

namespace fa {

inline bool head_dim_ok(int D) { return D == 32 || D == 64 || D == 128; }

// a * b * c (each >= 0) is at most INT_MAX.
inline bool fits_int(int64_t a, int64_t b, int64_t c) { return (__int128)a * b * c <= INT_MAX; }

// Elements from the first to one past the last; 0 when that (or an offset)
// does not fit 62 bits or a stride is negative.
inline int64_t extent(const fa_tensor& t, int B, int H, int N, int D) {
  const long long strides[3] = {t.stride_b, t.stride_h, t.stride_n};
  const int sizes[3] = {B, H, N};
  __int128 e = D;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0) return 0;
    e += (__int128)strides[i] * (sizes[i] - 1);
  }
  return e > ((__int128)1 << 58) ? 0 : (int64_t)e;
}

// One axis of a difference of two rows' offsets: a multiple of `stride` from
// lo to hi times.
struct Step {
  int64_t stride, lo, hi;
};

// Whether some choice of multiples brings `at` + their sum within a row's D
// elements of 0 (`moved`: a multiple other than 0 has been chosen, or need not
// be).  Steps go from the largest stride to the smallest; a multiple that the
// rest cannot bring back is left out, which leaves two or three for axes that
// nest.  Layouts of which `budget` choices do not decide count as meeting.
inline bool meets(const Step* t, int n, __int128 at, int D, bool moved, int& budget) {
  if (--budget < 0) return true;
  if (n == 0) return moved && at > -D && at < D;
  __int128 rest_lo = 0, rest_hi = 0;
  for (int i = 1; i < n; ++i) {
    rest_lo += (__int128)t[i].stride * t[i].lo;
    rest_hi += (__int128)t[i].stride * t[i].hi;
  }
  // -D < at + z * stride + rest < D
  const __int128 from = -D + 1 - at - rest_hi, to = D - 1 - at - rest_lo;
  auto floor_div = [](__int128 a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
  __int128 lo = floor_div(from + t->stride - 1, t->stride), hi = floor_div(to, t->stride);
  if (lo < t->lo) lo = t->lo;
  if (hi > t->hi) hi = t->hi;
  for (__int128 z = lo; z <= hi; ++z)
    if (meets(t + 1, n - 1, at + z * t->stride, D, moved || z != 0, budget)) return true;
  return false;
}

constexpr int kMeetsBudget = 20000;

inline bool meets(const Step* t, int n, __int128 at, int D, bool moved) {
  int budget = kMeetsBudget;
  return meets(t, n, at, D, moved, budget);
}

inline void sort_steps(Step* t, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (t[j].stride > t[i].stride) {
        const Step s = t[i]; t[i] = t[j]; t[j] = s;
      }
}

// No element is written twice.
inline bool writes_once(const fa_tensor& x, int B, int H, int N, int D) {
  const long long st[3] = {x.stride_b, x.stride_h, x.stride_n};
  const int size[3] = {B, H, N};
  Step t[6];
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (st[i] < D) return false;
    t[n++] = Step{st[i], -(int64_t)(size[i] - 1), size[i] - 1};
  }
  sort_steps(t, n);
  int64_t span = D;  // axes that nest, each stepping over all that the smaller ones span, need no search
  int i = n;
  while (i > 0 && t[i - 1].stride >= span) {
    span += t[i - 1].stride * t[i - 1].hi;
    --i;
  }
  return i == 0 || !meets(t, n, 0, D, false);
}

// Two tensors of one element type share no element: their ranges are apart, or
// their rows interleave without meeting (slices of one buffer, in any order of
// its axes).
inline bool apart(const fa_tensor& a, int Ha, const fa_tensor& b, int Hb, int B, int N, int D, int size) {
  if (!ranges_overlap(a.data, (size_t)extent(a, B, Ha, N, D) * size, b.data,
                      (size_t)extent(b, B, Hb, N, D) * size))
    return true;
  const long long sa[3] = {a.stride_b, a.stride_h, a.stride_n}, sb[3] = {b.stride_b, b.stride_h, b.stride_n};
  const int na[3] = {B, Ha, N}, nb[3] = {B, Hb, N};
  Step t[6];
  int n = 0;
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {  // (equal strides of the two tensors are one step)
    if (stride == 0 || lo == hi) return;
    for (int i = 0; i < n; ++i)
      if (t[i].stride == stride) {
        t[i].lo += lo;
        t[i].hi += hi;
        return;
      }
    t[n++] = Step{stride, lo, hi};
  };
  for (int i = 0; i < 3; ++i) {
    add(sa[i], 0, na[i] - 1);
    add(sb[i], -(int64_t)(nb[i] - 1), 0);
  }
  sort_steps(t, n);
  const __int128 bytes = (__int128) reinterpret_cast<uintptr_t>(a.data) - reinterpret_cast<uintptr_t>(b.data);
  return !meets(t, n, bytes / size, D, true);  // (both are aligned to their elements)
}

// One tensor in one place.
inline bool same(const fa_tensor& a, const fa_tensor& b, int B, int H, int N) {
  return a.data == b.data && (B == 1 || a.stride_b == b.stride_b) && (H == 1 || a.stride_h == b.stride_h) &&
         (N == 1 || a.stride_n == b.stride_n);
}

// Every row starts 16-byte aligned.
inline bool rows16(const fa_tensor& t, int B, int H, int N, int size) {
  const int e = 16 / size;
  return aligned16(t.data) && (B == 1 || t.stride_b % e == 0) && (H == 1 || t.stride_h % e == 0) &&
         (N == 1 || t.stride_n % e == 0);
}

// The axes of rotary positions as the kernels take them: turns per unit of
// position of each of the D / 2 pairs, modulo one, as a 64-bit fraction, and the
// axis that each pair belongs to.  FA_OK or FA_ERR_INVALID_ARGUMENT.
inline int rope_pairs(const fa_rope_axes* axes, int D, unsigned long long* freq, unsigned char* axis) {
  if (axes->count < 1 || axes->count > FA_ROPE_MAX_AXES) return FA_ERR_INVALID_ARGUMENT;
  int sum = 0;
  for (int a = 0; a < axes->count; ++a) {
    if (axes->dims[a] < 2 || axes->dims[a] % 2 || axes->dims[a] > D) return FA_ERR_INVALID_ARGUMENT;
    if (!(axes->theta[a] > 0.0) || !std::isfinite(axes->theta[a]) || !std::isfinite(axes->scale[a]))
      return FA_ERR_INVALID_ARGUMENT;
    sum += axes->dims[a];
  }
  if (sum != D) return FA_ERR_INVALID_ARGUMENT;
  int pair = 0;
  for (int a = 0; a < axes->count; ++a)
    for (int j = 0; j < axes->dims[a] / 2; ++j, ++pair) {
      const double f = axes->scale[a] * std::pow(axes->theta[a], -2.0 * j / axes->dims[a]) * 0.15915494309189535;
      if (!std::isfinite(f)) return FA_ERR_INVALID_ARGUMENT;
      const double frac = f - std::floor(f);  // in [0, 1]; 1 only for a tiny negative f
      freq[pair] = frac < 1.0 ? (unsigned long long)(frac * 18446744073709551616.0) : 0ull;
      axis[pair] = (unsigned char)a;
    }
  return FA_OK;
}

// Elements of an int32 position array [B][N][count] with batch stride
// pos_stride_b, from the first to one past the last; -1 when they are too many.
inline int64_t rope_positions(long long pos_stride_b, int B, int N, int count) {
  const __int128 n = (__int128)pos_stride_b * (B - 1) + (__int128)N * count;
  return n > ((__int128)1 << 58) ? -1 : (int64_t)n;
}

}  // namespace fa
