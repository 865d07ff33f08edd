// cache_device.cuh -- what the kernels that read a paged cache share: the rows of a
// sequence, checked, and the keys they see.
#pragma once

#include <stdint.h>

#include "cache_kernels.h"
#include "ptx.cuh"
#include "softmax_math.cuh"
#include "swa_kernels.h"

namespace swa {

// The new tokens of one sequence: rows [from, from + count) of the packed tensors at
// positions pos0, pos0 + 1, ...; keys exist at positions [0, limit).
struct CacheSeq {
  int from, count, pos0, limit;
  bool bad;                                // something of the call's bounds does not hold
};

// An entry of the call's index arrays (on the host, of a self-test's own).
__host__ __device__ __forceinline__ int load_index(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

__host__ __device__ __forceinline__ CacheSeq cache_seq(const CacheAttendParams& p, int b) {
  CacheSeq s;
  s.bad = false;
  int to;
  if (p.cu_tokens) {
    s.from = load_index(p.cu_tokens + b);
    to = load_index(p.cu_tokens + b + 1);
    if (s.from < 0 || to < s.from || to > p.T) {
      s.bad = true;
      s.from = to = 0;
    }
  } else {
    const int c = p.T / p.B;
    s.from = b * c;
    to = s.from + c;
  }
  const int len = load_index(p.seq_lens + b);
  const int all = to - s.from;
  s.count = min(all, p.max_tokens);
  // positions of tokens before the start of the sequence attend nothing
  s.pos0 = (int)max((long long)len - all, -(1LL << 30));
  s.limit = max(0, min(len, p.max_len));
  s.bad = s.bad || all > p.max_tokens || (all > 0 && (len > p.max_len || len < all));
  return s;
}

// Keys [lo, hi) that token i of the sequence attends (empty: lo >= hi). Neither end passes
// the limit, whatever length the device memory holds: a page of either exists in the table.
__host__ __device__ __forceinline__ int key_begin(const CacheAttendParams& p, const CacheSeq& s, int i) {
  return p.window < 0 ? 0 : (int)min((long long)s.limit, max(0LL, (long long)s.pos0 + i - p.window));
}
__host__ __device__ __forceinline__ int key_end(const CacheSeq& s, int i) { return min(s.pos0 + i + 1, s.limit); }

// ------------------------------------------------------------------ capped scores (bf16 kernels)
// cap tanh(s / cap) in units of log2 (s: the product, scaled inside). Two ways:
//  kCapUsual  cap - 2 cap / (1 + e^(2 s / cap)), two MUFU operations and few others. It takes
//             the difference of numbers of the size of the cap, so its error is cap 2^-22
//             whatever the score: 2^-15 for caps up to kCapUsualMost, far below what P in
//             bf16 costs.
//  kCapAny    the same where |s| >= cap / 8, so that the error is below |s| 2^-19; below that
//             the odd series s (1 - t^2 / 3 + 2 t^4 / 15), t = s / cap, whose first term left
//             out is 17 t^6 / 315 < 2^-22.
// A 4096-token chunk over 16384 keys, 32/8 heads, D = 128, takes 1600 us the first way and 1750 the
// second (802 without a cap); single tokens, bound by bytes, take the same either way.
constexpr int kCapNone = 0, kCapUsual = 1, kCapAny = 2;
constexpr float kCapUsualMost = 128.f;

__host__ __forceinline__ int cap_kind(float softcap) {
  return !(softcap > 0.f) ? kCapNone : softcap <= kCapUsualMost ? kCapUsual : kCapAny;
}

template <int CAP>
struct ScoreCap {
  float in, top, sl2;                      // 2 log2(e) scale / cap, cap log2(e), scale log2(e)
  __device__ __forceinline__ ScoreCap(float scale_log2, float softcap)
      // the smallest caps: a score of 0 must stay 0
      : in(CAP ? fminf(2.f * scale_log2 / softcap, 3.4e38f) : 0.f), top(softcap * 1.4426950408889634f), sl2(scale_log2) {}

  __device__ __forceinline__ void pair(float& s0, float& s1) const {
    float u0, u1, d0, d1, y0, y1;
    fmul2(u0, u1, s0, s1, in, in);
    fadd2(d0, d1, ex2_approx(u0), ex2_approx(u1), 1.f, 1.f);
    ffma2(y0, y1, rcp_approx(d0), rcp_approx(d1), -2.f * top, -2.f * top, top, top);
    if (CAP == kCapAny) {
      constexpr double kHalfLn2 = 0.34657359027997265;               // t = u ln(2) / 2
      constexpr float c1 = static_cast<float>(-kHalfLn2 * kHalfLn2 / 3);
      constexpr float c2 = static_cast<float>(2 * kHalfLn2 * kHalfLn2 * kHalfLn2 * kHalfLn2 / 15);
      constexpr float bend = static_cast<float>(0.125 / kHalfLn2);
      float w0, w1, p0, p1;
      fmul2(w0, w1, u0, u1, u0, u1);
      ffma2(p0, p1, w0, w1, c2, c2, c1, c1);
      fmul2(p0, p1, p0, p1, w0, w1);
      fmul2(w0, w1, s0, s1, sl2, sl2);
      ffma2(p0, p1, w0, w1, p0, p1, w0, w1);
      y0 = fabsf(u0) < bend ? p0 : y0;
      y1 = fabsf(u1) < bend ? p1 : y1;
    }
    s0 = y0;
    s1 = y1;
  }
};

}  // namespace swa
