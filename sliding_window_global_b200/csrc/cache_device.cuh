// cache_device.cuh -- what the kernels that read a paged cache share: the rows of a
// sequence, checked, and the keys they see.
#pragma once

#include <stdint.h>

#include "cache_kernels.h"
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

}  // namespace swa
