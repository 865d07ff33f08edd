// rotary_math.cuh -- rotation of a head row by its position and the RMS norm of the
// row, for one thread that owns two 8-element chunks of it.
//
// A head row of D elements is shared by D / 16 threads.  Thread p owns the chunks
// (groups of 8 consecutive elements) p and p + D / 16 in the interleaved layout, whose
// pairs (2j, 2j + 1) lie inside a chunk; in the half layout it owns p and p + R / 16,
// which hold both elements of the pairs 8p .. 8p + 7, or two of the chunks behind the
// rotated part.  Either way a pair never leaves its thread, the threads of a row read
// consecutive 16 bytes, and a norm costs log2(D / 16) shuffles.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "softmax_math.cuh"

namespace swa {

constexpr int kMaxPairs = 64;              // rotated pairs of a head (head_dim <= 128)

// What every kernel that rotates or norms head rows needs of swa_rotation and
// swa_head_norm.
struct RotaryMath {
  uint64_t turn[kMaxPairs];                // turns per position of each pair, in units of 2^-64, modulo one turn
  float amp;
  float eps;
  int rot;                                 // R
  int weight_bf16;                         // element type of the norm's weights
};

// sin and cos of pi x for |x| <= 1/4, by their series: the first terms left out are below
// (pi / 4)^11 / 11! = 1.8e-9 and (pi / 4)^12 / 12! = 1.2e-10.
__device__ __forceinline__ void sincos_quarter(float x, float& s, float& c) {
  constexpr double kPi = 3.14159265358979323846, kPi2 = kPi * kPi;
  constexpr double kPi4 = kPi2 * kPi2, kPi6 = kPi4 * kPi2, kPi8 = kPi4 * kPi4;
  constexpr float pi_hi = static_cast<float>(kPi), pi_lo = static_cast<float>(kPi - static_cast<double>(pi_hi));
  const float y = x * x;
  float p = static_cast<float>(kPi8 * kPi / 362880);
  p = fmaf(p, y, static_cast<float>(-kPi6 * kPi / 5040));
  p = fmaf(p, y, static_cast<float>(kPi4 * kPi / 120));
  p = fmaf(p, y, static_cast<float>(-kPi2 * kPi / 6));
  p = fmaf(p, y, pi_lo);
  s = fmaf(x, pi_hi, x * p);
  float q = static_cast<float>(-kPi8 * kPi2 / 3628800);
  q = fmaf(q, y, static_cast<float>(kPi8 / 40320));
  q = fmaf(q, y, static_cast<float>(-kPi6 / 720));
  q = fmaf(q, y, static_cast<float>(kPi4 / 24));
  q = fmaf(q, y, static_cast<float>(-kPi2 / 2));
  c = fmaf(q, y, 1.f);
}

// cos and sin of t * freq, times amp. The position is a whole number, so the angle in turns
// can be formed modulo one in fixed point, exactly but for the frequency, which is cut to
// 2^-64 turns: with |t| up to 2^31 an error of at most 2^-33 turns. (32-bit floats would leave
// no digit of it at far positions, and 64-bit ones are slow.) The angle is then cut to 2^-32
// turns, and its rest to the nearest quarter turn rounded to 24 bits, an error below 2^-25
// of it.
__device__ __forceinline__ void rotary_angle(int t, uint64_t turn, float amp, float& c, float& s) {
  const uint32_t at = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(t)) * turn) >> 32);
  const uint32_t k = (at + 0x20000000u) >> 30;             // nearest quarter turn
  const int rest = static_cast<int>(at - (k << 30));
  float sf, cf;
  sincos_quarter(static_cast<float>(rest) * 0x1p-31f, sf, cf);
  const float cr = (k & 1) ? sf : cf;
  const float sr = (k & 1) ? cf : sf;
  c = (k == 1 || k == 2) ? -cr * amp : cr * amp;
  s = (k >= 2) ? -sr * amp : sr * amp;
}

// The two chunks of a thread and which of them rotate.
struct ChunkPair {
  int a, b;                                // chunk indexes
  bool ra, rb;                             // chunk a / b rotates (half layout: both or none)
};

template <int D, bool INTER>
__device__ __forceinline__ ChunkPair chunk_pair(int p, int rot) {
  ChunkPair c;
  if (INTER) {
    c.a = p;
    c.b = p + D / 16;
    c.ra = c.a * 8 < rot;
    c.rb = c.b * 8 < rot;
  } else {
    const int half = rot / 16;             // chunks of one half of the rotated part
    const bool r = p < half;
    c.a = r ? p : 2 * half + 2 * (p - half);
    c.b = r ? p + half : c.a + 1;
    c.ra = c.rb = r;
  }
  return c;
}

// cs[i], sn[i] of the thread's eight pairs: interleaved, 0-3 of chunk a and 4-7 of
// chunk b; half, the pairs 8p .. 8p + 7.
template <int D, bool INTER>
__device__ __forceinline__ void rotary_table(const RotaryMath& m, const ChunkPair& cp, int t, float (&cs)[8],
                                             float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool on = INTER ? (i < 4 ? cp.ra : cp.rb) : cp.ra;
    const int j = INTER ? (i < 4 ? 4 * cp.a + i : 4 * cp.b + i - 4) : 8 * cp.a + i;
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (on) rotary_angle(t, m.turn[j], m.amp, cs[i], sn[i]);
  }
}

// Rotate in place (BACK: by the opposite angle).  Elements that do not rotate are not
// touched, so that an infinity in one never meets the other of a would-be pair.
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const ChunkPair& cp, const float (&cs)[8],
                                       const float (&sn)[8]) {
  if (INTER) {
    if (cp.ra) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = BACK ? -sn[i] : sn[i];
        const float x = a[2 * i], y = a[2 * i + 1];
        a[2 * i] = x * cs[i] - y * s;
        a[2 * i + 1] = x * s + y * cs[i];
      }
    }
    if (cp.rb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = BACK ? -sn[4 + i] : sn[4 + i];
        const float x = b[2 * i], y = b[2 * i + 1];
        b[2 * i] = x * cs[4 + i] - y * s;
        b[2 * i + 1] = x * s + y * cs[4 + i];
      }
    }
  } else if (cp.ra) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {       // two pairs an instruction
      float x0, x1, y0, y1;
      const float s0 = BACK ? -sn[i] : sn[i], s1 = BACK ? -sn[i + 1] : sn[i + 1];
      fmul2(x0, x1, b[i], b[i + 1], -s0, -s1);
      fmul2(y0, y1, a[i], a[i + 1], s0, s1);
      ffma2(x0, x1, a[i], a[i + 1], cs[i], cs[i + 1], x0, x1);
      ffma2(b[i], b[i + 1], b[i], b[i + 1], cs[i], cs[i + 1], y0, y1);
      a[i] = x0;
      a[i + 1] = x1;
    }
  }
}

// Sum of the squares of a thread's elements.
__device__ __forceinline__ float squares(const float (&a)[8], const float (&b)[8]) {
  float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    ffma2(s0, s1, a[i], a[i + 1], a[i], a[i + 1], s0, s1);
    ffma2(t0, t1, b[i], b[i + 1], b[i], b[i + 1], t0, t1);
  }
  return (s0 + s1) + (t0 + t1);
}

// Sum over the D / 16 threads of a row (every lane of the warp takes part).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// ------------------------------------------------------------------ chunks in memory
// A chunk of 8 elements as it lies in memory: one 16-byte vector (bf16) or two (fp32).
template <typename T>
struct Chunk {
  static constexpr int kVec = sizeof(T) * 8 / 16;
  uint4 v[kVec];
};

template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < Chunk<T>::kVec; ++i) c.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return c;
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, const Chunk<T>& c) {
#pragma unroll
  for (int i = 0; i < Chunk<T>::kVec; ++i) reinterpret_cast<uint4*>(p)[i] = c.v[i];
}

__device__ __forceinline__ void unpack(const Chunk<float>& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(c.v[i].x);
    x[4 * i + 1] = __uint_as_float(c.v[i].y);
    x[4 * i + 2] = __uint_as_float(c.v[i].z);
    x[4 * i + 3] = __uint_as_float(c.v[i].w);
  }
}

__device__ __forceinline__ void unpack(const Chunk<__nv_bfloat16>& c, float (&x)[8]) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {            // bf16 is the upper half of an fp32
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void pack(const float (&x)[8], Chunk<float>& c) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    c.v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
}

__device__ __forceinline__ void pack(const float (&x)[8], Chunk<__nv_bfloat16>& c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  c.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}

// The norm's weights of a chunk (all ones without weights).
__device__ __forceinline__ void load_weights(const void* w, int weight_bf16, int chunk, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  } else if (weight_bf16) {
    unpack(load_chunk(static_cast<const __nv_bfloat16*>(w) + 8 * chunk), x);
  } else {
    unpack(load_chunk(static_cast<const float*>(w) + 8 * chunk), x);
  }
}

}  // namespace swa
