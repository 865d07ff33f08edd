// cache_attend.cu -- attention over a paged cache: the entry points, and the fp32 kernel
// with the merge of its split sequences.  bf16 runs in cache_token.cu (few new tokens a
// sequence) and cache_chunk.cu (many).  The definition stands in include/swa.h.
//
// A row is one (new token, query head) pair; the rows of a KV head's query heads are
// packed token by token (row r = token * G + head in the group), so that a key tile is
// read once for the whole group.
#include <math.h>

#include <algorithm>

#include "cache_device.cuh"
#include "ptx.cuh"
#include "rotary_math.cuh"
#include "softmax_math.cuh"
#include "swa_host.h"

namespace swa {
namespace {

constexpr int kKeys = 64;                  // keys of a step of the CUDA-core kernel
constexpr int kCoreThreads = 256;
constexpr int kRowsMost = 32;              // rows of a sequence and KV head up to which the few-row kernel runs
constexpr int kRowsWarps = 4, kRowsBlocks = 3;                      // warps of its blocks, blocks an SM

template <int D, int RT>
constexpr int core_smem_bytes() {
  constexpr int kRows = 16 * RT;
  return (kRows * (D + 4) + 2 * kKeys * (D + 4) + kRows * (kKeys + 4)) * 4 + 2 * kKeys * 8;
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 RT rows x 64 keys a step in fp32 on the FMA pipe, each thread RT x 4 scores and RT x D/16
// outputs (two products an instruction; reads of shared memory bound it, which more rows a
// thread make fewer).  K of a step is fetched while V of the step before is used, and V
// while K is, both with cp.async; where each key lies is looked up a step ahead, by one
// thread a key.  The tile is 64 rows where those of a sequence fit, else 128: 2 x 256 tokens of 40
// heads, 8 KV heads, over 4096 keys, D = 128, take 1.40 ms with 128 (30 TFLOP/s) and 1.78 ms
// with 64 rows.
template <int D, int RT>
__global__ void __launch_bounds__(kCoreThreads) cache_core_kernel(const __grid_constant__ CacheAttendParams p,
                                                                  int row_tiles) {
  constexpr int kRows = 16 * RT;
  constexpr int LD = D + 4, LP = kKeys + 4;
  constexpr int NC = D / 64;               // float4 columns of a thread
  extern __shared__ float smem[];
  float* sQ = smem;
  float* sK = sQ + kRows * LD;
  float* sV = sK + kKeys * LD;
  float* sP = sV + kKeys * LD;
  long long* sAt = reinterpret_cast<long long*>(sP + kRows * LP);   // [2][keys] element offset of a key, < 0: none

  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int hk = blockIdx.y;
  const int split = blockIdx.x % p.nsplit;
  const int rt = blockIdx.x / p.nsplit % row_tiles;
  const int b = blockIdx.x / p.nsplit / row_tiles;
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && tid == 0 && rt == 0 && split == 0 && hk == 0) atomicOr(p.err, kDevErrCheck);
  const int rows = s.count * p.G;
  const int r0 = rt * kRows;
  if (r0 >= rows) return;

  // Q rows (zeros behind the last one)
  for (int e = tid; e < kRows * (D / 8); e += kCoreThreads) {
    const int r = e / (D / 8), c = e % (D / 8) * 8;
    float x[8];
    if (r0 + r < rows) {
      const int tok = (r0 + r) / p.G, h = hk * p.G + (r0 + r) % p.G;
      unpack(load_chunk(static_cast<const float*>(p.q) + (long long)(s.from + tok) * p.q_token + h * p.q_head + c), x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sQ[r * LD + c + i] = x[i];
  }

  const int t0 = r0 / p.G, t1 = min((r0 + kRows - 1) / p.G, s.count - 1);
  int lo = key_begin(p, s, t0);
  const int hi = key_end(s, t1);
  const int tiles = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;
  const int j0 = (int)((long long)tiles * split / p.nsplit), j1 = (int)((long long)tiles * (split + 1) / p.nsplit);

  int klo[RT], khi[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + ty * RT + i;
    klo[i] = r < rows ? key_begin(p, s, r / p.G) : 0;
    khi[i] = r < rows ? key_end(s, r / p.G) : 0;
  }
  float m[RT], l[RT], o[RT][4 * NC];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.f;
  }

  // a key exists if it lies in the tile's range and its page in the pool
  auto look_up = [&](int j) {
    if (tid >= kKeys) return;
    const int pos = lo + j * kKeys + tid;
    long long at = -1;
    if (j < j1 && pos < hi) {
      const int page = __ldg(p.block_table + (long long)b * p.max_pages + pos / p.page_size);
      if (page >= 0 && page < p.num_pages)
        at = (((long long)page * p.Hkv + hk) * p.page_size + pos % p.page_size) * D;
      else
        atomicOr(p.err, kDevErrCheck);
    }
    sAt[(j & 1) * kKeys + tid] = at;
  };
  auto fetch = [&](const void* pages, float* dst, int j) {         // zeros for a key that does not exist
#pragma unroll
    for (int e = tid; e < kKeys * (D / 4); e += kCoreThreads) {
      const int k = e / (D / 4), c = e % (D / 4) * 4;
      const long long at = sAt[(j & 1) * kKeys + k];
      copy16(dst + k * LD + c, static_cast<const float*>(pages) + (at < 0 ? 0 : at) + c, at >= 0);
    }
    copy_commit();
  };
  if (j0 < j1) {
    look_up(j0);
    __syncthreads();
    fetch(p.k_pages, sK, j0);
    fetch(p.v_pages, sV, j0);
  }
  for (int j = j0; j < j1; ++j) {
    const int key0 = lo + j * kKeys;
    look_up(j + 1);
    copy_wait<1>();                        // K of this step (V may be on its way)
    __syncthreads();
    float sc[RT][4], odd[RT][4];             // sums over even and odd d: two products an instruction
    bool there[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) there[k] = sAt[(j & 1) * kKeys + tx + 16 * k] >= 0;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[i][k] = odd[i][k] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 q4[RT], k4[4];
#pragma unroll
      for (int i = 0; i < RT; ++i) q4[i] = *reinterpret_cast<const float4*>(sQ + (ty * RT + i) * LD + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) k4[k] = *reinterpret_cast<const float4*>(sK + (tx + 16 * k) * LD + d);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ffma2(sc[i][k], odd[i][k], q4[i].x, q4[i].y, k4[k].x, k4[k].y, sc[i][k], odd[i][k]);
          ffma2(sc[i][k], odd[i][k], q4[i].z, q4[i].w, k4[k].z, k4[k].w, sc[i][k], odd[i][k]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float mx = m[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pos = key0 + tx + 16 * k;
        float x = (sc[i][k] + odd[i][k]) * p.scale;
        if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
        sc[i][k] = (pos >= klo[i] && pos < khi[i] && there[k]) ? x : -INFINITY;
        mx = fmaxf(mx, sc[i][k]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float alpha = m[i] == -INFINITY ? 0.f : expf(m[i] - ref);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float e = expf(sc[i][k] - ref);
        sP[(ty * RT + i) * LP + tx + 16 * k] = e;
        sum += e;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) o[i][c] *= alpha;
    }
    __syncthreads();                       // K has been read, P is written
    fetch(p.k_pages, sK, j + 1);           // behind the last step: zeros that nobody reads
    copy_wait<1>();                        // V of this step
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kKeys; k += 4) {
      float4 pr[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) pr[i] = *reinterpret_cast<const float4*>(sP + (ty * RT + i) * LP + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(sV + (k + kk) * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float w = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
            ffma2(o[i][4 * c], o[i][4 * c + 1], w, w, v.x, v.y, o[i][4 * c], o[i][4 * c + 1]);
            ffma2(o[i][4 * c + 2], o[i][4 * c + 3], w, w, v.z, v.w, o[i][4 * c + 2], o[i][4 * c + 3]);
          }
        }
      }
    }
    __syncthreads();                       // V has been read
    fetch(p.v_pages, sV, j + 1);
  }
  copy_wait<0>();

#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + ty * RT + i;
    if (r >= rows) continue;
    const long long row = (long long)(s.from + r / p.G) * p.Hq + hk * p.G + r % p.G;
    const bool has = l[i] != 0.f;          // also where every score is NaN
    const float inv = has ? 1.f / l[i] : 0.f;
    const float lse = has ? m[i] + logf(l[i]) : -INFINITY;
    if (p.nsplit > 1) {
      const long long pr = (long long)split * p.T * p.Hq + row;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4*>(p.part_o + pr * D + tx * 4 + 64 * c) =
            make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
      if (tx == 0) p.part_lse[pr] = lse;
    } else {
      float* out = static_cast<float*>(p.out) + row * D;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[tx * 4 + 64 * c + e] = o[i][4 * c + e] * inv;
      if (p.lse && tx == 0) p.lse[row] = lse;
    }
  }
}

template <int D>
constexpr int kRowsStages = 256 / D;       // steps of a warp's ring: 16 KB

// Few rows (single tokens) in fp32, RT at a time: the keys' bytes bound it, so a warp works on
// its own and keeps copies of the next step in flight. Sixteen lanes hold a key, each D/16 of its
// elements, and a warp takes eight keys a step (two halves of four). A lane reads only what
// it copied itself, so its own cp.async wait is all the order there is. RT x 4 partial dot
// products a lane are summed over the lanes by halving the list at each exchange, which
// leaves every lane RT/4 scores of its own to mask and exponentiate; the weights then go
// back to all lanes for the V products. A block's warps take its steps in turn and are
// joined through shared memory. Tiles of 4 or of 8 rows: more would not fit the registers.
// 8 sequences of 4000 keys, 32/8 heads, D = 128: 53 us (5.0 TB/s; 59 with K and V loaded into
// registers, 218 with cache_core_kernel); 32 ragged ones up to 16000 keys 272 us (86% of the
// copy rate). Two blocks of three stages take 51 and 328 us, one of eight warps 59 and 294.
// More rows read the keys anew a tile, from L2: 4 tokens (16 rows) of the first case 121 us, 8 tokens
// 198 us, where cache_core_kernel takes 219 and 371.
template <int D, int RT>
__global__ void __launch_bounds__(kRowsWarps * 32, kRowsBlocks)
cache_rows_kernel(const __grid_constant__ CacheAttendParams p, int row_tiles) {
  constexpr int U = 4, kStepKeys = 2 * U;  // keys of a half warp and of a step, which divide every page
  constexpr int E = D / 16, F4 = E / 4;    // elements of a lane, in float4s 64 elements apart
  constexpr int NL = U * RT / 16;          // scores a lane keeps: key lane / LR, rows (lane % LR) NL + i
  constexpr int LR = 16 / U;
  constexpr int kWarps = kRowsWarps, kThreads = kWarps * 32;
  constexpr int NST = kRowsStages<D>;
  __shared__ __align__(16) float sQ[RT * D];
  extern __shared__ float smem[];          // rings of the warps, afterwards their outputs
  __shared__ float sM[kWarps][RT], sL[kWarps][RT];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 15, half = lane >> 4;
  const int hk = blockIdx.y;
  const int split = blockIdx.x % p.nsplit;
  const int rt = blockIdx.x / p.nsplit % row_tiles;
  const int b = blockIdx.x / p.nsplit / row_tiles;
  grid_launch_dependents();
  const CacheSeq s = cache_seq(p, b);
  if (s.bad && tid == 0 && rt == 0 && split == 0 && hk == 0) atomicOr(p.err, kDevErrCheck);
  const int rows = s.count * p.G;
  const int r0 = rt * RT;
  if (r0 >= rows) return;

  const int lo = key_begin(p, s, r0 / p.G), hi = key_end(s, min((r0 + RT - 1) / p.G, s.count - 1));
  const int base = lo / kStepKeys * kStepKeys;
  const int steps = hi > lo ? (hi - base + kStepKeys - 1) / kStepKeys : 0;
  const int j0 = (int)((long long)steps * split / p.nsplit), j1 = (int)((long long)steps * (split + 1) / p.nsplit);

  int klo[NL], khi[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = r0 + (lane % LR) * NL + i;
    klo[i] = r < rows ? key_begin(p, s, r / p.G) : 0;
    khi[i] = r < rows ? key_end(s, r / p.G) : 0;
  }
  float m[NL], l[NL], o[RT][E];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) o[r][e] = 0.f;

  // a step's keys lie in one page: where they begin for this lane, < 0 if it does not exist
  const int32_t* table = p.block_table + (long long)b * p.max_pages;
  auto look_up = [&](int j) -> long long {
    if (j >= j1) return -1;
    const int pos = base + j * kStepKeys;
    const int page = __ldg(table + pos / p.page_size);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(p.err, kDevErrCheck);
      return -1;
    }
    return (((long long)page * p.Hkv + hk) * p.page_size + pos % p.page_size + half * U) * D + c * 4;
  };
  // a lane copies what it reads itself, so that its own wait is all it needs
  float* ring = smem + warp * NST * (2 * U * F4 * 128) + lane * 4;
  auto fetch = [&](int slot, long long at, int j) {          // zeros for keys outside [lo, hi)
    float* dst = ring + slot * (2 * U * F4 * 128);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = base + j * kStepKeys + half * U + u;
        const bool on = at >= 0 && pos >= lo && pos < hi;
        const float* src = static_cast<const float*>(kv ? p.v_pages : p.k_pages) + (on ? at + u * D : 0);
#pragma unroll
        for (int f = 0; f < F4; ++f) copy16(dst + ((kv * U + u) * F4 + f) * 128, src + f * 64, on);
      }
    copy_commit();
  };
  uint32_t exists = 0;                     // a bit a slot
  long long ahead;
  {
    long long at[NST];
#pragma unroll
    for (int st = 0; st < NST; ++st) at[st] = look_up(j0 + warp + st * kWarps);
#pragma unroll
    for (int st = 0; st < NST - 1; ++st) {
      fetch(st, at[st], j0 + warp + st * kWarps);
      exists |= (at[st] >= 0 ? 1u : 0u) << st;
    }
    ahead = at[NST - 1];
  }
  for (int e = tid; e < RT * (D / 4); e += kThreads) {
    const int r = e / (D / 4), at = e % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < rows)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                           (long long)(s.from + (r0 + r) / p.G) * p.q_token +
                                           (hk * p.G + (r0 + r) % p.G) * p.q_head + at);
    *reinterpret_cast<float4*>(sQ + r * D + at) = x;
  }
  __syncthreads();

  int slot = 0;
  for (int j = j0 + warp; j < j1; j += kWarps) {
    const int refill = slot == 0 ? NST - 1 : slot - 1;
    fetch(refill, ahead, j + (NST - 1) * kWarps);
    exists = (exists & ~(1u << refill)) | (ahead >= 0 ? 1u : 0u) << refill;
    ahead = look_up(j + NST * kWarps);
    copy_wait<NST - 1>();
    const float* now = ring + slot * (2 * U * F4 * 128);
    float4 k4[U][F4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < F4; ++f) k4[u][f] = *reinterpret_cast<const float4*>(now + (u * F4 + f) * 128);
    float x[U * RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float4 q4[F4];
#pragma unroll
      for (int f = 0; f < F4; ++f) q4[f] = *reinterpret_cast<const float4*>(sQ + r * D + f * 64 + c * 4);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float even = 0.f, odd = 0.f;
#pragma unroll
        for (int f = 0; f < F4; ++f) {
          ffma2(even, odd, q4[f].x, q4[f].y, k4[u][f].x, k4[u][f].y, even, odd);
          ffma2(even, odd, q4[f].z, q4[f].w, k4[u][f].z, k4[u][f].w, even, odd);
        }
        x[u * RT + r] = even + odd;
      }
    }
#pragma unroll
    for (int n = U * RT / 2, bit = 8; bit > 0; n >>= 1, bit >>= 1) {
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    const int pos = base + j * kStepKeys + half * U + c / LR;
    float mx[NL], alpha[NL];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      x[i] *= p.scale;
      if (p.softcap > 0.f) x[i] = p.softcap * tanhf(x[i] / p.softcap);
      x[i] = ((exists >> slot & 1) && pos >= klo[i] && pos < khi[i]) ? x[i] : -INFINITY;
      mx[i] = fmaxf(x[i], m[i]);
#pragma unroll
      for (int w = LR; w < 32; w <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], w));
      moved = moved || mx[i] != m[i];
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        alpha[i] = m[i] == -INFINITY ? 0.f : expf(m[i] - mx[i]);
        m[i] = mx[i];
        l[i] *= alpha[i];
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float f = __shfl_sync(0xffffffffu, alpha[r % NL], r / NL);
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] *= f;
      }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      x[i] = expf(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
      l[i] += x[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float4 v4[F4];
#pragma unroll
      for (int f = 0; f < F4; ++f) v4[f] = *reinterpret_cast<const float4*>(now + ((U + u) * F4 + f) * 128);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float w = __shfl_sync(0xffffffffu, x[r % NL], half * 16 + u * LR + r / NL);
#pragma unroll
        for (int f = 0; f < F4; ++f) {
          ffma2(o[r][4 * f], o[r][4 * f + 1], w, w, v4[f].x, v4[f].y, o[r][4 * f], o[r][4 * f + 1]);
          ffma2(o[r][4 * f + 2], o[r][4 * f + 3], w, w, v4[f].z, v4[f].w, o[r][4 * f + 2], o[r][4 * f + 3]);
        }
      }
    }
    slot = slot == NST - 1 ? 0 : slot + 1;
  }
  copy_wait<0>();
  __syncthreads();                         // the rings are read

#pragma unroll
  for (int i = 0; i < NL; ++i) {
#pragma unroll
    for (int w = LR; w < 32; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (lane < LR) {
      sM[warp][lane * NL + i] = m[i];
      sL[warp][lane * NL + i] = l[i];
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 16);
      if (half == 0) smem[(warp * RT + r) * D + e / 4 * 64 + c * 4 + e % 4] = o[r][e];
    }
  __syncthreads();
  for (int e = tid; e < RT * D; e += kThreads) {
    const int r = e / D, d = e % D;
    if (r0 + r >= rows) break;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sM[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sL[w][r] == 0.f ? 0.f : expf(sM[w][r] - top);
      sum += f * sL[w][r];
      acc += f * smem[(w * RT + r) * D + d];
    }
    const bool has = sum != 0.f;           // also where every score is NaN
    const float value = has ? acc / sum : 0.f, lse = has ? top + logf(sum) : -INFINITY;
    const long long row = (long long)(s.from + (r0 + r) / p.G) * p.Hq + hk * p.G + (r0 + r) % p.G;
    if (p.nsplit > 1) {
      const long long pr = (long long)split * p.T * p.Hq + row;
      p.part_o[pr * D + d] = value;
      if (d == 0) p.part_lse[pr] = lse;
    } else {
      static_cast<float*>(p.out)[row * D + d] = value;
      if (p.lse && d == 0) p.lse[row] = lse;
    }
  }
}

// out = sum_s exp(lse_s - lse) out_s over the splits in order, lse = log sum_s exp(lse_s):
// one warp a row.
template <int D>
__global__ void __launch_bounds__(128) cache_merge_kernel(const __grid_constant__ CacheAttendParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  grid_dependency_wait();
  const int h = (int)(id % p.Hq);
  const int i = (int)(id / p.Hq % p.max_tokens);
  const long long b = id / p.Hq / p.max_tokens;
  if (b >= p.B) return;
  const CacheSeq s = cache_seq(p, (int)b);
  if (i >= s.count) return;
  const long long row = (long long)(s.from + i) * p.Hq + h, step = (long long)p.T * p.Hq;
  float top = -INFINITY;
  for (int k = lane; k < p.nsplit; k += 32) top = fmaxf(top, p.part_lse[k * step + row]);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int k0 = 0; k0 < p.nsplit; k0 += 32) {
    const float w = k0 + lane < p.nsplit ? p.part_lse[(k0 + lane) * step + row] : -INFINITY;
    const float mine = w == -INFINITY ? 0.f : expf(w - top);   // a split without keys has zeros (NaN goes on)
    const int n = min(32, p.nsplit - k0);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float f = __shfl_sync(0xffffffffu, mine, k);
      sum += f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += f * p.part_o[((k0 + k) * step + row) * D + lane * E + e];
    }
  }
  const bool has = sum != 0.f;
  const float inv = has ? 1.f / sum : 0.f;
  float* out = static_cast<float*>(p.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = acc[e] * inv;
  if (p.lse && lane == 0) p.lse[row] = has ? top + logf(sum) : -INFINITY;
}

// ------------------------------------------------------------------ launches
template <int D, int RT>
cudaError_t launch_core(const CacheAttendParams& p, int row_tiles, cudaStream_t s) {
  constexpr int smem = core_smem_bytes<D, RT>();
  const cudaError_t e = allow_smem<&cache_core_kernel<D, RT>>(smem);
  if (e != cudaSuccess) return e;
  cache_core_kernel<D, RT><<<dim3((unsigned)((long long)p.B * row_tiles * p.nsplit), p.Hkv), kCoreThreads, smem, s>>>(
      p, row_tiles);
  return cudaGetLastError();
}

template <int D, int RT>
cudaError_t launch_rows(const CacheAttendParams& p, int row_tiles, cudaStream_t s) {
  constexpr int ring = kRowsWarps * kRowsStages<D> * 16 * D * 4, out = kRowsWarps * RT * D * 4;
  constexpr int smem = ring > out ? ring : out;
  static_assert(kRowsBlocks * (smem + RT * D * 4 + 8 * kRowsWarps * RT + 1024) <= 228 * 1024, "blocks an SM");
  const cudaError_t e = allow_smem<&cache_rows_kernel<D, RT>>(smem);
  if (e != cudaSuccess) return e;
  cache_rows_kernel<D, RT><<<dim3((unsigned)((long long)p.B * row_tiles * p.nsplit), p.Hkv), kRowsWarps * 32, smem, s>>>(
      p, row_tiles);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_core(const CacheAttendParams& p, int tile_rows, int row_tiles, cudaStream_t s) {
  return tile_rows == 4 ? launch_rows<D, 4>(p, row_tiles, s)
         : tile_rows == 8 ? launch_rows<D, 8>(p, row_tiles, s)
         : tile_rows == 64 ? launch_core<D, 4>(p, row_tiles, s) : launch_core<D, 8>(p, row_tiles, s);
}

cudaError_t launch_merge(const CacheAttendParams& p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.max_tokens * p.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.D == 64 ? cache_merge_kernel<64> : cache_merge_kernel<128>, p);
}

// A call that allows no sequence a token computes nothing: its bounds are checked all the same.
__global__ void cache_bounds_kernel(const __grid_constant__ CacheAttendParams p) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x)
    if (cache_seq(p, b).bad) atomicOr(p.err, kDevErrCheck);
}

cudaError_t launch_bounds(const CacheAttendParams& p, cudaStream_t s) {
  cache_bounds_kernel<<<1, 256, 0, s>>>(p);
  return cudaGetLastError();
}

// How a call is cut up, from sizes only: which kernel, and its parts.
struct AttendSplit {
  enum { kToken, kChunk, kCore } kernel;
  TokenSplit token;
  ChunkSplit chunk;
  int tile_rows, row_tiles, nsplit;        // CUDA-core kernel: rows of a tile, tiles, parts of the keys
  size_t bytes;                            // workspace
};

AttendSplit attend_split(const swa_cache& c, const swa_cache_batch& b, const swa_cache_attend_args& a, int max_tokens,
                         int max_len) {
  AttendSplit r = {};
  const int G = a.num_q_heads / c.num_kv_heads;
  // keys a sequence's new tokens can reach
  const long long reach = a.window < 0 ? max_len : std::min<long long>(max_len, (long long)a.window + max_tokens);
  // fp32 stays on the FMA pipe: the tensor core's products would keep 11 bits of it
  if (c.dtype == SWA_BF16) {
    if ((long long)max_tokens * G <= kTokenRows) {
      r.kernel = AttendSplit::kToken;
      r.token = token_split(b.batch, c.num_kv_heads, c.head_dim, max_tokens * G, reach);
      r.bytes = r.token.bytes;
    } else {
      r.kernel = AttendSplit::kChunk;
      r.chunk = chunk_split(b.batch, b.num_tokens, c.num_kv_heads, G, c.head_dim, c.page_size, max_tokens, max_len,
                            a.window);
      r.bytes = r.chunk.bytes;
    }
    return r;
  }
  r.kernel = AttendSplit::kCore;
  const long long rows = (long long)max_tokens * G;
  r.tile_rows = rows <= 4 ? 4 : rows <= kRowsMost ? 8 : rows <= 64 ? 64 : 128;
  r.row_tiles = (int)((rows + r.tile_rows - 1) / r.tile_rows);
  const long long blocks = std::max<long long>(1, (long long)b.batch * r.row_tiles * c.num_kv_heads);
  if (r.tile_rows > 8) {
    // parts of a step of keys at least, two blocks an SM
    r.nsplit = (int)std::max<long long>(1, std::min<long long>({(148 * 2 + blocks - 1) / blocks, reach / kKeys, 64}));
  } else {
    // One wave of blocks, in parts of 128 keys (four steps a warp) at least. Several sequences may
    // differ in length, so up to four waves in parts of 512 keys where these fill the GPU better
    // than 80%: 32 ragged sequences of up to 16000 keys 476 us in one wave, 328 in four (two
    // blocks an SM).
    const long long slots = 148 * kRowsBlocks;
    const auto fill = [&](long long n) { return (double)(n * blocks) / ((n * blocks + slots - 1) / slots * slots); };
    long long n = std::max<long long>(1, std::min(reach / 128, slots / blocks));
    double best = std::min(fill(n), 0.8);
    for (int waves = 2; waves <= 4 && b.batch > 1; ++waves) {
      const long long m = std::min(reach / 512, slots * waves / blocks);
      if (m > n && fill(m) > best * 1.03) {
        best = fill(m);
        n = m;
      }
    }
    r.nsplit = (int)n;
  }
  if (r.nsplit > 1) r.bytes = (size_t)r.nsplit * b.num_tokens * a.num_q_heads * (c.head_dim + 1) * 4;
  return r;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The longest sequence: the kernels' key numbers run past a sequence's end by less than
// 256 (a tile, or the steps fetched ahead) and have to stay in an int.
constexpr long long kLongest = 0x7fffffffLL - 255;

// Sizes of an attend call, checked: the status, and the bounds the kernels use.
swa_status attend_bounds(const swa_cache& c, const swa_cache_batch& b, const swa_cache_attend_args& a, int* max_tokens,
                         int* max_len) {
  swa_status st = check_cache(c);
  if (st == SWA_OK) st = check_batch(b);
  if (st != SWA_OK) return st;
  if (a.num_q_heads < 1 || a.num_q_heads % c.num_kv_heads != 0 || a.window < -1 || a.max_len < 0 ||
      !(a.softcap >= 0.f) || !isfinite(a.softcap) || !(a.scale >= 0.f) || !isfinite(a.scale) ||
      (b.cu_tokens && a.max_tokens < 0))
    return SWA_ERR_INVALID_ARG;
  if (a.num_q_heads > kMaxHeads) return SWA_ERR_UNSUPPORTED;
  const long long capacity = (long long)b.max_pages * c.page_size;
  *max_tokens = b.cu_tokens ? std::min(a.max_tokens, b.num_tokens) : (b.batch ? b.num_tokens / b.batch : 0);
  *max_len = (int)std::min<long long>({a.max_len ? a.max_len : capacity, capacity, kLongest});
  if ((long long)b.batch * *max_tokens * a.num_q_heads > 0x7fffffffLL ||
      (long long)b.num_tokens * a.num_q_heads > 0x7fffffffLL)
    return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

// The parameter block of a checked call but for the bounds and the workspace.
void fill_params(const swa_cache& c, const swa_cache_batch& b, const swa_cache_attend_args& a, CacheAttendParams* p) {
  p->k_pages = c.k_pages;
  p->v_pages = c.v_pages;
  p->q = a.q;
  p->out = a.out;
  p->lse = a.lse;
  p->block_table = b.block_table;
  p->seq_lens = b.seq_lens;
  p->cu_tokens = b.cu_tokens;
  p->err = c.error_word;
  p->q_token = a.q_stride[0];
  p->q_head = a.q_stride[1];
  p->B = b.batch;
  p->T = b.num_tokens;
  p->Hq = a.num_q_heads;
  p->Hkv = c.num_kv_heads;
  p->G = p->Hq / p->Hkv;
  p->D = c.head_dim;
  p->num_pages = c.num_pages;
  p->page_size = c.page_size;
  p->max_pages = b.max_pages;
  p->window = a.window;
  p->scale = a.scale == 0.f ? 1.f / sqrtf((float)p->D) : a.scale;
  p->softcap = a.softcap;
}

}  // namespace

swa_status check_cache(const swa_cache& c) {
  if (!c.k_pages || !c.v_pages || !c.error_word || !aligned16(c.k_pages) || !aligned16(c.v_pages) ||
      !aligned4(c.error_word) || c.num_pages < 1 || c.num_kv_heads < 1 || c.page_size < 1 || c.head_dim < 1 ||
      (c.dtype != SWA_BF16 && c.dtype != SWA_FP32))
    return SWA_ERR_INVALID_ARG;
  if ((c.head_dim != 64 && c.head_dim != 128) || c.page_size % 16 != 0 || c.num_kv_heads > kMaxHeads ||
      (long long)c.num_pages * c.num_kv_heads > 0x7fffffffLL)
    return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

swa_status check_batch(const swa_cache_batch& b) {
  if (b.batch < 0 || b.num_tokens < 0 || b.max_pages < 1) return SWA_ERR_INVALID_ARG;
  if (b.batch > 0 && b.num_tokens > 0 &&
      (!b.block_table || !b.seq_lens || !aligned4(b.block_table) || !aligned4(b.seq_lens) || !aligned4(b.cu_tokens) ||
       (!b.cu_tokens && b.num_tokens % b.batch != 0)))
    return SWA_ERR_INVALID_ARG;
  if (b.num_tokens > 0x7fffffff - 64) return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

}  // namespace swa

extern "C" {

size_t swa_cache_attend_workspace_bytes(const swa_cache* c, const swa_cache_batch* b, const swa_cache_attend_args* a) {
  int max_tokens, max_len;
  if (!c || !b || !a || swa::attend_bounds(*c, *b, *a, &max_tokens, &max_len) != SWA_OK) return 0;
  if (b->batch == 0 || b->num_tokens == 0 || max_tokens == 0) return 0;
  return swa::attend_split(*c, *b, *a, max_tokens, max_len).bytes;
}

swa_status swa_cache_attend(const swa_cache* c, const swa_cache_batch* b, const swa_cache_attend_args* a,
                            void* stream) {
  if (!c || !b || !a) return SWA_ERR_INVALID_ARG;
  swa::CacheAttendParams p = {};
  const swa_status st = swa::attend_bounds(*c, *b, *a, &p.max_tokens, &p.max_len);
  if (st != SWA_OK) return st;
  if (b->batch == 0 || b->num_tokens == 0) return SWA_OK;
  if (p.max_tokens == 0) {
    swa::fill_params(*c, *b, *a, &p);
    const cudaError_t e = swa::launch_bounds(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
  }
  const int64_t unit = c->dtype == SWA_FP32 ? 4 : 8;
  if (!a->q || !a->out || !swa::aligned16(a->q) || !swa::aligned16(a->out) || !swa::aligned4(a->lse) ||
      (b->num_tokens > 1 && (a->q_stride[0] <= 0 || a->q_stride[0] % unit)) ||
      (a->num_q_heads > 1 && (a->q_stride[1] <= 0 || a->q_stride[1] % unit)))
    return SWA_ERR_INVALID_ARG;
  const swa::AttendSplit sp = swa::attend_split(*c, *b, *a, p.max_tokens, p.max_len);
  swa::fill_params(*c, *b, *a, &p);
  p.nsplit = sp.nsplit;
  if (sp.bytes && (!a->workspace || !swa::aligned16(a->workspace) || a->workspace_bytes < sp.bytes))
    return SWA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (sp.kernel == swa::AttendSplit::kToken) {
    if (!sp.token.ok) return SWA_ERR_UNSUPPORTED;
    e = swa::launch_cache_token(p, sp.token, a->workspace, s);
    return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
  }
  if (sp.kernel == swa::AttendSplit::kChunk) {
    e = swa::launch_cache_chunk(p, sp.chunk, a->workspace, s);
    return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
  }
  if (p.nsplit > 1) {
    p.part_o = static_cast<float*>(a->workspace);
    p.part_lse = p.part_o + (size_t)p.nsplit * p.T * p.Hq * p.D;
  }
  e = p.D == 64 ? swa::launch_core<64>(p, sp.tile_rows, sp.row_tiles, s)
                : swa::launch_core<128>(p, sp.tile_rows, sp.row_tiles, s);
  if (e == cudaSuccess && p.nsplit > 1) e = swa::launch_merge(p, s);
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

swa_status swa_selftest_token_columns(const swa_cache* c, const swa_cache_batch* b, const swa_cache_attend_args* a,
                                      int32_t* columns) {
  swa::CacheAttendParams p = {};
  if (!c || !b || !a || !columns) return SWA_ERR_INVALID_ARG;
  const swa_status st = swa::attend_bounds(*c, *b, *a, &p.max_tokens, &p.max_len);
  if (st != SWA_OK) return st;
  if (b->batch == 0 || b->num_tokens == 0) return SWA_OK;
  swa::fill_params(*c, *b, *a, &p);
  swa::token_columns(p, columns);
  return SWA_OK;
}

swa_status swa_cache_check(const swa_cache* c, void* stream) {
  if (!c || !c->error_word || !swa::aligned4(c->error_word)) return SWA_ERR_INVALID_ARG;
  return swa::read_and_clear_error(c->error_word, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
