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
// thread a key.  The tile is the smallest of 16, 64 and 128 rows that the rows of a sequence
// fill: 2 x 256 tokens of 40 heads, 8 KV heads, over 4096 keys, D = 128, take 1.40 ms with 128
// (30 TFLOP/s) and 1.78 ms with 64 rows; one token of 8 sequences of 4000 keys 218 us with 16
// and 370 us with 64.
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
    const bool has = m[i] != -INFINITY;
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

// out = sum_s exp(lse_s - lse) out_s over the splits in order, lse = log sum_s exp(lse_s):
// one warp a row.
template <int D>
__global__ void __launch_bounds__(128) cache_merge_kernel(const __grid_constant__ CacheAttendParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(id % p.Hq);
  const int i = (int)(id / p.Hq % p.max_tokens);
  const long long b = id / p.Hq / p.max_tokens;
  if (b >= p.B) return;
  const CacheSeq s = cache_seq(p, (int)b);
  if (i >= s.count) return;
  const long long row = (long long)(s.from + i) * p.Hq + h, step = (long long)p.T * p.Hq;
  float top = -INFINITY;
  for (int k = 0; k < p.nsplit; ++k) top = fmaxf(top, p.part_lse[k * step + row]);
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int k = 0; k < p.nsplit; ++k) {
    const float w = p.part_lse[k * step + row];
    if (w == -INFINITY) continue;          // a split without keys (NaN goes on)
    const float f = expf(w - top);
    sum += f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * p.part_o[(k * step + row) * D + lane * E + e];
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

template <int D>
cudaError_t launch_core(const CacheAttendParams& p, int tile_rows, int row_tiles, cudaStream_t s) {
  return tile_rows == 16 ? launch_core<D, 1>(p, row_tiles, s)
         : tile_rows == 64 ? launch_core<D, 4>(p, row_tiles, s) : launch_core<D, 8>(p, row_tiles, s);
}

cudaError_t launch_merge(const CacheAttendParams& p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.max_tokens * p.Hq;
  const unsigned blocks = (unsigned)((rows + 3) / 4);
  if (p.D == 64) cache_merge_kernel<64><<<blocks, 128, 0, s>>>(p);
  else cache_merge_kernel<128><<<blocks, 128, 0, s>>>(p);
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
      r.chunk = chunk_split(b.batch, b.num_tokens, c.num_kv_heads, G, c.head_dim, c.page_size, max_len, a.window);
      r.bytes = r.chunk.bytes;
    }
    return r;
  }
  r.kernel = AttendSplit::kCore;
  const long long rows = (long long)max_tokens * G;
  r.tile_rows = rows <= 16 ? 16 : rows <= 64 ? 64 : 128;
  r.row_tiles = (int)((rows + r.tile_rows - 1) / r.tile_rows);
  // parts of a step of keys at least, two blocks an SM
  const long long blocks = (long long)b.batch * r.row_tiles * c.num_kv_heads;
  const long long want = (148 * 2 + blocks - 1) / std::max<long long>(blocks, 1);
  r.nsplit = (int)std::max<long long>(1, std::min<long long>({want, reach / kKeys, 64}));
  if (r.nsplit > 1) r.bytes = (size_t)r.nsplit * b.num_tokens * a.num_q_heads * (c.head_dim + 1) * 4;
  return r;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

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
  *max_len = (int)std::min<long long>(a.max_len ? a.max_len : capacity, capacity);
  if ((long long)b.batch * *max_tokens * a.num_q_heads > 0x7fffffffLL ||
      (long long)b.num_tokens * a.num_q_heads > 0x7fffffffLL)
    return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
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
  if (b->batch == 0 || b->num_tokens == 0 || p.max_tokens == 0) return SWA_OK;
  const int64_t unit = c->dtype == SWA_FP32 ? 4 : 8;
  if (!a->q || !a->out || !swa::aligned16(a->q) || !swa::aligned16(a->out) || !swa::aligned4(a->lse) ||
      (b->num_tokens > 1 && (a->q_stride[0] <= 0 || a->q_stride[0] % unit)) ||
      (a->num_q_heads > 1 && (a->q_stride[1] <= 0 || a->q_stride[1] % unit)))
    return SWA_ERR_INVALID_ARG;
  const swa::AttendSplit sp = swa::attend_split(*c, *b, *a, p.max_tokens, p.max_len);
  p.k_pages = c->k_pages;
  p.v_pages = c->v_pages;
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  p.block_table = b->block_table;
  p.seq_lens = b->seq_lens;
  p.cu_tokens = b->cu_tokens;
  p.err = c->error_word;
  p.q_token = a->q_stride[0];
  p.q_head = a->q_stride[1];
  p.B = b->batch;
  p.T = b->num_tokens;
  p.Hq = a->num_q_heads;
  p.Hkv = c->num_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.D = c->head_dim;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.max_pages = b->max_pages;
  p.window = a->window;
  p.nsplit = sp.nsplit;
  p.scale = a->scale == 0.f ? 1.f / sqrtf((float)p.D) : a->scale;
  p.softcap = a->softcap;
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

swa_status swa_cache_check(const swa_cache* c, void* stream) {
  if (!c || !c->error_word || !swa::aligned4(c->error_word)) return SWA_ERR_INVALID_ARG;
  return swa::read_and_clear_error(c->error_word, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
