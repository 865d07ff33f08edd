// rotary.cu -- rotary positions and per-head RMS norms of queries and keys ("SWAN-GPT"
// §3.3(1): the sliding-window layers rotate q and k by position), their gradients, and
// the append into a paged cache, which rotates on the way.  The formulas stand in
// include/swa.h.
//
// What bounds it: every element is read once and written once for a handful of
// operations, so memory does.  A block takes 16 (D = 128) or 32 (D = 64) tokens and a
// run of heads; a thread keeps the cosines and sines of its eight pairs in registers
// for all those heads (they depend on the token only), and loads a group of heads ahead of
// the arithmetic, which keeps enough bytes in flight.  Rows may lie anywhere: a
// projection's token-major output is read in place and written head-major, in runs of
// 16 bytes a thread and 128 or more a row.
#include <math.h>

#include <algorithm>

#include "cache_kernels.h"
#include "ptx.cuh"
#include "rotary_kernels.h"
#include "swa_kernels.h"

namespace swa {
namespace {

constexpr int kRotaryThreads = 128;
// Heads of a block at most. Forward, a 2 x 8191-token normed prompt: 57.5 us with 32, 59.7 with
// 16. Backward, a normed 16384-token prompt: 131 us with 16, whose items the blocks share
// out evenly, 134 with 8, 143 with 32 (before the products went two an instruction: 56 and
// 129 us now).
constexpr int kForwardRun = 32, kBackwardRun = 16;
// Blocks of an SM that the registers must allow. Forward: four (128 registers; 104.5 us for
// the plain 32768-token prompt, 106.7 without the bound). Backward: five without a norm; with
// one the compiler's own choice, since four blocks would spill (131 to 163 us). That is 158 to
// 168 registers and three blocks an SM for bf16 heads in the interleaved layout, and in the half
// layout with bf16 upstream gradients; 176 to 186 registers and two blocks in the half layout
// with fp32 upstream gradients and for fp32 heads. 16384 tokens of 32 + 8 heads, D = 128, bf16
// heads and fp32 gradients: 129 us interleaved, 164 in the half layout.
// Append: three, whose look-ups need more registers (normed prompts 45.9 us, 51.6 with four).
constexpr int kForwardBlocks = 4, kBackwardBlocks = 5, kAppendBlocks = 3;

template <typename T>
__host__ __device__ constexpr int unroll_heads() {
  return sizeof(T) == 2 ? 4 : 1;
}

// Which kind of rows block `y` works on, and which run of its heads.
struct Segment {
  int kind, run;
};

__device__ __forceinline__ Segment segment_of(const int* segs, int kinds, int y) {
  Segment s;
  s.kind = 0;
  while (s.kind + 1 < kinds && y >= segs[s.kind]) y -= segs[s.kind++];
  s.run = y;
  return s;
}

// A packed token of a cache call: its position and the row of its page.  ok is false
// for a row that belongs to no sequence and for one whose place does not exist (which
// also sets the error bit).
struct CacheToken {
  bool ok;
  int pos;
  long long page_row;                      // row of (page, head 0, slot) in the pools
};

__device__ __forceinline__ CacheToken cache_token(const RotaryParams& p, int tok) {
  CacheToken t;
  t.ok = false;
  t.pos = 0;
  t.page_row = 0;
  if (tok >= p.tokens) return t;
  int b, from, to;
  if (p.cu_tokens) {
    // the first sequence that ends behind the token
    int lo = 0, hi = p.batch;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_tokens + mid + 1) <= tok) lo = mid + 1;
      else hi = mid;
    }
    b = lo;
    if (b >= p.batch) return t;                           // behind the last sequence
    from = __ldg(p.cu_tokens + b);
    to = __ldg(p.cu_tokens + b + 1);
    if (from < 0 || tok < from || to > p.tokens) {
      atomicOr(p.err, kDevErrCheck);
      return t;
    }
  } else {
    const int c = p.tokens / p.batch;
    b = tok / c;
    from = b * c;
    to = from + c;
  }
  const long long pos = (long long)__ldg(p.seq_lens + b) - (to - tok);
  if (pos < 0 || pos >= (long long)p.max_pages * p.page_size) {
    atomicOr(p.err, kDevErrCheck);
    return t;
  }
  const int page = __ldg(p.block_table + (long long)b * p.max_pages + pos / p.page_size);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.err, kDevErrCheck);
    return t;
  }
  t.ok = true;
  t.pos = (int)pos;
  t.page_row = (long long)page * p.num_kv_heads * p.page_size + pos % p.page_size;
  return t;
}

template <typename T, int D, bool NORM, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kRotaryThreads, CACHE ? kAppendBlocks : kForwardBlocks) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kPer = D / 16;                             // threads of a row
  constexpr int U = unroll_heads<T>();
  const int th = threadIdx.x % kPer;
  const long long tok = (long long)blockIdx.x * (kRotaryThreads / kPer) + threadIdx.x / kPer;
  const Segment sg = segment_of(p.segs, CACHE ? 3 : 2, blockIdx.y);
  const HeadRows& r = p.rows[sg.kind];
  const int h_begin = sg.run * p.heads_per_seg, h_end = min(r.heads, h_begin + p.heads_per_seg);
  const bool live = tok < p.tokens;
  const int batch = live && !CACHE ? (int)tok / p.n : 0, at = live && !CACHE ? (int)tok % p.n : 0;
  const ChunkPair cp = chunk_pair<D, INTER>(th, p.m.rot);
  const T* src = static_cast<const T*>(r.src) + (CACHE ? tok * r.st : batch * r.sb + at * r.st);
  // The loads run one group of heads ahead of the arithmetic, the first one ahead of the
  // token's place and its cosines.
  Chunk<T> na[U], nb[U];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      na[u] = Chunk<T>{};
      nb[u] = Chunk<T>{};
      if (live && h0 + u < h_end) {
        const T* x = src + (h0 + u) * r.sh;
        na[u] = load_chunk(x + 8 * cp.a);
        nb[u] = load_chunk(x + 8 * cp.b);
      }
    }
  };
  fetch(h_begin);
  bool ok = live;
  int pos = 0;
  long long dst_off = 0, dst_head = r.dh;
  if (CACHE) {
    const CacheToken t = cache_token(p, (int)min(tok, (long long)p.tokens));
    ok = t.ok;
    pos = t.pos;
    if (sg.kind == 0) {
      dst_off = tok * r.dt;
    } else {
      dst_off = t.page_row * D;
      dst_head = (long long)p.page_size * D;
    }
  } else if (live) {
    pos = p.positions ? __ldg(p.positions + tok) : (int)((unsigned)p.start + (unsigned)at);
    dst_off = batch * r.db + at * r.dt;
  }
  T* dst = static_cast<T*>(r.dst) + dst_off;
  const bool copy = CACHE && sg.kind == 2;                 // values are stored as they come
  float cs[8], sn[8], wa[8], wb[8];
  if (!copy) {
    if (NORM) {
      load_weights(r.weight, p.m.weight_bf16, cp.a, wa);
      load_weights(r.weight, p.m.weight_bf16, cp.b, wb);
    }
    rotary_table<D, INTER>(p.m, cp, pos, cs, sn);
  }
  for (int h0 = h_begin; h0 < h_end; h0 += U) {
    Chunk<T> a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u] = na[u];
      b[u] = nb[u];
    }
    fetch(h0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!copy) {
        float xa[8], xb[8];
        unpack(a[u], xa);
        unpack(b[u], xb);
        if (NORM) {
          const float inv = __frsqrt_rn(row_sum<D>(squares(xa, xb)) * (1.f / D) + p.m.eps);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            fmul2(xa[i], xa[i + 1], xa[i], xa[i + 1], inv, inv);
            fmul2(xa[i], xa[i + 1], xa[i], xa[i + 1], wa[i], wa[i + 1]);
            fmul2(xb[i], xb[i + 1], xb[i], xb[i + 1], inv, inv);
            fmul2(xb[i], xb[i + 1], xb[i], xb[i + 1], wb[i], wb[i + 1]);
          }
        }
        rotate<INTER, false>(xa, xb, cp, cs, sn);
        pack(xa, a[u]);
        pack(xb, b[u]);
      }
      if (ok && h0 + u < h_end) {
        T* y = dst + (h0 + u) * dst_head;
        store_chunk(y + 8 * cp.a, a[u]);
        store_chunk(y + 8 * cp.b, b[u]);
      }
    }
  }
}

// With u = x r, r = 1 / rms, and h the upstream gradient turned back:
//   dw = sum of h u over all rows,  dx = r (w h - u mean(w h u)).
// Each block adds up its rows' dw in registers and writes one partial row; the
// reduction below adds the partials in a fixed order.
template <typename T, typename G, typename O, int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads, NORM ? 1 : kBackwardBlocks) rotary_backward_kernel(const __grid_constant__
                                                                             RotaryBackwardParams p) {
  constexpr int kPer = D / 16;
  constexpr int kTok = kRotaryThreads / kPer;
  constexpr int U = 1;
  const int th = threadIdx.x % kPer, row = threadIdx.x / kPer;
  grid_launch_dependents();
  const int kind = blockIdx.x >= p.blocks[0];
  const int first = kind ? blockIdx.x - p.blocks[0] : blockIdx.x;
  const HeadRows& r = p.grad[kind];
  const ChunkPair cp = chunk_pair<D, INTER>(th, p.m.rot);
  float wa[8], wb[8], da[8], db[8];
  if (NORM) {
    load_weights(r.weight, p.m.weight_bf16, cp.a, wa);
    load_weights(r.weight, p.m.weight_bf16, cp.b, wb);
#pragma unroll
    for (int i = 0; i < 8; ++i) da[i] = db[i] = 0.f;
  }
  const long long tiles = ((long long)p.tokens + kTok - 1) / kTok;
  const long long items = tiles * p.segs[kind];
  for (long long it = first; it < items; it += p.blocks[kind]) {
    const long long tok = it / p.segs[kind] * kTok + row;
    const int hs = (int)(it % p.segs[kind]) * p.heads_per_seg;
    const int he = min(r.heads, hs + p.heads_per_seg);
    const bool ok = tok < p.tokens;
    int pos = 0;
    long long g_off = 0, o_off = 0, x_off = 0;
    if (ok) {
      const int b = (int)tok / p.n, i = (int)tok % p.n;
      pos = p.positions ? __ldg(p.positions + tok) : (int)((unsigned)p.start + (unsigned)i);
      g_off = b * r.sb + i * r.st;
      o_off = b * r.db + i * r.dt;
      x_off = b * p.xb[kind] + i * p.xt[kind];
    }
    const G* g = static_cast<const G*>(r.src) + g_off;
    O* o = static_cast<O*>(r.dst) + o_off;
    const T* x = static_cast<const T*>(p.x[kind]) + x_off;
    Chunk<G> nga[U], ngb[U];
    Chunk<T> nxa[U], nxb[U];
    auto fetch = [&](int h0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        nga[u] = ngb[u] = Chunk<G>{};
        nxa[u] = nxb[u] = Chunk<T>{};
        if (ok && h0 + u < he) {
          const G* gp = g + (h0 + u) * r.sh;
          nga[u] = load_chunk(gp + 8 * cp.a);
          ngb[u] = load_chunk(gp + 8 * cp.b);
          if (NORM) {
            const T* xp = x + (h0 + u) * p.xh[kind];
            nxa[u] = load_chunk(xp + 8 * cp.a);
            nxb[u] = load_chunk(xp + 8 * cp.b);
          }
        }
      }
    };
    fetch(hs);                             // as in the forward kernel, ahead of the arithmetic
    float cs[8], sn[8];
    rotary_table<D, INTER>(p.m, cp, pos, cs, sn);
    for (int h0 = hs; h0 < he; h0 += U) {
      Chunk<G> ga[U], gb[U];
      Chunk<T> xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ga[u] = nga[u];
        gb[u] = ngb[u];
        xa[u] = nxa[u];
        xb[u] = nxb[u];
      }
      fetch(h0 + U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float ha[8], hb[8];
        unpack(ga[u], ha);
        unpack(gb[u], hb);
        rotate<INTER, true>(ha, hb, cp, cs, sn);
        if (NORM) {
          float ua[8], ub[8];
          unpack(xa[u], ua);
          unpack(xb[u], ub);
          const float inv = __frsqrt_rn(row_sum<D>(squares(ua, ub)) * (1.f / D) + p.m.eps);
          const bool live = ok && h0 + u < he;             // a row of zeros with eps 0 has no norm
          float d0 = 0.f, d1 = 0.f, e0 = 0.f, e1 = 0.f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            fmul2(ua[i], ua[i + 1], ua[i], ua[i + 1], inv, inv);
            fmul2(ub[i], ub[i + 1], ub[i], ub[i + 1], inv, inv);
            if (live) {
              ffma2(da[i], da[i + 1], ha[i], ha[i + 1], ua[i], ua[i + 1], da[i], da[i + 1]);
              ffma2(db[i], db[i + 1], hb[i], hb[i + 1], ub[i], ub[i + 1], db[i], db[i + 1]);
            }
            fmul2(ha[i], ha[i + 1], ha[i], ha[i + 1], wa[i], wa[i + 1]);
            fmul2(hb[i], hb[i + 1], hb[i], hb[i + 1], wb[i], wb[i + 1]);
            ffma2(d0, d1, ha[i], ha[i + 1], ua[i], ua[i + 1], d0, d1);
            ffma2(e0, e1, hb[i], hb[i + 1], ub[i], ub[i + 1], e0, e1);
          }
          const float dot = -row_sum<D>((d0 + d1) + (e0 + e1)) * (1.f / D);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            ffma2(ha[i], ha[i + 1], ua[i], ua[i + 1], dot, dot, ha[i], ha[i + 1]);
            ffma2(hb[i], hb[i + 1], ub[i], ub[i + 1], dot, dot, hb[i], hb[i + 1]);
            fmul2(ha[i], ha[i + 1], ha[i], ha[i + 1], inv, inv);
            fmul2(hb[i], hb[i + 1], hb[i], hb[i + 1], inv, inv);
          }
        }
        if (ok && h0 + u < he) {
          Chunk<O> c;
          O* op = o + (h0 + u) * r.dh;
          pack(ha, c);
          store_chunk(op + 8 * cp.a, c);
          pack(hb, c);
          store_chunk(op + 8 * cp.b, c);
        }
      }
    }
  }
  if (NORM && p.partial) {
    // over the tokens of a warp (lanes of one column are kPer apart), then the warps
    __shared__ float sum[kRotaryThreads / 32][D];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int s = 16; s >= kPer; s >>= 1) {
        da[i] += __shfl_xor_sync(0xffffffffu, da[i], s);
        db[i] += __shfl_xor_sync(0xffffffffu, db[i], s);
      }
      if ((threadIdx.x & 31) < kPer) {
        sum[threadIdx.x >> 5][8 * cp.a + i] = da[i];
        sum[threadIdx.x >> 5][8 * cp.b + i] = db[i];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kRotaryThreads / 32; ++w) t += sum[w][threadIdx.x];
      p.partial[(long long)blockIdx.x * D + threadIdx.x] = t;
    }
  }
}

// dweight[kind][column] = sum of the kind's partial rows: a block takes 8 columns, each of
// its 128 rows of threads a strided run of partials (all its loads in flight at once), and
// the runs are added up in a tree: one order, whatever the timing.
__global__ void __launch_bounds__(1024) rotary_weight_kernel(const float* partial, int blocks_q, int blocks_k, int D,
                                                             float* dq_weight, float* dk_weight) {
  __shared__ double run[128][9];
  const int kind = blockIdx.y;
  float* out = kind ? dk_weight : dq_weight;
  if (!out) return;
  const int col = blockIdx.x * 8 + threadIdx.x;
  const float* src = partial + (kind ? (long long)blocks_q * D : 0) + col;
  const int n = kind ? blocks_k : blocks_q;
  grid_dependency_wait();
  double t = 0.0;
#pragma unroll 8
  for (int i = threadIdx.y; i < n; i += 128) t += src[(long long)i * D];
  run[threadIdx.y][threadIdx.x] = t;
  for (int s = 64; s > 0; s >>= 1) {
    __syncthreads();
    if ((int)threadIdx.y < s) run[threadIdx.y][threadIdx.x] += run[threadIdx.y + s][threadIdx.x];
  }
  if (threadIdx.y == 0) out[col] = (float)run[0][threadIdx.x];
}

__global__ void zero_weight_kernel(float* a, float* b, int n) {
  if ((int)threadIdx.x < n) {
    if (a) a[threadIdx.x] = 0.f;
    if (b) b[threadIdx.x] = 0.f;
  }
}

// ------------------------------------------------------------------ dispatch
template <typename T, int D, bool NORM, bool CACHE>
cudaError_t launch_rotary_layout(const RotaryParams& p, bool inter, cudaStream_t s) {
  const long long tiles = ((long long)p.tokens + kRotaryThreads / (D / 16) - 1) / (kRotaryThreads / (D / 16));
  const dim3 grid((unsigned)tiles, (unsigned)(p.segs[0] + p.segs[1] + (CACHE ? p.segs[2] : 0)));
  if (inter) rotary_kernel<T, D, NORM, true, CACHE><<<grid, kRotaryThreads, 0, s>>>(p);
  else rotary_kernel<T, D, NORM, false, CACHE><<<grid, kRotaryThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, bool CACHE>
cudaError_t launch_rotary(const RotaryParams& p, int D, bool norm, bool inter, cudaStream_t s) {
  if (D == 64)
    return norm ? launch_rotary_layout<T, 64, true, CACHE>(p, inter, s)
                : launch_rotary_layout<T, 64, false, CACHE>(p, inter, s);
  return norm ? launch_rotary_layout<T, 128, true, CACHE>(p, inter, s)
              : launch_rotary_layout<T, 128, false, CACHE>(p, inter, s);
}

template <typename T, typename G, typename O, int D>
cudaError_t launch_backward_layout(const RotaryBackwardParams& p, bool norm, bool inter, cudaStream_t s) {
  const dim3 grid(p.blocks[0] + p.blocks[1]);
  if (norm && inter) rotary_backward_kernel<T, G, O, D, true, true><<<grid, kRotaryThreads, 0, s>>>(p);
  else if (norm) rotary_backward_kernel<T, G, O, D, true, false><<<grid, kRotaryThreads, 0, s>>>(p);
  else if (inter) rotary_backward_kernel<T, G, O, D, false, true><<<grid, kRotaryThreads, 0, s>>>(p);
  else rotary_backward_kernel<T, G, O, D, false, false><<<grid, kRotaryThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(D / 8, 2);
  cfg.blockDim = dim3(8, 128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_weight_kernel, static_cast<const float*>(p.partial), p.blocks[0], p.blocks[1], D,
                            p.dweight[0], p.dweight[1]);
}

template <typename T, typename G, typename O>
cudaError_t launch_backward(const RotaryBackwardParams& p, int D, bool norm, bool inter, cudaStream_t s) {
  return D == 64 ? launch_backward_layout<T, G, O, 64>(p, norm, inter, s)
                 : launch_backward_layout<T, G, O, 128>(p, norm, inter, s);
}

// ------------------------------------------------------------------ argument checks
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem(swa_dtype t) { return t == SWA_FP32 ? 4 : 2; }
bool known(swa_dtype t) { return t == SWA_BF16 || t == SWA_FP32; }

// Strides of `dims` axes that a 16-byte access can follow: none negative, each a
// multiple of 16 bytes where its axis is longer than one.
bool strides_ok(const int64_t* st, const long long* size, int dims, swa_dtype t) {
  for (int i = 0; i < dims; ++i)
    if (size[i] > 1 && (st[i] < 0 || st[i] % (16 / elem(t)) != 0)) return false;
  return true;
}

// No two elements of an output share memory: axes in the order of their strides, each
// stride at least the extent of the axes below it.
bool no_overlap(const int64_t* st, const long long* size, int dims, int D) {
  bool used[3] = {false, false, false};
  long long extent = D;
  for (int k = 0; k < dims; ++k) {
    int best = -1;
    for (int i = 0; i < dims; ++i)
      if (!used[i] && (best < 0 || st[i] < st[best] || (st[i] == st[best] && size[i] < size[best]))) best = i;
    used[best] = true;
    if (size[best] <= 1) continue;
    if (st[best] < extent) return false;
    extent = st[best] * (size[best] - 1) + extent;
  }
  return true;
}

// Positions counted from `start` have to stay in an int32.
bool positions_ok(const int32_t* positions, int start, int n) {
  return positions || (long long)start + n - 1 <= 0x7fffffffLL;
}

swa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA; }

}  // namespace

int rotary_tile_tokens(int D) { return kRotaryThreads / (D / 16); }

swa_status make_rotary_math(const swa_rotation& r, const swa_head_norm& n, int D, RotaryMath* m) {
  if (r.rotary_dim < 0 || r.rotary_dim > D || (r.interleaved != 0 && r.interleaved != 1) ||
      (r.rotary_dim > 0 && !r.freq) || !isfinite(r.amplitude) || (n.norm != 0 && n.norm != 1))
    return SWA_ERR_INVALID_ARG;
  if (n.norm && (!(n.eps >= 0.f) || !isfinite(n.eps) || !known(n.weight_dtype) || !aligned16(n.q_weight) ||
                 !aligned16(n.k_weight)))
    return SWA_ERR_INVALID_ARG;
  if (r.rotary_dim % 16 != 0) return SWA_ERR_UNSUPPORTED;
  for (int i = 0; i < r.rotary_dim / 2; ++i) {
    if (!isfinite(r.freq[i])) return SWA_ERR_INVALID_ARG;
    // turns modulo one, as a fraction of 2^64
    const long double turns = static_cast<long double>(r.freq[i]) * 0.159154943091895335768883763372514362L;
    const long double part = turns - floorl(turns);
    m->turn[i] = part >= 1.0L ? 0 : static_cast<uint64_t>(ldexpl(part, 64));
  }
  m->amp = r.amplitude == 0.f ? 1.f : r.amplitude;
  m->eps = n.norm ? n.eps : 0.f;
  m->rot = r.rotary_dim;
  m->weight_bf16 = n.weight_dtype == SWA_BF16;
  return SWA_OK;
}

int split_heads(long long token_tiles, const int* heads, int kinds, int longest, int* segs) {
  // Longer runs of heads reuse a token's cosines and keep loads in flight; shorter ones make
  // more blocks. Halve the runs until the call has two blocks an SM. Measured with two and
  // with eight: 8 + 2 normed heads of 5935 tokens 10.6 and 16.6 us, 64 sequences of 8 new tokens
  // 8.4 and 12.5 us, gradients of 16 + 8 normed heads of 7 x 435 tokens 18.6 and 24.7 us.
  int per = 1;
  for (int i = 0; i < kinds; ++i)
    while (per < heads[i] && per < longest) per *= 2;
  while (true) {
    long long blocks = 0;
    for (int i = 0; i < kinds; ++i) {
      segs[i] = (heads[i] + per - 1) / per;
      blocks += token_tiles * segs[i];
    }
    if (per == 1 || blocks >= 148 * 2) return per;
    per /= 2;
  }
}

}  // namespace swa

using swa::HeadRows;

extern "C" {

swa_status swa_rotary_forward(const swa_rotary_args* a, void* stream) {
  if (!a) return SWA_ERR_INVALID_ARG;
  const int D = a->head_dim, Hk = a->num_kv_heads;
  if (a->batch < 0 || a->seq_len < 0 || a->num_q_heads < 1 || Hk < 0 || D < 1 || !swa::known(a->dtype))
    return SWA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
  swa::RotaryParams p = {};
  const swa_status st = swa::make_rotary_math(a->rotation, a->head_norm, D, &p.m);
  if (st != SWA_OK) return st;
  const long long tokens = (long long)a->batch * a->seq_len;
  if (tokens > 0x7fffffffLL - 64) return SWA_ERR_UNSUPPORTED;
  if (tokens == 0) return SWA_OK;
  if (!swa::positions_ok(a->positions, a->start, a->seq_len)) return SWA_ERR_INVALID_ARG;
  const long long qs[3] = {a->batch, a->num_q_heads, a->seq_len}, ks[3] = {a->batch, Hk, a->seq_len};
  if (!a->q || !a->q_out || !swa::aligned16(a->q) || !swa::aligned16(a->q_out) || !swa::aligned4(a->positions) ||
      !swa::strides_ok(a->q_stride, qs, 3, a->dtype) || !swa::strides_ok(a->q_out_stride, qs, 3, a->dtype) ||
      !swa::no_overlap(a->q_out_stride, qs, 3, D))
    return SWA_ERR_INVALID_ARG;
  if (Hk > 0 && (!a->k || !a->k_out || !swa::aligned16(a->k) || !swa::aligned16(a->k_out) ||
                 !swa::strides_ok(a->k_stride, ks, 3, a->dtype) || !swa::strides_ok(a->k_out_stride, ks, 3, a->dtype) ||
                 !swa::no_overlap(a->k_out_stride, ks, 3, D)))
    return SWA_ERR_INVALID_ARG;
  p.rows[0] = HeadRows{a->q, a->q_out, a->head_norm.q_weight, a->q_stride[0], a->q_stride[1], a->q_stride[2],
                       a->q_out_stride[0], a->q_out_stride[1], a->q_out_stride[2], a->num_q_heads};
  p.rows[1] = HeadRows{a->k, a->k_out, a->head_norm.k_weight, a->k_stride[0], a->k_stride[1], a->k_stride[2],
                       a->k_out_stride[0], a->k_out_stride[1], a->k_out_stride[2], Hk};
  p.tokens = (int)tokens;
  p.n = a->seq_len;
  p.positions = a->positions;
  p.start = a->start;
  const int heads[2] = {a->num_q_heads, Hk};
  const int tile = swa::rotary_tile_tokens(D);
  p.heads_per_seg = swa::split_heads((tokens + tile - 1) / tile, heads, 2, swa::kForwardRun, p.segs);
  if (p.segs[0] + p.segs[1] > 65535) return SWA_ERR_UNSUPPORTED;
  const bool norm = a->head_norm.norm, inter = a->rotation.interleaved;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return swa::cuda_status(a->dtype == SWA_FP32 ? swa::launch_rotary<float, false>(p, D, norm, inter, s)
                                               : swa::launch_rotary<__nv_bfloat16, false>(p, D, norm, inter, s));
}

}  // extern "C"

namespace swa {
namespace {

constexpr long long kMaxNormBlocks = 148 * 6;

// Blocks of the backward kernel: one an item (tile of tokens, run of heads); with a norm, whose
// weights' partial sums each block leaves, six an SM at most, shared between q and k by their
// heads.  Depends on sizes only.
void backward_split(const swa_rotary_backward_args& a, int* segs, int* blocks, int* per) {
  const int tile = rotary_tile_tokens(a.head_dim);
  const long long tiles = ((long long)a.batch * a.seq_len + tile - 1) / tile;
  const int heads[2] = {a.num_q_heads, a.num_kv_heads};
  *per = split_heads(tiles, heads, 2, kBackwardRun, segs);
  const long long items[2] = {tiles * segs[0], tiles * segs[1]};
  const long long all = items[0] + items[1], cap = std::min<long long>(all, a.head_norm.norm ? kMaxNormBlocks : 1LL << 30);
  // shares in proportion to the heads, then as few blocks as keep the longest block's items
  const long long share[2] = {cap * heads[0] / (heads[0] + heads[1]), cap * heads[1] / (heads[0] + heads[1])};
  for (int i = 0; i < 2; ++i) {
    const long long rounds = (items[i] + std::max<long long>(share[i], 1) - 1) / std::max<long long>(share[i], 1);
    blocks[i] = rounds == 0 ? 0 : (int)((items[i] + rounds - 1) / rounds);
  }
}

bool backward_sizes_ok(const swa_rotary_backward_args& a) {
  return a.batch >= 0 && a.seq_len >= 0 && a.num_q_heads >= 1 && a.num_kv_heads >= 0 &&
         (a.head_dim == 64 || a.head_dim == 128) && (long long)a.batch * a.seq_len <= 0x7fffffffLL - 64;
}

}  // namespace
}  // namespace swa

extern "C" {

size_t swa_rotary_workspace_bytes(const swa_rotary_backward_args* a) {
  if (!a || !swa::backward_sizes_ok(*a) || a->head_norm.norm != 1 || (!a->dq_weight && !a->dk_weight)) return 0;
  if (a->batch == 0 || a->seq_len == 0) return 0;
  int segs[2], blocks[2], per;
  swa::backward_split(*a, segs, blocks, &per);
  return (size_t)(blocks[0] + blocks[1]) * a->head_dim * 4;
}

swa_status swa_rotary_backward(const swa_rotary_backward_args* a, void* stream) {
  if (!a) return SWA_ERR_INVALID_ARG;
  const int D = a->head_dim, Hk = a->num_kv_heads;
  if (a->batch < 0 || a->seq_len < 0 || a->num_q_heads < 1 || Hk < 0 || D < 1 || !swa::known(a->dtype) ||
      !swa::known(a->grad_dtype) || !swa::known(a->out_dtype) ||
      (a->dtype == SWA_FP32 && (a->grad_dtype != SWA_FP32 || a->out_dtype != SWA_FP32)))
    return SWA_ERR_INVALID_ARG;
  if (!swa::backward_sizes_ok(*a)) return SWA_ERR_UNSUPPORTED;
  swa::RotaryBackwardParams p = {};
  const swa_status st = swa::make_rotary_math(a->rotation, a->head_norm, D, &p.m);
  if (st != SWA_OK) return st;
  const bool norm = a->head_norm.norm, inter = a->rotation.interleaved;
  if (!swa::aligned4(a->dq_weight) || !swa::aligned4(a->dk_weight)) return SWA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long tokens = (long long)a->batch * a->seq_len;
  float* dweight[2] = {norm ? a->dq_weight : nullptr, norm ? a->dk_weight : nullptr};
  if (tokens == 0) {
    if (!dweight[0] && !dweight[1]) return SWA_OK;
    swa::zero_weight_kernel<<<1, 128, 0, s>>>(dweight[0], dweight[1], D);
    return swa::cuda_status(cudaGetLastError());
  }
  if (!swa::positions_ok(a->positions, a->start, a->seq_len)) return SWA_ERR_INVALID_ARG;
  const long long qs[3] = {a->batch, a->num_q_heads, a->seq_len}, ks[3] = {a->batch, Hk, a->seq_len};
  if (!a->dq_out || !a->dq || !swa::aligned16(a->dq_out) || !swa::aligned16(a->dq) || !swa::aligned4(a->positions) ||
      !swa::strides_ok(a->dq_out_stride, qs, 3, a->grad_dtype) || !swa::strides_ok(a->dq_stride, qs, 3, a->out_dtype) ||
      !swa::no_overlap(a->dq_stride, qs, 3, D) ||
      (norm && (!a->q || !swa::aligned16(a->q) || !swa::strides_ok(a->q_stride, qs, 3, a->dtype))))
    return SWA_ERR_INVALID_ARG;
  if (Hk > 0 &&
      (!a->dk_out || !a->dk || !swa::aligned16(a->dk_out) || !swa::aligned16(a->dk) ||
       !swa::strides_ok(a->dk_out_stride, ks, 3, a->grad_dtype) || !swa::strides_ok(a->dk_stride, ks, 3, a->out_dtype) ||
       !swa::no_overlap(a->dk_stride, ks, 3, D) ||
       (norm && (!a->k || !swa::aligned16(a->k) || !swa::strides_ok(a->k_stride, ks, 3, a->dtype)))))
    return SWA_ERR_INVALID_ARG;
  p.grad[0] = HeadRows{a->dq_out, a->dq, a->head_norm.q_weight, a->dq_out_stride[0], a->dq_out_stride[1],
                       a->dq_out_stride[2], a->dq_stride[0], a->dq_stride[1], a->dq_stride[2], a->num_q_heads};
  p.grad[1] = HeadRows{a->dk_out, a->dk, a->head_norm.k_weight, a->dk_out_stride[0], a->dk_out_stride[1],
                       a->dk_out_stride[2], a->dk_stride[0], a->dk_stride[1], a->dk_stride[2], Hk};
  p.x[0] = a->q;
  p.x[1] = a->k;
  for (int i = 0; i < 2; ++i) {
    const int64_t* xs = i ? a->k_stride : a->q_stride;
    p.xb[i] = xs[0];
    p.xh[i] = xs[1];
    p.xt[i] = xs[2];
    p.dweight[i] = dweight[i];
  }
  p.tokens = (int)tokens;
  p.n = a->seq_len;
  p.positions = a->positions;
  p.start = a->start;
  swa::backward_split(*a, p.segs, p.blocks, &p.heads_per_seg);
  if (dweight[0] || dweight[1]) {
    const size_t need = (size_t)(p.blocks[0] + p.blocks[1]) * D * 4;
    if (!a->workspace || !swa::aligned16(a->workspace) || a->workspace_bytes < need) return SWA_ERR_INVALID_ARG;
    p.partial = static_cast<float*>(a->workspace);
  }
  using B16 = __nv_bfloat16;
  cudaError_t e;
  if (a->dtype == SWA_FP32) e = swa::launch_backward<float, float, float>(p, D, norm, inter, s);
  else if (a->grad_dtype == SWA_FP32 && a->out_dtype == SWA_FP32)
    e = swa::launch_backward<B16, float, float>(p, D, norm, inter, s);
  else if (a->grad_dtype == SWA_FP32) e = swa::launch_backward<B16, float, B16>(p, D, norm, inter, s);
  else if (a->out_dtype == SWA_FP32) e = swa::launch_backward<B16, B16, float>(p, D, norm, inter, s);
  else e = swa::launch_backward<B16, B16, B16>(p, D, norm, inter, s);
  return swa::cuda_status(e);
}

swa_status swa_cache_append(const swa_cache* cache, const swa_cache_batch* batch, const swa_cache_append_args* a,
                            void* stream) {
  if (!cache || !batch || !a) return SWA_ERR_INVALID_ARG;
  swa_status st = swa::check_cache(*cache);
  if (st != SWA_OK) return st;
  const int D = cache->head_dim, Hq = a->num_q_heads, Hk = cache->num_kv_heads;
  if (Hq < 0) return SWA_ERR_INVALID_ARG;
  swa::RotaryParams p = {};
  st = swa::make_rotary_math(a->rotation, a->head_norm, D, &p.m);
  if (st != SWA_OK) return st;
  st = swa::check_batch(*batch);
  if (st != SWA_OK) return st;
  if (batch->batch == 0 || batch->num_tokens == 0) return SWA_OK;
  const long long T = batch->num_tokens;
  const long long qs[2] = {T, Hq}, ks[2] = {T, Hk};
  if (!a->k || !a->v || !swa::aligned16(a->k) || !swa::aligned16(a->v) ||
      !swa::strides_ok(a->k_stride, ks, 2, cache->dtype) || !swa::strides_ok(a->v_stride, ks, 2, cache->dtype))
    return SWA_ERR_INVALID_ARG;
  if (Hq > 0 && (!a->q || !a->q_out || !swa::aligned16(a->q) || !swa::aligned16(a->q_out) ||
                 !swa::strides_ok(a->q_stride, qs, 2, cache->dtype) ||
                 !swa::strides_ok(a->q_out_stride, qs, 2, cache->dtype) || !swa::no_overlap(a->q_out_stride, qs, 2, D)))
    return SWA_ERR_INVALID_ARG;
  p.rows[0] = HeadRows{a->q, a->q_out, a->head_norm.q_weight, 0, a->q_stride[1], a->q_stride[0], 0, a->q_out_stride[1],
                       a->q_out_stride[0], Hq};
  p.rows[1] = HeadRows{a->k, cache->k_pages, a->head_norm.k_weight, 0, a->k_stride[1], a->k_stride[0], 0, 0, 0, Hk};
  p.rows[2] = HeadRows{a->v, cache->v_pages, nullptr, 0, a->v_stride[1], a->v_stride[0], 0, 0, 0, Hk};
  p.tokens = batch->num_tokens;
  p.n = 1;
  p.batch = batch->batch;
  p.max_pages = batch->max_pages;
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.num_kv_heads = Hk;
  p.block_table = batch->block_table;
  p.seq_lens = batch->seq_lens;
  p.cu_tokens = batch->cu_tokens;
  p.err = cache->error_word;
  const int heads[3] = {Hq, Hk, Hk};
  const int tile = swa::rotary_tile_tokens(D);
  p.heads_per_seg = swa::split_heads((T + tile - 1) / tile, heads, 3, swa::kForwardRun, p.segs);
  if (p.segs[0] + p.segs[1] + p.segs[2] > 65535) return SWA_ERR_UNSUPPORTED;
  const bool norm = a->head_norm.norm, inter = a->rotation.interleaved;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return swa::cuda_status(cache->dtype == SWA_FP32 ? swa::launch_rotary<float, true>(p, D, norm, inter, s)
                                                   : swa::launch_rotary<__nv_bfloat16, true>(p, D, norm, inter, s));
}

}  // extern "C"
