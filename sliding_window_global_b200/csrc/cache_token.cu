// cache_token.cu -- attention over a paged cache when a sequence brings few new tokens
// (bf16; new tokens x heads of a group <= 32 rows): decoding, and checking guessed tokens.
//
// The bound is the read of K and V once.  A KV head of a sequence is one unit: its rows
// (new tokens x query heads of the group) fill one or two 16-row fragments, so that one
// pass over the keys serves the whole group.  All units' keys, cut into steps of 16 (D =
// 128) or 32 (D = 64) keys = 8 KB of K and V, form one list; every warp of the grid takes
// an equal, contiguous run of it, whatever the lengths (the host does not know them).  A
// warp works alone: it fetches its steps with cp.async into its own ring of three, and
// keeps scores, running maximum, sum and output in registers (mma.sync m16n8k16: with 16
// rows the tensor work is an eighth of the time that the bytes take, so that the
// 128-row tcgen05 products would only compute padding).  A unit that lies in one warp's run
// is stored directly; one that is split leaves a partial result a warp, which the merge
// kernel joins in the order of the keys.
//
// Where the keys in reach are few, the second launch and the search for a warp's run cost
// more than uneven work does: then a unit belongs to a cluster of one to eight blocks, its
// steps are shared out among their warps, and the parts are joined through shared memory of
// the block and of the cluster (UNIT; the rule stands at token_split).
#include <cuda_bf16.h>

#include <algorithm>

#include "cache_device.cuh"
#include "ptx.cuh"

namespace swa {
namespace {

constexpr int kStages = 3;
constexpr int kMaxWarps = 8;               // warps of a block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D>
struct Step {
  static constexpr int kKeys = 2048 / D;               // 16 or 32
  static constexpr int kGroups = kKeys / 16;           // 16-key groups: each lies in one page
  static constexpr int kHalf = kKeys * D * 2;          // bytes of K (or V) of a step
  static constexpr int kBytes = 2 * kHalf;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The steps of a sequence (the same for each of its KV heads): keys [lo, hi) of interest,
// steps from the step-aligned start on.  A sequence with new tokens has one at least, so
// that rows without a key are written too; without any key at all (a length beyond the
// call's bounds can put the windows there) nothing is looked up for it.
struct TokenUnit {
  CacheSeq s;
  int lo, hi, base, steps;
};

template <int D>
__host__ __device__ __forceinline__ TokenUnit token_unit(const CacheAttendParams& p, int b) {
  TokenUnit u;
  u.s = cache_seq(p, b);
  u.lo = u.hi = u.base = u.steps = 0;
  if (u.s.count > 0) {
    u.lo = key_begin(p, u.s, 0);
    u.hi = key_end(u.s, u.s.count - 1);
    if (u.hi <= u.lo) u.lo = u.hi = 0;
    u.base = u.lo / Step<D>::kKeys * Step<D>::kKeys;
    u.steps = max(1, (u.hi - u.base + Step<D>::kKeys - 1) / Step<D>::kKeys);
  }
  return u;
}

// The block-table column of the 16-key group that begins at `key`, < 0: nothing to look up,
// since none of its keys is in reach. A step's first group may lie wholly before a window, in
// a page of its own whose entry means nothing any more.
__host__ __device__ __forceinline__ int group_column(const CacheAttendParams& p, const TokenUnit& u, int key) {
  return key < u.hi && key + 16 > u.lo ? key / p.page_size : -1;
}

// Sum of the steps of all units, by one warp (below 2^31, checked on the host); each lane
// calls each(b, the first step of sequence b's units, their number, whether something of b's
// bounds does not hold).
template <int D, typename F>
__device__ __forceinline__ int scan_steps(const CacheAttendParams& p, int lane, F each) {
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int mine = 0;
    bool bad = false;
    if (b < p.B) {
      const TokenUnit u = token_unit<D>(p, b);
      mine = u.steps * p.Hkv;
      bad = u.s.bad;
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    each(b, before + sum - mine, mine, bad);
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return before;
}

// The runs of W warps over n steps: the first n % W of n / W + 1 steps, the rest of n / W.
struct Runs {
  int each, extra;
  __device__ __forceinline__ Runs(int n, int W) : each(n / W), extra(n % W) {}
  __device__ __forceinline__ int begin(int w) const { return w * each + min(w, extra); }
  __device__ __forceinline__ int of(int step) const {    // the run that holds a step
    const int head = extra * (each + 1);
    return step < head ? step / (each + 1) : extra + (step - head) / each;
  }
};

// Shared memory of another block of the cluster.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  uint32_t at;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
  uint32_t at;
  float4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(at)
               : "memory");
  return x;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// UNIT: joins the warps' parts of a unit, first those of a block, then the blocks', both in
// the order of the keys, and writes the unit's rows.  Every thread of the cluster calls it.
// The rings are free: each warp has computed what it fetched.
template <int D, int MT>
__device__ __forceinline__ void join_unit(const CacheAttendParams& p, const CacheSeq& s, int hk, int rows, int cluster,
                                          uint8_t* smem, float (&o)[MT][D / 8][4], float (&m)[MT][2],
                                          float (&l)[MT][2]) {
  constexpr int R = 16 * MT, LD = D + 8;               // rows 32 bytes apart in the banks
  __shared__ float sM[kMaxWarps][R], sL[kMaxWarps][R], sTop[R], sSum[R];
  __shared__ float sTops[8][R], sSums[8][R];           // the blocks' of the cluster
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, wb = blockDim.x >> 5;
  float* parts = reinterpret_cast<float*>(smem);       // [warps][R][LD]
  cp_async_wait<0>();
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float sum = l[mt][x];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = mt * 16 + (lane >> 2) + 8 * x;
      if (r >= rows) continue;
      float2* part = reinterpret_cast<float2*>(parts + (wid * R + r) * LD + 2 * (lane & 3));
#pragma unroll
      for (int e = 0; e < D / 8; ++e) part[4 * e] = make_float2(o[mt][e][2 * x], o[mt][e][2 * x + 1]);
      if ((lane & 3) == 0) {
        sM[wid][r] = m[mt][x];
        sL[wid][r] = sum;
      }
    }
  }
  __syncthreads();
  // each row's maximum and sum over n parts, and in place of their maxima the parts' weights
  // (0 for a part without keys; a NaN sum goes on)
  auto weigh = [&](float (*top)[R], float (*sum)[R], int n) {
    if ((int)threadIdx.x < rows) {
      const int r = threadIdx.x;
      float t = -INFINITY, total = 0.f;
      for (int k = 0; k < n; ++k) t = fmaxf(t, top[k][r]);
      for (int k = 0; k < n; ++k) {
        const float f = top[k][r] == -INFINITY ? 0.f : ex2_approx(top[k][r] - t);
        top[k][r] = f;
        total += f * sum[k][r];
      }
      sTop[r] = t;
      sSum[r] = total;
    }
    __syncthreads();
  };
  constexpr int Q = D / 4;                             // 16-byte pieces of a row
  auto store = [&](int r, int c, float4 acc) {
    const bool has = sSum[r] != 0.f;       // also where every score is NaN
    const float inv = has ? 1.f / sSum[r] : 0.f;
    const long long row = (long long)(s.from + r / p.G) * p.Hq + hk * p.G + r % p.G;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + c) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse && c == 0) p.lse[row] = has ? (sTop[r] + log2f(sSum[r])) * kLn2 : -INFINITY;
  };
  weigh(sM, sL, wb);
  for (int i = threadIdx.x; i < rows * Q; i += blockDim.x) {
    const int r = i / Q, c = i % Q * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < wb; ++k) {
      const float f = sM[k][r];
      const float4 x = *reinterpret_cast<const float4*>(parts + (k * R + r) * LD + c);
      acc = make_float4(acc.x + f * x.x, acc.y + f * x.y, acc.z + f * x.z, acc.w + f * x.w);
    }
    if (cluster == 1) store(r, c, acc);
    else *reinterpret_cast<float4*>(parts + r * LD + c) = acc;   // over warp 0's part: read by this thread alone
  }
  if (cluster == 1) return;
  cluster_sync();
  for (int i = threadIdx.x; i < cluster * rows; i += blockDim.x) {
    sTops[i / rows][i % rows] = ld_cluster(&sTop[i % rows], i / rows);
    sSums[i / rows][i % rows] = ld_cluster(&sSum[i % rows], i / rows);
  }
  cluster_sync();                                      // sTop and sSum are read before they are written again
  weigh(sTops, sSums, cluster);
  for (int i = cluster_rank() * blockDim.x + threadIdx.x; i < rows * Q; i += cluster * blockDim.x) {
    const int r = i / Q, c = i % Q * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < cluster; ++k) {
      const float f = sTops[k][r];
      const float4 x = ld_cluster4(parts + r * LD + c, k);
      acc = make_float4(acc.x + f * x.x, acc.y + f * x.y, acc.z + f * x.z, acc.w + f * x.w);
    }
    store(r, c, acc);
  }
  cluster_sync();                                      // nobody leaves while its memory is read
}

template <int D, int MT, int CAP, bool UNIT>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) cache_token_kernel(const __grid_constant__ CacheAttendParams p,
                                                                         int cluster) {
  using S = Step<D>;
  constexpr int NG = S::kGroups;
  constexpr int CH = D / 8;                            // 16-byte chunks of a row
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, wb = blockDim.x >> 5;
  const int w = blockIdx.x * wb + wid, W = gridDim.x * wb;
  const uint32_t ring = smem_u32(smem) + wid * kStages * S::kBytes;

  // ---- this warp's run, and the sequence, head and step it starts at
  int b = 0, hk = 0, j = 0, total = 0;
  TokenUnit unit = {};                                 // UNIT: the cluster's
  if (UNIT) {
    const int id = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    b = id / p.Hkv;
    hk = id % p.Hkv;
    unit = token_unit<D>(p, b);
    if (unit.s.bad && hk == 0 && rank == 0 && threadIdx.x == 0) atomicOr(p.err, kDevErrCheck);
    if (unit.steps == 0) return;                       // no new tokens: the whole cluster leaves
    const Runs runs(unit.steps, cluster * wb);
    j = runs.begin(rank * wb + wid);
    total = runs.begin(rank * wb + wid + 1) - j;
  } else {
    grid_launch_dependents();
    int last_first = 0, last_mine = 0;       // of the last 32 sequences: with B <= 32, of all
    const int n = scan_steps<D>(p, lane, [&](int bb, int first, int mine, bool bad) {
      last_first = first;
      last_mine = mine;
      if (w != 0 || bb >= p.B) return;
      p.prefix[bb] = first;
      if (bad) atomicOr(p.err, kDevErrCheck);
    });
    if (w == 0 && lane == 0) p.prefix[p.B] = n;
    const Runs runs(n, W);
    const int begin = runs.begin(w);
    total = runs.begin(w + 1) - begin;
    if (total == 0) return;
    int first = 0, steps = 1;
    auto look = [&](int bb, int ff, int mine, bool) {
      const unsigned hit = __ballot_sync(0xffffffffu, ff <= begin && begin < ff + mine);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = __shfl_sync(0xffffffffu, bb, src);
        first = __shfl_sync(0xffffffffu, ff, src);
        steps = __shfl_sync(0xffffffffu, mine, src) / p.Hkv;
      }
    };
    if (p.B <= 32) look(lane, last_first, last_mine, false);
    else scan_steps<D>(p, lane, look);
    hk = (begin - first) / steps;
    j = (begin - first) % steps;
  }

  // ---- fetching side: its own place in the list, kStages - 1 steps ahead
  TokenUnit fu = UNIT ? unit : token_unit<D>(p, b);
  int fb = b, fhk = hk, fj = j;
  int fpage[NG];
  unsigned history = 0;                    // per group of a fetched step: its page exists (newest lowest)
  auto look_up = [&]() {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int col = group_column(p, fu, fu.base + fj * S::kKeys + 16 * g);
      fpage[g] = col < 0 ? 0 : load_index(p.block_table + (long long)fb * p.max_pages + col);
    }
  };
  if (total > 0) look_up();
  int fetched = 0;
  auto fetch = [&]() {
    if (fetched < total) {
      const uint32_t dst = ring + fetched % kStages * S::kBytes;
      const int key0 = fu.base + fj * S::kKeys;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int key = key0 + 16 * g;
        const bool ok = fpage[g] >= 0 && fpage[g] < p.num_pages;
        if (!ok && lane == 0) atomicOr(p.err, kDevErrCheck);
        history = history << 1 | (ok ? 1u : 0u);
        const long long off = (((long long)(ok ? fpage[g] : 0) * p.Hkv + fhk) * p.page_size + key % p.page_size) * D;
        const __nv_bfloat16* ks = static_cast<const __nv_bfloat16*>(p.k_pages) + off;
        const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(p.v_pages) + off;
#pragma unroll
        for (int i = 0; i < 16 * CH / 32; ++i) {
          const int c = lane + 32 * i, row = c / CH, col = c % CH;
          const bool on = ok && key + row >= fu.lo && key + row < fu.hi;   // else zeros: V times p = 0 must stay 0
          const uint32_t at = dst + ((16 * g + row) * CH + (col ^ (row & 7))) * 16;
          cp_async16(at, ks + c * 8, on);
          cp_async16(at + S::kHalf, vs + c * 8, on);
        }
      }
      ++fetched;
      if (++fj == fu.steps && !UNIT) {
        fj = 0;
        if (++fhk == p.Hkv) {
          fhk = 0;
          do {
            ++fb;
          } while (fb < p.B && (fu = token_unit<D>(p, fb)).steps == 0);
        }
      }
      if (fetched < total) look_up();
    } else {
      history <<= NG;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch();

  // ---- computing side
  const float sl2 = p.scale * kLog2e;
  const ScoreCap<CAP> score_cap(sl2, p.softcap);
  int done = 0;
  while (UNIT || done < total) {
    const TokenUnit u = UNIT ? unit : token_unit<D>(p, b);
    const int rows = u.s.count * p.G;
    uint32_t qf[MT][D / 16][4];
    int klo[MT][2], khi[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const __nv_bfloat16* src[2];
      bool live[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + (lane >> 2) + 8 * x;
        live[x] = r < rows;
        const int tok = live[x] ? r / p.G : 0, h = hk * p.G + (live[x] ? r % p.G : 0);
        klo[mt][x] = live[x] ? key_begin(p, u.s, tok) : 0;
        khi[mt][x] = live[x] ? key_end(u.s, tok) : 0;
        src[x] = static_cast<const __nv_bfloat16*>(p.q) + (long long)(u.s.from + tok) * p.q_token + h * p.q_head +
                 2 * (lane & 3);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qf[mt][kk][x] = live[x & 1] ? *reinterpret_cast<const uint32_t*>(src[x & 1] + 16 * kk + 8 * (x >> 1)) : 0u;
      }
    }
    // keys that every row of the unit sees need no mask
    const int full_lo = key_begin(p, u.s, u.s.count - 1);
    const int full_hi = key_end(u.s, 0);
    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 8; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[mt][e][c] = 0.f;
    }
    const bool from_start = j == 0;
    while (done < total) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fetch();                             // into the slot of the step before, which every lane has read
      const uint32_t at = ring + done % kStages * S::kBytes;
      const unsigned pages = history >> ((kStages - 1) * NG) & ((1u << NG) - 1);
      const int key0 = u.base + j * S::kKeys;

      float s[MT][2 * NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][t][c] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t kf[4];
          const int row = (lane & 7) + ((lane >> 4) << 3), col = 2 * kk + ((lane >> 3) & 1);
          ldmatrix4(kf, at + ((16 * g + row) * CH + (col ^ (row & 7))) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(s[mt][2 * g], qf[mt][kk], kf[0], kf[1]);
            mma_bf16(s[mt][2 * g + 1], qf[mt][kk], kf[2], kf[3]);
          }
        }
      }
      const bool masked = key0 < full_lo || key0 + S::kKeys > full_hi || pages != (1u << NG) - 1;
      uint32_t pf[MT][NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float mx[2] = {m[mt][0], m[mt][1]};
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t) {
          if (CAP) {
            score_cap.pair(s[mt][t][0], s[mt][t][1]);
            score_cap.pair(s[mt][t][2], s[mt][t][3]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x = CAP ? s[mt][t][c] : s[mt][t][c] * sl2;
            if (masked) {
              const int key = key0 + 8 * t + 2 * (lane & 3) + (c & 1);
              const bool see = key >= klo[mt][c >> 1] && key < khi[mt][c >> 1] && (pages >> (NG - 1 - t / 2) & 1);
              x = see ? x : -INFINITY;
            }
            s[mt][t][c] = x;
            mx[c >> 1] = fmaxf(mx[c >> 1], x);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[mt][0] || mx[1] > m[mt][1])) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float alpha = m[mt][x] == -INFINITY ? 0.f : ex2_approx(m[mt][x] - mx[x]);
            m[mt][x] = mx[x];
            l[mt][x] *= alpha;
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              o[mt][e][2 * x] *= alpha;
              o[mt][e][2 * x + 1] *= alpha;
            }
          }
        }
        const float ref[2] = {m[mt][0] == -INFINITY ? 0.f : m[mt][0], m[mt][1] == -INFINITY ? 0.f : m[mt][1]};
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e[c] = ex2_approx(s[mt][t][c] - ref[c >> 1]);
            l[mt][c >> 1] += e[c];
          }
          // p in bf16: the type of the tensor product that follows; the sum keeps 32 bits, which
          // the lse shows. Root mean square error of the outputs against 64 bits: 1.8e-3 of
          // their size, 1.7e-3 of it their own rounding to bf16.
          pf[mt][t / 2][2 * (t & 1)] = pack_bf16x2(e[0], e[1]);
          pf[mt][t / 2][2 * (t & 1) + 1] = pack_bf16x2(e[2], e[3]);
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          uint32_t vf[4];
          const int row = (lane & 7) + (((lane >> 3) & 1) << 3), col = 2 * e + (lane >> 4);
          ldmatrix4_trans(vf, at + S::kHalf + ((16 * g + row) * CH + (col ^ (row & 7))) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(o[mt][2 * e], pf[mt][g], vf[0], vf[1]);
            mma_bf16(o[mt][2 * e + 1], pf[mt][g], vf[2], vf[3]);
          }
        }
      }
      ++done;
      ++j;
      if (j == u.steps) break;
    }

    if (UNIT) {
      join_unit<D, MT>(p, u.s, hk, rows, cluster, smem, o, m, l);
      return;
    }

    // ---- the unit (or this run's part of it) is done
    const bool whole = from_start && j == u.steps;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[mt][x];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = mt * 16 + (lane >> 2) + 8 * x;
        if (r >= rows) continue;
        const bool has = sum != 0.f;       // also where every score is NaN
        const float inv = has ? 1.f / sum : 0.f;
        const float lse = has ? (m[mt][x] + log2f(sum)) * kLn2 : -INFINITY;
        if (whole) {
          const long long row = (long long)(u.s.from + r / p.G) * p.Hq + hk * p.G + r % p.G;
          uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + row * D + 2 * (lane & 3));
#pragma unroll
          for (int e = 0; e < D / 8; ++e) out[4 * e] = pack_bf16x2(o[mt][e][2 * x] * inv, o[mt][e][2 * x + 1] * inv);
          if (p.lse && (lane & 3) == 0) p.lse[row] = lse;
        } else {
          const long long row = (2LL * w + (from_start ? 1 : 0)) * (16 * MT) + r;
          float2* part = reinterpret_cast<float2*>(p.part_o + row * D + 2 * (lane & 3));
#pragma unroll
          for (int e = 0; e < D / 8; ++e) part[4 * e] = make_float2(o[mt][e][2 * x] * inv, o[mt][e][2 * x + 1] * inv);
          if ((lane & 3) == 0) p.part_lse[row] = lse;
        }
      }
    }
    if (j == u.steps) {
      j = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        if (done < total) {
          do {
            ++b;
          } while (token_unit<D>(p, b).steps == 0);
        }
      }
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of every row whose unit was split, a block a row: the parts' weights first,
// then its warps add up the parts in turn, and the warps are added up in order, so the same
// call gives the same bits. A unit has a part in every run that holds some of its steps, at
// most all of them: blocks of 16 warps where the units are few, of four where they are many.
template <int D, int kMergeThreads>
__global__ void __launch_bounds__(kMergeThreads) cache_token_merge_kernel(const __grid_constant__ CacheAttendParams p,
                                                                           int W, int row_pad) {
  constexpr int kWarps = kMergeThreads / 32, E = D / 32;
  __shared__ float sW[148 * kMaxWarps], sRed[kWarps], sSum[kWarps], sO[kWarps][D];
  grid_dependency_wait();
  const int max_rows = p.max_tokens * p.G;
  const int r = blockIdx.x % max_rows;
  const int hk = blockIdx.x / max_rows % p.Hkv;
  const int b = blockIdx.x / max_rows / p.Hkv;
  const CacheSeq s = cache_seq(p, b);
  const int first = p.prefix[b], steps = (p.prefix[b + 1] - first) / p.Hkv, n = p.prefix[p.B];
  if (steps == 0 || r >= s.count * p.G) return;
  const int u0 = first + hk * steps, u1 = u0 + steps;
  // the runs that hold the unit's first and last step (none between them is empty)
  const Runs runs(n, W);
  const int w0 = runs.of(u0), parts = runs.of(u1 - 1) - w0 + 1;
  if (parts == 1) return;                  // stored whole
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // part k lies in slot 0 of its run, the first one in slot 1 (its unit began there)
  auto row_of = [&](int k) { return (2LL * (w0 + k) + (k == 0 ? 1 : 0)) * row_pad + r; };
  float top = -INFINITY;
  for (int k = threadIdx.x; k < parts; k += kMergeThreads) {
    sW[k] = p.part_lse[row_of(k)];
    top = fmaxf(top, sW[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sRed[warp] = top;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sRed[i]);
  float sum = 0.f;
  for (int k = threadIdx.x; k < parts; k += kMergeThreads) {
    const float f = sW[k] == -INFINITY ? 0.f : ex2_approx((sW[k] - top) * kLog2e);   // no key: 0 (a NaN goes on)
    sW[k] = f;
    sum += f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sSum[warp] = sum;
  __syncthreads();
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int k = warp; k < parts; k += kWarps) {
    const float f = sW[k];
    const float2* src = reinterpret_cast<const float2*>(p.part_o + row_of(k) * D) + lane;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = src[16 * e];
      acc[e] += f * x.x;
      acc[e + 1] += f * x.y;
    }
  }
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(&sO[warp][32 * e + 2 * lane]) = make_float2(acc[e], acc[e + 1]);
  __syncthreads();
  if (threadIdx.x >= D) return;
  const int c = threadIdx.x;
  float out = 0.f;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    out += sO[i][c];
    sum += sSum[i];
  }
  const bool has = sum != 0.f;
  const long long row = (long long)(s.from + r / p.G) * p.Hq + hk * p.G + r % p.G;
  static_cast<__nv_bfloat16*>(p.out)[row * D + c] = __float2bfloat16_rn(has ? out / sum : 0.f);
  if (p.lse && c == 0) p.lse[row] = has ? top + log2f(sum) * kLn2 : -INFINITY;
}

template <int D, int MT, int CAP>
cudaError_t launch_token(const CacheAttendParams& p, const TokenSplit& t, cudaStream_t s) {
  const int smem = t.warps * kStages * Step<D>::kBytes;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (t.cluster) {
    cudaError_t e = allow_smem<&cache_token_kernel<D, MT, CAP, true>>(kMaxWarps * kStages * Step<D>::kBytes);
    if (e != cudaSuccess) return e;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = t.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(t.blocks);
    cfg.blockDim = dim3(t.warps * 32);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, cache_token_kernel<D, MT, CAP, true>, p, t.cluster);
  }
  cudaError_t e = allow_smem<&cache_token_kernel<D, MT, CAP, false>>(kMaxWarps * kStages * Step<D>::kBytes);
  if (e != cudaSuccess) return e;
  cache_token_kernel<D, MT, CAP, false><<<t.blocks, t.warps * 32, smem, s>>>(p, 0);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hkv * p.max_tokens * p.G));
  const bool many = (long long)p.B * p.Hkv * 16 > t.blocks * t.warps;      // fewer than 16 parts a unit
  cfg.blockDim = dim3(many ? 128 : 512);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, many ? cache_token_merge_kernel<D, 128> : cache_token_merge_kernel<D, 512>, p,
                            t.blocks * t.warps, 16 * MT);
}

template <int D, int MT>
cudaError_t launch_token(const CacheAttendParams& p, const TokenSplit& t, cudaStream_t s) {
  const int cap = cap_kind(p.softcap);
  return cap == kCapAny     ? launch_token<D, MT, kCapAny>(p, t, s)
         : cap == kCapUsual ? launch_token<D, MT, kCapUsual>(p, t, s)
                            : launch_token<D, MT, kCapNone>(p, t, s);
}

// Shared memory of the joined parts fits into the rings they replace.
static_assert(32 * (128 + 8) * 4 <= kStages * Step<128>::kBytes && 32 * (64 + 8) * 4 <= kStages * Step<64>::kBytes,
              "parts of a warp");

}  // namespace

TokenSplit token_split(int B, int Hkv, int D, int rows, long long reach) {
  TokenSplit t = {};
  t.row_pad = rows <= 16 ? 16 : 32;
  const int keys = 2048 / D;
  const long long unit_steps = (reach + keys - 1) / keys + 1, units = (long long)B * Hkv;
  const long long steps = units * unit_steps;
  t.ok = steps < (1LL << 31);
  // A cluster for each unit, as many blocks as the GPU holds at once, two steps a warp at
  // least; with more units than SMs, blocks of four warps, two of them on an SM.
  int cluster = 1, warps = units > 148 ? 4 : kMaxWarps;
  while (cluster < 8 && units * cluster * 2 <= 148 && unit_steps > cluster * warps * 2) cluster *= 2;
  if (unit_steps <= 4) warps = 4;        // not fewer: they share the join of the rows too
  const long long slots = 148 * (kMaxWarps / warps);
  const long long waves = (units * cluster + slots - 1) / slots;
  // Equal runs of all steps: balanced whatever the lengths, but a launch and a search more
  // (about six steps' time). Lengths may be anything below the bound, so that clusters are
  // for few steps a warp only: three sequences of 4000 to 9656 keys, 12 heads, D = 128, take
  // 37 us in runs and 44 us with clusters of four blocks, of 19 steps a warp.
  const long long per_warp = (unit_steps + cluster * warps - 1) / (cluster * warps);
  const long long per_run = (steps + 148 * kMaxWarps - 1) / (148 * kMaxWarps);
  if (per_warp <= 16 && waves * per_warp <= per_run + 6 && units * cluster < (1LL << 31)) {
    t.cluster = cluster;
    t.warps = warps;
    t.blocks = (int)(units * cluster);
    return t;
  }
  // Two steps a warp at least; one block an SM, of as few warps as that allows.
  const long long want = std::min<long long>((steps + 1) / 2, 148 * kMaxWarps);
  t.warps = 1;
  while (t.warps < kMaxWarps && 148 * t.warps < want) t.warps *= 2;
  t.blocks = (int)((want + t.warps - 1) / t.warps);
  t.bytes = (((size_t)B + 1) * 4 + 15) / 16 * 16 + (size_t)2 * t.blocks * t.warps * t.row_pad * (D + 1) * 4;
  return t;
}

template <int D>
static void unit_columns(const CacheAttendParams& p, int b, int32_t* first_last) {
  const TokenUnit u = token_unit<D>(p, b);
  first_last[0] = first_last[1] = -1;
  for (int j = 0; j < u.steps; ++j)
    for (int g = 0; g < Step<D>::kGroups; ++g) {
      const int col = group_column(p, u, u.base + j * Step<D>::kKeys + 16 * g);
      if (col < 0) continue;
      if (first_last[0] < 0) first_last[0] = col;
      first_last[1] = col;
    }
}

void token_columns(const CacheAttendParams& p, int32_t* columns) {
  for (int b = 0; b < p.B; ++b) p.D == 64 ? unit_columns<64>(p, b, columns + 2 * b) : unit_columns<128>(p, b, columns + 2 * b);
}

cudaError_t launch_cache_token(CacheAttendParams p, const TokenSplit& t, void* workspace, cudaStream_t s) {
  p.prefix = static_cast<int*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + (((size_t)p.B + 1) * 4 + 15) / 16 * 16);
  p.part_lse = p.part_o + (size_t)2 * t.blocks * t.warps * t.row_pad * p.D;
  if (p.D == 64) return t.row_pad == 16 ? launch_token<64, 1>(p, t, s) : launch_token<64, 2>(p, t, s);
  return t.row_pad == 16 ? launch_token<128, 1>(p, t, s) : launch_token<128, 2>(p, t, s);
}

}  // namespace swa
