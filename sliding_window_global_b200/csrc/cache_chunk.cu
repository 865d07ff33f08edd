// cache_chunk.cu -- attention over a paged cache when sequences bring many new tokens
// (bf16): prompts and their chunks.
//
// The bound is the tensor core. A query tile holds floor(128 / G) tokens with the G query
// heads of one KV head, so its 128 TMEM lanes share every key; a unit is two such tiles (A
// and B, consecutive tokens) of one KV head, which share every key tile they both see. Key
// tiles of 128 positions come from the pages by TMA, in boxes that never cross a page
// (16 to 128 keys); positions that do not exist are asked for outside the tensor map,
// which fills them with zeros. As in the band kernel (band_tc.cu): S = Q K^T by
// tcgen05.mma into TMEM, one thread per row for the softmax, P written over S, O += P V with
// P read from TMEM, a lazy rescale of O.
//
// Sequences' lengths are known on the device only, so a small kernel first lists the token
// tiles and cuts the list of all units' key tiles into one equal run for each block. A unit
// that a cut goes through leaves a partial result in each of its runs, joined afterwards in
// the order of the keys; short units are never cut. Where the units are few and short enough
// for a block each, there is no list: each block finds its own unit (of one query tile, if
// even these are few enough). Sequences that fill one query tile each run two blocks an SM
// (ONE), with one buffer of K and one of V that are freed apart, so that one block's softmax
// runs beside the other's products: see chunk_split.
//
// Measured: a 4096-token chunk over 16384 keys, 32/8 heads, D = 128, 804 us (1.20 PFLOP/s, 73% of
// the measured burst rate); six ragged chunks of up to 2048 tokens in a 512-key window 105 us.
//
// A capped score (ScoreCap) takes three operations of the MUFU instead of one: the long chunk
// 1600 us, the MUFU 83% active. Exponentials by a polynomial on the FMA pipe (1e-4 off) would
// gain a few per cent and show in the lse: they stay on the MUFU. The one-tile form has fewer
// registers a thread and spills with capped scores (34 x 76 tokens over 3713 keys, 12 heads,
// D = 64: 221 us, 115 uncapped).
//
// Warp roles (ONE has no tile B: 4 loads and so on): 0-3 softmax of tile A, 4-7 of tile B, 8 loads, 9 MMAs, 10 zeroes the values at
// positions outside the unit's keys (P is 0 there, but 0 times a NaN would not be).
#include <cuda_bf16.h>

#include <algorithm>

#include "cache_device.cuh"
#include "ptx.cuh"
#include "softmax_math.cuh"
#include "swa_host.h"

namespace swa {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsControl = 72;
constexpr int kOneThreads = 256, kOneRegsSoftmax = 192, kOneRegsControl = 64;   // units of one query tile, two blocks an SM
static_assert(128 * (kOneRegsSoftmax + kOneRegsControl) <= kOneThreads * 128, "setmaxnreg split exceeds the launch budget");
static_assert(256 * kRegsSoftmax + 128 * kRegsControl <= kThreads * 168 && 2 * kRegsSoftmax + kRegsControl <= 3 * 168,
              "setmaxnreg split exceeds the launch budget or a sub-partition's registers");
constexpr int kStages = 2;
constexpr uint32_t kSub = 128 * 128;                      // 128 rows of 128 bytes, swizzled
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;                 // log2 units
constexpr int kShortUnit = 16;                            // units of up to so many key tiles are not cut,
constexpr int kShortIfFew = 6, kDirectIfFew = 12;         // where they fill half the GPU at most: see chunk_split
constexpr int kMinPiece = 4;                              // nor is a unit cut this close to its ends
constexpr int kUnitRows = 2 * kTile;

// The tokens of a unit: a pair of query tiles of a sequence, or one (unit_tokens).
struct ChunkEntry {
  long long first;                 // first step (key tile) of its units: KV head 0, 1, ...
  int b;
  int row0;                        // row of the first token in the packed tensors
  int tokens;
  int pos0;                        // position of the first token
  int limit;                       // keys exist below this
  int base, tiles;                 // first key of key tile 0, key tiles
  int pad;
};

// Where a run starts; the entry behind the last run is the end of the list.
struct ChunkRun {
  long long step;
  int entry, hk, j;
  int inside;                      // the cut goes through a unit
};

struct ChunkParams {
  CUtensorMap mq, mk, mv;
  CacheAttendParams a;
  int* entry_first;                // [B] first entry of each sequence (many sequences)
  ChunkEntry* entries;
  ChunkRun* runs;                  // [runs + 1]
  float* part_o;                   // [runs, 2, 256, D]
  float* part_lse;                 // [runs, 2, 256]
  int num_runs, tile_tokens, unit_tokens, box, max_entries;
  int short_unit;                  // units of up to so many key tiles are not cut
  int direct;                      // a block a unit, no list
  float scale_log2;
};

// ------------------------------------------------------------------ the list of work
constexpr int kPlanThreads = 512;

// Inclusive sums over the block's threads; every thread calls it.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  __syncthreads();                                       // the sums of the call before are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  total = all;
  return x + before;
}

// The entry of sequence b's tokens from t0 on.
__device__ __forceinline__ ChunkEntry make_entry(const ChunkParams& p, int b, const CacheSeq& s, int t0) {
  ChunkEntry r = {};
  r.b = b;
  r.row0 = s.from + t0;
  r.tokens = min(p.unit_tokens, s.count - t0);
  r.pos0 = s.pos0 + t0;
  r.limit = s.limit;
  const int k0 = key_begin(p.a, s, t0), k1 = key_end(s, t0 + r.tokens - 1);
  r.base = k0 / p.box * p.box;
  r.tiles = k1 > k0 ? (k1 - r.base + kTile - 1) / kTile : 1;
  return r;
}

// The first kPlanThreads sequences and entries are searched in shared memory, more of them
// in the workspace.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ long long warp_sums[kPlanThreads / 32], s_step[kPlanThreads];
  __shared__ int s_entry[kPlanThreads + 1], s_tiles[kPlanThreads];
  const CacheAttendParams& a = p.a;
  const int pair = p.unit_tokens;
  grid_launch_dependents();
  // units' tokens of each sequence
  const bool few = a.B <= kPlanThreads;
  int* entry_first = few ? s_entry : p.entry_first;
  long long total, before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long long n = 0;
    if (b < a.B) {
      const CacheSeq s = cache_seq(a, b);
      if (s.bad) atomicOr(a.err, kDevErrCheck);
      n = (s.count + pair - 1) / pair;
    }
    const long long upto = block_scan(n, warp_sums, total);
    if (b < a.B) entry_first[b] = (int)min(before + upto - n, (long long)p.max_entries);
    before += total;
  }
  const int entries = (int)min(before, (long long)p.max_entries);   // overlapping cu_tokens may name more rows than T
  __syncthreads();
  // their keys, and the first step of each
  long long steps = 0;
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    ChunkEntry r = {};
    long long n = 0;
    if (e < entries) {
      int lo = 0, hi = a.B - 1;                          // the last sequence that starts at or before e
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (entry_first[mid] <= e) lo = mid;
        else hi = mid - 1;
      }
      r = make_entry(p, lo, cache_seq(a, lo), (e - entry_first[lo]) * pair);
      n = (long long)r.tiles * a.Hkv;
    }
    const long long upto = block_scan(n, warp_sums, total);
    r.first = steps + upto - n;
    if (e < entries) p.entries[e] = r;
    if (e0 == 0) {
      s_step[threadIdx.x] = r.first;
      s_tiles[threadIdx.x] = r.tiles;
    }
    steps += total;
  }
  __syncthreads();
  // equal runs, their cuts moved to a unit's edge where the unit is short or the edge near
  const bool listed = entries <= kPlanThreads;
  for (int c = threadIdx.x; c <= p.num_runs; c += kPlanThreads) {
    const long long x = steps * c / p.num_runs;
    ChunkRun r = {x, entries, 0, 0, 0};
    if (x < steps) {
      int lo = 0, hi = entries - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((listed ? s_step[mid] : p.entries[mid].first) <= x) lo = mid;
        else hi = mid - 1;
      }
      const int tiles = listed ? s_tiles[lo] : p.entries[lo].tiles;
      const long long in = x - (listed ? s_step[lo] : p.entries[lo].first);
      r.entry = lo;
      r.hk = (int)(in / tiles);
      r.j = (int)(in % tiles);
      const bool to_start = tiles <= p.short_unit ? 2 * r.j < tiles : r.j < kMinPiece;
      const bool to_end = tiles <= p.short_unit ? !to_start : tiles - r.j < kMinPiece;
      if (to_start) {
        r.step -= r.j;
        r.j = 0;
      } else if (to_end) {
        r.step += tiles - r.j;
        r.j = 0;
        if (++r.hk == a.Hkv) {
          r.hk = 0;
          ++r.entry;
        }
      }
      r.inside = r.j > 0;
    }
    p.runs[c] = r;
  }
}

// ------------------------------------------------------------------ a run's pieces
// Key tiles [j0, j1) of one unit.
struct Piece {
  ChunkEntry en;
  int hk, j0, j1;
};

// One query tile of a piece: its rows and the key tiles [a, e) it uses.
struct Half {
  int tok0, tokens;                // first token in the entry, tokens
  int lo, hi;                      // keys its rows see
  int a, e;
};

__device__ __forceinline__ Half half_of(const ChunkParams& p, const Piece& pc, int x) {
  Half h;
  h.tok0 = x * p.tile_tokens;
  h.tokens = min(max(pc.en.tokens - h.tok0, 0), p.tile_tokens);
  const int pos = pc.en.pos0 + h.tok0;
  h.lo = p.a.window < 0 ? 0 : (int)max(0LL, (long long)pos - p.a.window);
  h.hi = min(pos + h.tokens, pc.en.limit);
  // rows without a key still take part in one tile, so that they are written
  int a = min(max(h.lo - pc.en.base, 0) / kTile, pc.en.tiles - 1);
  int e = h.hi > h.lo ? min((h.hi - pc.en.base + kTile - 1) / kTile, pc.en.tiles) : a + 1;
  h.a = max(a, pc.j0);
  h.e = h.tokens > 0 ? max(h.a, min(e, pc.j1)) : h.a;
  return h;
}

// Direct calls: the entry of this block's unit, found by one warp (no tiles: there is none).
__device__ __forceinline__ void find_unit(const ChunkParams& p, int lane, ChunkEntry* own) {
  const int e = blockIdx.x / p.a.Hkv;
  int before = 0;
  if (lane == 0) *own = ChunkEntry{};
  __syncwarp();
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    const int b = b0 + lane;
    CacheSeq s = {};
    if (b < p.a.B) {
      s = cache_seq(p.a, b);
      if (s.bad && blockIdx.x == 0) atomicOr(p.a.err, kDevErrCheck);
    }
    const int n = (s.count + p.unit_tokens - 1) / p.unit_tokens;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const int first = before + upto - n;
    if (e >= first && e < first + n) *own = make_entry(p, b, s, (e - first) * p.unit_tokens);
    before += __shfl_sync(0xffffffffu, upto, 31);
    if (before > e && blockIdx.x > 0) break;
  }
}

// The pieces of a block's run, in order; every warp role walks them alike. The entry behind
// a piece's own is fetched a piece ahead.
struct Walk {
  long long left;
  int entry, hk, j;
  ChunkEntry ahead;
  __device__ __forceinline__ Walk(const ChunkParams& p, const ChunkEntry& own) {
    if (p.direct) {
      left = own.tiles;
      entry = 0;
      hk = blockIdx.x % p.a.Hkv;
      j = 0;
      ahead = own;
      return;
    }
    const ChunkRun& r = p.runs[blockIdx.x];
    left = p.runs[blockIdx.x + 1].step - r.step;
    entry = r.entry;
    hk = r.hk;
    j = r.j;
    if (left > 0) ahead = p.entries[entry];
  }
  __device__ __forceinline__ bool next(const ChunkParams& p, Piece& pc) {
    if (left <= 0) return false;
    pc.en = ahead;
    pc.hk = hk;
    pc.j0 = j;
    pc.j1 = (int)min((long long)pc.en.tiles, j + left);
    left -= pc.j1 - pc.j0;
    j = 0;
    if (++hk == p.a.Hkv) {
      hk = 0;
      ++entry;
      if (left > 0) ahead = p.entries[entry];
    }
    return true;
  }
};

struct ChunkShared {
  ChunkEntry own;                  // direct calls: this block's unit
  uint32_t missing[kStages];       // 16-key groups of a key tile whose page does not exist
  uint32_t tmem_slot;
  int abort_flag;
};

template <int D, bool ONE>
struct ChunkCfg {
  static constexpr int kTiles = ONE ? 1 : 2;                // query tiles
  static constexpr int kBuffers = ONE ? 1 : kStages;        // of K and of V
  static constexpr uint32_t kTileBytes = 128u * D * 2u;
  static constexpr uint32_t kKOff = kTiles * kTileBytes;
  static constexpr uint32_t kVOff = kKOff + kBuffers * kTileBytes;
  static constexpr uint32_t kOutOff = kVOff + kBuffers * kTileBytes;   // 4 KB a softmax warp: 32 rows x 64 columns
  static constexpr uint32_t kBarOff = kOutOff + kTiles * 4 * 4096;
  static constexpr int kNumBars = 2 + 2 + 5 * kStages + 2 + 2 + 2 + 2;
  static constexpr uint32_t kUnitOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr uint32_t kSmemBytes = kUnitOff + sizeof(ChunkShared);
  static constexpr uint32_t kTmemCols = ONE ? 256 : 512;
  // TMEM columns: S_A | S_B | O_A | O_B, P over S
  __host__ __device__ static constexpr uint32_t s_col(int x) { return x ? 128u : 0u; }
  __host__ __device__ static constexpr uint32_t o_col(int x) { return ONE ? 128u : 256u + (x ? D : 0); }
};
static_assert(ChunkCfg<128, false>::kSmemBytes <= 227 * 1024 && 2 * (ChunkCfg<128, true>::kSmemBytes + 1024) <= 228 * 1024,
              "shared memory");

// A value that is the same in every lane, said so to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ float row_max(const float (&x)[kTile]) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fmaxf(x[i], x[8 + i]);
#pragma unroll
  for (int e = 16; e < kTile; e += 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmax3(m[i], x[e + i], x[e + 8 + i]);
  }
  return fmax3(fmax3(m[0], m[1], m[2]), fmax3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

template <int D, int CAP, bool ONE>
__global__ void __launch_bounds__(ONE ? kOneThreads : kThreads, ONE ? 2 : 1)
cache_chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = ChunkCfg<D, ONE>;
  constexpr int NX = C::kTiles, NB = C::kBuffers;
  constexpr int kLoads = 4 * NX, kMma = kLoads + 1, kClear = kLoads + 2;   // warp roles behind the softmax's
  constexpr int kInc = ONE ? kOneRegsSoftmax : kRegsSoftmax, kDec = ONE ? kOneRegsControl : kRegsControl;
  // no static shared memory lies before it, so it begins on a 1024-byte boundary
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kKOff;
  uint8_t* sV = smem + C::kVOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_full = bars;                 // [2]
  uint64_t* q_empty = bars + 2;            // [2]
  uint64_t* k_full = bars + 4;             // [kStages] K of a key tile has landed
  uint64_t* v_full = k_full + kStages;     // V has landed
  uint64_t* v_ready = v_full + kStages;    // V is free of values outside the unit's keys
  uint64_t* kv_empty = v_ready + kStages;  // V has been used, and K with two buffers
  uint64_t* k_empty = kv_empty + kStages;  // one buffer: K has been used
  uint64_t* s_full = k_empty + kStages;    // [2]
  uint64_t* p_half = s_full + 2;           // [2] P of keys 0-63 written
  uint64_t* p_full = p_half + 2;           // [2]
  uint64_t* o_full = p_full + 2;           // [2]
  ChunkShared& shared = *reinterpret_cast<ChunkShared*>(smem + C::kUnitOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) % 1024 != 0) {        // the swizzled tiles rest on it
    if (tid == 0) atomicOr(p.a.err, kDevErrCheck);
    return;
  }
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_half[x], kTile);
      mbar_init(&p_full[x], kTile);
      mbar_init(&o_full[x], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_ready[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    shared.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMma) {
    tmem_alloc(&shared.tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (p.direct && warp == kLoads) find_unit(p, lane, &shared.own);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = shared.tmem_slot;
  const ChunkEntry& own = shared.own;
  volatile int* abort_v = &shared.abort_flag;
  grid_dependency_wait();                  // the list of work
  grid_launch_dependents();

  if (warp == kLoads) {
    // ------------------------------------------------------------ loads
    setmaxnreg_dec<kDec>();
    const int halves = D / 64, boxes = kTile / p.box;
    const int box = lane / halves, sub = lane % halves;    // of a key tile: this lane's box
    const bool loads = lane < boxes * halves;
    const uint32_t box_off = sub * kSub + box * p.box * 128;
    const int nowhere = p.a.num_pages * p.a.Hkv;           // a plane outside the maps: zeros
    const uint32_t q_bytes = (uint32_t)(p.tile_tokens * p.a.G) * D * 2;
    int qloads[2] = {0, 0};
    int kv = 0;
    bool ok = true;
    Walk walk(p, own);
    Piece pc;
    while (ok && walk.next(p, pc)) {
      const Half ha = half_of(p, pc, 0), hb = half_of(p, pc, 1);
      const int lo = ha.lo, hi = hb.tokens > 0 ? hb.hi : ha.hi;
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const Half& h = x ? hb : ha;
        if (!ok || h.e <= h.a) continue;
        if (qloads[x] > 0) ok = mbar_wait_bounded(&q_empty[x], (qloads[x] - 1) & 1, abort_v, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[x], q_bytes);
          for (int c = 0; c < halves; ++c)
            tma_load_3d(sQ + x * C::kTileBytes + c * kSub, &p.mq, &q_full[x], 64 * c, pc.hk * p.a.G,
                        pc.en.row0 + h.tok0);
        }
        __syncwarp();
        ++qloads[x];
      }
      const int32_t* table = p.a.block_table + (long long)pc.en.b * p.a.max_pages;
      for (int j = pc.j0; ok && j < pc.j1; ++j, ++kv) {
        const int st = kv % kStages;
        const int key = pc.en.base + j * kTile + box * p.box;
        int y = 0, z = nowhere;
        uint32_t miss = 0;
        if (loads && key < hi && key + p.box > lo) {
          const int page = __ldg(table + key / p.a.page_size);
          if (page >= 0 && page < p.a.num_pages) {
            y = key % p.a.page_size;
            z = page * p.a.Hkv + pc.hk;
          } else {
            miss = ((1u << (p.box / 16)) - 1) << (box * p.box / 16);
          }
        }
        miss = __reduce_or_sync(0xffffffffu, miss);
        // the step whose buffers these are
        const int from = kv - NB, fs = (from + kStages) % kStages;
        if (from >= 0) ok = mbar_wait_bounded(ONE ? &k_empty[fs] : &kv_empty[fs], (from / kStages) & 1, abort_v, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          shared.missing[st] = miss;
          if (miss) atomicOr(p.a.err, kDevErrCheck);
          mbar_arrive_expect_tx(&k_full[st], C::kTileBytes);
        }
        __syncwarp();
        if (loads) tma_load_3d(sK + kv % NB * C::kTileBytes + box_off, &p.mk, &k_full[st], 64 * sub, y, z);
        if (ONE && from >= 0) {
          ok = mbar_wait_bounded(&kv_empty[fs], (from / kStages) & 1, abort_v, kWaitLimitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&v_full[st], C::kTileBytes);
        __syncwarp();
        if (loads) tma_load_3d(sV + kv % NB * C::kTileBytes + box_off, &p.mv, &v_full[st], 64 * sub, y, z);
      }
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMAs
    // The whole warp walks the steps and one thread issues, see elect_one.
    setmaxnreg_dec<kDec>();
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, true);
    const uint32_t q_lo = sdesc_lo(smem_u32(sQ), 16);
    const uint32_t k_lo = sdesc_lo(smem_u32(sK), 16);
    const uint32_t v_lo = sdesc_lo(smem_u32(sV), kSub);
    const uint32_t tm = uniform(tmem);
    int qwaits[2] = {0, 0}, pwaits[2] = {0, 0};
    int kv = 0;                            // ring position of the step
    bool ok = true;
    Walk walk(p, own);
    Piece pc;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_v, kWaitLimitNs));
    };
    auto issue_qk = [&](int x, int g, bool last) -> bool {
      const int st = g % kStages;
      if (!wait(&k_full[st], (g / kStages) & 1)) return false;
      tc_fence_after();
      const uint32_t qd = q_lo + x * (C::kTileBytes >> 4), kd = k_lo + g % NB * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kSub + (kk & 3) * 32) >> 4;
          umma_ss_lo(tm + C::s_col(x), qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[x]);
        if (ONE) umma_commit(&k_empty[st]);
        if (last) umma_commit(&q_empty[x]);
      }
      __syncwarp();
      return true;
    };
    while (ok && walk.next(p, pc)) {
      int a[2] = {0, 0}, e[2] = {0, 0};
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const Half h = half_of(p, pc, x);
        a[x] = uniform(h.a);
        e[x] = uniform(h.e);
      }
      const int j0 = uniform(pc.j0), j1 = uniform(pc.j1);
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        if (!ok || e[x] <= a[x]) continue;
        ok = wait(&q_full[x], qwaits[x]++ & 1);
      }
      for (int j = j0; ok && j < j1; ++j, ++kv) {
        const int st = kv % kStages;
#pragma unroll
        for (int x = 0; x < NX; ++x)
          if (ok && j == a[x] && a[x] < e[x]) ok = issue_qk(x, kv, j == e[x] - 1);
        if (!ok) break;
        if (!wait(&v_ready[st], (kv / kStages) & 1)) { ok = false; break; }
        const bool any = (j >= a[0] && j < e[0]) || (j >= a[1] && j < e[1]);
        if (!any) {                        // nobody reads the tile; its K must have landed too
          ok = wait(&k_full[st], (kv / kStages) & 1);
          if (lane == 0) {
            mbar_arrive(&kv_empty[st]);
            if (ONE) mbar_arrive(&k_empty[st]);
          }
          continue;
        }
        const uint32_t vd = v_lo + kv % NB * (C::kTileBytes >> 4);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          if (!ok || j < a[x] || j >= e[x]) continue;
          const uint32_t add = j > a[x] ? 1u : 0u;
          if (!wait(&p_half[x], pwaits[x] & 1)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)
              umma_ts_lo(tm + C::o_col(x), tm + C::s_col(x) + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv, kk > 0 ? 1u : add);
          }
          __syncwarp();
          if (!wait(&p_full[x], pwaits[x] & 1)) { ok = false; break; }
          ++pwaits[x];
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = kTile / 32; kk < kTile / 16; ++kk)
              umma_ts_lo(tm + C::o_col(x), tm + C::s_col(x) + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv, 1u);
            if (j == e[x] - 1) umma_commit(&o_full[x]);
            if (ONE) umma_commit(&kv_empty[st]);
          }
          __syncwarp();
          if (j < e[x] - 1) ok = issue_qk(x, kv + 1, j + 1 == e[x] - 1);
        }
        if (!ONE && elect_one()) umma_commit(&kv_empty[st]);
        __syncwarp();
      }
    }
  } else if (warp == kClear) {
    // ------------------------------------------------------------ values outside the unit's keys
    setmaxnreg_dec<kDec>();
    int kv = 0;
    bool ok = true;
    Walk walk(p, own);
    Piece pc;
    while (ok && walk.next(p, pc)) {
      const Half ha = half_of(p, pc, 0), hb = half_of(p, pc, 1);
      const int lo = ha.lo, hi = hb.tokens > 0 ? hb.hi : ha.hi;
      for (int j = pc.j0; j < pc.j1; ++j, ++kv) {
        const int st = kv % kStages;
        ok = mbar_wait_bounded(&v_full[st], (kv / kStages) & 1, abort_v, kWaitLimitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int key0 = pc.en.base + j * kTile;
        if (key0 < lo || key0 + kTile > hi) {
          for (int i = lane; i < kTile * (D / 8); i += 32) {
            const int row = i / (D / 8), c = i % (D / 8);
            if (key0 + row < lo || key0 + row >= hi)       // a whole row: its swizzle does not matter
              *reinterpret_cast<uint4*>(sV + kv % NB * C::kTileBytes + (c / 8) * kSub + row * 128 + (c % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ready[st]);
      }
    }
  } else if (warp > kClear) {
    setmaxnreg_dec<kDec>();
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kInc>();
    const int x = warp >> 2;
    const int row = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_base + C::s_col(x), o_addr = lane_base + C::o_col(x);
    const int tok = row / p.a.G, head = row % p.a.G;
    const float sl2 = p.scale_log2;
    const ScoreCap<CAP> score_cap(sl2, p.a.softcap);
    int it = 0, oc = 0, kv = 0;
    bool ok = true;
    Walk walk(p, own);
    Piece pc;
    while (ok && walk.next(p, pc)) {
      const Half h = half_of(p, pc, x);
      const int kv0_piece = kv;
      kv += pc.j1 - pc.j0;
      const bool whole = pc.j0 == 0 && pc.j1 == pc.en.tiles;
      const bool row_valid = tok < h.tokens;             // rows behind the last token of the tile hold nothing
      // partial results: slot 0 where the unit began in an earlier run, else slot 1
      const long long part = ((long long)blockIdx.x * 2 + (pc.j0 == 0 ? 1 : 0)) * kUnitRows + x * kTile + row;
      if (h.e <= h.a) {
        if (!whole && row_valid) p.part_lse[part] = -INFINITY;
        continue;
      }
      const int pos = pc.en.pos0 + h.tok0 + tok;
      int klo = p.a.window < 0 ? 0 : max(0, pos - p.a.window);
      int khi = min(pos + 1, pc.en.limit);
      if (!row_valid) khi = klo = 0;
      const int all_lo = __reduce_max_sync(0xffffffffu, klo);  // keys [all_lo, all_hi) need no mask in this warp
      const int all_hi = __reduce_min_sync(0xffffffffu, khi);
      float m = -INFINITY, l = 0.f;
      for (int j = h.a; j < h.e; ++j) {
        const int g = kv0_piece + j - pc.j0;
        if (!mbar_wait_bounded(&s_full[x], it & 1, abort_v, kWaitLimitNs)) { ok = false; break; }
        // the phase that published `missing` is over: this orders the read below after it
        if (!mbar_wait_bounded(&k_full[g % kStages], (g / kStages) & 1, abort_v, kWaitLimitNs)) { ok = false; break; }
        const uint32_t miss = shared.missing[g % kStages];
        tc_fence_after();
        uint32_t xr[kTile];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld32(s_addr + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(xr + ch * 32));
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_wait_ld_dep(*reinterpret_cast<uint32_t(*)[32]>(xr + ch * 32));
        float s[kTile];
#pragma unroll
        for (int e = 0; e < kTile; e += 2) {
          s[e] = __uint_as_float(xr[e]);
          s[e + 1] = __uint_as_float(xr[e + 1]);
          if (CAP) score_cap.pair(s[e], s[e + 1]);
        }
        const int key0 = pc.en.base + j * kTile;
        const int lo_t = klo - key0, hi_t = khi - key0;
        uint32_t live = 0xF;               // 32-column chunks with a key for any row of the warp
        if (key0 < all_lo || key0 + kTile > all_hi || miss) {
          // One path for every kind of mask (a bit a key): the loop has to stay small, since
          // its instructions are fetched anew on every way around.
          live = 0;
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t keep = lo_t <= 32 * ch ? ~0u : lo_t >= 32 * ch + 32 ? 0u : ~0u << (lo_t - 32 * ch);
            keep &= hi_t >= 32 * ch + 32 ? ~0u : hi_t <= 32 * ch ? 0u : ~(~0u << (hi_t - 32 * ch));
            keep &= ((miss >> (2 * ch)) & 1 ? 0u : 0xffffu) | ((miss >> (2 * ch + 1)) & 1 ? 0u : 0xffff0000u);
            if (__any_sync(0xffffffffu, keep != 0)) live |= 1u << ch;
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * ch + e] = (keep >> e & 1) ? s[32 * ch + e] : -INFINITY;
          }
        }
        const float mul = CAP ? 1.f : sl2;
        const float m_new = fmaxf(m, row_max(s) * mul);
        const bool need = (m == -INFINITY) ? (m_new > -INFINITY) : (m_new > m + kRescaleThreshold);
        const bool rescale = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (rescale) {
          alpha = (m == -INFINITY) ? 0.f : ex2_approx(m - m_new);
          l *= alpha;
          m = m_new;
        }
        const float neg_m = (m == -INFINITY) ? 0.f : -m;
        if (rescale && j > h.a) {
          // O is stable: its previous product was issued before this S, and they end in order
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t rr[16];
            tmem_ld16(o_addr + ch * 16, rr);
            tmem_wait_ld_dep16(rr);
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st16(o_addr + ch * 16, rr);
          }
        }
        float acc0 = 0.f, acc1 = 0.f, acc2 = 0.f, acc3 = 0.f;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
          if (!(live & (1u << ch))) {
#pragma unroll
            for (int q = 0; q < 16; ++q) pk[q] = 0u;
          } else {
#pragma unroll
            for (int q = 0; q < 32; q += 4) {
              const int e = ch * 32 + q;
              float a0, a1, a2, a3;
              ffma2(a0, a1, s[e], s[e + 1], mul, mul, neg_m, neg_m);
              ffma2(a2, a3, s[e + 2], s[e + 3], mul, mul, neg_m, neg_m);
              a0 = ex2_approx(a0);
              a1 = ex2_approx(a1);
              a2 = ex2_approx(a2);
              a3 = ex2_approx(a3);
              fadd2(acc0, acc1, acc0, acc1, a0, a1);
              fadd2(acc2, acc3, acc2, acc3, a2, a3);
              // P in bf16, the type of the product that follows; the sum keeps 32 bits, which the
              // lse shows. Root mean square error of the outputs against 64 bits: 2.3e-3 of
              // their size, 1.7e-3 of it their own rounding to bf16.
              pk[q / 2] = pack_bf16x2(a0, a1);
              pk[q / 2 + 1] = pack_bf16x2(a2, a3);
            }
          }
          tmem_st16(s_addr + ch * 16, pk);
          if (ch == 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_half[x]);
          }
        }
        l += (acc0 + acc1) + (acc2 + acc3);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[x]);
        ++it;
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      // O is read before this group's next p_half arrival, which the MMA warp waits for
      // before it writes O again.
      if (!mbar_wait_bounded(&o_full[x], oc & 1, abort_v, kWaitLimitNs)) { ok = false; break; }
      ++oc;
      tc_fence_after();
      const bool has = l != 0.f;           // also where every score is NaN
      const float inv = has ? 1.f / l : 0.f;
      const float lse = has ? (m + __log2f(l)) * kLn2 : -INFINITY;
      // Rows leave through shared memory, so that eight lanes write 128 bytes of a row: 64 bf16
      // or 32 fp32 columns at a time, the 16-byte chunks of a row swizzled by its number.
      const int out_row = (pc.en.row0 + h.tok0 + tok) * p.a.Hq + pc.hk * p.a.G + head;
      const int rows_here = min(h.tokens * p.a.G - (warp & 3) * 32, 32);       // rows of this warp that exist
      uint8_t* stage = smem + C::kOutOff + warp * 4096;
      const int sw_row = lane >> 3, sw_chunk = lane & 7;
#pragma unroll 1
      for (int half = 0; half < (whole ? D / 64 : D / 32); ++half) {
        if (whole) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t rr[32];
            tmem_ld32(o_addr + half * 64 + ch * 32, rr);
            tmem_wait_ld_dep(rr);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 v;
              v.x = pack_bf16x2(__uint_as_float(rr[q * 8 + 0]) * inv, __uint_as_float(rr[q * 8 + 1]) * inv);
              v.y = pack_bf16x2(__uint_as_float(rr[q * 8 + 2]) * inv, __uint_as_float(rr[q * 8 + 3]) * inv);
              v.z = pack_bf16x2(__uint_as_float(rr[q * 8 + 4]) * inv, __uint_as_float(rr[q * 8 + 5]) * inv);
              v.w = pack_bf16x2(__uint_as_float(rr[q * 8 + 6]) * inv, __uint_as_float(rr[q * 8 + 7]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((ch * 4 + q) ^ (lane & 7)) << 4)) = v;
            }
          }
        } else {
          uint32_t rr[32];
          tmem_ld32(o_addr + half * 32, rr);
          tmem_wait_ld_dep(rr);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 v = make_float4(__uint_as_float(rr[q * 4 + 0]) * inv, __uint_as_float(rr[q * 4 + 1]) * inv,
                                         __uint_as_float(rr[q * 4 + 2]) * inv, __uint_as_float(rr[q * 4 + 3]) * inv);
            *reinterpret_cast<float4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = v;
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + sw_row;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((sw_chunk ^ (r & 7)) << 4));
          const int to = __shfl_sync(0xffffffffu, out_row, r);
          uint4* dst = whole ? reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + (long long)to * D) + half * 8
                             : reinterpret_cast<uint4*>(p.part_o + (part - lane + r) * D) + half * 8;
          if (r < rows_here) dst[sw_chunk] = v;
        }
        __syncwarp();
      }
      if (row_valid && whole && p.a.lse) p.a.lse[out_row] = lse;
      if (row_valid && !whole) p.part_lse[part] = lse;
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (shared.abort_flag) {
    // A bounded wait expired: report it, then give copies and MMAs still in flight time to
    // land before TMEM and shared memory are released.
    if (tid == 0) {
      atomicOr(p.a.err, kDevErrTimeout);
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 2000000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == kMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of a unit that cuts go through: block row c belongs to the first cut
// inside its unit, one warp to a row; parts are added in the order of the keys.
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int E = D / 32;
  grid_dependency_wait();
  const int c = blockIdx.x + 1;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const ChunkRun cut = p.runs[c];
  if (!cut.inside) return;
  const ChunkEntry en = p.entries[cut.entry];
  const long long u0 = cut.step - cut.j, u1 = u0 + en.tiles;
  if (p.runs[c - 1].step > u0) return;                    // not the first cut of its unit
  const int x = r / kTile, row = r % kTile, tok = x * p.tile_tokens + row / p.a.G;
  if (row >= p.tile_tokens * p.a.G || tok >= en.tokens) return;
  // a lane a part, 32 of them at a time: first their largest lse, then their weights
  auto part_of = [&](int k) { return ((long long)k * 2 + (k == c - 1 ? 1 : 0)) * kUnitRows + r; };
  auto lse_of = [&](int k, bool& more) {                  // -inf: no part, or no key in it
    const long long step = k < p.num_runs ? p.runs[k].step : u1;
    more = __all_sync(0xffffffffu, step < u1);
    return step < u1 && p.runs[k + 1].step > step ? p.part_lse[part_of(k)] : -INFINITY;
  };
  bool more = true;
  float top = -INFINITY, first = 0.f;
  for (int k = c - 1; more; k += 32) {
    const float lse = lse_of(k + lane, more);
    if (k == c - 1) first = lse;
    top = fmaxf(top, lse);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  more = true;
  for (int k0 = c - 1; more; k0 += 32) {
    float lse = first;
    if (k0 == c - 1) more = __all_sync(0xffffffffu, k0 + lane < p.num_runs && p.runs[min(k0 + lane, p.num_runs)].step < u1);
    else lse = lse_of(k0 + lane, more);
    const float mine = lse == -INFINITY ? 0.f : ex2_approx((lse - top) * kLog2e);      // a NaN goes on
    const uint32_t parts = __ballot_sync(0xffffffffu, lse != -INFINITY);
    const int n = 32 - __clz(parts);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float f = __shfl_sync(0xffffffffu, mine, k);
      const bool on = parts >> k & 1;                    // else nothing was written there
      const float2* src = reinterpret_cast<const float2*>(p.part_o + part_of(k0 + k) * D) + lane;
      l += f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = on ? src[16 * e] : make_float2(0.f, 0.f);
        o[e] += f * v.x;
        o[e + 1] += f * v.y;
      }
    }
  }
  const bool has = l != 0.f;
  const float inv = has ? 1.f / l : 0.f;
  const long long out_row = (long long)(en.row0 + tok) * p.a.Hq + cut.hk * p.a.G + row % p.a.G;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.out) + out_row * D) + lane;
#pragma unroll
  for (int e = 0; e < E; e += 2) out[16 * e] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (p.a.lse && lane == 0) p.a.lse[out_row] = has ? top + __log2f(l) * kLn2 : -INFINITY;
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

template <int D, int CAP, bool ONE>
cudaError_t launch_units(const ChunkParams& p, cudaLaunchConfig_t cfg) {
  const cudaError_t e = allow_smem<&cache_chunk_kernel<D, CAP, ONE>>((int)ChunkCfg<D, ONE>::kSmemBytes);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(ONE ? kOneThreads : kThreads);
  cfg.dynamicSmemBytes = ChunkCfg<D, ONE>::kSmemBytes;
  return cudaLaunchKernelEx(&cfg, cache_chunk_kernel<D, CAP, ONE>, p);
}

template <int D, bool ONE>
cudaError_t launch_units(const ChunkParams& p, int cap, const cudaLaunchConfig_t& cfg) {
  return cap == kCapAny     ? launch_units<D, kCapAny, ONE>(p, cfg)
         : cap == kCapUsual ? launch_units<D, kCapUsual, ONE>(p, cfg)
                            : launch_units<D, kCapNone, ONE>(p, cfg);
}

template <int D>
cudaError_t launch_chunk(const ChunkParams& p, const ChunkSplit& t, cudaStream_t s) {
  cudaError_t e;
  if (!p.direct) {
    chunk_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int cap = cap_kind(p.a.softcap);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_runs);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.direct ? 0 : 1;
  e = t.one ? launch_units<D, true>(p, cap, cfg) : launch_units<D, false>(p, cap, cfg);
  if (e != cudaSuccess || !t.split || p.num_runs < 2) return e;
  cfg.gridDim = dim3(p.num_runs - 1, kUnitRows / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D>, p);
}

}  // namespace

ChunkSplit chunk_split(int B, int T, int Hkv, int G, int D, int page_size, int max_tokens, int max_len,
                       int window) {
  ChunkSplit t = {};
  t.tile_tokens = kTile / G;
  t.box = 16;
  while (t.box < kTile && page_size % (2 * t.box) == 0) t.box *= 2;
  // Units of one query tile, a block each, where all of them fit on the GPU at once; else
  // of two, which share their keys' loads and hide each other's latencies. A block a unit
  // without a list needs units that are short and sequences that one warp can look through.
  // Where the units leave half the GPU idle, the long ones among them are cut after all: 256
  // tokens over 1900 keys (8/8 heads) 43 -> 27 us, 16 over 2000 (32/8) 39 -> 23, while 900
  // over 950 (4/1, 8 tiles a unit) take 23 a block each and 29 cut.
  // Sequences of one query tile each (small) have units of one, two blocks an SM, where these are
  // enough for all blocks uncut or leave each a long run: 34 x 76 tokens over 3713 keys, 12
  // heads, D = 64, 174 -> 118 us, 8 x 16 over 8192 (32/8) 76 -> 70; 16 x 64 over 2000 (8 heads) 39,
  // with the cuts that two blocks an SM would need 49.
  const bool small = max_tokens <= t.tile_tokens;
  for (int tiles_per_unit = 1; tiles_per_unit <= 2; ++tiles_per_unit) {
    t.unit_tokens = tiles_per_unit * t.tile_tokens;
    t.max_entries = small ? std::min(B, T) : (int)(T / t.unit_tokens + std::min<long long>(B, T));
    // key tiles of a unit at most
    const long long reach = window < 0 ? max_len : std::min<long long>(max_len, (long long)window + t.unit_tokens);
    const long long tiles = (reach + t.box + kTile - 1) / kTile + 1;
    const long long units = (long long)t.max_entries * Hkv;
    t.one = small && tiles_per_unit == 2 && (units >= 296 || units * tiles >= 12 * 296);
    if (t.one) t.unit_tokens = t.tile_tokens;
    const bool few = units <= 74;
    t.short_unit = few ? kShortIfFew : kShortUnit;
    t.direct = units <= 148 && B <= 1024 && tiles <= (few ? kDirectIfFew : kShortUnit);
    t.split = !t.direct && tiles > t.short_unit;
    // two key tiles a run at least
    t.runs = (int)std::min<long long>(t.one ? 296 : 148, t.direct ? units : std::max<long long>(1, units * tiles / 2));
    if (t.direct) break;
  }
  if (t.direct) return t;
  const size_t rows = t.split ? (size_t)t.runs * 2 * kUnitRows : 0;
  t.bytes = up16((size_t)B * 4) + up16((size_t)t.max_entries * sizeof(ChunkEntry)) +
            up16((size_t)(t.runs + 1) * sizeof(ChunkRun)) + rows * (D + 1) * 4;
  return t;
}

cudaError_t launch_cache_chunk(const CacheAttendParams& a, const ChunkSplit& t, void* workspace, cudaStream_t s) {
  ChunkParams p = {};
  const uint64_t e = 2;                    // bytes of an element
  // strides of axes of length one are free: give the map one it accepts
  const uint64_t qh = a.Hq > 1 ? (uint64_t)a.q_head * e : (uint64_t)a.D * e;
  const uint64_t qt = a.T > 1 ? (uint64_t)a.q_token * e : (uint64_t)a.D * e;
  const uint64_t row = (uint64_t)a.D * e, plane = (uint64_t)a.page_size * row;
  if (!make_load_map(&p.mq, a.q, a.D, a.Hq, a.T, qh, qt, a.G, t.tile_tokens) ||
      !make_load_map(&p.mk, a.k_pages, a.D, a.page_size, (uint64_t)a.num_pages * a.Hkv, row, plane, t.box, 1) ||
      !make_load_map(&p.mv, a.v_pages, a.D, a.page_size, (uint64_t)a.num_pages * a.Hkv, row, plane, t.box, 1))
    return cudaErrorInvalidValue;
  p.a = a;
  p.direct = t.direct;
  p.short_unit = t.short_unit;
  p.unit_tokens = t.unit_tokens;
  if (!t.direct) {
    char* ws = static_cast<char*>(workspace);
    p.entry_first = reinterpret_cast<int*>(ws);
    ws += up16((size_t)a.B * 4);
    p.entries = reinterpret_cast<ChunkEntry*>(ws);
    ws += up16((size_t)t.max_entries * sizeof(ChunkEntry));
    p.runs = reinterpret_cast<ChunkRun*>(ws);
    ws += up16((size_t)(t.runs + 1) * sizeof(ChunkRun));
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = p.part_o + (t.split ? (size_t)t.runs * 2 * kUnitRows * a.D : 0);
  }
  p.num_runs = t.runs;
  p.tile_tokens = t.tile_tokens;
  p.box = t.box;
  p.max_entries = t.max_entries;
  p.scale_log2 = a.scale * kLog2e;
  return a.D == 64 ? launch_chunk<64>(p, t, s) : launch_chunk<128>(p, t, s);
}

}  // namespace swa
