// cache_kernels.h -- checks, parameter block and launchers of the attention over a paged
// cache.  Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/swa.h"

namespace swa {

// Allow Kern `bytes` of dynamic shared memory; asked of the driver once a device.
template <auto Kern>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

// Checks of a cache and of a batch: SWA_ERR_INVALID_ARG for a null or misaligned pointer
// or a bad size, SWA_ERR_UNSUPPORTED for a shape the kernels do not implement.
swa_status check_cache(const swa_cache& c);
swa_status check_batch(const swa_cache_batch& b);

struct CacheAttendParams {
  const void* k_pages;
  const void* v_pages;
  const void* q;
  void* out;                        // [T, Hq, D]
  float* lse;                       // [T, Hq] or null
  const int32_t* block_table;       // [B, max_pages]
  const int32_t* seq_lens;          // [B]
  const int32_t* cu_tokens;         // [B + 1] or null
  int* err;
  float* part_o;                    // partial results, each the softmax over its own keys
  float* part_lse;
  int* prefix;                      // few-token kernel: [B + 1] first steps of the sequences
  long long q_token, q_head;        // strides of q, elements
  int B, T, Hq, Hkv, G, D;
  int num_pages, page_size, max_pages;
  int max_tokens, max_len;          // bounds on a sequence's new tokens and length
  int window;                       // < 0: none
  int nsplit;                       // parts of a sequence's keys
  float scale, softcap;
};

// The few-token kernel (bf16, new tokens of a sequence x heads of a group <= kTokenRows):
// how its warps are laid out, from sizes only.
constexpr int kTokenRows = 32;
struct TokenSplit {
  int cluster;                      // blocks that share a unit; 0: runs of equal length instead
  int warps, blocks;                // warps of a block, blocks
  int row_pad;                      // rows of a partial result
  bool ok;                          // the steps can be counted in 31 bits
  size_t bytes;                     // workspace
};
TokenSplit token_split(int B, int Hkv, int D, int rows, long long reach);
cudaError_t launch_cache_token(CacheAttendParams p, const TokenSplit& t, void* workspace, cudaStream_t s);

// First and last block-table column that kernel looks up for each sequence (-1, -1: none),
// computed on the host; p's index arrays are host memory.
void token_columns(const CacheAttendParams& p, int32_t* columns);

// The many-token kernel (bf16): how its work is laid out, from sizes only.
struct ChunkSplit {
  int runs;                         // blocks, each with an equal run of key tiles
  int tile_tokens;                  // tokens of a query tile: 128 rows / heads of a group
  int unit_tokens;                  // tokens of a unit: one query tile's or two's
  int short_unit;                   // units of up to so many key tiles are not cut
  bool direct;                      // a block a unit, no list of work
  bool one;                         // units of one query tile, two blocks an SM
  int box;                          // keys of one load: they lie in one page
  int max_entries;                  // units of all sequences, for one KV head
  bool split;                       // units long enough to be parted between blocks
  size_t bytes;                     // workspace
};
ChunkSplit chunk_split(int B, int T, int Hkv, int G, int D, int page_size, int max_tokens, int max_len, int window);
cudaError_t launch_cache_chunk(const CacheAttendParams& p, const ChunkSplit& t, void* workspace, cudaStream_t s);

}  // namespace swa
