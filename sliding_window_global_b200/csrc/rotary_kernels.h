// rotary_kernels.h -- parameter blocks and launchers of the rotation / head-norm
// kernels (rotary.cu), shared with the cache entry points.  Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/swa.h"
#include "rotary_math.cuh"

namespace swa {

// One kind of head rows (queries, keys, or values that are only copied).
struct HeadRows {
  const void* src;
  void* dst;
  const void* weight;
  long long sb, sh, st;              // source strides over (batch, head, token), elements
  long long db, dh, dt;              // destination strides (unused for cache pages)
  int heads;
};

struct RotaryParams {
  RotaryMath m;
  HeadRows rows[3];                  // q, k, v
  int segs[3];                       // blocks along the heads of each kind
  int heads_per_seg;
  int tokens;                        // rows of one head over all batches
  int n;                             // tokens of a batch (dense calls)
  const int32_t* positions;          // [tokens] or null: start + index in the batch
  int start;
  // cache calls: where a packed token lies
  int batch, max_pages, num_pages, page_size, num_kv_heads;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;
  int* err;
};

struct RotaryBackwardParams {
  RotaryMath m;
  HeadRows grad[2];                  // dq_out -> dq, dk_out -> dk; weight: the norm's
  const void* x[2];                  // the forward's q and k (norm only)
  long long xb[2], xh[2], xt[2];
  int segs[2];
  int blocks[2];                     // blocks that work on q, on k
  int heads_per_seg;
  int tokens, n;
  const int32_t* positions;
  int start;
  float* partial;                    // [blocks[0] + blocks[1], D] sums of the weights' gradients, or null
  float* dweight[2];                 // [D] or null
};

// Check a rotation and a head norm for heads of D elements and fill in *m.
swa_status make_rotary_math(const swa_rotation& r, const swa_head_norm& n, int D, RotaryMath* m);

// Heads per block, `longest` at most, so that a call of few tokens still spreads over the
// GPU, and the resulting blocks along each kind's heads.
int split_heads(long long token_tiles, const int* heads, int kinds, int longest, int* segs);

// Tokens of one block.
int rotary_tile_tokens(int D);

}  // namespace swa
