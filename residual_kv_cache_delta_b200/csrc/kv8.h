// Host-side arguments, launch choices and workspace layout of the 8-bit paged cache (deltakv_kv8_*) and of
// deltakv_merge_attention.  The workspace query and the attention call both derive the layout from here.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/deltakv.h"
#include "layout.h"

namespace dkv {

constexpr int kKv8MaxSplits = 128;      // key ranges one query row may be cut into
constexpr int kKv8CellKeys = 16;        // keys of one unit of split work: every block size is a multiple
constexpr int kKv8MinSplitCells = 16;   // a split covers at least 256 keys (or all there are)

struct Kv8AppendArgs {
  const dkv_kv8_shape* shape;
  const dkv_kv8_cache* cache;
  const dkv_kv8_rope* rope;  // nullptr: no rotation
  const void* k_new;
  const void* v_new;
  int64_t k_stride, v_stride;
  const int* cu_new;
  const int* start_pos;
  const int* block_tables;
  int max_blocks, num_seqs;
  int64_t total_new;
  int max_new;
  const void* q;
  int64_t q_stride;
  void* q_out;
};

struct Kv8AttnArgs {
  const dkv_kv8_shape* shape;
  const dkv_kv8_cache* cache;
  const dkv_kv8_score* score;  // nullptr: plain causal attention
  const void* q;
  int64_t q_stride;
  const int* cu_q;
  const int* context_lens;
  const int* block_tables;
  int max_blocks, num_seqs;
  int64_t total_q;
  int max_q, max_ctx;
  float softmax_scale;
  void* out;
  float* lse;
};

// Workspace of an attention call: per split and query row the running maximum and sum (log2 domain) and the
// unnormalised output row, all fp32.  One split: nothing is staged.
struct Kv8AttnWs {
  size_t ml = 0, o = 0, total = 0;
};

inline Kv8AttnWs kv8_attn_layout(const dkv_kv8_shape& sh, int64_t staged_rows) {
  Kv8AttnWs w;
  if (staged_rows > 0) {
    const size_t rows = static_cast<size_t>(staged_rows);
    w.o = align_up(rows * 8, kWsAlign);
    w.total = align_up(w.o + rows * sh.head_dim * 4, kWsAlign);
  }
  return w;
}

dkv_status launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st);
int kv8_attn_splits(const dkv_kv8_shape& sh, int num_seqs, int max_q, int span);
int64_t kv8_attn_staged(const dkv_kv8_shape& sh, int64_t total_q, int max_q, int max_ctx);
dkv_status launch_kv8_attention(const Kv8AttnArgs& a, int nsplit, const Kv8AttnWs& w, void* workspace, cudaStream_t st);
dkv_status launch_merge(int dtype, int64_t rows, int head_dim, int n, const void* const* outs,
                        const float* const* lses, void* out, float* lse, cudaStream_t st);

}  // namespace dkv
