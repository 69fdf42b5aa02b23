// Launch of attention over the 8-bit cache: the split plan and the choice of kernel.
#pragma once

#include "kv8_attn_simple.cuh"
#include "kv8_tile.cuh"

namespace dkv {

// Up to so many rows per kv head the streaming kernel is taken (in row tiles of 16), above it the tcgen05 one, whose time
// hardly depends on the rows below its tile.  Microseconds of the first and the second, both from one build, which takes either
// by a switch; 8 kv heads, int8:
//                      16 rows         32 rows         64 rows         80 rows         96 rows         128 rows
//   d 128,  8 x  5000   30.9 and  94.4  49.6 and  95.6  95.2 and  97.8   139 and  98.3   141 and  97.6   188 and  99.3
//           8 x 32768    153 and   534   283 and   536   511 and   538   662 and   539   779 and   541   980 and   542
//           1 x  2000   12.0 and  16.9  12.3 and  17.2  14.5 and  18.4  16.0 and  18.9  16.4 and  19.9  18.1 and  20.5
//           1 x 32768   26.9 and  73.6  40.5 and  73.8  76.1 and  75.1  95.7 and  75.7  99.6 and  76.5   144 and  77.7
//   d  64,  8 x  5000   23.4 and  78.7  35.2 and  78.8  57.1 and  80.9  84.4 and  80.9  90.7 and  80.9   112 and  81.2
//           8 x 32768   91.0 and   452   169 and   452   308 and   453   383 and   453   449 and   453   589 and   454
//           1 x  2000   11.1 and  15.9  11.6 and  16.4  13.5 and  16.7  15.2 and  16.8  15.2 and  17.7  15.9 and  17.8
//           1 x 32768   22.9 and  62.0  30.4 and  62.4  46.7 and  63.3  64.3 and  63.4  65.2 and  63.6  86.2 and  64.0
// e4m3 takes up to 10% less in the first column and 3% in the second.  With one kv head, where neither fills the GPU, the first
// leads further (d 128, 8 x 5000, 64 rows: 20.5 and 25.8; d 64, 80 rows: 19.8 and 23.3).  Capped scores take the second longer
// (8 x 32768: 589 and 896 at 64 rows of d 128, 463 and 802 at 80 of d 64).
template <int D>
constexpr int kStreamMaxRows = D == 64 ? 80 : 64;

// The kernel of a call: how many query rows a CTA (tcgen05: a pair) takes, how many of them an SM holds, and the most CTAs
// that a call with splits may have.  That limit bounds the workspace (most x tile staged rows).  It is 16 rounds of CTAs (12
// of the tcgen05 kernel's, whose CTAs stage 512 rows): by the split plan's model, a call that it keeps from splitting loses a
// tenth at most, at 524288 keys.
struct Kv8Kind {
  bool tiles;
  int tile, per_sm;
  int64_t slots, most;
};

static Kv8Kind kv8_kind(const dkv_kv8_shape& sh, int max_q) {
  const int64_t rows = static_cast<int64_t>(max_q) * (sh.num_q_heads / sh.num_kv_heads);
  Kv8Kind k;
  k.tiles = sh.dtype != DKV_F32 && rows > (sh.head_dim == 64 ? kStreamMaxRows<64> : kStreamMaxRows<128>);
  k.tile = sh.dtype == DKV_F32 ? kSimpleRows : k.tiles ? kTileRows : rows <= 8 ? 8 : 16;
  k.per_sm = sh.dtype == DKV_F32 ? 4 : k.tiles ? 1 : sh.head_dim == 64 ? stream_ctas<64>(k.tile / 8) : stream_ctas<128>(k.tile / 8);
  k.slots = k.tiles ? num_sms() / 2 : num_sms();  // the tcgen05 kernel's CTAs come in pairs
  k.most = (k.tiles ? 12 : 16) * k.slots * k.per_sm;
  return k;
}

// Most key ranges that a row of up to `span` keys is cut into.
static int kv8_most_splits(int span) {
  const int64_t cells = ceil_div64(span, kKv8CellKeys);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kKv8MaxSplits, ceil_div64(cells, kKv8MinSplitCells))));
}

// Key ranges that a row is cut into.  span: most keys that a query token sees.
int kv8_attn_splits(const dkv_kv8_shape& sh, int num_seqs, int max_q, int span) {
  const Kv8Kind k = kv8_kind(sh, max_q);
  const int64_t rows = static_cast<int64_t>(max_q) * (sh.num_q_heads / sh.num_kv_heads);
  const int64_t base = ceil_div64(rows, k.tile) * sh.num_kv_heads * std::max(num_seqs, 1);
  const int64_t cells = ceil_div64(span, kKv8CellKeys);
  const int most = kv8_most_splits(span);
  // Time in cells of one SM: the fullest SM's share of the cells, a start and an end for each of its rounds of CTAs, and
  // with splits the join (tcgen05 kernel: 256 rows of fp32 written and read again per CTA).
  int nsplit = 1;
  double best = 0;
  for (int n = 1; n <= most && (n == 1 || n * base <= k.most); ++n) {
    const int64_t ctas = base * n;
    // (a CTA alone on its SM waits for its own latencies and is hardly faster than two that share one)
    double t = static_cast<double>(std::max<int64_t>(ceil_div64(ctas, k.slots), std::min(k.per_sm, 2))) *
                   (static_cast<double>(cells) / n) +
               24.0 * static_cast<double>(ceil_div64(ctas, k.slots * k.per_sm));
    if (n > 1) t += 20.0 + (k.tiles ? 40.0 * static_cast<double>(ceil_div64(ctas, k.slots)) : 0.0);
    if (n == 1 || t < best) best = t, nsplit = n;
  }
  return nsplit;
}

// Query rows times splits that no call within these bounds exceeds.  The splits of a call go up and down with its batch, so
// this is not the plan's own number but one that grows with every bound: a workspace for a program's largest step serves
// its smaller ones.  (A call stages splits x total_q x H_q rows; they fill at most its CTAs' tiles.)
int64_t kv8_attn_staged(const dkv_kv8_shape& sh, int64_t total_q, int max_q, int max_ctx) {
  const int splits = kv8_most_splits(max_ctx);
  if (splits == 1) return 0;
  const Kv8Kind k = kv8_kind(sh, max_q);
  return std::min<int64_t>(splits * total_q * sh.num_q_heads, k.most * k.tile);
}

// Joins the splits of each row; starts while the attention kernel's last CTAs run.  With more than 8 splits four warps share
// a row: for one sequence of 131072 tokens, 64 rows, the join took 31 us with one warp a row and 8 us with four (both from a
// profiler's launch list, caches cold).  With few splits one warp reads them in few steps, and a CTA of four rows serves.
template <typename T, int D>
static dkv_status launch_combine(const Kv8Attn& p, cudaStream_t st) {
  if (p.nsplit == 1) return DKV_OK;
  const int64_t rows = p.total_q * p.heads * p.group;
  const cudaError_t e =
      p.nsplit > 8 ? launch_programmatic(kv8_combine_kernel<T, D, 4>, dim3(static_cast<unsigned>(rows)), dim3(128), 0, st, p)
                   : launch_programmatic(kv8_combine_kernel<T, D, 1>, dim3(static_cast<unsigned>(ceil_div64(rows, 4))),
                                         dim3(128), 0, st, p);
  return e == cudaSuccess ? DKV_OK : DKV_ERR_CUDA;
}

template <int D, bool E4M3, int NT, bool BIAS>
static dkv_status attn_stream(const Kv8Attn& p, cudaStream_t st) {
  constexpr auto kKernel = kv8_stream_kernel<D, E4M3, NT, BIAS>;
  if (!ensure_max_dynamic_smem<kKernel, true>()) return DKV_ERR_CUDA;
  CUtensorMap map;
  if (!make_map_codes(&map, p.codes, static_cast<uint64_t>(p.num_blocks) * p.heads * 2 * p.block, D)) return DKV_ERR_CUDA;
  const int row_tiles = static_cast<int>(ceil_div64(static_cast<int64_t>(p.max_q) * p.group, 8 * NT));
  const int64_t ctas = static_cast<int64_t>(p.nsplit) * row_tiles * p.heads * p.num_seqs;
  if (ctas > INT32_MAX) return DKV_ERR_UNSUPPORTED;
  kKernel<<<static_cast<unsigned>(ctas), kStreamWarps * 32, stream_smem<D>(NT), st>>>(map, p, row_tiles);
  if (cudaGetLastError() != cudaSuccess) return DKV_ERR_CUDA;
  return launch_combine<__nv_bfloat16, D>(p, st);
}

template <int D, bool E4M3, bool BIAS>
static dkv_status attn_tile(const Kv8Attn& p, cudaStream_t st) {
  constexpr auto kKernel = kv8_tile_kernel<D, E4M3, BIAS>;
  if (!ensure_max_dynamic_smem<kKernel>()) return DKV_ERR_CUDA;
  const int row_tiles = static_cast<int>(ceil_div64(static_cast<int64_t>(p.max_q) * p.group, kTileRows));
  const int64_t ctas = static_cast<int64_t>(p.nsplit) * row_tiles * p.heads * p.num_seqs;  // pairs
  if (ctas > INT32_MAX / 2) return DKV_ERR_UNSUPPORTED;
  kKernel<<<static_cast<unsigned>(2 * ctas), kTileThreads, TileSmem<D>::bytes, st>>>(p, row_tiles);
  if (cudaGetLastError() != cudaSuccess) return DKV_ERR_CUDA;
  return launch_combine<__nv_bfloat16, D>(p, st);
}

template <int D, bool E4M3, bool BIAS>
static dkv_status attn_rows(const Kv8Attn& p, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group;
  if (rows <= 8) return attn_stream<D, E4M3, 1, BIAS>(p, st);
  if (rows <= kStreamMaxRows<D>) return attn_stream<D, E4M3, 2, BIAS>(p, st);
  return attn_tile<D, E4M3, BIAS>(p, st);
}

template <int D, bool E4M3>
static dkv_status attn_bf16(const Kv8Attn& p, cudaStream_t st) {
  return p.softcap > 0.f || p.slopes ? attn_rows<D, E4M3, true>(p, st) : attn_rows<D, E4M3, false>(p, st);
}

template <int D, bool E4M3>
static dkv_status attn_simple(const Kv8Attn& p, cudaStream_t st) {
  const int row_tiles = static_cast<int>(ceil_div64(static_cast<int64_t>(p.max_q) * p.group, kSimpleRows));
  const int64_t ctas = static_cast<int64_t>(p.nsplit) * row_tiles * p.heads * p.num_seqs;
  if (ctas > INT32_MAX) return DKV_ERR_UNSUPPORTED;
  kv8_attn_simple_kernel<D, E4M3><<<static_cast<unsigned>(ctas), 128, 0, st>>>(p, row_tiles);
  if (cudaGetLastError() != cudaSuccess) return DKV_ERR_CUDA;
  return launch_combine<float, D>(p, st);
}

dkv_status launch_kv8_attention(const Kv8AttnArgs& a, int nsplit, const Kv8AttnWs& w, void* workspace, cudaStream_t st) {
  const dkv_kv8_shape& sh = *a.shape;
  Kv8Attn p = {};
  p.codes = static_cast<const uint8_t*>(a.cache->codes);
  p.scales = a.cache->scales;
  p.num_blocks = a.cache->num_blocks;
  p.heads = sh.num_kv_heads, p.group = sh.num_q_heads / sh.num_kv_heads, p.block = sh.block_tokens;
  p.q = a.q, p.q_stride = a.q_stride, p.cu_q = a.cu_q, p.context_lens = a.context_lens;
  p.block_tables = a.block_tables, p.max_blocks = a.max_blocks, p.num_seqs = a.num_seqs;
  p.total_q = a.total_q, p.max_q = a.max_q, p.max_ctx = a.max_ctx;
  p.scale = a.softmax_scale > 0.f ? a.softmax_scale : 1.0f / sqrtf(static_cast<float>(sh.head_dim));
  if (a.score) {
    // a window of at least the longest context hides nothing
    p.softcap = a.score->softcap, p.window = a.score->window < a.max_ctx ? a.score->window : 0, p.slopes = a.score->alibi_slopes;
    p.prefix_lens = a.score->prefix_lens, p.first_key = a.score->first_key;
  }
  p.out = a.out, p.lse = a.lse, p.nsplit = nsplit;
  if (p.window > 0)  // fewer keys to share out
    p.nsplit = std::min(p.nsplit, kv8_attn_splits(sh, a.num_seqs, a.max_q, static_cast<int>(std::min<int64_t>(
                                               a.max_ctx, int64_t{a.max_q} + p.window))));
  p.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + w.ml);
  p.o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.o);
  const bool e4 = sh.code == DKV_KV8_E4M3, d64 = sh.head_dim == 64;
  if (sh.dtype == DKV_F32) {
    if (d64) return e4 ? attn_simple<64, true>(p, st) : attn_simple<64, false>(p, st);
    return e4 ? attn_simple<128, true>(p, st) : attn_simple<128, false>(p, st);
  }
  if (d64) return e4 ? attn_bf16<64, true>(p, st) : attn_bf16<64, false>(p, st);
  return e4 ? attn_bf16<128, true>(p, st) : attn_bf16<128, false>(p, st);
}

}  // namespace dkv
