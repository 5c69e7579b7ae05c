// paged.cuh -- what the two paths of attn_fwd_paged share.  A request whose K/V heads have at most
// ROWS_MAX packed rows (query tokens times group size) takes the memory-bound path of
// paged_attn.cu, a longer one the tcgen05 path of paged_tile.cu; each path's kernels pass over the
// other's requests, so the lengths need not be known on the host.  Two rules move the border:
//  * where max_seqlen_q allows no request more than ROWS_ONLY rows, all take the memory-bound path, with
//    32 rows to an item.  24 requests of 32 rows against 4000 keys (d = 128 / 64): 53 / 21 us, by the
//    tcgen05 path 55 / 31; above 32 rows the order turns (48 rows: 78 us against 57 at d = 128);
//  * few-row requests beside chunks join the chunks' units while they have few key tiles altogether
//    (FOLD_TILES in paged_attn.cu);
//  * where no request may have more rows than a Q tile, and the call gives them room for more than ROWS_MAX on the
//    average (total_q over B; the lengths themselves are on the device), all take the tcgen05 path, which
//    then needs neither the other path's kernel nor its plan (NO_PLAN_B).  32 query heads on 4, room for 16
//    tokens to a request, 4000 keys: with 16 tokens 64 requests take 119 / 105 us (d = 128 / 64), with a plan
//    124 / 109, 16 requests 44 / 37 and 51 / 40.  Where the room is not used it costs at d = 64: with one
//    token to a request 64 take 109 / 102, with a plan 115 / 51.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn.h"
#include "host.h"
#include "ptx.cuh"

namespace attn {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr long long MAX_STRIDE = 1ll << 38;  // elements: no memory holds two entries that far apart, and tensor maps end there
// attn_fwd_paged_tree without a plan: units that its requests, and that one of them, may have at most (what the lanes of a CTA look at in turn).
// 24 trees of 8 - 16 nodes x 4 heads on 4000 keys beside a chunk of 512 / 1900 / 2040 rows (8, 30 and 32 units): 85 / 109 / 113 us at d = 128,
// with a plan 97 / 137 / 139; 73 / 100 / 104 at d = 64, with a plan 85 / 119 / 120.  Beside few rows the order can turn, as above: 60 single tokens on
// 4000 keys and a chunk of 400 rows (32/8 heads) 181 and 182 us at d = 128, but 156 and 104 at d = 64; 30 chains of 4 on 2000 and one of 512: 61 and
// 69, 53 and 47.  Trees alone (60 nodes x 8 heads on 1000 keys, d = 128): 100 units 113 us, with a plan 116; 200 units 211 and 201, 400 units 407 and 379,
// 1000 units 1013 and 932, so from some 150 units on the plan would take 5 - 10 % less; 2000 units (100 nodes on 300 keys, d = 64) 489 and 474.
constexpr int NO_PLAN_UNITS = 2048, NO_PLAN_CHUNK = 32;
constexpr int NO_PLAN_B = 512;  // requests at most whose lengths every CTA looks at (16 to a lane)
constexpr int ROWS_MAX = 16, ROWS_ONLY = 32;
constexpr int TILE_QT = 2, TILE_ROWS = 128, TILE_KEYS = 128;  // Q tiles of a unit, rows of a Q tile, keys of a key tile

// Written by the plan (the joins by the tcgen05 kernel).  Line coordinates count steps over all (unit, head) pairs in order, heads inside: a
// pair is UNIT_COST steps for its start and end, then a step for each key tile.  (Measured with 1 / 2 / 3 / 4:
// checking 3 - 6 tokens of 24 requests 43.1 / 41.0 / 39.0 / 39.6 us, a mixed batch of 13 requests 77.4 /
// 74.3 / 66.7 / 66.0, four prompts of 4k 438 / 438 / 436 / 431.)
constexpr int UNIT_COST = 4;
constexpr int MIN_RUN = 4 + UNIT_COST;  // steps of a run at least
struct TileQueue {
  unsigned int next;    // next queue entry (a CTA starts with that of its own number)
  int whole, runs;      // entries: whole (unit, head) pairs, then runs
  int njoins;             // counted by the tcgen05 kernel
  int units;
  long long line0, line;  // where the runs' line begins, its length
};
struct TileUnit {
  int b, blk;
  int j0, w;      // key tiles j0 .. j0 + w - 1 (one where no key is seen: the unit still writes its rows)
  long long cum;  // steps of the units before
  int row0, sq, sk, pad;
};
struct TileJoin {  // up to JOIN_ROWS packed rows of a cut (unit, head) pair
  int row0, row, rows;  // request's first query row, first packed row, rows
  int h, run, parts;    // pieces in slots 2 run + 1, 2 (run + 1), 2 (run + 2), ...
  int in, pad;          // first row within the slot
};
constexpr int JOIN_ROWS = 16;
constexpr int JOINS_OF_RUN = TILE_ROWS / JOIN_ROWS;  // without a plan (attn_fwd_paged_tree: as many as a unit may have rows)

// Scratch of the tcgen05 path.
struct TileWork {
  TileQueue* queue;
  TileUnit* units;   // [max_units + 1], longest first
  TileJoin* joins;   // [max runs * 256 / JOIN_ROWS]: every cut pair holds a run's beginning
  float* part_o;     // [2 max runs][D / 4][256][4]: unscaled O of a piece (part_at)
  float2* part_ml;   // [2 max runs][256]: its exponent base (exp2 domain) and sum of weights
  int T;             // tokens of a Q tile
  int max_units;     // 0: no request takes this path
  int sms;
  int no_plan;       // not 0: every CTA finds its run by itself (NO_PLAN_B), and lists joins at places of its own, this many in all
};

struct PagedParams {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  float* lse;
  const int *table, *cu_q, *lens_k;
  long long q_row, q_head, o_row, o_head;  // strides in elements
  long long c_page, c_head, c_row;
  int B, Hq, Hkv, g, total_q, max_q, num_pages, page_size, width, table_stride;
  int wl, er;  // band: keys pos - wl .. pos + er (-1: unbounded)
  float scale_log2;
  unsigned int* status;
  uint32_t timeout_us;  // longest barrier wait (microseconds)
  TileWork tile;
  // attn_fwd_paged_tree: masks of the new rows, [total_q][tree_stride] words of which tree_words count, and positions
  const uint32_t* tree;
  const int* pos;
  int tree_words, tree_stride;
};

// Query rows, keys and first query row of request b, whatever the arrays hold.
__device__ __forceinline__ void request_span(const PagedParams& p, int b, int& row0, int& sq, int& sk) {
  row0 = min(max(p.cu_q[b], 0), p.total_q);
  sq = min(min(max(p.cu_q[b + 1], row0), p.total_q) - row0, p.max_q);
  sk = (int)min((long long)max(p.lens_k[b], 0), (long long)p.width * p.page_size);
}

// Keys that query row i (of sq, against sk keys) keeps: [lo, hi).
__device__ __forceinline__ int row_lo(const PagedParams& p, int i, int off) {
  return p.wl < 0 ? 0 : (int)max(0ll, (long long)i + off - p.wl);
}
__device__ __forceinline__ int row_hi(const PagedParams& p, int i, int off, int sk) {
  return p.er < 0 ? sk : (int)min((long long)sk, (long long)i + off + p.er + 1);
}

// A request with a mask among its new rows; a longer one is a chunk (kernels of attn_fwd_paged_tree; others: none).
template <bool TREE>
__device__ __forceinline__ bool has_mask(const PagedParams& p, int sq) { return TREE && sq <= 32 * p.tree_words; }
// First key of the context that a masked request's query row t may see.
__device__ __forceinline__ int masked_lo(const PagedParams& p, int t, int off) {
  return p.wl < 0 ? 0 : (int)max(0ll, (long long)max(p.pos[t], off) - p.wl);
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Tokens and keys of Q tiles [t0, t1) of block blk: false where it has no token.
template <bool TREE>
__device__ __forceinline__ bool tile_keys(const PagedParams& p, int sq, int sk, int blk, int t0, int t1, int& lo, int& hi) {
  const int i0 = (blk * TILE_QT + t0) * p.tile.T, i1 = min((blk * TILE_QT + t1) * p.tile.T, sq) - 1;
  lo = hi = 0;
  if (i0 > i1) return false;
  // (a mask may keep any new row, and its rows' positions begin at the context's end)
  const bool masked = has_mask<TREE>(p, sq);
  const int a = row_lo(p, masked ? 0 : i0, sk - sq), e = masked ? sk : row_hi(p, i1, sk - sq, sk);
  if (e > a) lo = a, hi = e;
  return true;
}

// Where four columns of a row of a slot begin.  A thread of the tcgen05 kernel has a row, so neighbouring rows
// lie side by side (with the columns of a row side by side a full piece took 6 - 11k cycles to write).
template <int D>
__device__ __forceinline__ long long part_at(int slot, int row, int col) {
  return (((long long)slot * (D / 4) + col / 4) * (TILE_QT * TILE_ROWS) + row) * 4;
}

// First step of run i out of n over a line, and the run that holds step x of it.
__host__ __device__ __forceinline__ long long run_begin(long long line, int n, int i) { return line * i / n; }
__device__ __forceinline__ int run_of(long long line, int n, long long x) { return (int)(((x + 1) * n - 1) / line); }

// Parameters of the tcgen05 path's kernel.
struct TileParams : PagedParams {
  CUtensorMap tm_q, tm_k, tm_v;
  int box_rows;   // rows of one K/V box
  int z_page, z_head, z_extent;  // the maps' page-and-head coordinate: page * z_page + h * z_head, below z_extent
  unsigned int g_inverse;  // 65536 / g + 1: row / g = row * g_inverse >> 16 for rows below 128
  unsigned int unit_inverse;  // 2^32 over a unit's tokens, rounded up
  int inject;
};
// Fills them in (ahead of any launch: a tensor map may fail), and launches the kernel.
int tile_prepare(const PagedParams& base, const attn_fwd_paged_params_t& a, TileParams& p);
int tile_launch(const TileParams& p, const attn_fwd_paged_params_t& a, int sms, int dev, cudaStream_t st);

// Launches a kernel (in clusters of `cluster` CTAs) that may start before the one ahead of it on the stream has
// finished; it waits for that one (griddepcontrol.wait) before it touches memory.
template <class P>
int launch_dependent(void (*kern)(P), dim3 grid, unsigned int threads, size_t smem, cudaStream_t st, const P& p, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// What attn_fwd_paged and attn_fwd_paged_tree (tree not NULL) run.
int paged_fwd_impl(const attn_fwd_paged_params_t& a, const attn_fwd_paged_tree_params_t* tree);

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace attn
