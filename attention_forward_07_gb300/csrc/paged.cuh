// paged.cuh -- what the two paths of attn_fwd_paged share.  A request whose K/V heads have at most
// ROWS_MAX packed rows (query tokens times group size) takes the memory-bound path of
// paged_attn.cu, a longer one the tcgen05 path of paged_tile.cu; each path's kernels pass over the
// other's requests, so the lengths need not be known on the host.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn.h"
#include "ptx.cuh"

namespace attn {

constexpr int ROWS_MAX = 16;

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
};

// Query rows, keys and first query row of request b, whatever the arrays hold.
__device__ __forceinline__ void request_span(const PagedParams& p, int b, int& row0, int& sq, int& sk) {
  row0 = min(max(__ldg(p.cu_q + b), 0), p.total_q);
  sq = min(min(max(__ldg(p.cu_q + b + 1), row0), p.total_q) - row0, p.max_q);
  sk = (int)min((long long)max(__ldg(p.lens_k + b), 0), (long long)p.width * p.page_size);
}

// Keys that query row i (of sq, against sk keys) keeps: [lo, hi).
__device__ __forceinline__ int row_lo(const PagedParams& p, int i, int off) {
  return p.wl < 0 ? 0 : (int)max(0ll, (long long)i + off - p.wl);
}
__device__ __forceinline__ int row_hi(const PagedParams& p, int i, int off, int sk) {
  return p.er < 0 ? sk : (int)min((long long)sk, (long long)i + off + p.er + 1);
}

// Scratch of the tcgen05 path behind the other path's, and its launches (plan, attention, join).
size_t tile_workspace(const attn_fwd_paged_params_t& a, int sms);
int tile_launch(const PagedParams& p, const attn_fwd_paged_params_t& a, void* workspace, int sms, int dev, cudaStream_t st);

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace attn
