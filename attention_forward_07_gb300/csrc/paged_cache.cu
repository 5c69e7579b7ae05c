// paged_cache.cu -- the bookkeeping of a paged key/value cache: block tables and slot maps
// from request lengths, and the write of new key / value rows into their slots.

#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "attn.h"
#include "host.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------ tables
// With held_b = ceil(ctx_b / P), want_b = ceil((ctx_b + new_b) / P), need_b = want_b - held_b and
// N_b, C_b the sums of need and new over the requests before b, the n-th page handed out is
// free[count - 1 - n], request b's page held_b + i is the (N_b + i)-th, and new row t of request
// b is at position ctx_b + t - C_b.
//
// One launch and nothing kept between calls: every CTA sums all lengths by itself (a block-wide scan
// of two counters, kept in shared memory), then the threads of all CTAs share out the pages and
// the rows (four neighbours to a thread where there are more rows than threads) and find their request
// by bisection.  A slot on a page added in this call comes
// straight from the free list, so no CTA waits for another's table entries.  The CTAs are one
// cluster, and its barrier orders the reads of free_count before its one write, which may be in
// place.  What bounds it is latency: the chain lengths -> scan -> bisection -> free list -> slot.
// Measured: 64 requests that grow by a token 3.4 us; 509 requests, 12 prompts of up to 8000 tokens among
// them (0.45 MB to read and write, 0.07 us of bandwidth) 6.8 us.
constexpr int TABLES_THREADS = 1024;
constexpr int TABLES_MAX_B = 16384;

struct TablesParams {
  attn_paged_tables_params_t a;
  unsigned int* status;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ceil(n / P) for every n >= 0 that 31 bits hold (n + P - 1 may not fit).
__device__ __forceinline__ int pages_of(int n, int P) {
  const int q = n / P;
  return q + (q * P != n);
}

// Last request b with pre[b] <= x (pre[0] = 0, non-decreasing, x < pre[B]): the one that holds x.
__device__ __forceinline__ int holder(const int* pre, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(TABLES_THREADS) paged_tables_kernel(const __grid_constant__ TablesParams p) {
  const attn_paged_tables_params_t& a = p.a;
  extern __shared__ int pre[];       // rows_pre[B + 1], need_pre[B + 1], ctx[B]
  __shared__ int2 warp_sum[32];
  const int B = a.B, P = a.page_size;
  int* rows_pre = pre;
  int* need_pre = pre + B + 1;
  int* ctx_s = pre + 2 * (B + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();
  grid_dependency_wait();
  const int count_in = *a.free_count, count = min(max(count_in, 0), a.max_free);

  // block-wide exclusive scan of (new, need), `per` neighbouring requests to a thread
  const int per = (B + TABLES_THREADS - 1) / TABLES_THREADS;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  int2 sum = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    const int ctx = max(a.ctx_lens[b], 0), add = max(a.new_lens[b], 0);
    ctx_s[b] = ctx;
    rows_pre[b] = sum.x;
    need_pre[b] = sum.y;
    sum.x += add;
    sum.y += pages_of(ctx + add, P) - pages_of(ctx, P);
    if (blockIdx.x == 0) a.seqlens_k[b] = ctx + add;
  }
  int2 incl = sum;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, s), y = __shfl_up_sync(0xffffffffu, incl.y, s);
    if (lane >= s) incl.x += x, incl.y += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int2 w = warp_sum[lane];
    const int2 own = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, w.x, s), y = __shfl_up_sync(0xffffffffu, w.y, s);
      if (lane >= s) w.x += x, w.y += y;
    }
    warp_sum[lane] = make_int2(w.x - own.x, w.y - own.y);
    if (lane == 31) rows_pre[B] = w.x, need_pre[B] = w.y;
  }
  __syncthreads();
  const int2 before = make_int2(warp_sum[warp].x + incl.x - sum.x, warp_sum[warp].y + incl.y - sum.y);
  for (int b = b0; b < b1; ++b) rows_pre[b] += before.x, need_pre[b] += before.y;
  __syncthreads();
  cluster_arrive();  // free_count has been read (the wait stands before its write)
  const int total = rows_pre[B], need = need_pre[B];

  bool bad = count_in != count || need > count || total > a.max_rows;
  const auto free_page = [&](int n) {
    const int id = (unsigned)n < (unsigned)count ? a.free_pages[count - 1 - n] : -1;
    return id >= 0 && id < a.num_pages ? id : -1;
  };
  const int nthr = gridDim.x * TABLES_THREADS, gid = blockIdx.x * TABLES_THREADS + tid;
  if (blockIdx.x == 0)
    for (int b = tid; b <= B; b += TABLES_THREADS) a.cu_seqlens_q[b] = rows_pre[b];
  for (int n = nthr - 1 - gid; n < need; n += nthr) {  // (from the far end: the near threads have rows)
    const int b = holder(need_pre, B, n);
    const int i = pages_of(ctx_s[b], P) + (n - need_pre[b]);
    const int id = free_page(n);
    const bool fits = (unsigned)i < (unsigned)a.table_width;
    if (fits) a.block_table[(long long)b * a.table_stride + i] = id;
    bad |= id < 0 || !fits;
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  const int each = a.max_rows > nthr ? 4 : 1;
  for (int t0 = each * gid; t0 < a.max_rows; t0 += each * nthr) {
    int slot[4] = {-1, -1, -1, -1}, at[4] = {-1, -1, -1, -1};
    int b = -1, page = -1, id = -1;  // request, page (of the request) and its id, of the row before
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + k;
      if (k >= each || t >= min(total, a.max_rows)) break;
      if (b < 0) b = holder(rows_pre, B, t);
      while (t >= rows_pre[b + 1]) ++b, page = -1;
      const int pos = ctx_s[b] + (t - rows_pre[b]), i = pos / P;
      if (i != page) {
        page = i;
        id = -1;
        if ((unsigned)i < (unsigned)a.table_width) {
          const int held = pages_of(ctx_s[b], P);
          id = i < held ? a.block_table[(long long)b * a.table_stride + i] : free_page(need_pre[b] + i - held);
          if (id >= a.num_pages) id = -1;
        }
      }
      at[k] = pos;
      if (id >= 0) slot[k] = id * P + (pos - i * P);
      else bad = true;
    }
    if (each == 4 && wide && t0 + 4 <= a.max_rows) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(at[0], at[1], at[2], at[3]);
    } else {
      for (int k = 0; k < each && t0 + k < a.max_rows; ++k) {
        a.slots[t0 + k] = slot[k];
        if (a.positions) a.positions[t0 + k] = at[k];
      }
    }
  }
  if (bad) atomicOr(p.status, STATUS_PAGE);
  __syncwarp();
  cluster_wait();
  if (gid == 0) *a.free_count_out = max(count - need, 0);
}

// ------------------------------------------------------------------ append
// cache[slot / P][h][slot % P][:] = new[h][t][:].  One warp takes a row t, reads its slot once
// (the division by P is the row's, not each chunk's) and moves the row's 2 * Hkv * d / 8 chunks of 16
// bytes of K and V, up to eight in flight to a lane.  Memory-bound: every byte is read and written once.
// Measured: 16.9 thousand rows of 8 heads, d = 128: 23.8 us, 5.81 TB/s (0.86 of measured copy bandwidth);
// 64 rows: 2.8 us, a launch's time.  All is read past L1, which nothing here uses twice: with plain loads the
// wait for the kernel ahead empties L1 first, and 64 rows take 3.4 us.
constexpr int APPEND_WARPS = 4;

struct AppendParams {
  attn_paged_append_params_t a;
  unsigned int* status;
};

template <int D>
__global__ void __launch_bounds__(32 * APPEND_WARPS) paged_append_kernel(const __grid_constant__ AppendParams p) {
  const attn_paged_append_params_t& a = p.a;
  constexpr int CPR = D / 8, UNROLL = 8;  // 16-byte chunks of a row
  const int lane = threadIdx.x & 31;
  const int nwarps = gridDim.x * APPEND_WARPS;
  const int per_side = a.Hkv * CPR;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int t = blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5); t < a.rows; t += nwarps) {
    const int slot = load_cg(a.slots + t);
    const int page = slot / a.page_size;
    if (slot < 0) continue;
    if (page >= a.num_pages) {
      if (lane == 0) atomicOr(p.status, STATUS_PAGE);
      continue;
    }
    const long long dst0 = (long long)page * a.cache_page_stride + (long long)(slot - page * a.page_size) * a.cache_row_stride;
    for (int c0 = lane; c0 < 2 * per_side; c0 += 32 * UNROLL) {
      uint4 x[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int c = c0 + 32 * u;
        if (c < 2 * per_side) {
          const bool v = c >= per_side;
          const int e = v ? c - per_side : c;
          const uint16_t* src = static_cast<const uint16_t*>(v ? a.v_new : a.k_new);
          x[u] = load_cg_x4(src + (long long)(e / CPR) * (v ? a.v_head_stride : a.k_head_stride) +
                            (long long)t * (v ? a.v_row_stride : a.k_row_stride) + (e % CPR) * 8);
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int c = c0 + 32 * u;
        if (c < 2 * per_side) {
          const bool v = c >= per_side;
          const int e = v ? c - per_side : c;
          uint16_t* dst = static_cast<uint16_t*>(v ? a.v_cache : a.k_cache);
          *reinterpret_cast<uint4*>(dst + dst0 + (long long)(e / CPR) * a.cache_head_stride + (e % CPR) * 8) = x[u];
        }
      }
    }
  }
}

size_t tables_smem(int B) { return (3 * (size_t)B + 2) * sizeof(int); }

// CTAs of a cluster of paged_tables_kernel at most: 16 where the device has that many SMs side by side for it
// (509 requests, 52 thousand rows: 7.5 us against 9.5 with the portable 8, a step's worth of rows less to a thread).  Asked once per device.
int widest_cluster(int dev, int& ctas) {
  static std::atomic<int> known[64];
  if ((ctas = known[dev].load()) != 0) return ATTN_OK;
  const size_t smem = tables_smem(TABLES_MAX_B);
  if (cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(TABLES_THREADS);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  ctas = 8;
  if (cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, paged_tables_kernel, &cfg) == cudaSuccess && clusters > 0)
    ctas = 16;
  else
    cudaGetLastError();  // (the answer was no)
  known[dev].store(ctas);
  return ATTN_OK;
}

bool misaligned(const void* ptr, unsigned int to) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }

}  // namespace
}  // namespace attn

extern "C" {

int attn_paged_tables(const attn_paged_tables_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_paged_tables_params_t& a = *params;
    // (no page list where it holds no page, no slot map where it holds no row)
    if (!a.ctx_lens || !a.new_lens || !a.block_table || (!a.free_pages && a.max_free != 0) || !a.free_count || !a.free_count_out ||
        !a.cu_seqlens_q || !a.seqlens_k || (!a.slots && (a.max_rows != 0 || a.positions)))
      return ATTN_ERR_INVALID;
    for (const void* ptr : {(const void*)a.ctx_lens, (const void*)a.new_lens, (const void*)a.block_table, (const void*)a.free_pages,
                            (const void*)a.free_count, (const void*)a.free_count_out, (const void*)a.cu_seqlens_q,
                            (const void*)a.seqlens_k, (const void*)a.slots, (const void*)a.positions})
      if (misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    if (a.B < 1 || a.B > TABLES_MAX_B || a.table_width < 1 || a.table_stride < a.table_width || a.max_free < 0 ||
        a.max_rows < (a.slots ? 1 : 0) || a.max_rows > (1 << 30) ||
        a.page_size < 16 || a.page_size % 16 != 0 || a.num_pages < 1 || (long long)a.num_pages * a.page_size > INT_MAX)
      return ATTN_ERR_INVALID;
    int sms = 0, dev = 0;
    int rc = host_device(sms, dev);
    if (rc != ATTN_OK) return rc;
    TablesParams p{a, nullptr};
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    int widest = 0;
    if ((rc = widest_cluster(dev, widest)) != ATTN_OK) return rc;
    const size_t smem = tables_smem(a.B);
    // a CTA for every four rows of its threads, up to the widest cluster
    int ctas = 1;
    while (ctas < widest && (long long)ctas * 4 * TABLES_THREADS < a.max_rows) ctas *= 2;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(a.stream);
    return launch_dependent(paged_tables_kernel, dim3(ctas), TABLES_THREADS, smem, st, p, ctas);
  });
}

int attn_paged_append(const attn_paged_append_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_paged_append_params_t& a = *params;
    if (!a.k_new || !a.v_new || !a.k_cache || !a.v_cache || !a.slots) return ATTN_ERR_INVALID;
    for (const void* ptr : {a.k_new, a.v_new, (const void*)a.k_cache, (const void*)a.v_cache})
      if (misaligned(ptr, 16)) return ATTN_ERR_INVALID;
    if (misaligned(a.slots, 4)) return ATTN_ERR_INVALID;
    if (a.d != 64 && a.d != 128) return ATTN_ERR_UNSUPPORTED;
    if (a.dtype != ATTN_F16 && a.dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
    if (a.rows < 1 || a.rows > (1 << 30) || a.Hkv < 1 || a.Hkv > (1 << 16) || a.num_pages < 1 || a.page_size < 16 || a.page_size % 16 != 0 ||
        (long long)a.num_pages * a.page_size > INT_MAX)
      return ATTN_ERR_INVALID;
    for (long long s : {a.k_row_stride, a.k_head_stride, a.v_row_stride, a.v_head_stride, a.cache_page_stride, a.cache_head_stride,
                        a.cache_row_stride})
      if (s < 0 || s % 8 != 0 || s > MAX_STRIDE) return ATTN_ERR_INVALID;
    if (a.cache_row_stride == 0 || (a.num_pages > 1 && a.cache_page_stride == 0) || (a.Hkv > 1 && a.cache_head_stride == 0))
      return ATTN_ERR_INVALID;
    int sms = 0, dev = 0;
    int rc = host_device(sms, dev);
    if (rc != ATTN_OK) return rc;
    AppendParams p{a, nullptr};
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    const int grid = (a.rows + APPEND_WARPS - 1) / APPEND_WARPS;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(a.stream);
    return launch_dependent(a.d == 64 ? paged_append_kernel<64> : paged_append_kernel<128>, dim3(grid), 32 * APPEND_WARPS, 0, st, p);
  });
}

}  // extern "C"
