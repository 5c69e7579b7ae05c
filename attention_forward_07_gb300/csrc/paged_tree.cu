// paged_tree.cu -- drafted trees over a paged cache: masks and positions of their nodes, the walk along those that
// the model confirms, and the accepted rows' move to where a chain would have them.

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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Rows [row0, row0 + n) of request b, whatever the offsets hold.
__device__ __forceinline__ void rows_of(const int* cu, int b, int rows, int& row0, int& n) {
  const int x = load_cg(cu + b), y = load_cg(cu + b + 1);
  row0 = min(max(x, 0), rows);
  n = min(max(y, row0), rows) - row0;
}

// ------------------------------------------------------------------ masks and positions
// mask(i) = bits of i and of the nodes above it, depth(i) = their number less one, position = context + depth.  One CTA
// takes a request, its first warp the nodes, 32 at a time in order: within the 32 every node's mask joins that of the node
// it has got to and goes on from there, twice as far each time (shuffles); the topmost one's parent lies in an earlier 32, whose masks and
// depths are in shared memory.  So a chain takes no longer than a bush.  As the nodes above have descending numbers, those within a
// window are a mask's highest bits.  What bounds it is latency: offsets -> parents -> shuffles.  Measured: one tree of 26 nodes
// 1.3 us, 301 of up to 64 nodes with chunks of up to 2000 tokens among them 2.3, 46 chains of 256 nodes 11 (a thread walking up from every
// node: 1.7, 3.7 and 28).
constexpr int TREE_THREADS = 128, TREE_WORDS = 32, TREE_NODES = 32 * TREE_WORDS;

struct TreeParams {
  attn_paged_tree_params_t a;
  unsigned int* status;
};
size_t tree_smem(int words) { return (size_t)32 * words * (words + 1) * sizeof(uint32_t); }  // masks, depths

__global__ void __launch_bounds__(TREE_THREADS) paged_tree_kernel(const __grid_constant__ TreeParams p) {
  const attn_paged_tree_params_t& a = p.a;
  extern __shared__ uint32_t masks[];  // [nodes][mask_words]
  int* depths = reinterpret_cast<int*>(masks + 32 * a.mask_words * a.mask_words);
  const int lane = threadIdx.x, b = blockIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  int row0, n;
  const int keys = max(load_cg(a.seqlens_k + b), 0);
  rows_of(a.cu_seqlens_q, b, a.rows, row0, n);
  const int ctx = max(keys - n, 0);
  if (n > 32 * a.mask_words) {  // a chunk: a chain without a mask
    for (int i = threadIdx.x; i < n; i += TREE_THREADS) a.positions[row0 + i] = ctx + i;
    return;
  }
  if (threadIdx.x >= 32) return;
  bool bad = false;
  int next = lane < n ? load_cg(a.parents + row0 + lane) : -1;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    int up = next;
    if (i + 32 < n) next = load_cg(a.parents + row0 + i + 32);
    if (i >= n) up = -1;
    if (up >= i || up < -1) {  // (only a node ahead of it can be above it)
      up = -1;
      bad = true;
    }
    uint32_t bits = 1u << lane;
    int to = up - base;  // the lane that the node's mask ends ahead of; below 0: no more of these 32
    while (__any_sync(0xffffffffu, to >= 0)) {
      const uint32_t more = __shfl_sync(0xffffffffu, bits, max(to, 0));
      const int further = __shfl_sync(0xffffffffu, to, max(to, 0));
      if (to >= 0) {
        bits |= more;
        to = further;
      }
    }
    const int above = __shfl_sync(0xffffffffu, up, __ffs(bits) - 1);  // the topmost one's parent, ahead of these 32 (or none)
    if (i < n) {
      const int depth = __popc(bits) - 1 + (above >= 0 ? depths[above] + 1 : 0);
      uint32_t* out = a.tree_mask + (long long)(row0 + i) * a.mask_stride;
      int left = a.window_left < 0 ? INT_MAX : min(a.window_left, INT_MAX - 1) + 1;  // nodes that the mask may hold
      for (int w = a.mask_words - 1; w >= 0; --w) {
        uint32_t x = w == base >> 5 ? bits : above >= 0 && w < base >> 5 ? masks[above * a.mask_words + w] : 0u;
        for (int over = __popc(x) - left; over > 0; --over) x &= x - 1u;
        left -= __popc(x);
        masks[i * a.mask_words + w] = x;
        out[w] = x;
      }
      depths[i] = depth;
      a.positions[row0 + i] = (int)min((long long)ctx + depth, (long long)INT_MAX);
    }
    __syncwarp();
  }
  if (bad) atomicOr(p.status, STATUS_PAGE);
}

// ------------------------------------------------------------------ acceptance
// A walk: from the last confirmed node to its first child (the lowest number) whose token is the model's choice
// behind the node, and on from there.  A warp takes a request; the nodes from the last confirmed one on lie in its
// registers, ACCEPT_HELD of them, so a step is a few ballots; further ones are read again at each step.  Pages that hold no token any
// longer are counted, every warp tells every CTA of the cluster its requests' counts, and behind the cluster's barrier
// each CTA sums them up by itself and writes its requests' pages to the free list in the requests' order.
// What bounds it is latency: offsets -> nodes -> walk -> table entries -> barrier -> sum -> list.  Measured: 8 trees of 26 nodes 5.1 us, 301 of
// up to 64 nodes 6.6 (with 8 CTAs, two requests to some warps, and the table read again behind the barrier 10.1).
constexpr int ACCEPT_THREADS = 1024, ACCEPT_WARPS = ACCEPT_THREADS / 32, ACCEPT_MAX_B = 16384;
constexpr int ACCEPT_BLOCKS = 4, ACCEPT_HELD = 32 * ACCEPT_BLOCKS;

struct AcceptParams {
  attn_paged_accept_params_t a;
  unsigned int* status;
};

__device__ __forceinline__ void store_remote(const int* local, int cta, int x) {  // the same place of another CTA's shared memory
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(cta));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ int ceil_div(int n, int m) {
  const int q = n / m;
  return q + (q * m != n);
}

__global__ void __launch_bounds__(ACCEPT_THREADS) paged_accept_kernel(const __grid_constant__ AcceptParams p) {
  const attn_paged_accept_params_t& a = p.a;
  extern __shared__ int counts[];  // pages that go back, of every request; [B, 2 B): tokens that this CTA's requests keep
  __shared__ int warp_sum[ACCEPT_WARPS];
  int* after_s = counts + a.B;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = gridDim.x * ACCEPT_WARPS, gwarp = warp * gridDim.x + blockIdx.x;  // (neighbours in different CTAs)
  cluster_arrive();
  grid_launch_dependents();
  grid_dependency_wait();
  const bool pages_back = a.free_pages != nullptr;
  const int count_in = pages_back ? load_cg(a.free_count) : 0, have = min(max(count_in, 0), a.max_free);
  bool bad = count_in != have;

  const auto page_at = [&](int b, int idx) {  // (may be out of range)
    return (unsigned)idx < (unsigned)a.table_width ? load_cg(a.block_table + (long long)b * a.table_stride + idx) : -1;
  };
  // a request's tokens from now on, its entries whose pages go back and the first 32 of these pages: where a warp has no second
  // request, it keeps them over the cluster's barrier
  const bool alone = a.B <= nwarps;
  int after = 0, back0 = 0, back1 = 0, id = -1;
  for (int b = gwarp; b < a.B; b += nwarps) {
    int row0, n;
    id = -1;
    const int keys = max(load_cg(a.seqlens_k + b), 0);
    const int asked = a.confirmed ? load_cg(a.confirmed + b) : 1;
    rows_of(a.cu_seqlens_q, b, a.rows, row0, n);
    const int ctx = keys - n;  // (below 0 where the lengths contradict each other: rows ahead of position 0 have no slot)
    const int sure = min(max(asked, 1), n), base = sure - 1;
    int par[ACCEPT_BLOCKS], tok[ACCEPT_BLOCKS], want[ACCEPT_BLOCKS];
#pragma unroll
    for (int k = 0; k < ACCEPT_BLOCKS; ++k) {
      const int i = base + k * 32 + lane;
      par[k] = -2;
      tok[k] = want[k] = 0;
      if (n > 0 && i < n) {
        par[k] = load_cg(a.parents + row0 + i);
        tok[k] = load_cg(a.tokens + row0 + i);
        want[k] = load_cg(a.targets + row0 + i);
      }
    }
    const auto choice = [&](int node) {  // the model's behind a node
      const int at = node - base;
      if (at >= ACCEPT_HELD) return load_cg(a.targets + row0 + node);
      int x = want[0];
#pragma unroll
      for (int k = 1; k < ACCEPT_BLOCKS; ++k) x = at >> 5 == k ? want[k] : x;
      return __shfl_sync(0xffffffffu, x, at & 31);
    };
    int cur = base, taken = 0, next = n > 0 ? choice(cur) : -1;
    bool alive = n > 0;
    for (int c0 = 0; c0 < a.max_path; c0 += 32) {
      int mine = -1;
      for (int s = 0; alive && s < 32 && c0 + s < a.max_path; ++s) {
        int child = -1;
#pragma unroll
        for (int k = ACCEPT_BLOCKS - 1; k >= 0; --k) {
          const int i = base + k * 32 + lane;
          const unsigned int yes = __ballot_sync(0xffffffffu, par[k] == cur && tok[k] == next && i > cur && i < n);
          if (yes) child = base + k * 32 + __ffs(yes) - 1;
        }
        for (int i0 = base + ACCEPT_HELD; child < 0 && i0 < n; i0 += 32) {
          const int i = i0 + lane;
          const bool ok = i < n && i > cur && load_cg(a.parents + row0 + i) == cur && load_cg(a.tokens + row0 + i) == next;
          const unsigned int yes = __ballot_sync(0xffffffffu, ok);
          if (yes) child = i0 + __ffs(yes) - 1;
        }
        alive = child >= 0;
        if (!alive) break;
        if (lane == s) mine = child;
        cur = child;
        next = choice(cur);
        ++taken;
      }
      const int j = c0 + lane, from = ctx + mine, to = ctx + sure + j, i = from / a.page_size, o = to / a.page_size;
      const bool moves = mine >= 0 && mine != sure + j;
      int x = -1, y = -1;  // the pages (asked for before either is used)
      if (moves && to >= 0) x = page_at(b, i), y = page_at(b, o);
      if (c0 + 32 >= a.max_path) {
        // the walk has ended: the first pages that may go back, too
        after = max(ctx + sure + taken, 0);
        back0 = ceil_div(after, a.page_size);
        back1 = pages_back ? ceil_div(keys, a.page_size) : back0;
        if (back0 + lane < back1) id = page_at(b, back0 + lane);
      }
      if (j < a.max_path) {
        int src = -1, dst = -1;
        x = x < a.num_pages ? x : -1;
        y = y < a.num_pages ? y : -1;
        if (x >= 0 && y >= 0) {
          src = x * a.page_size + (from - i * a.page_size);
          dst = y * a.page_size + (to - o * a.page_size);
        }
        bad |= moves && src < 0;
        const long long at = (long long)b * a.max_path + j;
        a.path[at] = mine;
        a.src_slots[at] = src;
        a.dst_slots[at] = dst;
      }
    }
    if (lane == 0) {
      a.accepted[b] = sure + taken;
      a.ctx_lens[b] = after;
      a.next_tokens[b] = next;
      after_s[b] = after;
    }
    id = id < a.num_pages ? id : -1;
    const bool here = back0 + lane < back1;
    bad |= here && id < 0;
    int back = __popc(__ballot_sync(0xffffffffu, here && id >= 0));
    for (int i0 = back0 + 32; i0 < back1; i0 += 32) {
      const int later = i0 + lane < back1 ? page_at(b, i0 + lane) : -1;
      const bool ok = later >= 0 && later < a.num_pages;
      bad |= i0 + lane < back1 && !ok;
      back += __popc(__ballot_sync(0xffffffffu, ok));
    }
    if (b == gwarp) {  // (nobody writes to a CTA's shared memory before it runs)
      __syncwarp();
      cluster_wait();
    }
    if (lane < gridDim.x) store_remote(counts + b, lane, back);
  }
  if (gwarp >= a.B) cluster_wait();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (pages_back) {
    // requests before each one: neighbouring requests to a thread
    const int per = (a.B + ACCEPT_THREADS - 1) / ACCEPT_THREADS, b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    int own = 0;
    for (int b = b0; b < b1; ++b) own += counts[b];
    int incl = own;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < ACCEPT_WARPS; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    before += incl - own;
    for (int b = b0; b < b1; ++b) {
      const int x = counts[b];
      counts[b] = before;
      before += x;
    }
    __syncthreads();
    for (int b = gwarp; b < a.B; b += nwarps) {
      if (!alone) {
        back0 = ceil_div(after_s[b], a.page_size);
        back1 = ceil_div(max(load_cg(a.seqlens_k + b), 0), a.page_size);
      }
      int at = have + counts[b];
      for (int i0 = back0; i0 < back1; i0 += 32) {
        if (!alone || i0 > back0) id = i0 + lane < back1 ? page_at(b, i0 + lane) : -1;
        id = id < a.num_pages ? id : -1;
        const unsigned int yes = __ballot_sync(0xffffffffu, id >= 0);
        const int to = at + __popc(yes & ((1u << lane) - 1u));
        if (id >= 0) {
          if (to < a.max_free) a.free_pages[to] = id;
          else bad = true;
        }
        at += __popc(yes);
      }
    }
    // (every CTA has read free_count ahead of the cluster's barrier)
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_count_out = min(have + total, a.max_free);
  }
  if (bad) atomicOr(p.status, STATUS_PAGE);
}

// ------------------------------------------------------------------ moves
// cache[l][dst] = cache[l][src] for the moves of every list and every layer l.  A CTA takes a list and a layer,
// a thread 16-byte columns of K's and V's rows: it makes the list's moves in order, MOVE_AHEAD of them in flight, so
// that a row which a later move overwrites has been read, without any other order between threads.  61 lists of up to 8 moves in
// 32 layers of 8 heads, d = 128 (66 MB read and written) 12.9 us, 5.1 TB/s.  Half of what it reads and nearly all that it writes stays in L2 (DRAM at 33 % of
// its peak), and what it waits for is the latency of slots and rows: 1952 CTAs of lists of uneven lengths, 760 at a time.  Two or four layers
// to a CTA 13.7 and 14.6, four moves ahead 13.2, 128 threads 13.6.  8 lists in one layer: 2.3 us, a launch's time.
constexpr int MOVE_THREADS = 256, MOVE_AHEAD = 8, MOVE_LIST = 64;

struct MoveParams {
  attn_paged_move_params_t a;
  unsigned int* status;
};

template <int D>
__global__ void __launch_bounds__(MOVE_THREADS) paged_move_kernel(const __grid_constant__ MoveParams p) {
  const attn_paged_move_params_t& a = p.a;
  constexpr int CPR = D / 8;
  __shared__ long long from_s[MOVE_LIST], to_s[MOVE_LIST];
  const int tid = threadIdx.x, per_side = a.Hkv * CPR;
  grid_launch_dependents();
  grid_dependency_wait();
  const auto place = [&](int slot) {
    const int page = slot / a.page_size;
    return (long long)page * a.cache_page_stride + (long long)(slot - page * a.page_size) * a.cache_row_stride;
  };
  for (int list = blockIdx.x; list < a.lists; list += gridDim.x) {
    for (int m0 = 0; m0 < a.length; m0 += MOVE_LIST) {
      const int moves = min(MOVE_LIST, a.length - m0);
      if (tid < moves) {
        const long long at = (long long)list * a.length + m0 + tid;
        const int src = load_cg(a.src_slots + at), dst = load_cg(a.dst_slots + at);
        const int slots = a.num_pages * a.page_size;
        const bool ok = src >= 0 && dst >= 0 && src < slots && dst < slots;
        if (src >= slots || dst >= slots) atomicOr(p.status, STATUS_PAGE);
        from_s[tid] = ok ? place(src) : -1;
        to_s[tid] = ok ? place(dst) : 0;
      }
      __syncthreads();
      for (int layer = blockIdx.y; layer < a.layers; layer += gridDim.y)
        for (int c = tid; c < 2 * per_side; c += MOVE_THREADS) {
          const bool v = c >= per_side;
          const int e = v ? c - per_side : c;
          uint16_t* base = static_cast<uint16_t*>(v ? a.v_cache : a.k_cache) + layer * a.cache_layer_stride + (e / CPR) * a.cache_head_stride + e % CPR * 8;
          for (int j = 0; j < moves; j += MOVE_AHEAD) {
            uint4 x[MOVE_AHEAD];
#pragma unroll
            for (int u = 0; u < MOVE_AHEAD; ++u)
              if (j + u < moves && from_s[j + u] >= 0) x[u] = load_cg_x4(base + from_s[j + u]);
#pragma unroll
            for (int u = 0; u < MOVE_AHEAD; ++u)
              if (j + u < moves && from_s[j + u] >= 0) *reinterpret_cast<uint4*>(base + to_s[j + u]) = x[u];
          }
        }
      __syncthreads();  // the places have been read
    }
  }
}

// CTAs of a cluster of paged_accept_kernel at most: 16 where the device has that many SMs side by side for it, so that 512 requests have a
// warp each.  Asked once per device.
int widest_cluster(int dev, int& ctas) {
  static std::atomic<int> known[64];
  if ((ctas = known[dev].load()) != 0) return ATTN_OK;
  const size_t smem = 2 * (size_t)ACCEPT_MAX_B * sizeof(int);
  if (cudaFuncSetAttribute(paged_accept_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(ACCEPT_THREADS);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  ctas = 8;
  if (cudaFuncSetAttribute(paged_accept_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, paged_accept_kernel, &cfg) == cudaSuccess && clusters > 0)
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

int attn_paged_tree(const attn_paged_tree_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_paged_tree_params_t& a = *params;
    for (const void* ptr : {(const void*)a.parents, (const void*)a.cu_seqlens_q, (const void*)a.seqlens_k, (const void*)a.positions, (const void*)a.tree_mask})
      if (!ptr || misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    if (a.B < 1 || a.B > ACCEPT_MAX_B || a.rows < 1 || a.rows > (1 << 30) || a.mask_words < 1 || a.mask_words > TREE_WORDS ||
        a.mask_stride < a.mask_words || a.window_left < -1)
      return ATTN_ERR_INVALID;
    int sms = 0, dev = 0;
    int rc = host_device(sms, dev);
    if (rc != ATTN_OK) return rc;
    TreeParams p{a, nullptr};
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    const size_t smem = tree_smem(a.mask_words);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(paged_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tree_smem(TREE_WORDS)) != cudaSuccess)
      return ATTN_ERR_CUDA;
    return launch_dependent(paged_tree_kernel, dim3(a.B), TREE_THREADS, smem, reinterpret_cast<cudaStream_t>(a.stream), p);
  });
}

int attn_fwd_paged_tree(const attn_fwd_paged_tree_params_t* params) {
  return attn::entry([&]() -> int { return params ? attn::paged_fwd_impl(params->call, params) : ATTN_ERR_INVALID; });
}

int attn_paged_accept(const attn_paged_accept_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_paged_accept_params_t& a = *params;
    for (const void* ptr : {(const void*)a.cu_seqlens_q, (const void*)a.seqlens_k, (const void*)a.block_table, (const void*)a.accepted,
                            (const void*)a.ctx_lens, (const void*)a.next_tokens, (const void*)a.path, (const void*)a.src_slots, (const void*)a.dst_slots})
      if (!ptr || misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    for (const void* ptr : {(const void*)a.tokens, (const void*)a.targets, (const void*)a.parents})
      if ((!ptr && a.rows != 0) || misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    for (const void* ptr : {(const void*)a.confirmed, (const void*)a.free_pages, (const void*)a.free_count, (const void*)a.free_count_out})
      if (misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    if (a.free_pages ? !a.free_count || !a.free_count_out || a.max_free < 1 : a.max_free != 0) return ATTN_ERR_INVALID;
    if (a.B < 1 || a.B > ACCEPT_MAX_B || a.rows < 0 || a.rows > (1 << 30) || a.max_path < 1 || a.max_path > TREE_NODES || a.table_width < 1 ||
        a.table_stride < a.table_width || a.page_size < 16 || a.page_size % 16 != 0 || a.num_pages < 1 || (long long)a.num_pages * a.page_size > INT_MAX ||
        (long long)a.table_width * a.page_size > INT_MAX - 4096)
      return ATTN_ERR_INVALID;
    int sms = 0, dev = 0;
    int rc = host_device(sms, dev);
    if (rc != ATTN_OK) return rc;
    AcceptParams p{a, nullptr};
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    const size_t smem = 2 * (size_t)a.B * sizeof(int);
    int widest = 0;
    if ((rc = widest_cluster(dev, widest)) != ATTN_OK) return rc;
    int ctas = 1;
    while (ctas < widest && ctas * ACCEPT_WARPS < a.B) ctas *= 2;
    return launch_dependent(paged_accept_kernel, dim3(ctas), ACCEPT_THREADS, smem, reinterpret_cast<cudaStream_t>(a.stream), p, ctas);
  });
}

int attn_paged_move(const attn_paged_move_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_paged_move_params_t& a = *params;
    for (const void* ptr : {(const void*)a.k_cache, (const void*)a.v_cache})
      if (!ptr || misaligned(ptr, 16)) return ATTN_ERR_INVALID;
    for (const void* ptr : {(const void*)a.src_slots, (const void*)a.dst_slots})
      if (!ptr || misaligned(ptr, 4)) return ATTN_ERR_INVALID;
    if (a.d != 64 && a.d != 128) return ATTN_ERR_UNSUPPORTED;
    if (a.dtype != ATTN_F16 && a.dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
    if (a.layers < 1 || a.layers > (1 << 16) || a.lists < 1 || a.lists > (1 << 20) || a.length < 1 || a.length > (1 << 20) || a.Hkv < 1 ||
        a.Hkv > (1 << 16) || a.num_pages < 1 || a.page_size < 16 || a.page_size % 16 != 0 || (long long)a.num_pages * a.page_size > INT_MAX)
      return ATTN_ERR_INVALID;
    for (long long s : {a.cache_layer_stride, a.cache_page_stride, a.cache_head_stride, a.cache_row_stride})
      if (s < 0 || s % 8 != 0 || s > MAX_STRIDE) return ATTN_ERR_INVALID;
    if (a.cache_row_stride == 0 || (a.num_pages > 1 && a.cache_page_stride == 0) || (a.Hkv > 1 && a.cache_head_stride == 0) ||
        (a.layers > 1 && a.cache_layer_stride == 0))
      return ATTN_ERR_INVALID;
    int sms = 0, dev = 0;
    int rc = host_device(sms, dev);
    if (rc != ATTN_OK) return rc;
    MoveParams p{a, nullptr};
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    const dim3 grid(a.lists, a.layers < 65535 ? a.layers : 65535);
    return launch_dependent(a.d == 64 ? paged_move_kernel<64> : paged_move_kernel<128>, grid, MOVE_THREADS, 0, reinterpret_cast<cudaStream_t>(a.stream), p);
  });
}

}  // extern "C"
