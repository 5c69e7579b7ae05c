// paged_attn.cu -- attention of packed query rows over a paged key/value cache (attn_fwd_paged).
//
//     O[t, hq] = sum_j softmax_j( scale <Q[t, hq], K_j> ) V_j,   LSE[t, hq] = ln sum_j exp(...)
//
// over the keys j of row t's request that its position and window keep, K_j and V_j found
// through the request's block table.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "host.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "roles.cuh"

namespace attn {
namespace {

// An item whose tiles CTA c begins and others finish: the partial results to join.
struct Split {
  int row0, rows;  // the request's first query row, its packed rows (0: no such item)
  int h, parts;    // slots 2c + 1, 2(c + 1), 2(c + 2), ...
};

struct RowsParams : PagedParams {
  float* part_o;    // [2 * rows_grid][slot_rows][D] partial sums of V, not normalised
  float2* part_ml;  // [2 * rows_grid][slot_rows] their exponent base (exp2 domain) and sum of weights
  Split* split;     // [rows_grid]
  int rows_grid;    // CTAs of this path
  int slot_rows;    // rows of a slot: 16 or 32
};

// ------------------------------------------------------------------ few rows: the memory-bound path
// An item is (request, K/V head) with at most 16 MT packed rows, row r being query token r / g, query head
// r % g of the group: one pass over the keys serves the whole group.  Each key costs 4 d bytes and at most
// 16 MT * 4 d flops, below the machine's ratio, so the keys' stream from memory is the floor and
// everything else has to hide behind it:
//  * the items' key tiles, laid end to end, are cut into equal runs, one per CTA, whatever the
//    lengths: no CTA has more to read than another.  Items cut across CTAs leave partial results
//    (at most two to a CTA) that join_kernel puts together;
//  * the four warps of a CTA take a quarter of each tile's keys each, with a ring of asynchronous copies,
//    a running maximum, sum and accumulator of their own: nothing synchronises them before the item's end,
//    and the copies go on into the next item meanwhile;
//  * a lane holds the places of the next 32 page rows, so the table is read once per 32 copies;
//  * mma.sync with the keys as the N side: 16 rows are its smallest M, and its operands come by
//    ldmatrix straight from the copied rows (a tcgen05 tile's 128 rows would be an eighth full).
// Measured: 61 requests of 500 - 7200 keys, 32/8 heads, d = 128, bf16: 113 us, 6.1 TB/s of keys and values
// (0.90 of measured copy bandwidth); 3 of 84 - 106 thousand: 95 us, 6.0 TB/s; one of 1001: 9.3 us, latency (of
// launches, lengths -> table -> keys, and the join).  Ring depth, CTAs and keys to a stage were swept, with
// weights in one part: 2 stages and 3 CTAs 112 us, 2 and 4 (128 registers, spills) 166, 8 KiB in half the
// keys 126, this 110.
template <int D, int MT>
struct Rows {
  static constexpr int WARPS = 4, NTHREADS = 32 * WARPS;
  static constexpr int ROWS = 16 * MT;            // packed rows of an item at most
  static constexpr int KPW = D == 128 ? 16 : 32;  // keys of a warp's stage: 8 KiB of K and V
  static constexpr int NG = KPW / 16;             // groups of 16 keys: each lies in one page
  static constexpr int TK = WARPS * KPW;          // keys of a tile
  static constexpr int NST = 3;
  static constexpr int STAGE = 2 * KPW * D * 2;
  // Q operands in registers, or, where they and the accumulators would not fit, in shared memory
  static constexpr bool Q_SMEM = MT * D > 128;
  static constexpr int OFF_Q = WARPS * NST * STAGE;
  static constexpr int SMEM = OFF_Q + (Q_SMEM ? ROWS * D * 2 : 0);
  static constexpr int CTAS_PER_SM = 2;
  // Weights in two parts (see the product with V): 61 requests x 8k keys 112.5 us, with one part 111.5, and its
  // error the output rounding's alone (bf16 0.0017 of the norm, 0.0023 with one part).  With 32 rows at d =
  // 128 the products no longer hide behind the keys (64 requests x 2000 keys 121 us against 102).
  static constexpr bool TWO_PARTS = MT == 1 || D == 64;
  static constexpr int FOLD_TILES = D == 128 ? 128 : 12;  // (few_tiles_too)
  static_assert(STAGE >= 16 * D * 4, "a stage holds a 16-row accumulator of the warp at the item's end");
  static_assert(sizeof(TileUnit) % 8 == 0, "units are copied 8 bytes at a time");
  static_assert(NTHREADS == 128, "the plan and block_scan are written for four warps");
};

// What this path needs to know of a request: first query row, packed rows (0: not this path's), keys
// [lo, hi) that any of its rows keeps and the tiles [t0, t1) that hold them (one tile of nothing where no
// key is kept: the item still writes its rows).
struct RowsItem {
  int row0, R, off, sk;
  int lo, hi, t0, t1;
};
template <class C>
__device__ __forceinline__ RowsItem rows_request(const RowsParams& p, int b) {
  RowsItem it;
  int sq;
  request_span(p, b, it.row0, sq, it.sk);
  it.off = it.sk - sq;
  it.R = sq * p.g;
  it.lo = row_lo(p, 0, it.off);
  it.hi = row_hi(p, sq - 1, it.off, it.sk);
  if (it.hi <= it.lo) it.lo = it.hi = 0;
  it.t0 = it.lo / C::TK;
  it.t1 = it.hi > it.lo ? (it.hi - 1) / C::TK + 1 : it.t0 + 1;
  if (it.R > C::ROWS || it.R == 0) it.R = it.t0 = it.t1 = 0;
  return it;
}
// Its tiles, over all heads.
__device__ __forceinline__ long long rows_weight(const RowsParams& p, const RowsItem& it) { return (long long)(it.t1 - it.t0) * p.Hkv; }
// Whether the tcgen05 path takes the few-row requests as well, of `tiles` tiles (32 KiB each) altogether.  Two
// passes over the machine cost a start and an end each, one pass reads these keys more slowly (its step takes a
// 128-row tile's time), half as fast again at d = 64.  d = 128, 30 requests of 2000 keys beside a chunk of 512
// rows (50 tiles an SM): 98 us apart, 76 together; 16 of 8000 beside 2000 rows (108): 207 and 147; 64 of
// 4000 beside 256 (215): 198 and 224.  d = 64, 16 of 2000 beside 300 (7): 35 and 33; 30 of 2000 beside 512
// (13): 43 and 49.
template <class C>
__device__ __forceinline__ bool few_tiles_too(const RowsParams& p, long long tiles) {
  return p.tile.max_units > 0 && tiles < (long long)C::FOLD_TILES * p.tile.sms;
}
// The item after head h of request b.
template <class C>
__device__ __forceinline__ void rows_next(const RowsParams& p, int& b, int& h, RowsItem& it) {
  if (++h < p.Hkv) return;
  h = 0;
  do it = rows_request<C>(p, ++b);
  while (it.R == 0);
}

// ------------------------------------------------------------------ plan
// What the tcgen05 path works off, by one CTA of 128 threads while the others run the few-row path.  Units
// (of one head) are numbered request by request, requests of the other path having none, and sorted by
// weight into 32 classes, stably, so that equal inputs give equal cuts.  Bound by latency: one pass over the
// requests, then one over the units for each of weigh, sort, sum; the units stay in shared memory for these
// where they fit.
constexpr int PLAN_THREADS = 128, PLAN_WARPS = PLAN_THREADS / 32;
constexpr int MAX_SPLIT = 3; // runs per SM at most

// Exclusive sum over the block's threads of x, and the total.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* warp_sum, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += y;
  }
  __syncthreads();  // warp_sum may still be read from the scan before
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < PLAN_WARPS; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  return before + incl - x;
}

// `pre` is the CTA's shared memory: units before each request (B + 1 ints), then, where there is room, the
// units twice, as numbered and as sorted.
template <class C>
__device__ __forceinline__ void tile_plan(const RowsParams& p, int* pre) {
  __shared__ int sum_s[PLAN_WARPS], rank_s[PLAN_WARPS][33];
  __shared__ long long sum64_s[PLAN_WARPS];
  __shared__ int wmax_s, wmin_s;
  const TileWork& tw = p.tile;
  const int sms = tw.sms;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_tokens = TILE_QT * tw.T;
  const int per = (p.B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int own = 0, total;
  long long few = 0, few_all;
  for (int b = b0; b < b1; ++b) few += rows_weight(p, rows_request<C>(p, b));
  block_scan(few, sum64_s, few_all);
  const bool all_here = few_tiles_too<C>(p, few_all);
  for (int b = b0; b < b1; ++b) {
    int row0, sq, sk;
    request_span(p, b, row0, sq, sk);
    pre[b] = own;
    own += all_here || sq * p.g > ROWS_MAX ? (sq + unit_tokens - 1) / unit_tokens : 0;
  }
  if (tid == 0) wmax_s = 0, wmin_s = INT_MAX;
  for (int x = lane; x < 33; x += 32) rank_s[warp][x] = 0;
  const int before = block_scan(own, sum_s, total);
  for (int b = b0; b < b1; ++b) pre[b] += before;
  if (tid == 0) pre[p.B] = total;
  __syncthreads();
  const int units = min(total, tw.max_units);  // (more only where the row offsets overlap)
  const int at_units = (p.B + 1 + 3) & ~3;       // (ints)
  const bool near = (size_t)at_units * 4 + (size_t)(2 * units + 1) * sizeof(TileUnit) <= (size_t)C::SMEM;
  TileUnit* const sorted = near ? reinterpret_cast<TileUnit*>(pre + at_units) : tw.units;
  TileUnit* const numbered = sorted + units + 1;  // (only where near)
  const auto weigh = [&](int u) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u) lo = mid;
      else hi = mid;
    }
    TileUnit x;
    x.b = lo;
    x.blk = u - pre[lo];
    int row0, sq, sk, k0, k1;
    request_span(p, x.b, row0, sq, sk);
    tile_keys(p, sq, sk, x.blk, 0, TILE_QT, k0, k1);
    x.j0 = k0 / TILE_KEYS;
    x.w = max((k1 + TILE_KEYS - 1) / TILE_KEYS - x.j0, 1);
    x.cum = x.pad = 0;
    x.row0 = row0;
    x.sq = sq;
    x.sk = sk;
    return x;
  };
  // every warp takes a stretch of neighbouring units
  const int stretch = (units + PLAN_THREADS - 1) / PLAN_THREADS * 32;
  const int u0 = min(warp * stretch, units), u1 = min(u0 + stretch, units);
  int wmax = 0, wmin = INT_MAX;
  for (int u = u0 + lane; u < u1; u += 32) {
    const TileUnit x = weigh(u);
    if (near) numbered[u] = x;
    wmax = max(wmax, x.w);
    wmin = min(wmin, x.w);
  }
  wmax = __reduce_max_sync(0xffffffffu, wmax);
  wmin = __reduce_min_sync(0xffffffffu, wmin);
  if (lane == 0) {
    atomicMax(&wmax_s, wmax);
    atomicMin(&wmin_s, wmin);
  }
  __syncthreads();
  wmax = max(wmax_s, 1);
  const auto unit_at = [&](int u) { return near ? numbered[u] : weigh(u); };
  const auto class_of = [&](int w) { return 31 - (int)((unsigned)(w - 1) * 32u / (unsigned)wmax); };  // (w <= 2^24)
  for (int at = u0; at < u1; at += 32) {
    const int c = at + lane < u1 ? class_of(unit_at(at + lane).w) : 32;  // (class 32: no unit)
    const unsigned int same = __match_any_sync(0xffffffffu, c);
    if (lane == __ffs(same) - 1) rank_s[warp][c] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  {
    // where each warp's units of each class go: classes outside, warps inside
    const int c = tid / PLAN_WARPS, w = tid % PLAN_WARPS;
    const int x = rank_s[w][c];
    const int at = block_scan(x, sum_s, total);
    rank_s[w][c] = at;
  }
  __syncthreads();
  for (int at = u0; at < u1; at += 32) {
    TileUnit x = {};
    int c = 32;
    if (at + lane < u1) {
      x = unit_at(at + lane);
      c = class_of(x.w);
    }
    const unsigned int same = __match_any_sync(0xffffffffu, c);
    const int to = rank_s[warp][c] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (lane == __ffs(same) - 1) rank_s[warp][c] += __popc(same);
    __syncwarp();
    if (c < 32) sorted[to] = x;
  }
  __syncthreads();
  // steps before each unit, in the sorted order
  const int chunk = (units + PLAN_THREADS - 1) / PLAN_THREADS;
  const int s0 = min(tid * chunk, units), s1 = min(s0 + chunk, units);
  long long weight = 0, all;
  for (int s = s0; s < s1; ++s) weight += sorted[s].w + UNIT_COST;
  long long cum = block_scan(weight, sum64_s, all);
  for (int s = s0; s < s1; ++s) {
    sorted[s].cum = cum;
    cum += sorted[s].w + UNIT_COST;
  }
  if (tid == 0) sorted[units].cum = all;
  __syncthreads();
  if (near)
    for (int e = tid; e < (units + 1) * (int)(sizeof(TileUnit) / 8); e += PLAN_THREADS)
      reinterpret_cast<uint2*>(tw.units)[e] = reinterpret_cast<const uint2*>(sorted)[e];

  // Whole pairs: full waves of the longest, where none is longer than an SM's share.
  const long long pairs = (long long)units * p.Hkv, share = all * p.Hkv / sms;
  const int whole = wmax + UNIT_COST <= share ? (int)(pairs / sms * sms) : 0;
  const auto line_of = [&](long long x) {
    const int s = (int)(x / p.Hkv);
    return sorted[s].cum * p.Hkv + (s < units ? (x - (long long)s * p.Hkv) * (sorted[s].w + UNIT_COST) : 0);
  };
  const long long line0 = line_of(whole), line = all * p.Hkv - line0;
  // Runs: one per SM; more where the whole pairs before them differ, so that the SMs that are done
  // earlier take more.
  const long long len = line / sms + 1;
  const int split = whole ? (int)min((long long)MAX_SPLIT, 1 + 2ll * (wmax - wmin_s) / len) : 1;
  const int runs = line ? (int)max(1ll, min((long long)split * sms, line / MIN_RUN)) : 0;
  if (tid == 0) *tw.queue = TileQueue{(unsigned int)sms, whole, runs, 0, units, line0, line};
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t x, float& lo, float& hi) {
  if constexpr (BF16) {
    lo = __uint_as_float(x << 16);
    hi = __uint_as_float(x & 0xFFFF0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    lo = f.x;
    hi = f.y;
  }
}
// 16 bytes into shared memory, zeros where `bytes` is 0 (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(Rows<D, MT>::NTHREADS, Rows<D, MT>::CTAS_PER_SM) rows_kernel(const __grid_constant__ RowsParams p) {
  using C = Rows<D, MT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_launch_dependents();
  grid_dependency_wait();
  if (p.tile.max_units > 0 && blockIdx.x == 0) {
    tile_plan<C>(p, reinterpret_cast<int*>(smem));
    return;
  }
  __shared__ long long warp_sum[PLAN_WARPS];
  __shared__ int3 start_s;            // request, head and tile that the run begins with
  __shared__ float2 ml_s[C::WARPS][C::ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this CTA's run: sum the weights, find where it begins
  const int per = (p.B + C::NTHREADS - 1) / C::NTHREADS;
  const int rb0 = min(tid * per, p.B), rb1 = min(rb0 + per, p.B);
  long long own = 0, n;
  for (int b = rb0; b < rb1; ++b) own += rows_weight(p, rows_request<C>(p, b));
  const long long before = block_scan(own, warp_sum, n);
  const int ctas = (int)min((long long)p.rows_grid, n);
  const int cta = (int)blockIdx.x - ((int)gridDim.x - p.rows_grid);
  if (tid == 0) p.split[cta].rows = 0;
  if (cta >= ctas || few_tiles_too<C>(p, n)) return;
  const long long run0 = run_begin(n, ctas, cta);
  const int run = (int)(run_begin(n, ctas, cta + 1) - run0);  // tiles
  if (run0 >= before && run0 < before + own) {
    long long at = before;
    for (int b = rb0;; ++b) {
      const RowsItem it = rows_request<C>(p, b);
      const long long w = rows_weight(p, it);
      if (run0 < at + w) {
        const int tiles = it.t1 - it.t0, h = (int)((run0 - at) / tiles);
        start_s = make_int3(b, h, it.t0 + (int)(run0 - at - (long long)h * tiles));
        break;
      }
      at += w;
    }
  }
  __syncthreads();

  const uint32_t ring = smem_u32(smem) + warp * (C::NST * C::STAGE);
  constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte chunks of a row, rows of one copy of the warp
  const int crow = lane / CPR, cchunk = lane % CPR;
  const int fr = lane >> 2, fc = (lane & 3) * 2;  // fragment row and column pair

  // ---- the copies run ahead of the products, across items: their own place in the run
  int b = start_s.x, h = start_s.y, tile = start_s.z;
  RowsItem it = rows_request<C>(p, b);
  int cb = b, ch = h, ctile = tile, cleft = run, ccount = 0, cslot = 0;
  RowsItem cit = it;
  long long place = -1;  // lane's entry of the item's next 32 groups: element offset of its first row, -1 = none
  const auto issue = [&] {
    if (cleft > 0) {
      if (ctile == cit.t1) {
        rows_next<C>(p, cb, ch, cit);
        ctile = cit.t0;
        ccount = 0;
      }
      if (ccount % (32 / C::NG) == 0) {
        const int t = ctile + lane / C::NG, key = t * C::TK + warp * C::KPW + (lane % C::NG) * 16;
        place = -1;
        if (t < ctile + cleft && key < cit.hi && key + 16 > cit.lo) {
          const int idx = key / p.page_size;
          const int pg = p.table[(long long)cb * p.table_stride + idx];
          if ((unsigned)pg < (unsigned)p.num_pages)
            place = (long long)pg * p.c_page + (long long)(key - idx * p.page_size) * p.c_row;
          else
            atomicOr(p.status, STATUS_PAGE);
        }
      }
      const uint32_t st = ring + cslot * C::STAGE;
      const int key0 = ctile * C::TK + warp * C::KPW;
      const uint16_t* kh = p.k + ch * p.c_head;
      const uint16_t* vh = p.v + ch * p.c_head;
#pragma unroll
      for (int gq = 0; gq < C::NG; ++gq) {
        const long long at = __shfl_sync(0xffffffffu, place, (ccount * C::NG + gq) % 32);
#pragma unroll
        for (int x = 0; x < 16 / RPI; ++x) {
          const int r = gq * 16 + x * RPI + crow;
          const int key = key0 + r;
          const bool ok = at >= 0 && key >= cit.lo && key < cit.hi;
          const long long src = ok ? at + (long long)(x * RPI + crow) * p.c_row + cchunk * 8 : 0;
          const uint32_t dst = st + r * (D * 2) + ((cchunk ^ (r & 7)) * 16);
          copy16(dst, kh + src, ok ? 16u : 0u);
          copy16(dst + C::KPW * D * 2, vh + src, ok ? 16u : 0u);
        }
      }
      ++ctile;
      ++ccount;
      --cleft;
      if (++cslot == C::NST) cslot = 0;
    }
    copy_commit();
  };
#pragma unroll 1
  for (int s = 0; s < C::NST - 1; ++s) issue();

  int slot = 0;
  for (int left = run; left > 0;) {
    const int ntiles = min(it.t1 - tile, left);
    const bool begins = tile == it.t0, ends = tile + ntiles == it.t1;

    // Q operands of each 16-row tile (rows past the last one are copies of it), and the keys of rows fr, fr + 8
    const auto q_row = [&](int r) {
      const int rr = min(r, it.R - 1), i = rr / p.g;
      return p.q + (long long)(it.row0 + i) * p.q_row + (long long)(h * p.g + rr - i * p.g) * p.q_head;
    };
    uint32_t qf[C::Q_SMEM ? 1 : MT][D / 16][4];
    int klo[MT][2], khi[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = mt * 16 + fr + 8 * x, i = min(r, it.R - 1) / p.g;
        klo[mt][x] = row_lo(p, i, it.off);
        khi[mt][x] = row_hi(p, i, it.off, it.sk);
        if constexpr (!C::Q_SMEM) {
          const uint16_t* src = q_row(r) + fc;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            qf[mt][s][x] = *reinterpret_cast<const uint32_t*>(src + s * 16);
            qf[mt][s][x + 2] = *reinterpret_cast<const uint32_t*>(src + s * 16 + 8);
          }
        }
      }
    if constexpr (C::Q_SMEM) {
      for (int e = tid; e < C::ROWS * CPR; e += C::NTHREADS) {
        const int r = e / CPR, c = e % CPR;
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + r * (D * 2) + ((c ^ (r & 7)) * 16)) = reinterpret_cast<const uint4*>(q_row(r))[c];
      }
      __syncthreads();
    }
    // tiles whose every key is kept by every row need no mask
    const int lo_all = row_lo(p, (it.R - 1) / p.g, it.off), hi_all = row_hi(p, 0, it.off, it.sk);

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) o[mt][x][0] = o[mt][x][1] = o[mt][x][2] = o[mt][x][3] = 0.f;
    }
    float* exchange = nullptr;  // the slot of the last stage, which no copy takes before the join

    for (int s = 0; s < ntiles; ++s) {
      copy_wait<C::NST - 2>();
      __syncwarp();
      issue();
      const uint32_t st = ring + slot * C::STAGE;
      exchange = reinterpret_cast<float*>(smem + slot * C::STAGE);
      if (++slot == C::NST) slot = 0;
      const int key0 = (tile + s) * C::TK + warp * C::KPW;
      if (key0 >= it.hi || key0 + C::KPW <= it.lo) continue;  // no key of this warp's quarter

      // S = Q K^T: ROWS rows x KPW keys
      float sc[MT][2 * C::NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2 * C::NG; ++x) sc[mt][x][0] = sc[mt][x][1] = sc[mt][x][2] = sc[mt][x][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t qa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (C::Q_SMEM) {
            const int r = mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * ks + (lane >> 4);
            ldsm_x4(smem_u32(smem) + C::OFF_Q + r * (D * 2) + ((c ^ (r & 7)) * 16), qa[mt]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) qa[mt][e] = qf[mt][ks][e];
          }
        }
#pragma unroll
        for (int gq = 0; gq < C::NG; ++gq) {
          uint32_t kf[4];
          const int r = gq * 16 + (lane >> 4) * 8 + (lane & 7), c = 2 * ks + ((lane >> 3) & 1);
          ldsm_x4(st + r * (D * 2) + ((c ^ (r & 7)) * 16), kf);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_16816<BF16>(sc[mt][2 * gq], qa[mt], kf[0], kf[1]);
            mma_16816<BF16>(sc[mt][2 * gq + 1], qa[mt], kf[2], kf[3]);
          }
        }
      }
      uint32_t pf[MT][C::NG][4], pl[C::TWO_PARTS ? MT : 1][C::NG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (key0 < lo_all || key0 + C::KPW > hi_all) {
#pragma unroll
          for (int x = 0; x < 2 * C::NG; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + x * 8 + fc + (e & 1);
              if (key < klo[mt][e >> 1] || key >= khi[mt][e >> 1]) sc[mt][x][e] = -INFINITY;
            }
        }
        // running maximum (exp2 domain): it moves only when it grows by more than 8, so the
        // accumulator is rarely rescaled and weights stay below 2^8
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 2 * C::NG; ++x) {
          mx[0] = fmaxf(mx[0], fmaxf(sc[mt][x][0], sc[mt][x][1]));
          mx[1] = fmaxf(mx[1], fmaxf(sc[mt][x][2], sc[mt][x][3]));
        }
        bool grow = false;
        float mn[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
          mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * p.scale_log2;
          mn[x] = mx[x] > m[mt][x] + 8.f ? mx[x] : m[mt][x];
          grow |= mn[x] != m[mt][x];
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float alpha = mn[x] == m[mt][x] ? 1.f : ex2_approx(m[mt][x] - mn[x]);
            l[mt][x] *= alpha;
            m[mt][x] = mn[x];
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
              o[mt][y][2 * x] *= alpha;
              o[mt][y][2 * x + 1] *= alpha;
            }
          }
        }
        const float mu[2] = {m[mt][0] == -INFINITY ? 0.f : m[mt][0], m[mt][1] == -INFINITY ? 0.f : m[mt][1]};
#pragma unroll
        for (int x = 0; x < 2 * C::NG; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[mt][x][e] = ex2_approx(fmaf(sc[mt][x][e], p.scale_log2, -mu[e >> 1]));
            l[mt][e >> 1] += sc[mt][x][e];
          }
        // A matrix instruction takes the weights in the values' type.  That rounding alone would cost as
        // much as the output's own, so what it leaves goes through a second instruction, and they count to
        // twice as many bits (TWO_PARTS; else it is accepted).  The sum l has them in 32 bits.
#pragma unroll
        for (int gq = 0; gq < C::NG; ++gq)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& a = sc[mt][2 * gq + (e >> 1)][(e & 1) * 2];
            float& c = sc[mt][2 * gq + (e >> 1)][(e & 1) * 2 + 1];
            pf[mt][gq][e] = pack2<BF16>(a, c);
            if constexpr (C::TWO_PARTS) {
              float ah, ch;
              unpack2<BF16>(pf[mt][gq][e], ah, ch);
              pl[mt][gq][e] = pack2<BF16>(a - ah, c - ch);
            }
          }
      }
      // O += P V
#pragma unroll
      for (int gq = 0; gq < C::NG; ++gq) {
        const int r = gq * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t vf[4];
          const int c = 2 * x + (lane >> 4);
          ldsm_x4_trans(st + C::KPW * D * 2 + r * (D * 2) + ((c ^ (r & 7)) * 16), vf);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_16816<BF16>(o[mt][2 * x], pf[mt][gq], vf[0], vf[1]);
            mma_16816<BF16>(o[mt][2 * x + 1], pf[mt][gq], vf[2], vf[3]);
            if constexpr (C::TWO_PARTS) {
              mma_16816<BF16>(o[mt][2 * x], pl[mt][gq], vf[0], vf[1]);
              mma_16816<BF16>(o[mt][2 * x + 1], pl[mt][gq], vf[2], vf[3]);
            }
          }
        }
      }
    }
    __syncwarp();  // every lane has read the last stage

    // ---- join the four warps, 16 rows at a time, each through the slot of its last stage: row r's 8-column
    // chunk c at chunk c ^ (r & 7)
    float* mine = exchange + warp * (C::NST * C::STAGE / 4);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();  // the 16 rows before have been read
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
        const int r = fr + 8 * x;
        if (mt * 16 + r >= it.R) continue;
        if ((lane & 3) == 0) ml_s[warp][mt * 16 + r] = make_float2(m[mt][x], l[mt][x]);
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
          *reinterpret_cast<float2*>(mine + r * D + ((y ^ (r & 7)) * 8) + fc) = make_float2(o[mt][y][2 * x], o[mt][y][2 * x + 1]);
      }
      __syncthreads();
      const int rs = tid / 8, r = mt * 16 + rs;
      if (r < it.R) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) mm = fmaxf(mm, ml_s[w][r].x);
        float f[C::WARPS], ll = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          f[w] = ml_s[w][r].x == -INFINITY ? 0.f : ex2_approx(ml_s[w][r].x - mm);
          ll += f[w] * ml_s[w][r].y;
        }
        const bool whole = begins && ends;
        const int at = (2 * cta + (begins ? 1 : 0)) * C::ROWS + r;  // (a part's place)
        const int i = r / p.g, hq = h * p.g + r - i * p.g;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const int phys = (tid & 7) + 8 * j, col = (phys ^ (rs & 7)) * 8;
          float acc[8] = {};
#pragma unroll
          for (int w = 0; w < C::WARPS; ++w) {
            const float4* src = reinterpret_cast<const float4*>(exchange + w * (C::NST * C::STAGE / 4) + rs * D + phys * 8);
            const float4 a = src[0], c = src[1];
            acc[0] = fmaf(f[w], a.x, acc[0]);
            acc[1] = fmaf(f[w], a.y, acc[1]);
            acc[2] = fmaf(f[w], a.z, acc[2]);
            acc[3] = fmaf(f[w], a.w, acc[3]);
            acc[4] = fmaf(f[w], c.x, acc[4]);
            acc[5] = fmaf(f[w], c.y, acc[5]);
            acc[6] = fmaf(f[w], c.z, acc[6]);
            acc[7] = fmaf(f[w], c.w, acc[7]);
          }
          if (whole) {
            *reinterpret_cast<uint4*>(p.o + (long long)(it.row0 + i) * p.o_row + (long long)hq * p.o_head + col) =
                make_uint4(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[2] * inv, acc[3] * inv),
                           pack2<BF16>(acc[4] * inv, acc[5] * inv), pack2<BF16>(acc[6] * inv, acc[7] * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + (long long)at * D + col);
            dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
          }
        }
        if ((tid & 7) == 0) {
          if (!whole) p.part_ml[at] = make_float2(mm, ll);
          else if (p.lse) p.lse[(long long)hq * p.total_q + it.row0 + i] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * LN2;
        }
      }
    }
    if (begins && !ends && tid == 0) {
      // the CTAs that hold the item's other tiles: up to the one whose run reaches its end
      const long long last = run0 + (run - left) + (it.t1 - tile) - 1;
      p.split[cta] = Split{it.row0, it.R, h, run_of(n, ctas, last) - cta + 1};
    }
    __syncthreads();  // the exchange has been read

    left -= ntiles;
    if (left > 0) {
      rows_next<C>(p, b, h, it);
      tile = it.t0;
    }
  }
}

// ------------------------------------------------------------------ join
// Puts the partial results of cut items and units together: for a row of theirs
//     m = max m_k, O = sum 2^(m_k - m) O_k / sum 2^(m_k - m) l_k, LSE = ln2 (m + log2 sum).
// A CTA takes 16 rows of a cut item of the few-row path, whose warps share out the rows, and where there are
// fewer rows than warps, a row's parts; or 16 rows of a cut unit of the tcgen05 path, four columns of a
// row to a thread, as that path writes them.  The parts were just written and are mostly in L2; four are in
// flight at a time.
constexpr int JOIN_WARPS = JOIN_ROWS, JOIN_AHEAD = 4;

template <int D, bool BF16>
__device__ __forceinline__ void join_unit(const RowsParams& p, const TileJoin& jn) {
  const int r = threadIdx.x % JOIN_ROWS, col = threadIdx.x / JOIN_ROWS * 4;
  static_assert(D / 4 <= 32 * JOIN_WARPS / JOIN_ROWS, "a thread to four columns of a row");
  if (r >= jn.rows || col >= D) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < jn.parts; k0 += JOIN_AHEAD) {
    float2 ml[JOIN_AHEAD];
    float4 v[JOIN_AHEAD];
#pragma unroll
    for (int a = 0; a < JOIN_AHEAD; ++a) {
      const int k = k0 + a, slot = 2 * (jn.run + k) + (k == 0);
      ml[a] = make_float2(-INFINITY, 0.f);
      v[a] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < jn.parts) {
        ml[a] = p.tile.part_ml[(long long)slot * (TILE_QT * TILE_ROWS) + jn.in + r];
        v[a] = *reinterpret_cast<const float4*>(p.tile.part_o + part_at<D>(slot, jn.in + r, col));
      }
    }
    float mn = m;
#pragma unroll
    for (int a = 0; a < JOIN_AHEAD; ++a) mn = fmaxf(mn, ml[a].x);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
    l *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int a = 0; a < JOIN_AHEAD; ++a) {
      const float fa = ml[a].x == -INFINITY ? 0.f : ex2_approx(ml[a].x - mn);
      l = fmaf(ml[a].y, fa, l);
      acc = make_float4(fmaf(v[a].x, fa, acc.x), fmaf(v[a].y, fa, acc.y), fmaf(v[a].z, fa, acc.z), fmaf(v[a].w, fa, acc.w));
    }
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int rr = jn.row + r, i = rr / p.g, hq = jn.h * p.g + rr - i * p.g;
  *reinterpret_cast<uint2*>(p.o + (long long)(jn.row0 + i) * p.o_row + (long long)hq * p.o_head + col) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (col == 0 && p.lse) p.lse[(long long)hq * p.total_q + jn.row0 + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_kernel(const __grid_constant__ RowsParams p) {
  constexpr int E = D / 32;  // columns of a lane
  __shared__ float acc_s[JOIN_WARPS][D];
  __shared__ float2 ml_s[JOIN_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_launch_dependents();
  grid_dependency_wait();
  const int halves = p.slot_rows / JOIN_ROWS, items = p.tile.no_plan ? 0 : p.rows_grid * halves;
  const int total = items + (p.tile.no_plan ? p.tile.sms * JOINS_OF_RUN : p.tile.max_units > 0 ? p.tile.queue->njoins : 0);
  for (int x = blockIdx.x; x < total; x += gridDim.x) {
    if (x >= items) {
      join_unit<D, BF16>(p, p.tile.joins[x - items]);
      continue;
    }
    const int c = x / halves, prow = x % halves * JOIN_ROWS;
    const Split sp = p.split[c];
    const int rows = min(sp.rows - prow, JOIN_ROWS), row0 = sp.row0, h = sp.h, parts = sp.parts;
    if (rows <= 0) continue;
    // part k of row r: record (k ? slot0 + k * stride : first) + r
    const int first = (2 * c + 1) * p.slot_rows + prow, slot0 = 2 * c * p.slot_rows + prow, stride = 2 * p.slot_rows;
    int share = 1;  // warps to a row
    while (share * 2 * rows <= JOIN_WARPS) share *= 2;
    const int r = warp / share, sub = warp % share;
    float m = -INFINITY, l = 0.f, acc[E] = {};
    if (r < rows) {
      constexpr int AHEAD = JOIN_AHEAD;
      for (int k0 = sub; k0 < parts; k0 += share * AHEAD) {
        float2 ml[AHEAD];
        float v[AHEAD][E];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const int k = k0 + a * share;
          const long long at = (k ? slot0 + (long long)k * stride : first) + r;
          ml[a] = k < parts ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[a][e] = k < parts ? p.part_o[at * D + lane * E + e] : 0.f;
        }
        float mn = m;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) mn = fmaxf(mn, ml[a].x);
        const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const float fa = ml[a].x == -INFINITY ? 0.f : ex2_approx(ml[a].x - mn);
          l = fmaf(ml[a].y, fa, l);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(v[a][e], fa, acc[e]);
        }
        m = mn;
      }
    }
    if (share > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) acc_s[warp][lane * E + e] = acc[e];
      if (lane == 0) ml_s[warp] = make_float2(m, l);
      __syncthreads();
      if (sub == 0 && r < rows) {
        float mm = m;
        for (int w = 1; w < share; ++w) mm = fmaxf(mm, ml_s[warp + w].x);
        const float f = m == -INFINITY ? 0.f : ex2_approx(m - mm);
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
        for (int w = 1; w < share; ++w) {
          const float2 ml = ml_s[warp + w];
          const float fw = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
          l = fmaf(ml.y, fw, l);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(acc_s[warp + w][lane * E + e], fw, acc[e]);
        }
        m = mm;
      }
    }
    if (sub != 0 || r >= rows) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int rr = prow + r, i = rr / p.g, hq = h * p.g + rr - i * p.g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (long long)(row0 + i) * p.o_row + (long long)hq * p.o_head + lane * E);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[(long long)hq * p.total_q + row0 + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
  }
}

// ------------------------------------------------------------------ host side
// Workspace: the few-row path's partial results, then, where a request may take the tcgen05 path, that
// path's scratch.
struct Plan {
  int rows_grid, slot_rows, T, max_units;
  size_t off_ml, off_split, off_queue, off_units, off_joins, off_tile_ml, off_tile_o, bytes;
  Plan(const attn_fwd_paged_params_t& a, int sms) {
    const int g = a.Hq / a.Hkv;
    rows_grid = 2 * sms;
    const int longest = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
    const long long most = (long long)longest * g;  // packed rows of a request
    slot_rows = most > ROWS_MAX && most <= ROWS_ONLY ? 32 : 16;
    const size_t slots = 2 * (size_t)rows_grid * slot_rows;
    off_ml = round256(slots * a.d * sizeof(float));
    off_split = off_ml + round256(slots * sizeof(float2));
    off_queue = off_split + round256((size_t)rows_grid * sizeof(Split));
    T = TILE_ROWS / g;
    if (most <= ROWS_ONLY) {
      max_units = 0;
      bytes = off_queue;
      return;
    }
    // units of a head: every request's tokens over 2 T, rounded up
    const long long by_rows = (long long)a.total_q / (TILE_QT * T) + a.B;  // <= total_q / 2 + B
    const long long by_len = a.B * (((long long)longest + TILE_QT * T - 1) / (TILE_QT * T));
    max_units = (int)(by_rows < by_len ? by_rows : by_len);
    const size_t max_runs = (size_t)MAX_SPLIT * sms, pieces = 2 * max_runs * TILE_QT * TILE_ROWS;
    off_units = off_queue + 256;
    off_joins = off_units + round256((size_t)(max_units + 1) * sizeof(TileUnit));
    off_tile_ml = off_joins + round256(max_runs * (TILE_QT * TILE_ROWS / JOIN_ROWS) * sizeof(TileJoin));
    off_tile_o = off_tile_ml + round256(pieces * sizeof(float2));
    bytes = off_tile_o + round256(pieces * a.d * sizeof(float));
  }
};

bool misaligned(const void* ptr, unsigned int to) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }

int check_shape(const attn_fwd_paged_params_t& a) {
  if (a.B < 1 || a.B > 16384 || a.total_q < 1 || a.Hq < 1 || a.Hkv < 1 || a.Hq % a.Hkv != 0 || a.max_seqlen_q < 1) return ATTN_ERR_INVALID;
  if (a.d != 64 && a.d != 128) return ATTN_ERR_UNSUPPORTED;
  if (a.Hq / a.Hkv > 128) return ATTN_ERR_UNSUPPORTED;
  if ((long long)a.total_q * a.Hq > INT_MAX - (1 << 27)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

int check(const attn_fwd_paged_params_t& a) {
  if (!a.q || !a.k_cache || !a.v_cache || !a.o || !a.block_table || !a.cu_seqlens_q || !a.seqlens_k)
    return ATTN_ERR_INVALID;
  int rc = check_shape(a);
  if (rc != ATTN_OK) return rc;
  if (a.dtype != ATTN_F16 && a.dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
  if (a.num_pages < 1 || a.table_width < 1 || a.table_stride < a.table_width || a.page_size < 16 ||
      a.page_size % 16 != 0 || (long long)a.table_width * a.page_size > INT_MAX - 4096 ||
      a.window_left < -1 || a.window_right < -1)
    return ATTN_ERR_INVALID;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale * LOG2E)) return ATTN_ERR_INVALID;
  for (const void* ptr : {a.q, a.k_cache, a.v_cache, (const void*)a.o})
    if (misaligned(ptr, 16)) return ATTN_ERR_INVALID;
  for (const void* ptr : {(const void*)a.lse, (const void*)a.block_table, (const void*)a.cu_seqlens_q, (const void*)a.seqlens_k})
    if (misaligned(ptr, 4)) return ATTN_ERR_INVALID;
  if (misaligned(a.workspace, 256)) return ATTN_ERR_INVALID;
  for (long long s : {a.q_row_stride, a.q_head_stride, a.o_row_stride, a.o_head_stride, a.cache_page_stride, a.cache_head_stride,
                      a.cache_row_stride})
    if (s < 0 || s % 8 != 0 || s > MAX_STRIDE) return ATTN_ERR_INVALID;
  // one handle stands for a stream of every thread, which the library cannot keep a workspace for
  if (!a.workspace && a.stream == reinterpret_cast<void*>(cudaStreamPerThread)) return ATTN_ERR_INVALID;
  // the strides of dimensions with more than one entry
  if (a.cache_row_stride == 0 || (a.num_pages > 1 && a.cache_page_stride == 0) || (a.Hkv > 1 && a.cache_head_stride == 0) ||
      (a.Hq > 1 && (a.q_head_stride == 0 || a.o_head_stride == 0)) || (a.total_q > 1 && (a.q_row_stride == 0 || a.o_row_stride == 0)))
    return ATTN_ERR_INVALID;
  // the tensor maps of the caches take page and head as one coordinate
  if (a.num_pages > 1 && a.Hkv > 1) {
    const long long big = a.cache_page_stride > a.cache_head_stride ? a.cache_page_stride : a.cache_head_stride;
    const long long unit = a.cache_page_stride + a.cache_head_stride - big;
    if (big % unit != 0 || (big == a.cache_page_stride ? a.num_pages : a.Hkv) > (INT_MAX - (1 << 20)) / (big / unit)) return ATTN_ERR_UNSUPPORTED;
  }
  return ATTN_OK;
}

template <int D, int MT, bool BF16>
int launch(const RowsParams& p, const attn_fwd_paged_params_t& a, const Plan& plan, int sms, int dev, cudaStream_t st) {
  using C = Rows<D, MT>;
  static std::atomic<unsigned long long> attr_set{0};  // bit per device
  const unsigned long long bit = 1ull << dev;
  if (!(attr_set.load() & bit)) {
    if (cudaFuncSetAttribute(rows_kernel<D, MT, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_set.fetch_or(bit);
  }
  const bool tiles = p.tile.max_units > 0;
  TileParams tp = {};
  int rc = tiles ? tile_prepare(p, a, tp) : ATTN_OK;
  if (rc == ATTN_OK && !p.tile.no_plan) rc = launch_dependent(rows_kernel<D, MT, BF16>, dim3(plan.rows_grid + (tiles ? 1 : 0)), C::NTHREADS, C::SMEM, st, p);
  if (rc == ATTN_OK && tiles) rc = tile_launch(tp, a, sms, dev, st);
  if (rc != ATTN_OK) return rc;
  const int joins = p.tile.no_plan ? sms * JOINS_OF_RUN : plan.rows_grid;
  return launch_dependent(join_kernel<D, BF16>, dim3(joins), 32 * JOIN_WARPS, 0, st, p);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_paged_workspace(const attn_fwd_paged_params_t* params, unsigned long long* bytes) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params || !bytes) return ATTN_ERR_INVALID;
    int rc = check_shape(*params);
    if (rc != ATTN_OK) return rc;
    int sms = 0, dev = 0;
    if ((rc = host_device(sms, dev)) != ATTN_OK) return rc;
    *bytes = Plan(*params, sms).bytes;
    return ATTN_OK;
  });
}

int attn_fwd_paged(const attn_fwd_paged_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_fwd_paged_params_t& a = *params;
    int rc = check(a);
    if (rc != ATTN_OK) return rc;
    int sms = 0, dev = 0;
    if ((rc = host_device(sms, dev)) != ATTN_OK) return rc;
    const Plan plan(a, sms);
    if (a.workspace && a.workspace_bytes < plan.bytes) return ATTN_ERR_INVALID;
    RowsParams p = {};
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k_cache);
    p.v = static_cast<const uint16_t*>(a.v_cache);
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.table = a.block_table;
    p.cu_q = a.cu_seqlens_q;
    p.lens_k = a.seqlens_k;
    p.q_row = a.q_row_stride;
    p.q_head = a.q_head_stride;
    p.o_row = a.o_row_stride;
    p.o_head = a.o_head_stride;
    p.c_page = a.cache_page_stride;
    p.c_head = a.cache_head_stride;
    p.c_row = a.cache_row_stride;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.g = a.Hq / a.Hkv;
    p.total_q = a.total_q;
    p.max_q = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.width = a.table_width;
    p.table_stride = a.table_stride;
    p.wl = a.window_left;
    p.er = a.causal ? 0 : a.window_right;
    p.scale_log2 = a.scale * LOG2E;
    if ((rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(a.stream);
    void* scratch = a.workspace;
    std::unique_lock<std::mutex> hold;  // until the launches are enqueued
    if (!scratch) {
      // a captured call would share the stream's workspace with whatever runs beside its replays
      cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
      if (cudaStreamIsCapturing(st, &capture) != cudaSuccess) return ATTN_ERR_CUDA;
      if (capture != cudaStreamCaptureStatusNone) return ATTN_ERR_INVALID;
      if ((rc = host_workspace(dev, a.stream, plan.bytes, hold, &scratch)) != ATTN_OK) return rc;
    }
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
    p.split = reinterpret_cast<Split*>(ws + plan.off_split);
    p.timeout_us = host_timeout_us();
    p.rows_grid = plan.rows_grid;
    p.tile.T = plan.T;
    p.tile.max_units = plan.max_units;
    p.tile.sms = sms;
    p.tile.no_plan = plan.max_units > 0 && p.max_q <= plan.T && a.B <= NO_PLAN_B && (long long)a.total_q * p.g > (long long)ROWS_MAX * a.B;
    if (plan.max_units > 0) {
      p.tile.queue = reinterpret_cast<TileQueue*>(ws + plan.off_queue);
      p.tile.units = reinterpret_cast<TileUnit*>(ws + plan.off_units);
      p.tile.joins = reinterpret_cast<TileJoin*>(ws + plan.off_joins);
      p.tile.part_ml = reinterpret_cast<float2*>(ws + plan.off_tile_ml);
      p.tile.part_o = reinterpret_cast<float*>(ws + plan.off_tile_o);
    }
    p.slot_rows = plan.slot_rows;
    const bool bf16 = a.dtype == ATTN_BF16;
    const auto go = [&](auto launch) { return launch(p, a, plan, sms, dev, st); };
    if (plan.slot_rows == 16) {
      if (a.d == 64) return go(bf16 ? launch<64, 1, true> : launch<64, 1, false>);
      return go(bf16 ? launch<128, 1, true> : launch<128, 1, false>);
    }
    if (a.d == 64) return go(bf16 ? launch<64, 2, true> : launch<64, 2, false>);
    return go(bf16 ? launch<128, 2, true> : launch<128, 2, false>);
  });
}

}  // extern "C"
