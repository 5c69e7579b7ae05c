// paged_tile.cu -- chunks of many rows: the tcgen05 path of attn_fwd_paged.
//
// The rows of a request's K/V head are packed token by token, the group's heads side by side, so
// one stream of keys serves the whole group: a Q tile holds T = 128 / g tokens of all g heads (T g <= 128
// rows), a unit two Q tiles.  The keys of a unit come through the block table: a 128-key tile is
// assembled from TMA boxes of up to page_size rows, which land in the 128-byte-swizzled tile that the
// MMA warp of roles.cuh expects.  Roles, TMEM and barriers are those of attn_fwd.cu.
//
// Work: a plan kernel weighs every unit by its key tiles and lists them longest first.  The attention
// kernel takes from a queue first whole units, as many as give every SM the same number, then runs: the rest of the
// units laid end to end and cut into equal lengths, so no SM waits for another's last unit, and few units
// still fill the machine.  The results of cut units (at most two pieces to a run) are joined by a third kernel.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "attn.h"
#include "host.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "roles.cuh"

namespace attn {
namespace {

constexpr int FLAG_SCRUB = 16;  // the key tile holds rows that no query row of the unit sees

// Written by the plan.  Line coordinates count key tiles over all (unit, head) pairs in order, heads inside.
struct TileQueue {
  unsigned int next;    // next queue entry
  int whole, runs;      // entries: whole (unit, head) pairs, then runs
  int njoins;           // cut (unit, head) pairs
  int units;
  long long line0, line;  // where the runs' line begins, its length
};
struct TileUnit {
  int b, blk;
  int j0, w;      // key tiles j0 .. j0 + w - 1 (one where no key is seen: the unit still writes its rows)
  long long cum;  // weights of the units before
};
struct TileJoin {
  int unit, h;
  int run, parts;  // slots 2 run + 1, 2 (run + 1), 2 (run + 2), ...
};

struct TileParams : PagedParams {
  CUtensorMap tm_q, tm_k, tm_v;
  int T;          // tokens of a Q tile
  int box_rows;   // rows of one K/V box
  TileQueue* queue;
  TileUnit* units;   // [max_units + 1], longest first
  TileJoin* joins;   // [max runs]: every cut pair holds a run's beginning
  float* part_o;     // [2 max runs][256][D]
  float2* part_ml;   // [2 max runs][256]
  int max_units;
  int inject;
};

struct TileHdr {
  int j, flags;
  int row0, sq, sk;
  int h, blk, slot;
  int lo, hi;  // keys that any row of the unit sees
  int pad[2];
};
static_assert(sizeof(TileHdr) == 48, "descriptor slot size");

template <int D>
using TileLayout = Layout<D, MASK_BAND, TileHdr>;

// Tokens and keys of Q tiles [t0, t1) of block blk: false where it has no token.
__device__ __forceinline__ bool tile_keys(const TileParams& p, int sq, int sk, int blk, int t0, int t1, int& lo, int& hi) {
  const int i0 = (blk * QT + t0) * p.T, i1 = min((blk * QT + t1) * p.T, sq) - 1;
  lo = hi = 0;
  if (i0 > i1) return false;
  const int a = row_lo(p, i0, sk - sq), e = row_hi(p, i1, sk - sq, sk);
  if (e > a) lo = a, hi = e;
  return true;
}

// First tile of run i out of n over a line, and the run that holds tile x of it.
__device__ __forceinline__ long long run_begin(long long line, int n, int i) { return line * i / n; }
__device__ __forceinline__ int run_of(long long line, int n, long long x) { return (int)(((x + 1) * n - 1) / line); }

// ------------------------------------------------------------------ plan
// One CTA.  Units (of one head) are numbered request by request, requests of the other path having none,
// and sorted by weight into 32 classes, stably, so that equal inputs give equal cuts.  Bound by latency: two
// passes over the lengths, one over the units for each of weigh, sort, sum.
constexpr int PLAN_THREADS = 1024;
constexpr int MIN_RUN = 4;   // tiles of a run at least
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
  if (warp == 0) {
    const T w = warp_sum[lane];
    T y = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, y, s);
      if (lane >= s) y += z;
    }
    warp_sum[lane] = y - w;
    if (lane == 31) warp_sum[32] = y;
  }
  __syncthreads();
  total = warp_sum[32];
  return warp_sum[warp] + incl - x;
}

__global__ void __launch_bounds__(PLAN_THREADS) tile_plan_kernel(const __grid_constant__ TileParams p, int sms) {
  grid_launch_dependents();
  extern __shared__ int pre[];  // units before each request, [B + 1]
  __shared__ int sum_s[33], rank_s[32][33];
  __shared__ long long sum64_s[33];
  __shared__ int wmax_s, wmin_s, joins_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_tokens = QT * p.T;
  const int per = (p.B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int own = 0, total;
  for (int b = b0; b < b1; ++b) {
    int row0, sq, sk;
    request_span(p, b, row0, sq, sk);
    pre[b] = own;
    own += sq * p.g > ROWS_MAX ? (sq + unit_tokens - 1) / unit_tokens : 0;
  }
  if (tid == 0) wmax_s = joins_s = 0, wmin_s = INT_MAX;
  rank_s[warp][lane] = 0;
  if (lane == 0) rank_s[warp][32] = 0;
  const int before = block_scan(own, sum_s, total);
  for (int b = b0; b < b1; ++b) pre[b] += before;
  if (tid == 0) pre[p.B] = total;
  __syncthreads();
  const int units = min(total, p.max_units);  // (more only where the row offsets overlap)
  const auto unit_at = [&](int u) {
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
    tile_keys(p, sq, sk, x.blk, 0, QT, k0, k1);
    x.j0 = k0 / BN;
    x.w = max((k1 + BN - 1) / BN - x.j0, 1);
    x.cum = 0;
    return x;
  };
  // every warp takes a stretch of neighbouring units
  const int stretch = (units + PLAN_THREADS - 1) / PLAN_THREADS * 32;
  const int u0 = min(warp * stretch, units), u1 = min(u0 + stretch, units);
  int wmax = 0, wmin = INT_MAX;
  for (int u = u0 + lane; u < u1; u += 32) {
    const int w = unit_at(u).w;
    wmax = max(wmax, w);
    wmin = min(wmin, w);
  }
  wmax = __reduce_max_sync(0xffffffffu, wmax);
  wmin = __reduce_min_sync(0xffffffffu, wmin);
  if (lane == 0) {
    atomicMax(&wmax_s, wmax);
    atomicMin(&wmin_s, wmin);
  }
  __syncthreads();
  wmax = max(wmax_s, 1);
  const auto class_of = [&](int w) { return 31 - (int)((long long)(w - 1) * 32 / wmax); };
  for (int at = u0; at < u1; at += 32) {
    const int c = at + lane < u1 ? class_of(unit_at(at + lane).w) : 32;  // (class 32: no unit)
    const unsigned int same = __match_any_sync(0xffffffffu, c);
    if (lane == __ffs(same) - 1) rank_s[warp][c] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  {
    // where each warp's units of each class go: classes outside, warps inside
    const int c = tid >> 5, w = tid & 31;
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
    if (c < 32) p.units[to] = x;
  }
  __syncthreads();
  // weights before each unit, in the sorted order
  const int chunk = (units + PLAN_THREADS - 1) / PLAN_THREADS;
  const int s0 = min(tid * chunk, units), s1 = min(s0 + chunk, units);
  long long weight = 0, all;
  for (int s = s0; s < s1; ++s) weight += p.units[s].w;
  long long cum = block_scan(weight, sum64_s, all);
  for (int s = s0; s < s1; ++s) {
    p.units[s].cum = cum;
    cum += p.units[s].w;
  }
  if (tid == 0) p.units[units].cum = all;
  __syncthreads();

  // Whole pairs: full waves of the longest, where none is longer than an SM's share.
  const long long pairs = (long long)units * p.Hkv, share = all * p.Hkv / sms;
  const int whole = wmax <= share ? (int)(pairs / sms * sms) : 0;
  const auto line_of = [&](long long x) {
    const int s = (int)(x / p.Hkv);
    return p.units[s].cum * p.Hkv + (s < units ? (x - (long long)s * p.Hkv) * p.units[s].w : 0);
  };
  const long long line0 = line_of(whole), line = all * p.Hkv - line0;
  // Runs: one per SM; more where the whole pairs before them differ, so that the SMs that are done
  // earlier take more.
  const long long len = line / sms + 1;
  const int split = whole ? (int)min((long long)MAX_SPLIT, 1 + 2ll * (wmax - wmin_s) / len) : 1;
  const int runs = line ? (int)max(1ll, min((long long)split * sms, line / MIN_RUN)) : 0;
  for (long long x = whole + tid; x < pairs; x += PLAN_THREADS) {
    const int s = (int)(x / p.Hkv), h = (int)(x - (long long)s * p.Hkv);
    const long long at = line_of(x) - line0;
    const int first = run_of(line, runs, at), last = run_of(line, runs, at + p.units[s].w - 1);
    if (first != last) p.joins[atomicAdd(&joins_s, 1)] = TileJoin{s, h, first, last - first + 1};
  }
  __syncthreads();
  if (tid == 0) *p.queue = TileQueue{0u, whole, runs, joins_s, units, line0, line};
}

// ------------------------------------------------------------------ load warp
template <int D>
__device__ __forceinline__ void tile_load_role(const TileParams& p, uint32_t base, uint8_t* gbase, volatile int* abort_flag, int lane) {
  using L = TileLayout<D>;
  const uint32_t to = p.timeout_us;
  const uint32_t bars = base + L::OFF_BAR;
  volatile TileHdr* hdr = reinterpret_cast<volatile TileHdr*>(gbase + L::OFF_HDR);
  uint32_t q_empty_par = (1u << L::QBUF) - 1u, q_pend = 0, q_pend_par = 0;
  int kslot = 0, vslot = 0, ie = 0;
  uint32_t kpar = 1, vpar = 1, ie_par = 1;
  uint32_t kpend = 0, kpend_par = 0, vpend = 0, vpend_par = 0;
  bool inject = p.inject != 0;
  const int whole = p.queue->whole, runs = p.queue->runs;
  // the lane's box of a key tile: chunk of box_rows keys, 64-column half
  const int nbox = BN / p.box_rows * L::HALVES;
  const int chunk = lane / L::HALVES, half = lane % L::HALVES;

  unsigned int q_next = 0;
  if (lane == 0) q_next = atomicAdd(&p.queue->next, 1u);
  int s = 0, h = 0, run = 0;  // unit (in the plan's order), head; run being worked off
  long long left = 0;         // tiles of the run that are left
  for (int k = 0;; ++k) {
    TileUnit pt;
    int slot = -1, from = 0, tiles;  // this piece: tiles from .. from + tiles of the unit
    if (left > 0) {
      // the run's next unit
      if (++h == p.Hkv) {
        h = 0;
        ++s;
      }
      pt = p.units[s];
      tiles = (int)min((long long)pt.w, left);
      left -= tiles;
      if (tiles < pt.w) slot = 2 * run + 1;
    } else {
      const unsigned int x = __shfl_sync(0xffffffffu, q_next, 0);
      if (x >= (unsigned int)(whole + runs)) {
        if (!bwait_warp(bars + 8u * (L::B_IEMPTY + ie), ie_par, abort_flag, to)) goto drain;
        if (lane == 0) {
          hdr[ie].j = -1;
          hdr[ie].flags = FLAG_EXIT;
          mbar_arrive(bars + 8u * (L::B_IFULL + ie));
        }
        __syncwarp();
        break;
      }
      if (lane == 0) q_next = atomicAdd(&p.queue->next, 1u);
      if (x < (unsigned int)whole) {
        s = (int)(x / p.Hkv);
        h = (int)(x % p.Hkv);
        pt = p.units[s];
        tiles = pt.w;
      } else {
        run = (int)x - whole;
        const long long line = p.queue->line, at = run_begin(line, runs, run);
        left = run_begin(line, runs, run + 1) - at;
        const long long pos = p.queue->line0 + at;
        // the last unit whose pairs begin at or before pos, 32 probes at a time
        int lo = whole / p.Hkv, hi = p.queue->units;
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
          const unsigned int yes = __ballot_sync(0xffffffffu, probe < hi && p.units[probe].cum * p.Hkv <= pos);
          lo += (31 - __clz(yes)) * step;  // (lane 0 always says yes)
          hi = min(hi, lo + step);
        }
        s = lo;
        pt = p.units[s];
        const long long in = pos - pt.cum * p.Hkv;
        h = (int)(in / pt.w);
        from = (int)(in - (long long)h * pt.w);
        tiles = (int)min((long long)(pt.w - from), left);
        left -= tiles;
        if (tiles < pt.w) slot = from == 0 ? 2 * run + 1 : 2 * run;
      }
    }
    const int j0 = pt.j0 + from, j1 = j0 + tiles;
    int row0, sq, sk, lo, hi;
    request_span(p, pt.b, row0, sq, sk);
    tile_keys(p, sq, sk, pt.blk, 0, QT, lo, hi);
    int jlo[QT], jhi[QT];  // key tiles of each Q tile, [jlo, jhi)
    bool rows1 = false;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      int a, e;
      const bool any = tile_keys(p, sq, sk, pt.blk, t, t + 1, a, e);
      if (t == 1) rows1 = any;
      jlo[t] = a / BN;
      jhi[t] = (e + BN - 1) / BN;
    }
    const int tok0 = pt.blk * QT * p.T;
    const int* table = p.table + (long long)pt.b * p.table_stride;

    const int qbuf = k % L::QBUF;
    if (!bwait_warp(bars + 8u * (L::B_QEMPTY + qbuf), (q_empty_par >> qbuf) & 1u, abort_flag, to)) goto drain;
    q_empty_par ^= 1u << qbuf;
    if (!inject) {
      if (lane == 0) {
        const uint32_t fb = bars + 8u * (L::B_QFULL + qbuf);
        mbar_expect_tx(fb, (uint32_t)((rows1 ? 2 : 1) * p.T * p.g * D * 2));
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int hh = 0; hh < L::HALVES; ++hh)
            if (t == 0 || rows1)
              tma_load_4d(base + L::OFF_Q + qbuf * L::Q_BUF_BYTES + t * L::Q_TILE_BYTES + hh * BM * 128, &p.tm_q, fb, hh * 64, 0,
                          row0 + tok0 + t * p.T, h);
      }
      q_pend |= 1u << qbuf;
      q_pend_par = (q_pend_par & ~(1u << qbuf)) | ((((q_empty_par >> qbuf) & 1u)) << qbuf);
    }
    inject = false;

    const auto describe = [&](int j, int flags) {
      hdr[ie].j = j;
      hdr[ie].flags = flags;
      hdr[ie].row0 = row0;
      hdr[ie].sq = sq;
      hdr[ie].sk = sk;
      hdr[ie].h = h;
      hdr[ie].blk = pt.blk;
      hdr[ie].slot = slot;
      hdr[ie].lo = lo;
      hdr[ie].hi = hi;
      mbar_arrive(bars + 8u * (L::B_IFULL + ie));
    };
    // page and row of the lane's box of key tile j; the page past the last one where no row sees its keys
    const auto place = [&](int j, int& page, int& row) {
      const int key = j * BN + chunk * p.box_rows;
      page = p.num_pages;
      row = 0;
      if (lane < nbox && key < hi && key + p.box_rows > lo) {
        const int idx = key / p.page_size;
        row = key - idx * p.page_size;
        page = __ldg(table + idx);
        if ((unsigned)page >= (unsigned)p.num_pages) {
          atomicOr(p.status, STATUS_PAGE);
          page = p.num_pages;
        }
      }
    };
    int page, row, page_next = 0, row_next = 0;
    place(j0, page_next, row_next);
    for (int j = j0; j < j1; ++j) {
      page = page_next;
      row = row_next;
      if (j + 1 < j1) place(j + 1, page_next, row_next);  // the table's latency passes behind this tile's loads
      const bool a0 = j >= jlo[0] && j < jhi[0], a1 = j >= jlo[1] && j < jhi[1];
      if (!a0 && !a1) continue;
      if (!bwait_warp(bars + 8u * (L::B_IEMPTY + ie), ie_par, abort_flag, to)) goto drain;
      if (lane == 0) describe(j, (a0 ? 1 : 0) | (a1 ? 2 : 0) | (lo > j * BN || hi < (j + 1) * BN ? FLAG_SCRUB : 0));
      __syncwarp();
      if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }

      if (!bwait_warp(bars + 8u * (L::B_KEMPTY + kslot), kpar, abort_flag, to)) goto drain;
      {
        const uint32_t fb = bars + 8u * (L::B_KFULL + kslot);
        if (lane == 0) mbar_expect_tx(fb, L::KV_TILE_BYTES);
        __syncwarp();
        if (lane < nbox)
          tma_load_4d(base + L::OFF_K + kslot * L::KV_TILE_BYTES + half * BN * 128 + chunk * p.box_rows * 128, &p.tm_k, fb, half * 64, row, h,
                      page);
      }
      kpend |= 1u << kslot;
      kpend_par = (kpend_par & ~(1u << kslot)) | ((kpar ^ 1u) << kslot);
      if (++kslot == L::KSLOT) { kslot = 0; kpar ^= 1u; }
      if (!bwait_warp(bars + 8u * (L::B_VEMPTY + vslot), vpar, abort_flag, to)) goto drain;
      {
        const uint32_t fb = bars + 8u * (L::B_VFULL + vslot);
        if (lane == 0) mbar_expect_tx(fb, L::KV_TILE_BYTES);
        __syncwarp();
        if (lane < nbox)
          tma_load_4d(base + L::OFF_V + vslot * L::KV_TILE_BYTES + half * BN * 128 + chunk * p.box_rows * 128, &p.tm_v, fb, half * 64, row, h,
                      page);
      }
      vpend |= 1u << vslot;
      vpend_par = (vpend_par & ~(1u << vslot)) | ((vpar ^ 1u) << vslot);
      if (++vslot == L::VSLOT) { vslot = 0; vpar ^= 1u; }
    }
    if (!bwait_warp(bars + 8u * (L::B_IEMPTY + ie), ie_par, abort_flag, to)) goto drain;
    if (lane == 0) describe(-1, FLAG_END);
    __syncwarp();
    if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }
  }
  return;

drain:
  // Aborted: let the copies this warp started land before the CTA exits.
  if (lane == 0) {
    for (int s = 0; s < L::KSLOT; ++s)
      if ((kpend >> s) & 1u) wait_drain(bars + 8u * (L::B_KFULL + s), (kpend_par >> s) & 1u);
    for (int s = 0; s < L::VSLOT; ++s)
      if ((vpend >> s) & 1u) wait_drain(bars + 8u * (L::B_VFULL + s), (vpend_par >> s) & 1u);
    for (int s = 0; s < L::QBUF; ++s)
      if ((q_pend >> s) & 1u) wait_drain(bars + 8u * (L::B_QFULL + s), (q_pend_par >> s) & 1u);
  }
  __syncwarp();
}

// What the MMA warp does beside its multiplications: it zeroes the rows of a V tile that no query row
// of the unit sees (past the last key, ahead of the window), which may hold anything; their weights are 0,
// and 0 * NaN would not be.
template <int D>
struct TileEnv {
  static constexpr bool SCRUB = true;
  int lo = 0, hi = 0;
  __device__ __forceinline__ void unit(volatile TileHdr& h) {
    lo = h.lo;
    hi = h.hi;
  }
  __device__ __forceinline__ void computed(int, int, int) {}
  __device__ __forceinline__ void scrub(int flags, int j, uint8_t* v, int lane) {
    if (!(flags & FLAG_SCRUB)) return;
    const int r0 = lo - j * BN, r1 = hi - j * BN;
    for (int r = lane >> 3; r < BN; r += 4) {
      if (r >= r0 && r < r1) continue;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
        *reinterpret_cast<uint4*>(v + hh * BN * 128 + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
};

// ------------------------------------------------------------------ softmax warpgroup t
template <int D, bool BF16>
__device__ __forceinline__ void tile_softmax_role(const TileParams& p, uint32_t base, uint8_t* gbase, volatile int* abort_flag, uint32_t tmem,
                                                  int t, int quarter, int lane) {
  using L = TileLayout<D>;
  const uint32_t to = p.timeout_us;
  const uint32_t bars = base + L::OFF_BAR;
  volatile TileHdr* hdr = reinterpret_cast<volatile TileHdr*>(gbase + L::OFF_HDR);
  const int r = quarter * 32 + lane;
  const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
  const uint32_t o_addr = tmem + lane_off + L::O_COL + t * L::O_STRIDE;
  const float c = p.scale_log2;
  // packed row -> token of the tile, head of the group; rows past T g stand in for the last one
  const int rr = min(r, p.T * p.g - 1), my_tok = rr / p.g;

  uint32_t s_par = 0, o_par = 0, ie_par = 0;
  int ie = 0, nq = 0, np = 0;

  for (int k = 0;; ++k) {
    if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) return;
    if (hdr[ie].flags & FLAG_EXIT) {
      mbar_arrive(bars + 8u * (L::B_IEMPTY + ie));
      break;
    }
    const int row0 = hdr[ie].row0, sq = hdr[ie].sq, h = hdr[ie].h, slot_out = hdr[ie].slot;
    const int tok0 = (hdr[ie].blk * QT + t) * p.T;  // the tile's first token
    const int sk = hdr[ie].sk;
    const int i = min(tok0 + my_tok, sq - 1);
    const int klo = row_lo(p, i, sk - sq), khi = row_hi(p, i, sk - sq, sk);
    float m = -INFINITY, l = 0.f;
    int nact = 0;

    while (true) {
      if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) return;
      const int j = hdr[ie].j;
      const int flags = hdr[ie].flags;
      const bool end = (flags & FLAG_END) != 0;
      const bool act = !end && ((flags >> t) & 1);
      mbar_arrive(bars + 8u * (L::B_IEMPTY + ie));
      if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }
      if (end) break;
      int slot = t;
      uint32_t spar = s_par;
      if constexpr (L::RING) {
        const int before = nq + ((t == 1 && (flags & 1)) ? 1 : 0);
        slot = before % L::S_SLOTS;
        spar = (uint32_t)(before / L::S_SLOTS) & 1u;
        nq += (flags & 1) + ((flags >> 1) & 1);
      }
      if (!act) continue;
      const uint32_t s_addr = tmem + lane_off + slot * 128;
      if (!bwait_warp(bars + 8u * (L::B_STILE + slot), spar, abort_flag, to)) return;
      if constexpr (!L::RING) s_par ^= 1u;
      tc_fence_after();
      const auto make_mask = [&] {
        const int hi = khi - j * BN, lo = klo - j * BN;
        const bool edge = __any_sync(0xffffffffu, hi < BN || lo > 0);
        return [=](uint32_t(&x)[64], int c0) {
          if (edge) {
#pragma unroll
            for (int cc = 0; cc < 64; ++cc)
              if (c0 + cc >= hi || c0 + cc < lo) x[cc] = __float_as_uint(-INFINITY);
          }
        };
      };
      if (!softmax_tile<D, BF16, L>(s_addr, o_addr, c, make_mask, bars + 8u * (L::B_OPV + t), np, nact, abort_flag, to, m, l)) return;
      tc_fence_before();
      if constexpr (L::RING) named_bar_sync(1 + t, BM);
      mbar_arrive(bars + 8u * (L::B_PREADY + t));
      ++nact;
      ++np;
    }

    // Epilogue.  A whole unit writes O / l and LSE, a part its unscaled O in 32 bits, m and l.
    if (nact > 0) {
      if (!bwait_warp(bars + 8u * (L::B_ODONE + t), o_par, abort_flag, to)) return;
      o_par ^= 1u;
      tc_fence_after();
    }
    const int rows = min(p.T, sq - tok0) * p.g;  // of this tile (may be <= 0)
    const bool row_ok = r < rows;
    if (slot_out >= 0) {
      const long long at = (long long)slot_out * UNIT_ROWS + t * BM + r;
      float* dst = p.part_o + at * D;
#pragma unroll
      for (int ch = 0; ch < D / 16; ++ch) {
        uint32_t ob[16];
        if (nact > 0) {
          tmem_ld32x32b_x16_wait(o_addr + ch * 16, ob);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) ob[x] = 0u;
        }
        if (row_ok) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(dst + ch * 16 + x * 4) = make_uint4(ob[4 * x], ob[4 * x + 1], ob[4 * x + 2], ob[4 * x + 3]);
        }
      }
      if (row_ok) p.part_ml[at] = make_float2(m, l);
      if (L::STAGE_O && lane == 0) mbar_arrive(bars + 8u * (L::B_QEMPTY + (k % L::QBUF)));
      continue;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    // The warp's 32 rows go through a slice of shared memory, 128 bytes of every row at a time (d = 64: the
    // unit's Q buffer, whose last reader is done; a tile that computed nothing has not waited for its Q
    // load, and writes zeros without it), and are written out a whole 128-byte segment to eight lanes.
    const bool staged = !L::STAGE_O || nact > 0;
    uint8_t* stage = L::STAGE_O ? gbase + L::OFF_Q + (k % L::QBUF) * L::Q_BUF_BYTES + (t * 4 + quarter) * (32 * 128)
                                : gbase + L::OFF_STAGE + (t * 4 + quarter) * (32 * 128);
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      if (staged) {
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t ob[16];
          if (nact > 0) {
            tmem_ld32x32b_x16_wait(o_addr + hh * 64 + ch * 16, ob);
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) ob[x] = 0u;
          }
          uint32_t pk[8];
#pragma unroll
          for (int x = 0; x < 8; ++x)
            pk[x] = pack2<BF16>(__uint_as_float(ob[2 * x]) * inv, __uint_as_float(ob[2 * x + 1]) * inv);
#pragma unroll
          for (int hc = 0; hc < 2; ++hc) {
            const int cc = 2 * ch + hc;
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((cc ^ (lane & 7)) * 16)) =
                make_uint4(pk[4 * hc], pk[4 * hc + 1], pk[4 * hc + 2], pk[4 * hc + 3]);
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int q = kk * 4 + lane / 8, cc = lane % 8, row = quarter * 32 + q;
        if (row < rows) {
          const uint4 val = staged ? *reinterpret_cast<const uint4*>(stage + q * 128 + ((cc ^ (q & 7)) * 16)) : make_uint4(0u, 0u, 0u, 0u);
          const int tok = row / p.g, head = h * p.g + row - tok * p.g;
          *reinterpret_cast<uint4*>(p.o + (long long)(row0 + tok0 + tok) * p.o_row + (long long)head * p.o_head + hh * 64 + cc * 8) = val;
        }
      }
      __syncwarp();
    }
    if constexpr (L::STAGE_O) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8u * (L::B_QEMPTY + (k % L::QBUF)));
    }
    if (row_ok && p.lse)
      p.lse[(long long)(h * p.g + r - my_tok * p.g) * p.total_q + row0 + tok0 + my_tok] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
  }
}

// ------------------------------------------------------------------ the kernel
template <int D, bool BF16>
__global__ void __launch_bounds__(NTHREADS, 1) paged_tile_kernel(const __grid_constant__ TileParams p) {
  using L = TileLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + L::OFF_BAR;

  if (threadIdx.x == 0) {
    init_barriers<L>(bars);
    abort_flag[0] = 0;
    *reinterpret_cast<unsigned int* volatile*>(abort_flag + 1) = p.status;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&p.tm_q);
    tma_prefetch_map(&p.tm_k);
    tma_prefetch_map(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the plan

  if (warp < 4) {
    setmaxnreg_dec<L::REGS_LOADMMA>();
    if (warp == 0) {
      tile_load_role<D>(p, base, gbase, abort_flag, lane);
    } else if (warp == 1) {
      TileEnv<D> env;
      mma_role<D, BF16, L>(env, p.timeout_us, base, gbase, abort_flag, tmem, lane);
    }
  } else {
    setmaxnreg_inc<L::REGS_SOFTMAX>();
    tile_softmax_role<D, BF16>(p, base, gbase, abort_flag, tmem, (warp - 4) >> 2, warp & 3, lane);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ join
// One warp per row of a cut unit: out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k.  Memory-bound (the parts
// were just written and are largely in L2).
template <int D, bool BF16>
__global__ void __launch_bounds__(256) tile_join_kernel(const __grid_constant__ TileParams p) {
  constexpr int E = D / 32;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int rows = p.queue->njoins * UNIT_ROWS, nwarps = gridDim.x * 8;
  for (int x = blockIdx.x * 8 + (threadIdx.x >> 5); x < rows; x += nwarps) {
    const int row = x % UNIT_ROWS, rest = x / UNIT_ROWS;
    const TileJoin jn = p.joins[rest];
    const TileUnit un = p.units[jn.unit];
    const int h = jn.h, t = row / BM, r = row % BM;
    int row0, sq, sk;
    request_span(p, un.b, row0, sq, sk);
    const int tok0 = (un.blk * QT + t) * p.T;
    if (r >= min(p.T, sq - tok0) * p.g) continue;
    float m = -INFINITY, l = 0.f, acc[E] = {};
    for (int k = 0; k < jn.parts; ++k) {
      const long long at = (long long)(k == 0 ? 2 * jn.run + 1 : 2 * (jn.run + k)) * UNIT_ROWS + row;
      const float2 ml = p.part_ml[at];
      const float* src = p.part_o + at * D + lane * E;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = src[e];
      const float mn = fmaxf(m, ml.x);
      const float fa = m == -INFINITY ? 0.f : ex2_approx(m - mn), fb = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
      l = l * fa + ml.y * fb;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * fa + v[e] * fb;
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int tok = r / p.g, head = h * p.g + r - tok * p.g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (long long)(row0 + tok0 + tok) * p.o_row + (long long)head * p.o_head + lane * E);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dst[e] = pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[(long long)head * p.total_q + row0 + tok0 + tok] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
  }
}

// ------------------------------------------------------------------ host side
struct TilePlan {
  int T, max_units, max_runs;
  size_t off_units, off_joins, off_ml, off_o, bytes;
  TilePlan(const attn_fwd_paged_params_t& a, int sms) {
    const int g = a.Hq / a.Hkv;
    T = BM / g;
    const int longest = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
    // units of a head: every request's tokens over 2 T, rounded up
    const long long by_rows = (long long)a.total_q / (QT * T) + a.B;
    const long long by_len = (long long)a.B * ((longest + QT * T - 1) / (QT * T));
    max_units = (int)(by_rows < by_len ? by_rows : by_len);  // by_rows <= total_q / 2 + B
    max_runs = MAX_SPLIT * sms;
    const size_t slots = 2 * (size_t)max_runs;
    off_units = 256;
    off_joins = off_units + round256((size_t)(max_units + 1) * sizeof(TileUnit));
    off_ml = off_joins + round256((size_t)max_runs * sizeof(TileJoin));
    off_o = off_ml + round256(slots * UNIT_ROWS * sizeof(float2));
    bytes = off_o + round256(slots * UNIT_ROWS * a.d * sizeof(float));
  }
};

template <int D, bool BF16>
int launch_tiles(const TileParams& p, int sms, int dev, cudaStream_t st) {
  using L = TileLayout<D>;
  auto kern = paged_tile_kernel<D, BF16>;
  static std::atomic<unsigned long long> attr_set{0};  // bit per device
  const unsigned long long bit = 1ull << dev;
  if (!(attr_set.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_ALLOC) != cudaSuccess ||
        cudaFuncSetAttribute(tile_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 66 * 1024) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_set.fetch_or(bit);
  }
  tile_plan_kernel<<<1, PLAN_THREADS, ((size_t)p.B + 1) * sizeof(int), st>>>(p, sms);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = L::SMEM_ALLOC;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return ATTN_ERR_CUDA;
  cfg.gridDim = dim3(4 * sms);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tile_join_kernel<D, BF16>, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

size_t tile_workspace(const attn_fwd_paged_params_t& a, int sms) { return TilePlan(a, sms).bytes; }

int tile_launch(const PagedParams& base, const attn_fwd_paged_params_t& a, void* workspace, int sms, int dev, cudaStream_t st) {
  const TilePlan plan(a, sms);
  TileParams p = {};
  static_cast<PagedParams&>(p) = base;
  const bool bf16 = a.dtype == ATTN_BF16;
  p.T = plan.T;
  p.box_rows = 128;
  while (a.page_size % p.box_rows != 0) p.box_rows /= 2;
  // (the stride of a dimension of one entry is of no account: any valid one does)
  const auto stride = [&](long long s, int n) { return n > 1 ? s * 2 : (long long)a.d * 2; };
  const Map4 q{{a.d, p.g, a.total_q, a.Hkv},
               {stride(a.q_head_stride, p.g), stride(a.q_row_stride, a.total_q), stride(a.q_head_stride * p.g, a.Hkv)},
               {64, p.g, p.T, 1}};
  const Map4 kv{{a.d, a.page_size, a.Hkv, a.num_pages},
                {a.cache_row_stride * 2, stride(a.cache_head_stride, a.Hkv), stride(a.cache_page_stride, a.num_pages)},
                {64, p.box_rows, 1, 1}};
  int rc;
  if ((rc = host_map4(&p.tm_q, a.q, bf16, q)) != ATTN_OK || (rc = host_map4(&p.tm_k, a.k_cache, bf16, kv)) != ATTN_OK ||
      (rc = host_map4(&p.tm_v, a.v_cache, bf16, kv)) != ATTN_OK)
    return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.queue = reinterpret_cast<TileQueue*>(ws);
  p.units = reinterpret_cast<TileUnit*>(ws + plan.off_units);
  p.joins = reinterpret_cast<TileJoin*>(ws + plan.off_joins);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.max_units = plan.max_units;
  p.inject = host_take_inject();
  if (a.d == 64) return bf16 ? launch_tiles<64, true>(p, sms, dev, st) : launch_tiles<64, false>(p, sms, dev, st);
  return bf16 ? launch_tiles<128, true>(p, sms, dev, st) : launch_tiles<128, false>(p, sms, dev, st);
}

}  // namespace attn
