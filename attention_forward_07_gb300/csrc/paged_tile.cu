// paged_tile.cu -- chunks of many rows: the tcgen05 path of attn_fwd_paged.
//
// The rows of a request's K/V head are packed token by token, the group's heads side by side, so
// one stream of keys serves the whole group: a Q tile holds T = 128 / g tokens of all g heads (T g <= 128
// rows), a unit two Q tiles.  The keys of a unit come through the block table: a 128-key tile is
// assembled from TMA boxes of up to page_size rows, which land in the 128-byte-swizzled tile that the
// MMA warp of roles.cuh expects.  Roles, TMEM and barriers are those of attn_fwd.cu.
//
// Work: a plan kernel weighs every unit by its key tiles, cuts units along the keys where they are too few
// or too unequal to fill the machine, and lists the parts longest first; the attention kernel takes them from
// a queue; the results of cut units are joined by a third kernel.
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

struct TileQueue {
  int nparts;          // entries of the list; each stands for Hkv parts
  unsigned int next;   // next (entry, head) to hand out
  int njoins;          // cut units to join, times heads
  int nslots;
};
struct TilePart {
  int b, blk;
  int j0, j1;   // key tiles
  int slot;     // -1: the whole unit; else partial result slot + h
  int pad[3];
};
struct TileJoin {
  int b, blk;
  int slot, parts;  // part k of head h in slot + k * Hkv + h
};

struct TileParams : PagedParams {
  CUtensorMap tm_q, tm_k, tm_v;
  int T;          // tokens of a Q tile
  int box_rows;   // rows of one K/V box
  TileQueue* queue;
  TilePart* parts;
  TileJoin* joins;
  int* weights;    // [units per head]
  float* part_o;   // [slots][256][D]
  float2* part_ml; // [slots][256]
  int max_units, max_slots;
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

// ------------------------------------------------------------------ plan
// One CTA.  Units are numbered request by request (requests of the other path have none); a unit's
// weight is its key tiles.  Cutting every unit into parts of at most c tiles costs about
//     ceil(parts / SMs) * (weight of a part + 2)   key-tile steps, a part's start and end counting as two
// (measured), two more where it is a piece whose result has to be joined; c is chosen among
// ceil(largest / k) for 32 values of k, one to a warp.
constexpr int PLAN_THREADS = 1024, PLAN_BINS = 1024;
constexpr int MIN_PART = 4;  // tiles of a piece

__device__ __forceinline__ int plan_cut(int warp) {  // 1 .. 16, then wider steps to 152
  return warp < 16 ? warp + 1 : warp < 24 ? 18 + 2 * (warp - 16) : warp < 28 ? 36 + 8 * (warp - 24) : 76 + 25 * (warp - 28);
}

__global__ void __launch_bounds__(PLAN_THREADS) tile_plan_kernel(const __grid_constant__ TileParams p, int sms) {
  grid_launch_dependents();
  extern __shared__ int pre[];  // units before each request, [B + 1]
  __shared__ int warp_sum[32], bins[PLAN_BINS];
  __shared__ float est_s[32];
  __shared__ int best_s, wmax_s, slots_s, joins_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_tokens = QT * p.T;
  const auto units_of = [&](int b) {
    int row0, sq, sk;
    request_span(p, b, row0, sq, sk);
    return sq * p.g > ROWS_MAX ? (sq + unit_tokens - 1) / unit_tokens : 0;
  };
  const int per = (p.B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int own = 0;
  for (int b = b0; b < b1; ++b) pre[b] = own, own += units_of(b);
  int incl = own;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) wmax_s = slots_s = joins_s = 0;
  bins[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sum[lane];
    int x = w;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    warp_sum[lane] = x - w;
    if (lane == 31) pre[p.B] = x;
  }
  __syncthreads();
  const int before = warp_sum[warp] + incl - own;
  for (int b = b0; b < b1; ++b) pre[b] += before;
  __syncthreads();
  const int units = min(pre[p.B], p.max_units);  // (more only where the row offsets overlap)
  const auto find = [&](int u) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const auto key_tiles = [&](int b, int blk, int& j0, int& j1) {
    int row0, sq, sk, lo, hi;
    request_span(p, b, row0, sq, sk);
    tile_keys(p, sq, sk, blk, 0, QT, lo, hi);
    j0 = lo / BN;
    j1 = (hi + BN - 1) / BN;
  };
  int wmax = 0;
  for (int u = tid; u < units; u += PLAN_THREADS) {
    const int b = find(u);
    int j0, j1;
    key_tiles(b, u - pre[b], j0, j1);
    p.weights[u] = j1 - j0;
    wmax = max(wmax, j1 - j0);
  }
  wmax = __reduce_max_sync(0xffffffffu, wmax);
  if (lane == 0) atomicMax(&wmax_s, wmax);
  __syncthreads();
  wmax = max(wmax_s, 1);
  const auto cap_of = [&](int k) { return max((wmax + k - 1) / k, min(wmax, MIN_PART)); };
  {
    const int c = cap_of(plan_cut(warp));
    long long w = 0;
    int n = 0, cut = 0;
    for (int u = lane; u < units; u += 32) {
      const int x = p.weights[u], m = max((x + c - 1) / c, 1);
      w += x;
      n += m;
      if (m > 1) cut += m;
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, s);
      n += __shfl_xor_sync(0xffffffffu, n, s);
      cut += __shfl_xor_sync(0xffffffffu, cut, s);
    }
    if (lane == 0) {
      const float parts = (float)n * p.Hkv, cost = ((float)w * p.Hkv + 2.f * parts + 2.f * (float)cut * p.Hkv) / fmaxf(parts, 1.f);
      const float waves = ceilf(parts / sms);
      const float est = fmaxf(waves * cost, (float)c + 2.f);
      est_s[warp] = (long long)cut * p.Hkv <= p.max_slots ? est : INFINITY;  // (k = 1 cuts nothing)
    }
  }
  __syncthreads();
  if (warp == 0) {
    float e = est_s[lane];
    int k = lane;
#pragma unroll
    for (int s = 16; s; s >>= 1) {
      const float e2 = __shfl_xor_sync(0xffffffffu, e, s);
      const int k2 = __shfl_xor_sync(0xffffffffu, k, s);
      if (e2 < e || (e2 == e && k2 < k)) e = e2, k = k2;
    }
    if (lane == 0) best_s = cap_of(plan_cut(k));
  }
  __syncthreads();
  const int c = best_s;
  // counting sort of the parts, longest first
  const auto bin_of = [&](int x, int m) { return PLAN_BINS - 1 - (int)((long long)((x + m - 1) / m) * (PLAN_BINS - 1) / c); };
  for (int u = tid; u < units; u += PLAN_THREADS) {
    const int x = p.weights[u], m = max((x + c - 1) / c, 1);
    atomicAdd(&bins[bin_of(x, m)], m);
  }
  __syncthreads();
  {
    const int x = bins[tid];
    int in = x;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in, s);
      if (lane >= s) in += y;
    }
    if (lane == 31) warp_sum[warp] = in;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    bins[tid] = base + in - x;
  }
  __syncthreads();
  for (int u = tid; u < units; u += PLAN_THREADS) {
    const int b = find(u), blk = u - pre[b];
    int j0, j1;
    key_tiles(b, blk, j0, j1);
    const int x = j1 - j0, m = max((x + c - 1) / c, 1);
    const int at = atomicAdd(&bins[bin_of(x, m)], m);
    int slot = -1;
    if (m > 1) {
      slot = atomicAdd(&slots_s, m * p.Hkv);
      p.joins[atomicAdd(&joins_s, 1)] = TileJoin{b, blk, slot, m};
    }
    for (int k = 0; k < m; ++k)
      p.parts[at + k] = TilePart{b, blk, j0 + (int)((long long)x * k / m), j0 + (int)((long long)x * (k + 1) / m),
                                 m > 1 ? slot + k * p.Hkv : -1, {0, 0, 0}};
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int w = 0; w < 32; ++w) n += warp_sum[w];
    *p.queue = TileQueue{n, 0u, joins_s * p.Hkv, slots_s};
  }
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
  const unsigned int total = (unsigned int)p.queue->nparts * p.Hkv;
  // the lane's box of a key tile: chunk of box_rows keys, 64-column half
  const int nbox = BN / p.box_rows * L::HALVES;
  const int chunk = lane / L::HALVES, half = lane % L::HALVES;

  unsigned int q_next = 0;
  if (lane == 0) q_next = atomicAdd(&p.queue->next, 1u);
  for (int k = 0;; ++k) {
    const unsigned int x = __shfl_sync(0xffffffffu, q_next, 0);
    if (x >= total) {
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
    const TilePart pt = p.parts[x / p.Hkv];
    const int h = (int)(x % p.Hkv);
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
    const int slot = pt.slot < 0 ? -1 : pt.slot + h;
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
    if (pt.j0 < pt.j1) place(pt.j0, page_next, row_next);
    for (int j = pt.j0; j < pt.j1; ++j) {
      page = page_next;
      row = row_next;
      if (j + 1 < pt.j1) place(j + 1, page_next, row_next);  // the table's latency passes behind this tile's loads
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
    const TileJoin jn = p.joins[rest / p.Hkv];
    const int h = rest % p.Hkv, t = row / BM, r = row % BM;
    int row0, sq, sk;
    request_span(p, jn.b, row0, sq, sk);
    const int tok0 = (jn.blk * QT + t) * p.T;
    if (r >= min(p.T, sq - tok0) * p.g) continue;
    float m = -INFINITY, l = 0.f, acc[E] = {};
    for (int k = 0; k < jn.parts; ++k) {
      const long long at = (long long)(jn.slot + k * p.Hkv + h) * UNIT_ROWS + row;
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
  int T, max_units, max_slots, max_parts;
  size_t off_parts, off_joins, off_weights, off_ml, off_o, bytes;
  TilePlan(const attn_fwd_paged_params_t& a, int sms) {
    const int g = a.Hq / a.Hkv;
    T = BM / g;
    const int longest = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
    // units of a head: every request's tokens over 2 T, rounded up
    const long long by_rows = (long long)a.total_q / (QT * T) + a.B;
    const long long by_len = (long long)a.B * ((longest + QT * T - 1) / (QT * T));
    max_units = (int)(by_rows < by_len ? by_rows : by_len);  // by_rows <= total_q / 2 + B
    max_slots = 4 * sms;  // room for as many pieces
    max_parts = max_units + max_slots;
    off_parts = 256;
    off_joins = off_parts + round256((size_t)max_parts * sizeof(TilePart));
    off_weights = off_joins + round256((size_t)max_slots * sizeof(TileJoin));
    off_ml = off_weights + round256((size_t)max_units * sizeof(int));
    off_o = off_ml + round256((size_t)max_slots * UNIT_ROWS * sizeof(float2));
    bytes = off_o + round256((size_t)max_slots * UNIT_ROWS * a.d * sizeof(float));
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
  const long long most = ((long long)p.max_units + p.max_slots) * p.Hkv;
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
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
  p.parts = reinterpret_cast<TilePart*>(ws + plan.off_parts);
  p.joins = reinterpret_cast<TileJoin*>(ws + plan.off_joins);
  p.weights = reinterpret_cast<int*>(ws + plan.off_weights);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.max_units = plan.max_units;
  p.max_slots = plan.max_slots;
  p.inject = host_take_inject();
  if (a.d == 64) return bf16 ? launch_tiles<64, true>(p, sms, dev, st) : launch_tiles<64, false>(p, sms, dev, st);
  return bf16 ? launch_tiles<128, true>(p, sms, dev, st) : launch_tiles<128, false>(p, sms, dev, st);
}

}  // namespace attn
