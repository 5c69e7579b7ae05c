// paged_tile.cu -- chunks of many rows: the tcgen05 path of attn_fwd_paged.
//
// The rows of a request's K/V head are packed token by token, the group's heads side by side, so
// one stream of keys serves the whole group: a Q tile holds T = 128 / g tokens of all g heads (T g <= 128
// rows), a unit two Q tiles.  The keys of a unit come through the block table: a 128-key tile is
// assembled from TMA boxes of up to page_size rows, which land in the 128-byte-swizzled tile that the
// MMA warp of roles.cuh expects.  Roles, TMEM and barriers are those of attn_fwd.cu.
//
// Work: the plan (in rows_kernel) weighs every unit by its key tiles and lists them longest first.  The
// kernel here takes from a queue first whole units, as many as give every SM the same number, then runs: the
// rest of the units laid end to end and cut into equal lengths, so no SM waits for another's last unit, and
// few units still fill the machine.  The results of cut units (at most two pieces to a run) are joined by
// join_kernel.
//
// The weights enter the second product rounded to the values' type, as in attn_fwd: half a step each,
// which adds as much to the error as the output's own rounding (bf16 0.0023 of the norm, 0.0017 without).
// A second product with what the rounding leaves would cost chunks half as much again, and a few tokens of 24
// requests 54 us against 41.
//
// Bound by: the tensor path for chunks.  2037 rows x 32 heads against 32k keys, d = 128, pages of 16: 0.71 ms, 1450
// TFLOP/s (0.76 of the measured burst peak; contiguous attn_fwd_ex on the same shape, in turn with it, 0.77 ms); four
// prompts of 4k rows 0.43 ms, 1280 TFLOP/s, of which a unit's start and end (one Q buffer at d = 128) take a tenth.  At
// d = 64 the softmax, with as many exponentials for half the flops: the chunk 0.64 ms (contiguous 0.63), the prompts 0.35.
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

constexpr int FLAG_SCRUB = 16;  // the key tile holds rows that no query row of the request sees: those outside
                                // [flags >> 8 & 255, flags >> 16 & 255)

struct TileHdr {
  int j, flags;
  int row0, sq, sk;
  int h, blk, slot;
};
static_assert(sizeof(TileHdr) == 32, "descriptor slot size");

template <int D>
using TileLayout = Layout<D, MASK_BAND, TileHdr, true>;

// Keys that any query row of a request sees.
__device__ __forceinline__ void request_keys(const TileParams& p, int sq, int sk, int& lo, int& hi) {
  lo = row_lo(p, 0, sk - sq);
  hi = row_hi(p, sq - 1, sk - sq, sk);
}

// The lane's box of key tile j of request b: chunk of box_rows keys, its place in the cache (z: page and
// head as one coordinate, row group in the page).  Boxes with no key of [lo, hi) lie past the last page and
// read as zeros, as do those whose page is out of range.
struct TileBox {
  int chunk, z, group;
  __device__ __forceinline__ TileBox(const TileParams& p, int b, int h, int j, int lo, int hi, int lane) {
    chunk = lane * p.box_rows;
    z = p.z_extent;
    group = 0;
    const int key = j * BN + chunk;
    if (chunk < BN && key < hi && key + p.box_rows > lo) {
      const int idx = key / p.page_size;
      const int page = p.table[(long long)b * p.table_stride + idx];
      group = (key - idx * p.page_size) >> 3;
      if ((unsigned)page < (unsigned)p.num_pages) z = page * p.z_page + h * p.z_head;
      else atomicOr(p.status, STATUS_PAGE);
    }
  }
  template <int D>
  __device__ __forceinline__ void load(const TileParams& p, const CUtensorMap* map, uint32_t dst, uint32_t full, int lane) const {
    if (lane == 0) mbar_expect_tx(full, BN * D * 2);
    __syncwarp();
    if (chunk < BN) tma_load_5d(dst + chunk * D * 2, map, full, 0, 0, 0, group, z);
    __syncwarp();
  }
};

// The last unit, from that of the first pair after `whole` ones on, whose pairs begin at or before step pos: 32 probes at a time.
__device__ __forceinline__ int unit_holding(const TileParams& p, int whole, long long pos, int lane) {
  int lo = whole / p.Hkv, hi = p.tile.queue->units;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
    const unsigned int yes = __ballot_sync(0xffffffffu, probe < hi && p.tile.units[probe].cum * p.Hkv <= pos);
    lo += (31 - __clz(yes)) * step;  // (lane 0 always says yes)
    hi = min(hi, lo + step);
  }
  return lo;
}

// ------------------------------------------------------------------ runs without a plan
// Where no request has more rows than a Q tile, every request is one unit, and the units in their own order
// do for equal runs, one to a CTA: each finds its own from the lengths, and the plan's kernel is not needed
// (24 requests of 3 - 6 tokens x 8 heads against up to 6k keys: 34.5 us, with the plan 39.3 (33.4 now); 4 requests of
// 6 tokens against 16k: 38 and 45).  A run's beginning: request, head, steps of the pair that lie before it.
struct RunStart {
  int b, h, runs;
  long long in, line, pos, left;  // (pos: the run's first step, left: its steps)
};
__device__ __forceinline__ bool request_unit(const TileParams& p, int b, TileUnit& x) {
  int k0, k1;
  request_span(p, b, x.row0, x.sq, x.sk);
  tile_keys(p, x.sq, x.sk, 0, 0, TILE_QT, k0, k1);
  x.b = b;
  x.blk = 0;
  x.j0 = k0 / TILE_KEYS;
  x.w = max((k1 + TILE_KEYS - 1) / TILE_KEYS - x.j0, 1);
  return x.sq > 0;
}
// By a warp; false where there are fewer runs.
__device__ __forceinline__ bool run_start(const TileParams& p, int run, int lane, RunStart& r) {
  const int per = (p.B + 31) / 32, b0 = min(lane * per, p.B), b1 = min(b0 + per, p.B);
  TileUnit x;
  long long own = 0;
  for (int b = b0; b < b1; ++b)
    if (request_unit(p, b, x)) own += x.w + UNIT_COST;
  own *= p.Hkv;
  long long incl = own;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += y;
  }
  r.line = __shfl_sync(0xffffffffu, incl, 31);
  r.runs = r.line ? (int)max(1ll, min((long long)p.tile.sms, r.line / MIN_RUN)) : 0;
  if (run >= r.runs) return false;
  r.pos = run_begin(r.line, r.runs, run);
  r.left = run_begin(r.line, r.runs, run + 1) - r.pos;
  const bool mine = r.pos >= incl - own && r.pos < incl;
  r.b = r.h = 0;
  r.in = 0;
  if (mine) {
    long long at = incl - own;
    for (int b = b0; b < b1; ++b) {
      if (!request_unit(p, b, x)) continue;
      const int steps = x.w + UNIT_COST;
      if (r.pos < at + (long long)steps * p.Hkv) {
        r.b = b;
        r.h = (int)((r.pos - at) / steps);
        r.in = r.pos - at - (long long)r.h * steps;
        break;
      }
      at += (long long)steps * p.Hkv;
    }
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  r.b = __shfl_sync(0xffffffffu, r.b, from);
  r.h = __shfl_sync(0xffffffffu, r.h, from);
  r.in = __shfl_sync(0xffffffffu, r.in, from);
  return true;
}

// ------------------------------------------------------------------ join list
// One warp of each CTA lists the cut pairs for join_kernel while the others work (the plan, which all wait
// for, was 2.5 - 4 us longer with it).  Each pair is found by the run that takes its second piece.
__device__ __forceinline__ void run_join_list(const TileParams& p, int lane) {  // (without a plan)
  const int r = blockIdx.x;
  TileJoin* list = p.tile.joins + r * JOINS_OF_RUN;
  RunStart rs;
  TileJoin jn = {};
  if (run_start(p, r, lane, rs)) {
    TileUnit un;
    request_unit(p, rs.b, un);
    const long long at = rs.pos - rs.in;  // where the pair begins
    const int first = run_of(rs.line, rs.runs, at + UNIT_COST), last = run_of(rs.line, rs.runs, at + un.w + UNIT_COST - 1);
    if (r == first + 1 && r <= last)
      jn = TileJoin{un.row0, lane * JOIN_ROWS, max(min(un.sq * p.g - lane * JOIN_ROWS, JOIN_ROWS), 0), rs.h, first, last - first + 1, lane * JOIN_ROWS, 0};
  }
  if (lane < JOINS_OF_RUN) list[lane] = jn;
}
__device__ __forceinline__ void tile_join_list(const TileParams& p, int lane) {
  TileQueue* q = p.tile.queue;
  const int whole = q->whole, runs = q->runs;
  const long long line0 = q->line0, line = q->line;
  for (int r = blockIdx.x; r < runs; r += gridDim.x) {
    const long long begin = run_begin(line, runs, r);
    const TileUnit un = p.tile.units[unit_holding(p, whole, line0 + begin, lane)];
    const int steps = un.w + UNIT_COST, h = (int)((line0 + begin - un.cum * p.Hkv) / steps);
    const long long at = un.cum * p.Hkv + (long long)h * steps - line0;  // where the pair begins
    const int first = run_of(line, runs, at + UNIT_COST), last = run_of(line, runs, at + steps - 1);
    if (r != first + 1 || r > last) continue;
    int n[TILE_QT], rows[TILE_QT];
#pragma unroll
    for (int t = 0; t < TILE_QT; ++t) {
      rows[t] = max(min(p.tile.T, un.sq - (un.blk * TILE_QT + t) * p.tile.T), 0) * p.g;
      n[t] = (rows[t] + JOIN_ROWS - 1) / JOIN_ROWS;
    }
    static_assert(TILE_QT * TILE_ROWS / JOIN_ROWS <= 32, "a lane to an entry");
    int to = 0;
    if (lane == 0) to = atomicAdd(&q->njoins, n[0] + n[1]);
    to = __shfl_sync(0xffffffffu, to, 0);
    if (lane < n[0] + n[1]) {
      const int t = lane >= n[0], k = lane - (t ? n[0] : 0);
      p.tile.joins[to + lane] = TileJoin{un.row0, (un.blk * TILE_QT + t) * p.tile.T * p.g + k * JOIN_ROWS, min(rows[t] - k * JOIN_ROWS, JOIN_ROWS), h,
                                         first, last - first + 1, t * TILE_ROWS + k * JOIN_ROWS, 0};
    }
  }
}

// ------------------------------------------------------------------ load warp
template <int D, bool TURNS>
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
  const bool no_plan = TURNS && p.tile.no_plan;
  bool begun = false;  // (without a plan)
  const unsigned int whole = no_plan ? 0 : p.tile.queue->whole, entries = no_plan ? 0 : whole + p.tile.queue->runs;

  // The first entry is the CTA's own number, later ones come from the queue, one ahead and no more (an SM
  // that held two would leave another without).  While a unit's first tiles load, the next entry and,
  // where it is a whole pair, its unit arrive.
  unsigned int x_next = blockIdx.x, raw = 0;
  TileUnit u_next = {};
  if (x_next < whole) u_next = p.tile.units[x_next / p.Hkv];
  bool asked = false;  // raw is on its way
  const auto fetch = [&] {
    if (!asked) return;
    x_next = __shfl_sync(0xffffffffu, raw, 0);
    if (x_next < whole) u_next = p.tile.units[x_next / p.Hkv];
    asked = false;
  };
  int s = 0, h = 0, run = 0;  // unit (in the plan's order), head; run being worked off
  long long left = 0;         // steps of the run that are left
  TileUnit pt;
  for (int k = 0;; ++k) {
    int slot = -1, from = 0, tiles = 0;  // this piece: tiles from .. from + tiles of the unit
    while (tiles == 0) {
      long long in = 0;  // steps of the pair that lie before the run
      if (left > 0) {
        // the run's next unit
        if (++h == p.Hkv) {
          h = 0;
          ++s;
          if (no_plan)
            while (s < p.B && !request_unit(p, s, pt)) ++s;
        }
        if (!no_plan) pt = p.tile.units[s];
      } else {
        const unsigned int x = x_next;
        RunStart rs;
        const bool more = no_plan ? !begun && run_start(p, blockIdx.x, lane, rs) : x < entries;
        if (!more) {
          if (!bwait_warp(bars + 8u * (L::B_IEMPTY + ie), ie_par, abort_flag, to)) goto drain;
          if (lane == 0) {
            hdr[ie].j = -1;
            hdr[ie].flags = FLAG_EXIT;
            mbar_arrive(bars + 8u * (L::B_IFULL + ie));
          }
          __syncwarp();
          return;
        }
        if (no_plan) {
          run = blockIdx.x;
          s = rs.b;
          h = rs.h;
          in = rs.in;
          left = rs.left;
          request_unit(p, s, pt);
          begun = true;
        } else {
          pt = u_next;
          if (lane == 0) raw = atomicAdd(&p.tile.queue->next, 1u);
          asked = true;
          if (x < whole) {
            h = (int)(x % p.Hkv);
            tiles = pt.w;
            break;
          }
          run = (int)(x - whole);
          const int runs = (int)(entries - whole);
          const long long line = p.tile.queue->line, at = run_begin(line, runs, run);
          left = run_begin(line, runs, run + 1) - at;
          const long long pos = p.tile.queue->line0 + at;
          s = unit_holding(p, (int)whole, pos, lane);
          pt = p.tile.units[s];
          in = pos - pt.cum * p.Hkv;
          h = (int)(in / (pt.w + UNIT_COST));
          in -= (long long)h * (pt.w + UNIT_COST);
        }
      }
      // the run's steps of the pair; none of its tiles where the run ends ahead of them
      const long long out = min(in + left, (long long)(pt.w + UNIT_COST));
      left -= out - in;
      from = (int)max(in - UNIT_COST, 0ll);
      tiles = (int)max(out - UNIT_COST, 0ll) - from;
      slot = tiles == pt.w ? -1 : from == 0 ? 2 * run + 1 : 2 * run;
      if (tiles == 0) fetch();
    }
    const int j0 = pt.j0 + from, j1 = j0 + tiles;
    const int row0 = pt.row0, sq = pt.sq, sk = pt.sk;
    int lo, hi;
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
    int scrub_lo, scrub_hi;
    request_keys(p, sq, sk, scrub_lo, scrub_hi);
    const int tok0 = pt.blk * QT * p.tile.T;

    const int qbuf = k % L::QBUF;
    if (!bwait_warp(bars + 8u * (L::B_QEMPTY + qbuf), (q_empty_par >> qbuf) & 1u, abort_flag, to)) goto drain;
    q_empty_par ^= 1u << qbuf;
    if (!inject) {
      if (lane == 0) {
        const uint32_t fb = bars + 8u * (L::B_QFULL + qbuf);
        mbar_expect_tx(fb, (uint32_t)((rows1 || TURNS ? 2 : 1) * p.tile.T * p.g * D * 2));
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int hh = 0; hh < L::HALVES; ++hh)
            if (t == 0 || rows1 || TURNS)
              tma_load_5d(base + L::OFF_Q + qbuf * L::Q_BUF_BYTES + t * L::Q_TILE_BYTES + hh * BM * 128, &p.tm_q, fb, hh * 64, 0,
                          row0 + tok0 + (TURNS ? 0 : t * p.tile.T), h, 0);
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
      mbar_arrive(bars + 8u * (L::B_IFULL + ie));
    };
    for (int j = j0; j < j1; ++j) {
      bool a0 = j >= jlo[0] && j < jhi[0], a1 = j >= jlo[1] && j < jhi[1];
      if (!a0 && !a1) continue;
      if constexpr (TURNS) {
        a1 = (j - j0) & 1;
        a0 = !a1;
      }
      const TileBox box(p, pt.b, h, j, lo, hi, lane);  // looked up while the slots are still taken
      if (!bwait_warp(bars + 8u * (L::B_IEMPTY + ie), ie_par, abort_flag, to)) goto drain;
      if (lane == 0) {
        int flags = (a0 ? 1 : 0) | (a1 ? 2 : 0);
        const int r0 = max(scrub_lo - j * BN, 0), r1 = min(scrub_hi - j * BN, BN);
        if (r0 > 0 || r1 < BN) flags |= FLAG_SCRUB | r0 << 8 | r1 << 16;
        describe(j, flags);
      }
      __syncwarp();
      if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }

      if (!bwait_warp(bars + 8u * (L::B_KEMPTY + kslot), kpar, abort_flag, to)) goto drain;
      box.load<D>(p, &p.tm_k, base + L::OFF_K + kslot * L::KV_TILE_BYTES, bars + 8u * (L::B_KFULL + kslot), lane);
      kpend |= 1u << kslot;
      kpend_par = (kpend_par & ~(1u << kslot)) | ((kpar ^ 1u) << kslot);
      if (++kslot == L::KSLOT) { kslot = 0; kpar ^= 1u; }
      if (!bwait_warp(bars + 8u * (L::B_VEMPTY + vslot), vpar, abort_flag, to)) goto drain;
      box.load<D>(p, &p.tm_v, base + L::OFF_V + vslot * L::KV_TILE_BYTES, bars + 8u * (L::B_VFULL + vslot), lane);
      vpend |= 1u << vslot;
      vpend_par = (vpend_par & ~(1u << vslot)) | ((vpar ^ 1u) << vslot);
      if (++vslot == L::VSLOT) { vslot = 0; vpar ^= 1u; }
      if (j > j0) fetch();
    }
    fetch();
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
// of the request sees (past the last key, ahead of the window), which may hold anything; their weights are
// 0, and 0 * NaN would not be.
template <int D, bool TURNS>
struct TileEnv {
  static constexpr bool SCRUB = true, BY_TURNS = TURNS;
  __device__ __forceinline__ void unit(volatile TileHdr&) {}
  __device__ __forceinline__ void computed(int, int, int) {}
  __device__ __forceinline__ void scrub(int flags, uint8_t* v, int lane) {
    if (!(flags & FLAG_SCRUB)) return;
    const int r0 = flags >> 8 & 255, r1 = flags >> 16 & 255;
    for (int r = lane >> 3; r < BN; r += 4) {
      if (r >= r0 && r < r1) continue;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
        *reinterpret_cast<uint4*>(v + (r >> 3) * TileLayout<D>::KV_SBO + hh * 1024 + (r & 7) * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
};

// ------------------------------------------------------------------ softmax warpgroup t
template <int D, bool BF16, bool TURNS>
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
  const auto token_of = [&](int row) { return (int)(row * p.g_inverse >> 16); };

  uint32_t s_par = 0, o_par = 0, ie_par = 0;
  int ie = 0, nq = 0, np = 0;
  // both softmax warpgroups: what either wrote before is seen by the other after
  const auto meet = [&](bool second) -> bool {
    tc_fence_before();
    mbar_arrive(bars + 8u * L::B_XCHG);
    if (!bwait_warp(bars + 8u * L::B_XCHG, (uint32_t)second, abort_flag, to)) return false;
    tc_fence_after();
    return true;
  };

  for (int k = 0;; ++k) {
    if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) return;
    if (hdr[ie].flags & FLAG_EXIT) {
      mbar_arrive(bars + 8u * (L::B_IEMPTY + ie));
      break;
    }
    const auto first_token = [&](int e) { return (hdr[e].blk * QT + (TURNS ? 0 : t)) * p.tile.T; };
    int klo, khi;
    {
      const int sq = hdr[ie].sq, sk = hdr[ie].sk, i = min(first_token(ie) + token_of(min(r, p.tile.T * p.g - 1)), sq - 1);
      klo = row_lo(p, i, sk - sq);
      khi = row_hi(p, i, sk - sq, sk);
    }
    int row0 = 0, sq = 0, h = 0, slot_out = 0, tok0 = 0;  // the unit's place, read at its end
    float m = -INFINITY, l = 0.f;
    int nact = 0;

    while (true) {
      if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) return;
      const int j = hdr[ie].j;
      const int flags = hdr[ie].flags;
      const bool end = (flags & FLAG_END) != 0;
      const bool act = !end && ((flags >> t) & 1);
      if (end) {
        row0 = hdr[ie].row0;
        sq = hdr[ie].sq;
        h = hdr[ie].h;
        slot_out = hdr[ie].slot;
        tok0 = first_token(ie);
      }
      mbar_arrive(bars + 8u * (L::B_IEMPTY + ie));
      if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }
      if (end) break;
      int slot = t;
      uint32_t spar = s_par;
      if constexpr (L::RING) {
        const int before = nq + ((t == 1 && (flags & 1)) ? 1 : 0);
        slot = before % L::S_SLOTS;
        spar = L::sp_parity(np);
        nq += (flags & 1) + ((flags >> 1) & 1);
      }
      if (!act) continue;
      const uint32_t s_addr = tmem + lane_off + slot * 128;
      if (!bwait_warp(bars + 8u * (L::B_STILE + L::sp_bar(t, np)), spar, abort_flag, to)) return;
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
      mbar_arrive(bars + 8u * (L::B_PREADY + L::sp_bar(t, np)));
      ++nact;
      ++np;
    }

    // Epilogue.  A whole unit writes O / l and LSE, a part its unscaled O in 32 bits, m and l.  Its loops are not
    // unrolled: it runs once a unit, and fetching its instructions took longer than a loop's turns do.
    if (nact > 0) {
      if (!bwait_warp(bars + 8u * (L::B_ODONE + t), o_par, abort_flag, to)) return;
      o_par ^= 1u;
      tc_fence_after();
    }
    const int rows = min(p.tile.T, sq - tok0) * p.g;  // of this tile (may be <= 0)
    const bool row_ok = r < rows;
    const int my_tok = token_of(r);
    const int part_row = (TURNS ? 0 : t * BM) + r;
    const long long part = (long long)slot_out * UNIT_ROWS + part_row;
    if constexpr (TURNS) {
      // Both Q tiles hold results of the same rows: they exchange m and l through shared memory (d = 128:
      // the staging area, d = 64: the Q buffer, whose reads are over), then each warpgroup joins and
      // writes half of the columns, reading both accumulators.  They meet before the exchange is read
      // and again before either goes on to the next unit.
      constexpr int XCH = L::STAGE_O ? L::OFF_Q : L::OFF_STAGE, XCH_T = L::STAGE_O ? L::Q_TILE_BYTES : 4 * 32 * 128;
      uint8_t* xch = gbase + XCH + (L::STAGE_O ? (k % L::QBUF) * L::Q_BUF_BYTES : 0);
      if constexpr (L::STAGE_O) {  // (a Q tile that computed nothing may still be loading)
        if (nact == 0 && !bwait_warp(bars + 8u * (L::B_QFULL + (k % L::QBUF)), (uint32_t)(k / L::QBUF) & 1u, abort_flag, to)) return;
      }
      reinterpret_cast<float2*>(xch + t * XCH_T)[r] = make_float2(m, l);
      if (!meet(false)) return;
      const float2 other = reinterpret_cast<const float2*>(xch + (1 - t) * XCH_T)[r];
      const float mm = fmaxf(m, other.x);
      const float f_own = m == -INFINITY ? 0.f : ex2_approx(m - mm), f_other = other.x == -INFINITY ? 0.f : ex2_approx(other.x - mm);
      const float ll = l * f_own + other.y * f_other;
      const float inv = slot_out >= 0 ? 1.f : ll == 0.f ? 0.f : 1.f / ll;
      const float fa = (t ? f_other : f_own) * inv, fb = (t ? f_own : f_other) * inv;
      const uint32_t both = tmem + lane_off + L::O_COL + t * (D / 2);
      const int head = h * p.g + r - my_tok * p.g;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t oa[16], ob[16];
        tmem_ld32x32b_x16_wait(both + ch * 16, oa);
        tmem_ld32x32b_x16_wait(both + L::O_STRIDE + ch * 16, ob);
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)  // (an accumulator that nothing has gone into holds anything)
          x[e] = (fa != 0.f ? fa * __uint_as_float(oa[e]) : 0.f) + (fb != 0.f ? fb * __uint_as_float(ob[e]) : 0.f);
        const int col = t * (D / 2) + ch * 16;
        if (row_ok && slot_out >= 0) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(p.tile.part_o + part_at<D>(slot_out, part_row, col + e)) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else if (row_ok) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + (long long)(row0 + tok0 + my_tok) * p.o_row + (long long)head * p.o_head + col);
          dst[0] = make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
          dst[1] = make_uint4(pack2<BF16>(x[8], x[9]), pack2<BF16>(x[10], x[11]), pack2<BF16>(x[12], x[13]), pack2<BF16>(x[14], x[15]));
        }
        __syncwarp();
      }
      if (t == 0 && row_ok) {
        if (slot_out >= 0) p.tile.part_ml[part] = make_float2(mm, ll);
        else if (p.lse) p.lse[(long long)head * p.total_q + row0 + tok0 + my_tok] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * LN2;
      }
      if (!meet(true)) return;
      if constexpr (L::STAGE_O) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8u * (L::B_QEMPTY + (k % L::QBUF)));
      }
      continue;
    }
    if (slot_out >= 0) {
#pragma unroll 1
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
            *reinterpret_cast<uint4*>(p.tile.part_o + part_at<D>(slot_out, part_row, ch * 16 + x * 4)) =
                make_uint4(ob[4 * x], ob[4 * x + 1], ob[4 * x + 2], ob[4 * x + 3]);
        }
      }
      if (row_ok) p.tile.part_ml[part] = make_float2(m, l);
      if (L::STAGE_O && lane == 0) mbar_arrive(bars + 8u * (L::B_QEMPTY + (k % L::QBUF)));
      continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    // The warp's 32 rows go through a slice of shared memory, 128 bytes of every row at a time (d = 64: the
    // unit's Q buffer, whose last reader is done; a tile that computed nothing has not waited for its Q
    // load, and writes zeros without it), and are written out a whole 128-byte segment to eight lanes.
    const bool staged = !L::STAGE_O || nact > 0;
    uint8_t* stage = L::STAGE_O ? gbase + L::OFF_Q + (k % L::QBUF) * L::Q_BUF_BYTES + (t * 4 + quarter) * (32 * 128)
                                : gbase + L::OFF_STAGE + (t * 4 + quarter) * (32 * 128);
    uint16_t* out[8];  // where the lane's segments of rows kk * 4 + lane / 8 go
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const int row = quarter * 32 + kk * 4 + lane / 8, tok = token_of(row), head = h * p.g + row - tok * p.g;
      out[kk] = p.o + (long long)(row0 + tok0 + tok) * p.o_row + (long long)head * p.o_head + lane % 8 * 8;
    }
#pragma unroll 1
    for (int hh = 0; hh < D / 64; ++hh) {
      if (staged) {
#pragma unroll 1
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
          *reinterpret_cast<uint4*>(out[kk] + hh * 64) = val;
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
      p.lse[(long long)(h * p.g + r - my_tok * p.g) * p.total_q + row0 + tok0 + my_tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
  }
}

// ------------------------------------------------------------------ the kernel
template <int D, bool BF16, bool TURNS>
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
  grid_launch_dependents();
  grid_dependency_wait();  // the plan

  if (warp < 4) {
    setmaxnreg_dec<L::REGS_LOADMMA>();
    if (warp == 0) {
      tile_load_role<D, TURNS>(p, base, gbase, abort_flag, lane);
    } else if (warp == 1) {
      TileEnv<D, TURNS> env;
      mma_role<D, BF16, L>(env, p.timeout_us, base, gbase, abort_flag, tmem, lane);
    } else if (warp == 2) {
      if (TURNS && p.tile.no_plan) run_join_list(p, lane);
      else tile_join_list(p, lane);
    }
  } else {
    setmaxnreg_inc<L::REGS_SOFTMAX>();
    tile_softmax_role<D, BF16, TURNS>(p, base, gbase, abort_flag, tmem, (warp - 4) >> 2, warp & 3, lane);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ host side
template <int D, bool BF16, bool TURNS>
int launch_tiles(const TileParams& p, int sms, int dev, cudaStream_t st) {
  using L = TileLayout<D>;
  auto kern = paged_tile_kernel<D, BF16, TURNS>;
  static std::atomic<unsigned long long> attr_set{0};  // bit per device
  const unsigned long long bit = 1ull << dev;
  if (!(attr_set.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_ALLOC) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_set.fetch_or(bit);
  }
  return launch_dependent(kern, dim3(sms), NTHREADS, L::SMEM_ALLOC, st, p);
}

}  // namespace

int tile_prepare(const PagedParams& base, const attn_fwd_paged_params_t& a, TileParams& p) {
  static_cast<PagedParams&>(p) = base;
  const bool bf16 = a.dtype == ATTN_BF16;
  p.box_rows = 128;
  while (a.page_size % p.box_rows != 0) p.box_rows /= 2;
  // (the stride of a dimension of one entry is of no account: any valid one does)
  const auto stride = [&](long long s, int n) { return n > 1 ? s * 2 : (long long)a.d * 2; };
  const Map5 q{{a.d, p.g, a.total_q, a.Hkv, 1},
               {stride(a.q_head_stride, p.g), stride(a.q_row_stride, a.total_q), stride(a.q_head_stride * p.g, a.Hkv), a.d * 2ll},
               {64, p.g, p.tile.T, 1, 1}};
  // 64 columns, 8 rows, halves, groups of 8 rows, and page and head in the smaller of their strides
  const long long sp = a.num_pages > 1 ? a.cache_page_stride : 0, sh = a.Hkv > 1 ? a.cache_head_stride : 0;
  const long long unit = sp && sh ? (sp < sh ? sp : sh) : sp + sh;
  p.z_page = unit ? (int)(sp / unit) : 0;
  p.z_head = unit ? (int)(sh / unit) : 0;
  p.z_extent = (a.num_pages - 1) * p.z_page + (a.Hkv - 1) * p.z_head + 1;
  const Map5 kv{{64, 8, a.d / 64, a.page_size / 8, p.z_extent},
                {a.cache_row_stride * 2, 128, a.cache_row_stride * 16, unit ? unit * 2 : a.d * 2ll},
                {64, 8, a.d / 64, p.box_rows / 8, 1}};
  int rc;
  if ((rc = host_map5(&p.tm_q, a.q, bf16, q)) != ATTN_OK || (rc = host_map5(&p.tm_k, a.k_cache, bf16, kv)) != ATTN_OK ||
      (rc = host_map5(&p.tm_v, a.v_cache, bf16, kv)) != ATTN_OK)
    return rc;
  p.g_inverse = 65536u / p.g + 1;
  p.inject = host_take_inject();
  return ATTN_OK;
}

int tile_launch(const TileParams& p, const attn_fwd_paged_params_t& a, int sms, int dev, cudaStream_t st) {
  const bool bf16 = a.dtype == ATTN_BF16;
  // Where no request has more rows than one Q tile, both Q tiles take the same rows and the key tiles by turns,
  // so that one's products run while the other's softmax does.  24 requests of 3 - 6 tokens x 8 heads
  // against up to 6k keys, when their start took longer: 45 us by turns, 51 with the second Q tile idle.
  const bool turns = p.max_q <= p.tile.T;
  const auto go = [&](auto launch) { return launch(p, sms, dev, st); };
  if (a.d == 64) {
    if (turns) return go(bf16 ? launch_tiles<64, true, true> : launch_tiles<64, false, true>);
    return go(bf16 ? launch_tiles<64, true, false> : launch_tiles<64, false, false>);
  }
  if (turns) return go(bf16 ? launch_tiles<128, true, true> : launch_tiles<128, false, true>);
  return go(bf16 ? launch_tiles<128, true, false> : launch_tiles<128, false, false>);
}

}  // namespace attn
