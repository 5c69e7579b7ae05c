// roles.cuh -- what the tcgen05 attention kernels share: shared-memory and TMEM layout, tile
// descriptors, bounded barrier waits, the MMA warp and the softmax of a key tile.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "host.h"
#include "ptx.cuh"

namespace attn {

constexpr int BM = 128;        // query rows per Q tile = TMEM lanes
constexpr int QT = 2;          // Q tiles per work unit
constexpr int UNIT_ROWS = BM * QT;
constexpr int BN = 128;        // keys per K/V tile
constexpr int NTHREADS = 384;  // 12 warps
constexpr int REGS_LAUNCH = 168;
constexpr int NINFO = 4;       // depth of the tile-descriptor ring
constexpr int TMEM_COLS = 512;
constexpr int FLAG_END = 4;    // info entry marking the end of a work unit
constexpr int FLAG_EXIT = 8;   // info entry telling the consumers that no unit is left
constexpr float LN2 = 0.69314718055994530942f;

// NONE: every key; CAUSAL: keys up to the aligned position; BAND: keys in
// [key_lo(i), key_hi(i)) per query row (sliding windows); CUSTOM: kept-bit words from the
// mask pre-pass (which folds any band in).  The first two keep their bounds cheap.
enum MaskMode { MASK_NONE = 0, MASK_CAUSAL = 1, MASK_CUSTOM = 2, MASK_BAND = 3 };

struct InfoHdr {
  int j;      // key tile index
  int flags;  // bit t: Q tile t computes this key tile; FLAG_END: end of unit
  int sq, sk;  // the unit's query and key lengths (per batch entry with seqlens arrays)
  int qoff;    // packed layouts: the entry's first row in q / o / lse
  int bh, qb;  // the work unit this entry belongs to: b * Hq + hq, 256-row block
  int pad;
};
static_assert(sizeof(InfoHdr) == 32, "descriptor slot size");

// GROUPED: the 64-column halves of K / V rows stand side by side for every 8 rows (128-byte swizzle
// atoms of 1024 bytes) instead of one half-tile behind the other, so that one TMA box brings both.
template <int D, int MODE, class HDR = InfoHdr, bool GROUPED = false>
struct Layout {
  using Hdr = HDR;
  static constexpr int KV_HALF = GROUPED ? 1024 : BN * 128;  // from a half to the next
  static constexpr int KV_SBO = GROUPED ? 1024 * (D / 64) : 1024;  // from 8 rows to the next 8
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int HALVES = D / 64;                  // 128-byte swizzle spans per row
  static constexpr int Q_TILE_BYTES = BM * D * 2;
  static constexpr int KV_TILE_BYTES = BN * D * 2;
  // d = 64 (short sequences, many units per CTA) double-buffers the Q tiles so the next
  // unit's Q load overlaps the current unit; d = 128 spends that room on K/V slots.
  static constexpr int QBUF = (D == 64) ? 2 : 1;
  // With two Q buffers a unit's buffer is not refilled before the unit after next, so its
  // epilogue can stage O there and write it out coalesced (8 softmax warps x 32 rows x d
  // fp16/bf16 = exactly one buffer); the buffer is released when those warps are done.
  static constexpr bool STAGE_O = (QBUF == 2);
  static constexpr int QEMPTY_COUNT = 1 + (STAGE_O ? QT * 4 : 0);  // MMA commit + softmax warps
  // TMEM.  d = 128: S_t (fp32, 128 columns) at t * 128, P_t (fp16/bf16 pairs) over its first 64
  // columns, O_t at 256 + t * 128.  d = 64: a ring of three S slots at 0, 128, 256 shared by the
  // two Q tiles (the n-th Q.K^T of the CTA goes to slot n % 3, its P over the slot's first 64
  // columns), O_t at 384 + t * 64: a Q tile's next Q.K^T runs while its softmax works on the
  // current one.
  static constexpr bool RING = (D == 64);
  static constexpr int S_SLOTS = RING ? 3 : QT;
  // Barriers that say S or P is there.  A wait tells a phase from the next one by one bit, so it has to be
  // within a phase of what it waits for.  d = 64: two barriers to a Q tile, its n-th S and P by turns.  Whoever
  // waits for the n-th has waited for the (n - 2)-th, and the (n + 2)-th is not made before it is done with
  // the n-th.  That holds for arrivals as well: a warp that is ahead arrives for its (n + 1)-th P at the other
  // barrier, and gets no (n + 2)-th S before all have arrived for the n-th P, so the four warps of a
  // warpgroup need not meet ahead of their arrival (a meeting would wait without limit for a warp that has
  // given up).  (With S barriers to ring slots a softmax might have passed over key tiles of the other Q
  // tile alone, and taken an earlier phase for its own; with one P barrier to a Q tile the MMA warp, where
  // it lost time between a Q.K^T and the wait for the P before, found two phases gone by.)
  static constexpr int SP_BARS = RING ? 2 * QT : QT;
  __device__ static __forceinline__ int sp_bar(int t, uint32_t n) { return RING ? 2 * t + (int)(n & 1u) : t; }
  __device__ static __forceinline__ uint32_t sp_parity(uint32_t n) { return (RING ? n >> 1 : n) & 1u; }
  static constexpr int O_COL = RING ? 384 : 256;
  static constexpr int O_STRIDE = RING ? 64 : 128;
  static_assert(S_SLOTS * 128 + QT * O_STRIDE <= TMEM_COLS, "TMEM columns");
  // Registers per thread after setmaxnreg: the load / MMA warpgroup and the two softmax
  // warpgroups share the launch's 384 x 168 (the ring bookkeeping of d = 64 costs the MMA
  // warp a few; its softmax, with a 64-column O, needs fewer).
  static constexpr int REGS_LOADMMA = (D == 64) ? 96 : 88;
  static constexpr int REGS_SOFTMAX = (D == 64) ? 200 : 208;
  static_assert(128 * REGS_LOADMMA + 256 * REGS_SOFTMAX <= NTHREADS * REGS_LAUNCH, "register split");
  // With one Q buffer (d = 128) the epilogue stages O through a 32 KiB area of its own,
  // 4 KiB per softmax warp, one 64-column half at a time (custom masks need that room for
  // their mask words and write O directly).
  static constexpr bool STAGE_SEP = (D == 128 && MODE != MASK_CUSTOM);
  static constexpr int STAGE_BYTES = STAGE_SEP ? QT * 4 * 32 * 128 : 0;
  // Separate K and V rings: K(j) is read by the two QK^T of tile j, V(j) by the two P.V
  // one tile later, so each ring is released right after its own last reader.
  static constexpr int KSLOT = (D == 128) ? 2 : 4;
  static constexpr int VSLOT = (D == 128) ? 2 : 4;
  static constexpr int OFF_Q = 0;
  static constexpr int Q_BUF_BYTES = QT * Q_TILE_BYTES;
  static constexpr int OFF_K = OFF_Q + QBUF * Q_BUF_BYTES;
  static constexpr int OFF_V = OFF_K + KSLOT * KV_TILE_BYTES;
  static constexpr int OFF_STAGE = OFF_V + VSLOT * KV_TILE_BYTES;
  static constexpr int OFF_WORDS = OFF_STAGE + STAGE_BYTES;
  static constexpr int WORDS_PER_ENTRY = UNIT_ROWS * (BN / 32);
  static constexpr int OFF_HDR = OFF_WORDS + (MODE == MASK_CUSTOM ? NINFO * WORDS_PER_ENTRY * 4 : 0);
  static constexpr int OFF_BAR = OFF_HDR + NINFO * (int)sizeof(HDR);
  // barrier indices
  static constexpr int B_QFULL = 0, B_QEMPTY = QBUF, B_KFULL = 2 * QBUF,
                       B_KEMPTY = B_KFULL + KSLOT, B_VFULL = B_KEMPTY + KSLOT,
                       B_VEMPTY = B_VFULL + VSLOT, B_IFULL = B_VEMPTY + VSLOT,
                       B_IEMPTY = B_IFULL + NINFO,
                       B_STILE = B_IEMPTY + NINFO, B_PREADY = B_STILE + SP_BARS,
                       B_ODONE = B_PREADY + SP_BARS, B_OPV = B_ODONE + QT, B_DRAIN = B_OPV + QT,
                       B_XCHG = B_DRAIN + 1, NBAR = B_XCHG + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM_ALLOC = BYTES + 1024;  // slack for 1024-byte alignment
  static_assert(SMEM_ALLOC <= 232448, "shared memory");
  // Over half of the SM's shared memory: one CTA per SM, so TMEM (512 columns) never
  // has to be shared between resident CTAs.
  static_assert(SMEM_ALLOC > 116 * 1024, "one CTA per SM");
};

// Slow path of a bounded barrier wait (inlined: a shared non-inlined callee cannot serve
// warps running under different setmaxnreg budgets).  Gives up when another thread has aborted, when
// the wait has lasted timeout_us, or after an iteration cap, and then aborts the CTA and marks the
// launch's status word (its address stands behind the flag, set at kernel start).
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       uint32_t timeout_us) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0; it < (1u << 28); ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if ((it & 15u) == 15u && globaltimer_ns() - t0 > 1000ull * timeout_us) break;
  }
  *abort_flag = 1;
  atomicOr(*reinterpret_cast<unsigned int* volatile*>(abort_flag + 1), STATUS_TIMEOUT);
  return false;
}

__device__ __forceinline__ bool bwait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                      uint32_t timeout_us) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort_flag, timeout_us);
}

// Warp-uniform variant: every lane waits, and the warp only proceeds if all lanes did.
__device__ __forceinline__ bool bwait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           uint32_t timeout_us) {
  bool ok = bwait(bar, parity, abort_flag, timeout_us);
  return __all_sync(0xffffffffu, ok);
}

// Wait used only while draining after an abort: ignores the abort flag, short limit.
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0; it < (1u << 24); ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 15u) == 15u && globaltimer_ns() - t0 > 200000000ull) return;
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// Initialises the barriers of a layout (one thread).  `readers`: threads that read the tile descriptors
// beside the MMA warp's one and the softmax threads.
template <class L>
__device__ __forceinline__ void init_barriers(uint32_t bars, int readers = 0) {
  for (int qb2 = 0; qb2 < L::QBUF; ++qb2) {
    mbar_init(bars + 8u * (L::B_QFULL + qb2), 1);
    mbar_init(bars + 8u * (L::B_QEMPTY + qb2), L::QEMPTY_COUNT);
  }
  for (int s = 0; s < L::KSLOT; ++s) {
    mbar_init(bars + 8u * (L::B_KFULL + s), 1);
    mbar_init(bars + 8u * (L::B_KEMPTY + s), 1);
  }
  for (int s = 0; s < L::VSLOT; ++s) {
    mbar_init(bars + 8u * (L::B_VFULL + s), 1);
    mbar_init(bars + 8u * (L::B_VEMPTY + s), 1);
  }
  for (int e = 0; e < NINFO; ++e) {
    mbar_init(bars + 8u * (L::B_IFULL + e), 1);                 // load-warp lane 0
    mbar_init(bars + 8u * (L::B_IEMPTY + e), 1 + QT * BM + readers);  // MMA thread + softmax threads
  }
  for (int b = 0; b < L::SP_BARS; ++b) {
    mbar_init(bars + 8u * (L::B_STILE + b), 1);
    mbar_init(bars + 8u * (L::B_PREADY + b), BM);
  }
  for (int t = 0; t < QT; ++t) {
    mbar_init(bars + 8u * (L::B_ODONE + t), 1);
    mbar_init(bars + 8u * (L::B_OPV + t), 1);
  }
  mbar_init(bars + 8u * L::B_DRAIN, 1);
  mbar_init(bars + 8u * L::B_XCHG, QT * BM);
}

// ------------------------------------------------------------------ MMA issuer (warp 1)
// The whole warp runs this code converged (descriptors in uniform registers); elect.sync
// picks the lane that issues each tcgen05 instruction.  Per tile descriptor e (key tile j)
// and Q tile t:
//   d = 128:  O_t (+)= P_t(prev) . V(prev)   once softmax t has written P for the previous tile,
//             S_t     = Q_t . K(j)^T         then signal softmax t;
//             S_t / P_t share TMEM columns, so S_t is rewritten only after the P.V that reads it.
//   d = 64:   S(n)    = Q_t . K(j)^T         into ring slot n % 3 (the CTA's n-th Q.K^T),
//             O_t (+)= P_t(prev) . V(prev)   from the slot of the previous tile's S,
//             so the next S of a Q tile is computed while its softmax still works on the
//             current one.  At most two slots hold an S or P whose P.V is not yet issued when
//             a Q.K^T is issued, so the third is free; each P.V is followed by a commit on
//             OPV(t), which the softmax waits for before it rescales O_t.
// Each ring slot of K / V is released by a commit right after its last reader.
// `env` is what differs between the kernels: env.unit(descriptor) at a unit's start, env.computed(t, j,
// lane) for every (Q tile, key tile) block, Env::BY_TURNS (see below), and, where Env::SCRUB, env.scrub(flags, V tile, lane) once V(j) has landed and before any P.V reads it.
template <int D, bool BF16, class L, class Env>
__device__ __forceinline__ void mma_role(Env& env, uint32_t to, uint32_t base, uint8_t* gbase,
                                         volatile int* abort_flag, uint32_t tmem, int lane) {
  using Hdr = typename L::Hdr;
  const uint32_t bars = base + L::OFF_BAR;
  volatile Hdr* hdr = reinterpret_cast<volatile Hdr*>(gbase + L::OFF_HDR);
  constexpr uint32_t ID_QK = idesc_f16acc32(BF16, false, false, BM, BN);
  constexpr uint32_t ID_PV = idesc_f16acc32(BF16, false, true, BM, D);

  uint32_t q_par = 0, ie_par = 0, kpar = 0, vpar = 0, pn0 = 0, pn1 = 0;  // q_par: bit per Q buffer; pn: P tiles taken
  int kslot = 0, vslot = 0, ie = 0;
  int nqk = 0;                 // d = 64: ring slot of the next Q.K^T
  uint32_t odd = 0;            // d = 64: bit t: Q tile t has had an odd number of them
  int pslot0 = 0, pslot1 = 0;  // d = 64: ring slot holding P_t of the previous key tile

  for (int k = 0;; ++k) {
    // the unit's first descriptor names it (the loop below waits on it again, at once)
    if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) goto drain;
    if (hdr[ie].flags & FLAG_EXIT) {
      mbar_arrive_elect(bars + 8u * (L::B_IEMPTY + ie));
      break;
    }
    env.unit(hdr[ie]);
    const int qbuf = k % L::QBUF;
    if (!bwait_warp(bars + 8u * (L::B_QFULL + qbuf), (q_par >> qbuf) & 1u, abort_flag, to)) goto drain;
    q_par ^= 1u << qbuf;
    tc_fence_after();

    bool have_prev = false, pv0 = false, pv1 = false;
    int prev_flags = 0, prev_vslot = 0;
    uint32_t prev_vpar = 0;
    while (true) {
      if (!bwait_warp(bars + 8u * (L::B_IFULL + ie), ie_par, abort_flag, to)) goto drain;
      const int j = hdr[ie].j;
      const int flags = hdr[ie].flags;
      const bool end = (flags & FLAG_END) != 0;
      const int cur_kslot = kslot, cur_vslot = vslot;
      const uint32_t cur_kpar = kpar, cur_vpar = vpar;
      if (!end) {
        if (++kslot == L::KSLOT) { kslot = 0; kpar ^= 1u; }
        if (++vslot == L::VSLOT) { vslot = 0; vpar ^= 1u; }
      }
      // End of unit: every Q_t K^T of the unit is in the pipe, so the Q buffer is released
      // (to the next unit's load) before the last P.V, which does not read it.
      if (end) tc_commit_elect(bars + 8u * (L::B_QEMPTY + qbuf));
      if (have_prev) {
        if (!bwait_warp(bars + 8u * (L::B_VFULL + prev_vslot), prev_vpar, abort_flag, to)) goto drain;
        tc_fence_after();
        if constexpr (Env::SCRUB) env.scrub(prev_flags, gbase + L::OFF_V + prev_vslot * L::KV_TILE_BYTES, lane);
      }
      bool k_ready = false;
      int ahead = 0;  // by turns: the slot of Q tile 1's Q.K^T

      // d = 64 issues a Q tile's Q.K^T before its P.V, d = 128 its P.V first.  Where key tiles go to the
      // two Q tiles by turns (Env::BY_TURNS), Q tile 1's Q.K^T comes before all (turn -1), so that it does
      // not wait for Q tile 0's P of the key tile before (the other way round the order has it so already).
#pragma unroll
      for (int turn = Env::BY_TURNS ? -1 : 0; turn < QT; ++turn) {
        const int t = turn < 0 ? 1 : turn;
        int& pslot = t ? pslot1 : pslot0;
        int new_slot = Env::BY_TURNS && turn == 1 ? ahead : t;
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          if ((step == 0) == L::RING) {
            if (Env::BY_TURNS && turn == 1) continue;
            if (!end && ((flags >> t) & 1)) {
              if (!k_ready) {
                if (!bwait_warp(bars + 8u * (L::B_KFULL + cur_kslot), cur_kpar, abort_flag, to)) goto drain;
                tc_fence_after();
                k_ready = true;
              }
              if constexpr (L::RING) {
                new_slot = nqk;
                nqk = nqk == L::S_SLOTS - 1 ? 0 : nqk + 1;
              }
              const uint32_t s_col = tmem + new_slot * 128;
              const uint32_t qbase = base + L::OFF_Q + qbuf * L::Q_BUF_BYTES + t * L::Q_TILE_BYTES;
              const uint32_t kbase = base + L::OFF_K + cur_kslot * L::KV_TILE_BYTES;
              // Q and K as K-major operands: 16 elements (32 bytes) per step inside a
              // 128-byte swizzle row, the next 64 elements one half-tile further.
              if constexpr (D == 64) {
                // d = 64 issues twice the instructions per flop: the descriptors are built
                // once and stepped through their start-address field (address >> 4 in the
                // low 14 bits; every offset here keeps it below 2^14)
                const uint64_t qd = sdesc_sw128(qbase, 16, 1024), kd = sdesc_sw128(kbase, 16, L::KV_SBO);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
                  mma_ss_elect(s_col, qd + off, kd + off, ID_QK, kk > 0 ? 1u : 0u);
                }
              } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (kk >> 2) * (BM * 128) + (kk & 3) * 32;
                  const uint32_t koff = (kk >> 2) * L::KV_HALF + (kk & 3) * 32;
                  mma_ss_elect(s_col, sdesc_sw128(qbase + off, 16, 1024), sdesc_sw128(kbase + koff, 16, L::KV_SBO),
                               ID_QK, kk > 0 ? 1u : 0u);
                }
              }
              tc_commit_elect(bars + 8u * (L::B_STILE + L::sp_bar(t, odd >> t)));
              if constexpr (L::RING) odd ^= 1u << t;
              env.computed(t, j, lane);
              __syncwarp();
            }
          } else if (turn >= 0) {
            if (have_prev && ((prev_flags >> t) & 1)) {
              uint32_t& pn = t ? pn1 : pn0;
              if (!bwait_warp(bars + 8u * (L::B_PREADY + L::sp_bar(t, pn)), L::sp_parity(pn), abort_flag, to)) goto drain;
              ++pn;
              tc_fence_after();
              bool& started = t ? pv1 : pv0;
              const uint32_t p_col = tmem + (L::RING ? pslot : t) * 128;
              const uint32_t vbase = base + L::OFF_V + prev_vslot * L::KV_TILE_BYTES;
              // V tile as the MN-major B operand: 16 keys per step (two groups of 8), the two
              // 64-column halves of d KV_HALF apart, 8-key groups KV_SBO.
              if constexpr (D == 64) {
                const uint64_t vd = sdesc_sw128(vbase, L::KV_HALF, L::KV_SBO);
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                  mma_ts_elect(tmem + L::O_COL + t * L::O_STRIDE, p_col + kk * 8, vd + (uint64_t)(kk * 2 * L::KV_SBO >> 4),
                               ID_PV, (started || kk > 0) ? 1u : 0u);
              } else {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                  mma_ts_elect(tmem + L::O_COL + t * L::O_STRIDE, p_col + kk * 8,
                               sdesc_sw128(vbase + kk * 2 * L::KV_SBO, L::KV_HALF, L::KV_SBO), ID_PV,
                               (started || kk > 0) ? 1u : 0u);
              }
              started = true;
              if constexpr (L::RING) tc_commit_elect(bars + 8u * (L::B_OPV + t));
            }
            // end of unit: O_t is complete once its last P.V is -- signal it now, so softmax t
            // starts its epilogue without waiting for the other Q tile's P.V
            if (end && (t ? pv1 : pv0)) tc_commit_elect(bars + 8u * (L::B_ODONE + t));
            if (t == QT - 1 && have_prev) tc_commit_elect(bars + 8u * (L::B_VEMPTY + prev_vslot));
          }
        }
        if (turn < 0) ahead = new_slot;
        if constexpr (L::RING) {
          if (turn >= 0 && !end && ((flags >> t) & 1)) pslot = new_slot;
        }
      }
      if (!end) tc_commit_elect(bars + 8u * (L::B_KEMPTY + cur_kslot));
      mbar_arrive_elect(bars + 8u * (L::B_IEMPTY + ie));
      if (++ie == NINFO) { ie = 0; ie_par ^= 1u; }
      if (end) break;
      have_prev = true;
      prev_flags = flags;
      prev_vslot = cur_vslot;
      prev_vpar = cur_vpar;
    }
  }
  return;

drain:
  // Aborted: wait until every MMA this warp issued has finished before TMEM is freed.
  tc_commit_elect(bars + 8u * L::B_DRAIN);
  wait_drain(bars + 8u * L::B_DRAIN, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax of one key tile
// One thread per query row: the 128 scores of its row at s_addr (TMEM) become weights in place, the
// row's O at o_addr is rescaled when the exponent base moves, and m, l follow.  make_mask, called while the
// scores are on their way, gives mask_half(h, c0), which sets the excluded of the 64 scores h of columns
// c0.. to -inf.  np / nact: P tiles this thread's Q tile has produced (in all, in this unit).
// False when a wait ran out.
template <int D, bool BF16, class L, class MakeMask>
__device__ __forceinline__ bool softmax_tile(uint32_t s_addr, uint32_t o_addr, float c, MakeMask make_mask, uint32_t opv_bar,
                                             int np, int nact, volatile int* abort_flag, uint32_t to, float& m, float& l) {
  // Scores: the first 64 columns are loaded and reduced while the last 64 are in flight.
  uint32_t sr[128];
  uint32_t(&sa)[64] = *reinterpret_cast<uint32_t(*)[64]>(&sr[0]);
  uint32_t(&sb)[64] = *reinterpret_cast<uint32_t(*)[64]>(&sr[64]);
  tmem_ld32x32b_x64_wait(s_addr, sa);
  tmem_ld32x32b_x64(s_addr + 64, sb);

  // Mask: excluded scores become -inf (weight exactly 0).
  const auto mask_half = make_mask();
  // Row max of one half: four independent 3-input max chains, chain x over h[16x, 16x+16).
  auto max_half = [&](const uint32_t(&h)[64]) {
    float a4[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      a4[x] = fmaxf(__uint_as_float(h[16 * x]), __uint_as_float(h[16 * x + 1]));
#pragma unroll
      for (int e = 2; e < 16; e += 2)
        a4[x] = fmax3(a4[x], __uint_as_float(h[16 * x + e]), __uint_as_float(h[16 * x + e + 1]));
    }
    return fmax3(a4[0], a4[1], fmaxf(a4[2], a4[3]));
  };
  mask_half(sa, 0);
  const float mx_a = max_half(sa);
  tmem_wait_ld();
  tmem_fence_regs_x64(sb);
  mask_half(sb, 64);
  const float mx = fmaxf(mx_a, max_half(sb));

  // Lazy rescaling: the exponent base m only moves when the row max exceeds it by more
  // than 8 (weights stay <= 2^8); O and l are always scaled with the same base, so the
  // final O / l and LSE = ln2 * (m + log2 l) are exact.
  const float mx_s = mx * c;
  const bool grow = mx_s > m + 8.f;  // also true on the first kept key (m = -inf)
  const float m_new = grow ? mx_s : m;
  const float alpha = grow ? ex2_approx(m - m_new) : 1.f;
  const float m_use = (m_new == -INFINITY) ? 0.f : m_new;

  // Correction: rescale this row of O (only warps where some row moved its base).
  if (nact > 0 && __any_sync(0xffffffffu, grow)) {
    if constexpr (L::RING) {
      // d = 64: this tile's S was computed before the previous P.V was issued; wait
      // until that P.V (OPV phase np - 1, the latest that can have completed) is done
      if (!bwait_warp(opv_bar, (uint32_t)(np - 1) & 1u, abort_flag, to)) return false;
      tc_fence_after();
    }
    const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
    for (int ch = 0; ch < D / 16; ++ch) {
      uint32_t ob[16];
      tmem_ld32x32b_x16_wait(o_addr + ch * 16, ob);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float lo, hi;
        f2_unpack(fmul2(f2_pack(__uint_as_float(ob[2 * x]), __uint_as_float(ob[2 * x + 1])), a2), lo, hi);
        ob[2 * x] = __float_as_uint(lo);
        ob[2 * x + 1] = __float_as_uint(hi);
      }
      tmem_st32x32b_x16(o_addr + ch * 16, ob);
    }
  }

  // P = 2^(s*c - m): packed FMA for the arguments, MUFU ex2, four packed partial sums.
  const uint64_t c2 = f2_pack(c, c);
  const uint64_t nm2 = f2_pack(-m_use, -m_use);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  // P_t goes over the first 64 columns of S_t, in four stores so each overlaps the
  // exponentials of the next quarter (and few packed words are live at a time).
#pragma unroll
  for (int hh = 0; hh < 4; ++hh) {
    uint32_t pk[16];
#pragma unroll
    for (int cc = 0; cc < 16; ++cc) {
      const int e = hh * 16 + cc;
      float e0, e1;
      f2_unpack(ffma2(f2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), c2, nm2), e0, e1);
      const float p0 = ex2_approx(e0);
      const float p1 = ex2_approx(e1);
      acc[cc & 3] = fadd2(acc[cc & 3], f2_pack(p0, p1));
      pk[cc] = pack2<BF16>(p0, p1);
    }
    tmem_st32x32b_x16(s_addr + hh * 16, pk);
  }
  tmem_wait_st();
  float s0, s1, s2, s3, s4, s5, s6, s7;
  f2_unpack(acc[0], s0, s1);
  f2_unpack(acc[1], s2, s3);
  f2_unpack(acc[2], s4, s5);
  f2_unpack(acc[3], s6, s7);
  const float sum = ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
  l = l * alpha + sum;
  m = m_new;
  return true;
}

}  // namespace attn
