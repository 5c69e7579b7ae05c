// rope.cu -- norms of queries and keys for each head and their rotation by position, in one pass (attn_rope): into
// buffers, or the queries into a buffer and keys and values into their slots of a paged cache.
//
// For a head's row x of d elements with weights w, at positions n_a of A axes with frequencies f_a[i]:
//
//     y = x * rsqrt(mean(x^2) + eps) * w                 (y = x without weights)
//     phi_i = sum_a n_a f_a[i]
//     (y_a, y_b) -> (y_a cos phi_i - y_b sin phi_i, y_b cos phi_i + y_a sin phi_i)
//
// for pairs i < rot / 2, (a, b) = (i, i + rot / 2) or (2 i, 2 i + 1); elements from rot on are not turned.  All in 32 bits,
// rounded once at the end.  An angle is a part of a turn: f / 2 pi is held in 64 bits of fixed point, whose product with an integer position wraps at
// whole turns by itself and so keeps its accuracy at any position; its top 32 bits, as a float, go to sincospi.  An angle is off by A 2^-33 (f / 2 pi
// cut at 2^-64 of a turn, times a position), 2^-32 (the cut to 32 bits) and 2^-26 (half a step of a float of at most half a turn) of a turn at most.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "host.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int ROPE_WARPS = 8, ROPE_THREADS = 32 * ROPE_WARPS, ROPE_CTAS = 2, ROPE_AXES = 4;

struct RopeParams {
  attn_rope_params_t a;
  unsigned int* status;
  int q_items, k_items, v_items;  // items of a token
};

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t x) {
  if constexpr (BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool BF16>
__device__ __forceinline__ float weight_at(const void* w, bool f32, int i) {
  if (f32) return static_cast<const float*>(w)[i];
  const uint32_t x = static_cast<const uint16_t*>(w)[i];
  return widen2<BF16>(x).x;
}

// f / 2 pi in parts of a turn of 2^-64 (whole turns left out), in whole numbers, as 64-bit floating point is slow on this machine: f = m 2^e
// with 24 bits of m, times the first 128 bits of 1 / 2 pi.
__device__ __forceinline__ unsigned long long turn_of(float f) {
  constexpr unsigned long long HI = 0x28BE60DB9391054Aull, LO = 0x7F09D5F47D4D3770ull;
  const uint32_t x = __float_as_uint(f), exponent = x >> 23 & 255u;
  const unsigned long long m = exponent ? (x & 0x7FFFFFu) | 0x800000u : x & 0x7FFFFFu;
  const int shift = 64 + 150 - (int)max(exponent, 1u);  // the product's bits from here on count
  const unsigned long long p0 = m * LO, mid = m * HI, p1 = __umul64hi(m, LO) + mid, p2 = __umul64hi(m, HI) + (p1 < mid);
  unsigned long long t = 0;
  if (shift >= 128) t = shift < 192 ? p2 >> (shift - 128) : 0;
  else if (shift >= 64) t = shift == 64 ? p1 : p1 >> (shift - 64) | p2 << (128 - shift);
  else if (shift > 0) t = p0 >> shift | p1 << (64 - shift);
  return x >> 31 ? 0ull - t : t;
}

// A token's items are VECS heads of q, k or v each; all tokens' items, laid end to end, are cut into equal runs, one to a warp
// of as many CTAs as the machine holds.  A row is D / 16 lanes, eight pairs to a lane.  The loads run an item ahead of the rest, on into the
// next token, whose positions and slot have been read a token ahead: a warp always has loads in flight.  At a token's first
// item a warp works out the four products of weight and cosine or sine that turn its pairs (two pairs to a lane; the frequencies'
// parts of a turn and the weights are the CTA's) and leaves them in shared memory of its own, so no warp waits for another; a lane keeps
// its pairs' products for all heads of q, then of k.  The values' items are plain copies.
// Measured (d = 128): 16.9k rows of 32/8 heads into the cache 70.6 us, 5.9 TB/s (0.88 of measured copy bandwidth), neighbours' pairs 71.2; to buffers 58.3
// and 58.7 (0.88; at d = 64 32.8, 0.79).  8190 rows of 16/2 heads to buffers, three axes 18.8 us, one axis 18.4, neighbours' pairs 18.9 and 18.5, bound by
// its instructions (57 % of the issue slots: the angles and products of a token serve 18 rows only); 64 rows 3.8 us, a launch and a chain of loads.  16 warps an SM: 20 and 24, for which registers spill, take 74 and 90 us.
template <int D, bool BF16, bool ADJACENT>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_CTAS) rope_kernel(const __grid_constant__ RopeParams p) {
  const attn_rope_params_t& a = p.a;
  constexpr int LANES = D / 16, ROWS = 32 / LANES, UNROLL = 2, VECS = ROWS * UNROLL, PAIRS = D / 2;
  __shared__ unsigned long long turn[ROPE_AXES][PAIRS];
  __shared__ float weight[4][PAIRS];                              // of q: first and second of the pair; of k
  __shared__ __align__(16) float coef[ROPE_WARPS][2][4][PAIRS];   // [q, k][w_a cos, -w_b sin, w_b cos, w_a sin], lanes' first fours ahead of their second ones
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = a.rot_dim / 2;
  grid_launch_dependents();
  grid_dependency_wait();
  const int sub = lane / LANES, l = lane % LANES;
  // the lane's two chunks of eight elements
  int ca, cb;
  if (ADJACENT || l * 8 >= half) ca = ADJACENT ? l * 16 : a.rot_dim + (l * 8 - half) * 2, cb = ca + 8;
  else ca = l * 8, cb = ca + half;
  // Whether the lane's pairs are turned (eight of them, and half is a multiple of eight).  Those that are not are no pairs: an infinity or NaN in
  // one of the two times a sine of 0 would reach the other.
  const bool turned = l * 8 < half;
  const int qk_items = p.q_items + p.k_items, items = qk_items + p.v_items;
  float(&mine)[2][4][PAIRS] = coef[warp];
  // a token's positions (lane x: of axis x) and slot (lane ROPE_AXES)
  const auto read_token = [&](int t) {
    int x = 0;
    if (t < a.rows) {
      if (lane < a.axes && half > 0) x = load_cg(a.positions + lane * a.position_stride + t);
      else if (lane == ROPE_AXES && a.slots) x = load_cg(a.slots + t);
    }
    return x;
  };
  struct Item {
    int t, i, token;
    long long at;  // where the token's row of the cache begins
  };
  const long long all = (long long)a.rows * items, run = (long long)blockIdx.x * ROPE_WARPS + warp, runs = (long long)gridDim.x * ROPE_WARPS;
  const long long begin = all * run / runs;
  long long left = all * (run + 1) / runs - begin;  // the run's items, `next` the first of them
  Item next{(int)(begin / items), (int)(begin % items), 0, 0};
  int token_next = read_token(next.t);
  // reads a token that the run comes to, and skips it if it is left out
  const auto open = [&] {
    for (; left > 0; left -= items - next.i, ++next.t, next.i = 0) {
      next.token = token_next;
      token_next = read_token(next.t + 1);
      if (a.slots) {
        const int slot = __shfl_sync(0xffffffffu, next.token, ROPE_AXES), page = slot / a.page_size;
        if (slot < 0) continue;
        if (page >= a.num_pages) {
          if (lane == 0) atomicOr(p.status, STATUS_PAGE);
          continue;
        }
        next.at = (long long)page * a.cache_page_stride + (long long)(slot - page * a.page_size) * a.cache_row_stride;
      }
      return;
    }
  };
  const auto kind_of = [&](int i) { return i < p.q_items ? 0 : i < qk_items ? 1 : 2; };
  const auto head_of = [&](int i) { return (i < p.q_items ? i : i < qk_items ? i - p.q_items : i - qk_items) * VECS + sub; };
  const auto fetch = [&](uint4(&raw)[UNROLL][2]) {
    const int kind = kind_of(next.i), h0 = head_of(next.i), heads = kind == 0 ? a.Hq : a.Hkv;
    const void* from = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const long long row = kind == 0 ? a.q_row_stride : kind == 1 ? a.k_row_stride : a.v_row_stride;
    const long long head = kind == 0 ? a.q_head_stride : kind == 1 ? a.k_head_stride : a.v_head_stride;
    const uint16_t* src = static_cast<const uint16_t*>(from) + next.t * row + h0 * head + ca;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u, src += ROWS * head) {
      raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h0 + u * ROWS < heads) {
        raw[u][0] = load_cg_x4(src);
        raw[u][1] = load_cg_x4(src + (cb - ca));
      }
    }
  };
  const auto advance = [&] {
    --left;
    if (++next.i < items) return;
    ++next.t;
    next.i = 0;
    open();
  };

  uint64_t f[4][4];
  int f_kind = -1, f_token = -1, coef_token = -1;  // whose products f and the shared memory hold
  uint4 raw[UNROLL][2], ahead[UNROLL][2];
  open();
  bool more = left > 0;
  if (more) fetch(ahead);
  for (int x = tid; x < PAIRS * ROPE_AXES; x += ROPE_THREADS) {
    const int pair = x % PAIRS, axis = x / PAIRS;
    if (pair < half && axis < a.axes) turn[axis][pair] = turn_of(a.inv_freq[axis * half + pair]);
    // elements of the pair (those that are not turned: chunks of eight, paired off)
    int e;
    if (ADJACENT) e = 2 * pair + (axis & 1);
    else if (pair < half) e = pair + (axis & 1) * half;
    else e = a.rot_dim + (pair - half) / 8 * 16 + pair % 8 + (axis & 1) * 8;
    const void* w = axis < 2 ? a.q_weight : a.k_weight;
    weight[axis][pair] = w ? weight_at<BF16>(w, a.weight_f32, e) : 1.f;
  }
  __syncthreads();

  while (more) {
    const Item it = next;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) raw[u][0] = ahead[u][0], raw[u][1] = ahead[u][1];
    advance();
    more = left > 0;
    if (more) fetch(ahead);

    const int kind = kind_of(it.i), h0 = head_of(it.i), heads = kind == 0 ? a.Hq : a.Hkv;
    uint16_t* dst;
    long long dst_head;
    if (kind == 0) {
      dst = static_cast<uint16_t*>(a.q_out) + it.t * a.q_out_row_stride;
      dst_head = a.q_out_head_stride;
    } else if (a.slots) {
      dst = static_cast<uint16_t*>(kind == 1 ? a.k_cache : a.v_cache) + it.at;
      dst_head = a.cache_head_stride;
    } else {
      dst = static_cast<uint16_t*>(a.k_out) + it.t * a.k_out_row_stride;
      dst_head = a.k_out_head_stride;
    }
    dst += h0 * dst_head + ca;
    dst_head *= ROWS;
    if (kind == 2) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u, dst += dst_head)
        if (h0 + u * ROWS < heads) {
          *reinterpret_cast<uint4*>(dst) = raw[u][0];
          *reinterpret_cast<uint4*>(dst + (cb - ca)) = raw[u][1];
        }
      continue;
    }
    if (coef_token != it.t) {
      coef_token = it.t;
      __syncwarp();  // those of the token before have been read
      unsigned long long position[ROPE_AXES];
#pragma unroll
      for (int axis = 0; axis < ROPE_AXES; ++axis) position[axis] = (unsigned long long)(long long)__shfl_sync(0xffffffffu, it.token, axis);
#pragma unroll
      for (int x = 0; x < PAIRS / 32; ++x) {
        const int pair = lane + 32 * x, place = (pair & 4) * (PAIRS / 8) + pair / 8 * 4 + (pair & 3);
        float s = 0.f, c = 1.f;
        if (pair < half) {
          unsigned long long phi = 0;
#pragma unroll
          for (int axis = 0; axis < ROPE_AXES; ++axis)
            if (axis < a.axes) phi += turn[axis][pair] * position[axis];
          sincospif((float)(int)(phi >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float wa = weight[2 * k][pair], wb = weight[2 * k + 1][pair];
          mine[k][0][place] = wa * c;
          mine[k][1][place] = -wb * s;
          mine[k][2][place] = wb * c;
          mine[k][3][place] = wa * s;
        }
      }
      __syncwarp();
    }
    if (f_kind != kind || f_token != it.t) {
      f_kind = kind;
      f_token = it.t;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&mine[kind][x][y * (PAIRS / 2) + l * 4]);
          f[x][2 * y] = v.x, f[x][2 * y + 1] = v.y;
        }
    }
    const bool norm = (kind ? a.k_weight : a.q_weight) != nullptr;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u, dst += dst_head) {
      const int h = h0 + u * ROWS;
      if (h - sub >= heads) break;  // (the whole warp's)
      const uint32_t x0[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w}, x1[4] = {raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
      uint64_t va[4], vb[4];  // two of the lane's pairs each: their first elements, their second ones
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (ADJACENT) {  // (each word is a pair)
          const float2 lo = widen2<BF16>(e < 2 ? x0[2 * e] : x1[2 * e - 4]), hi = widen2<BF16>(e < 2 ? x0[2 * e + 1] : x1[2 * e - 3]);
          va[e] = f2_pack(lo.x, hi.x), vb[e] = f2_pack(lo.y, hi.y);
        } else {
          const float2 lo = widen2<BF16>(x0[e]), hi = widen2<BF16>(x1[e]);
          va[e] = f2_pack(lo.x, lo.y), vb[e] = f2_pack(hi.x, hi.y);
        }
      }
      float r = 1.f;
      if (norm) {
        uint64_t s2 = fmul2(va[0], va[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e > 0) s2 = ffma2(va[e], va[e], s2);
          s2 = ffma2(vb[e], vb[e], s2);
        }
        float ss, other;
        f2_unpack(s2, ss, other);
        ss += other;
#pragma unroll
        for (int y = 1; y < LANES; y <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, y);
        r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      }
      const uint64_t rr = f2_pack(r, r);
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t x = va[e];
          va[e] = ffma2(x, f[0][e], fmul2(vb[e], f[1][e]));
          vb[e] = ffma2(vb[e], f[2][e], fmul2(x, f[3][e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) va[e] = fmul2(va[e], f[0][e]), vb[e] = fmul2(vb[e], f[2][e]);
      }
      uint32_t y0[4], y1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a0, a1, b0, b1;
        f2_unpack(fmul2(rr, va[e]), a0, a1);
        f2_unpack(fmul2(rr, vb[e]), b0, b1);
        if (ADJACENT) {
          (e < 2 ? y0[2 * e] : y1[2 * e - 4]) = narrow2<BF16>(a0, b0);
          (e < 2 ? y0[2 * e + 1] : y1[2 * e - 3]) = narrow2<BF16>(a1, b1);
        } else {
          y0[e] = narrow2<BF16>(a0, a1);
          y1[e] = narrow2<BF16>(b0, b1);
        }
      }
      if (h < heads) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
        *reinterpret_cast<uint4*>(dst + (cb - ca)) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
      }
    }
  }
}

bool misaligned(const void* ptr, unsigned int to) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }

int check(const attn_rope_params_t& a) {
  if (!a.q || !a.k || !a.q_out) return ATTN_ERR_INVALID;
  if (a.slots ? !a.v || !a.k_cache || !a.v_cache : !a.k_out) return ATTN_ERR_INVALID;
  if (a.d != 64 && a.d != 128) return ATTN_ERR_UNSUPPORTED;
  if (a.dtype != ATTN_F16 && a.dtype != ATTN_BF16) return ATTN_ERR_UNSUPPORTED;
  if (a.rows < 1 || a.rows > (1 << 30) || a.Hq < 1 || a.Hkv < 1 || a.Hq > (1 << 16) || a.Hkv > (1 << 16)) return ATTN_ERR_INVALID;
  if (a.rot_dim < 0 || a.rot_dim > a.d || a.rot_dim % 16 != 0) return ATTN_ERR_INVALID;
  if (a.rot_dim > 0 && (!a.positions || !a.inv_freq || a.axes < 1 || a.axes > ROPE_AXES || (a.axes > 1 && a.position_stride != 0 && a.position_stride < a.rows)))
    return ATTN_ERR_INVALID;
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return ATTN_ERR_INVALID;
  const void *k_to = a.slots ? a.k_cache : a.k_out, *v_to = a.slots ? a.v_cache : nullptr;
  for (const void* ptr : {a.q, a.k, (const void*)a.q_out, k_to, v_to, a.slots ? a.v : nullptr})
    if (misaligned(ptr, 16)) return ATTN_ERR_INVALID;
  for (const void* ptr : {(const void*)a.slots, (const void*)a.positions, (const void*)a.inv_freq})
    if (misaligned(ptr, 4)) return ATTN_ERR_INVALID;
  for (const void* ptr : {a.q_weight, a.k_weight})
    if (misaligned(ptr, a.weight_f32 ? 4 : 2)) return ATTN_ERR_INVALID;
  const auto bad = [](long long s) { return s < 0 || s % 8 != 0 || s > MAX_STRIDE; };
  for (long long s : {a.q_row_stride, a.q_head_stride, a.k_row_stride, a.k_head_stride, a.q_out_row_stride, a.q_out_head_stride})
    if (bad(s)) return ATTN_ERR_INVALID;
  // (outputs: strides of dimensions with more than one entry)
  if ((a.rows > 1 && a.q_out_row_stride == 0) || (a.Hq > 1 && a.q_out_head_stride == 0)) return ATTN_ERR_INVALID;
  if (!a.slots) {
    if (bad(a.k_out_row_stride) || bad(a.k_out_head_stride) || (a.rows > 1 && a.k_out_row_stride == 0) || (a.Hkv > 1 && a.k_out_head_stride == 0))
      return ATTN_ERR_INVALID;
    return ATTN_OK;
  }
  for (long long s : {a.v_row_stride, a.v_head_stride, a.cache_page_stride, a.cache_head_stride, a.cache_row_stride})
    if (bad(s)) return ATTN_ERR_INVALID;
  if (a.num_pages < 1 || a.page_size < 16 || a.page_size % 16 != 0 || (long long)a.num_pages * a.page_size > INT_MAX) return ATTN_ERR_INVALID;
  if (a.cache_row_stride == 0 || (a.num_pages > 1 && a.cache_page_stride == 0) || (a.Hkv > 1 && a.cache_head_stride == 0)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

template <int D, bool BF16, bool ADJACENT>
int launch(RopeParams& p, int sms, cudaStream_t st) {
  constexpr int VECS = 32 / (D / 16) * 2;
  p.q_items = (p.a.Hq + VECS - 1) / VECS;
  p.k_items = (p.a.Hkv + VECS - 1) / VECS;
  p.v_items = p.a.slots ? p.k_items : 0;
  const int items = p.q_items + p.k_items + p.v_items, most = sms * ROPE_CTAS;
  const long long ctas = ((long long)p.a.rows * items + ROPE_WARPS - 1) / ROPE_WARPS;
  return launch_dependent(rope_kernel<D, BF16, ADJACENT>, dim3((unsigned int)(ctas < most ? ctas : most)), ROPE_THREADS, 0, st, p);
}

}  // namespace
}  // namespace attn

extern "C" int attn_rope(const attn_rope_params_t* params) {
  return attn::entry([&]() -> int {
    using namespace attn;
    if (!params) return ATTN_ERR_INVALID;
    const attn_rope_params_t& a = *params;
    int rc = check(a);
    if (rc != ATTN_OK) return rc;
    int sms = 0, dev = 0;
    if ((rc = host_device(sms, dev)) != ATTN_OK) return rc;
    RopeParams p{a, nullptr, 0, 0, 0};
    if (a.slots && (rc = host_status_word(dev, a.stream, &p.status)) != ATTN_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(a.stream);
    const bool bf16 = a.dtype == ATTN_BF16;
    const auto go = [&](auto launch) { return launch(p, sms, st); };
    if (a.d == 64) {
      if (a.interleaved) return go(bf16 ? launch<64, true, true> : launch<64, false, true>);
      return go(bf16 ? launch<64, true, false> : launch<64, false, false>);
    }
    if (a.interleaved) return go(bf16 ? launch<128, true, true> : launch<128, false, true>);
    return go(bf16 ? launch<128, true, false> : launch<128, false, false>);
  });
}
