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
// rounded once at the end.  An angle is a part of a turn: f / 2 pi is held in 64 bits of fixed point (f in 64 bits of
// floating point before), whose product with an integer position wraps at whole turns by itself and so keeps its
// accuracy at any position; its top 32 bits, as a float, go to sincospi.
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

constexpr int ROPE_WARPS = 8, ROPE_THREADS = 32 * ROPE_WARPS, ROPE_TOKENS = 8, ROPE_AXES = 4;

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

// f / 2 pi in parts of a turn of 2^-64 (whole turns left out).
__device__ __forceinline__ unsigned long long turn_of(float f) {
  double t = (double)f * 0.15915494309189533577;
  t -= rint(t);
  return (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
}

// A CTA takes TOKENS tokens.  First its threads work out, for every token and pair, the four products of weight and
// cosine or sine that turn a row (for q and for k), which all heads share, in shared memory.  Then its warps take
// items of VECS heads of a token: D / 16 lanes to a row, eight pairs to a lane, all of an item's loads in flight at
// once; the values' items are plain copies.
template <int D, bool BF16, bool ADJACENT, int TOKENS>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  const attn_rope_params_t& a = p.a;
  constexpr int LANES = D / 16, ROWS = 32 / LANES, UNROLL = 2, VECS = ROWS * UNROLL, PAIRS = D / 2;
  __shared__ __align__(16) float coef[TOKENS][2][4][PAIRS];  // [q, k][w_a cos, w_b sin, w_b cos, w_a sin]
  __shared__ long long dst_s[TOKENS];                        // where the token's row of the cache begins, -1: left out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();
  grid_dependency_wait();
  const int t0 = blockIdx.x * TOKENS, tokens = min(TOKENS, a.rows - t0);

  // ---- what the heads of a token share
  if (tid < tokens) {
    long long at = 0;
    if (a.slots) {
      const int slot = load_cg(a.slots + t0 + tid), page = slot / a.page_size;
      at = -1;
      if (slot >= 0 && page < a.num_pages)
        at = (long long)page * a.cache_page_stride + (long long)(slot - page * a.page_size) * a.cache_row_stride;
      else if (slot >= 0)
        atomicOr(p.status, STATUS_PAGE);
    }
    dst_s[tid] = at;
  }
  {
    const int pair = tid % PAIRS, half = a.rot_dim / 2;
    const bool turns = pair < half;
    // elements of the pair (those that are not turned: chunks of eight, paired off)
    int ea, eb;
    if (ADJACENT) ea = 2 * pair, eb = ea + 1;
    else if (turns) ea = pair, eb = pair + half;
    else ea = a.rot_dim + (pair - half) / 8 * 16 + pair % 8, eb = ea + 8;
    float wa[2] = {1.f, 1.f}, wb[2] = {1.f, 1.f};
    if (a.q_weight) {
      wa[0] = weight_at<BF16>(a.q_weight, a.weight_f32, ea);
      wb[0] = weight_at<BF16>(a.q_weight, a.weight_f32, eb);
    }
    if (a.k_weight) {
      wa[1] = weight_at<BF16>(a.k_weight, a.weight_f32, ea);
      wb[1] = weight_at<BF16>(a.k_weight, a.weight_f32, eb);
    }
    unsigned long long turn[ROPE_AXES] = {};
#pragma unroll
    for (int x = 0; x < ROPE_AXES; ++x)
      if (turns && x < a.axes) turn[x] = turn_of(a.inv_freq[x * half + pair]);
    for (int t = tid / PAIRS; t < tokens; t += ROPE_THREADS / PAIRS) {
      float s = 0.f, c = 1.f;
      if (turns) {
        unsigned long long phi = 0;
#pragma unroll
        for (int x = 0; x < ROPE_AXES; ++x)
          if (x < a.axes) phi += turn[x] * (unsigned long long)(long long)load_cg(a.positions + (long long)x * a.position_stride + t0 + t);
        sincospif((float)(int)(phi >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        coef[t][k][0][pair] = wa[k] * c;
        coef[t][k][1][pair] = wb[k] * s;
        coef[t][k][2][pair] = wb[k] * c;
        coef[t][k][3][pair] = wa[k] * s;
      }
    }
  }
  __syncthreads();

  // ---- the rows
  const int sub = lane / LANES, l = lane % LANES;
  // the lane's two chunks of eight elements
  const int half = a.rot_dim / 2;
  int ca, cb;
  if (ADJACENT || l * 8 >= half) ca = ADJACENT ? l * 16 : a.rot_dim + (l * 8 - half) * 2, cb = ca + 8;
  else ca = l * 8, cb = ca + half;
  const int per = p.q_items + p.k_items + p.v_items;
  for (int item = warp; item < tokens * per; item += ROPE_WARPS) {
    const int t = item / per, i = item - t * per;
    const long long at = dst_s[t];
    if (at < 0) continue;
    const int kind = i < p.q_items ? 0 : i < p.q_items + p.k_items ? 1 : 2;
    const int h0 = (kind == 0 ? i : kind == 1 ? i - p.q_items : i - p.q_items - p.k_items) * VECS + sub;
    const int heads = kind == 0 ? a.Hq : a.Hkv;
    const long long row = t0 + t;
    const uint16_t* src = kind == 0   ? static_cast<const uint16_t*>(a.q) + row * a.q_row_stride
                          : kind == 1 ? static_cast<const uint16_t*>(a.k) + row * a.k_row_stride
                                      : static_cast<const uint16_t*>(a.v) + row * a.v_row_stride;
    const long long src_head = kind == 0 ? a.q_head_stride : kind == 1 ? a.k_head_stride : a.v_head_stride;
    uint16_t* dst;
    long long dst_head;
    if (kind == 0) {
      dst = static_cast<uint16_t*>(a.q_out) + row * a.q_out_row_stride;
      dst_head = a.q_out_head_stride;
    } else if (a.slots) {
      dst = static_cast<uint16_t*>(kind == 1 ? a.k_cache : a.v_cache) + at;
      dst_head = a.cache_head_stride;
    } else {
      dst = static_cast<uint16_t*>(a.k_out) + row * a.k_out_row_stride;
      dst_head = a.k_out_head_stride;
    }
    uint4 raw[UNROLL][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
      const int h = h0 + u * ROWS;
      if (h < heads) {
        raw[u][0] = load_cg_x4(src + h * src_head + ca);
        raw[u][1] = load_cg_x4(src + h * src_head + cb);
      }
    }
    if (kind == 2) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = h0 + u * ROWS;
        if (h < heads) {
          *reinterpret_cast<uint4*>(dst + h * dst_head + ca) = raw[u][0];
          *reinterpret_cast<uint4*>(dst + h * dst_head + cb) = raw[u][1];
        }
      }
      continue;
    }
    float f[4][8];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float4 v = *reinterpret_cast<const float4*>(&coef[t][kind][x][l * 8 + y * 4]);
        f[x][4 * y] = v.x, f[x][4 * y + 1] = v.y, f[x][4 * y + 2] = v.z, f[x][4 * y + 3] = v.w;
      }
    const bool norm = (kind ? a.k_weight : a.q_weight) != nullptr;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = h0 + u * ROWS;
      const uint32_t x0[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w}, x1[4] = {raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
      float va[8], vb[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 lo = widen2<BF16>(x0[e]), hi = widen2<BF16>(x1[e]);
        if (ADJACENT) {  // (each word is a pair)
          va[e] = lo.x, vb[e] = lo.y;
          va[e + 4] = hi.x, vb[e + 4] = hi.y;
        } else {
          va[2 * e] = lo.x, va[2 * e + 1] = lo.y;
          vb[2 * e] = hi.x, vb[2 * e + 1] = hi.y;
        }
      }
      float r = 1.f;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(va[e], va[e], fmaf(vb[e], vb[e], ss));
#pragma unroll
        for (int s = 1; s < LANES; s <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
        r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      }
      float oa[8], ob[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        oa[e] = r * fmaf(va[e], f[0][e], -(vb[e] * f[1][e]));
        ob[e] = r * fmaf(vb[e], f[2][e], va[e] * f[3][e]);
      }
      uint32_t y0[4], y1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (ADJACENT) {
          y0[e] = narrow2<BF16>(oa[e], ob[e]);
          y1[e] = narrow2<BF16>(oa[e + 4], ob[e + 4]);
        } else {
          y0[e] = narrow2<BF16>(oa[2 * e], oa[2 * e + 1]);
          y1[e] = narrow2<BF16>(ob[2 * e], ob[2 * e + 1]);
        }
      }
      if (h < heads) {
        *reinterpret_cast<uint4*>(dst + h * dst_head + ca) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
        *reinterpret_cast<uint4*>(dst + h * dst_head + cb) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
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
  if (a.rot_dim > 0 && (!a.positions || !a.inv_freq || a.axes < 1 || a.axes > ROPE_AXES || (a.axes > 1 && a.position_stride < a.rows)))
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
  if (p.a.rows <= 2 * sms) return launch_dependent(rope_kernel<D, BF16, ADJACENT, 1>, dim3(p.a.rows), ROPE_THREADS, 0, st, p);
  return launch_dependent(rope_kernel<D, BF16, ADJACENT, ROPE_TOKENS>, dim3((p.a.rows + ROPE_TOKENS - 1) / ROPE_TOKENS), ROPE_THREADS, 0, st, p);
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
