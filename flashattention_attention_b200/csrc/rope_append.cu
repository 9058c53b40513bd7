// rope_append.cu -- append of any number of new tokens per sequence to a paged
// cache, keys and queries rotated to their positions on the way, and the
// read-back of cached rows (FlashRT QKV Cache RoPE, Kernels: rotation and
// cache write of the new K fused in one kernel).
//
// A row of d channels is held by W lanes (d / 8 rounded up to a power of two),
// eight channels per lane in two chunks of four.  Rotating channel pairs (i, i
// + rot/2), lane i takes the chunks [4i, 4i+4) and [rot/2 + 4i, +4), so both
// members of a pair sit in one lane; rotating pairs (2i, 2i+1), and for
// channels past rot_dim, the two chunks are adjacent.  Either way lane i's
// four pairs use angles 4i .. 4i+3.
//
// One launch does everything.  A group of W lanes takes one token and some of
// its rows: the token's sequence, slot, page and angles are found once and
// four rows' loads are in flight at a time.  Keys whose page bounds are kept
// go another way, since all new keys of a page have to meet: a CTA per page
// (of the first new token in it), its groups spread over KV heads and slices
// of the page's tokens, the slices' bounds joined in shared memory.  No page
// is touched by two CTAs, so there are no atomics and no order to depend on.
#include <type_traits>

#include "internal.h"
#include "quant.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

struct PoolArgs {
  const int32_t* block_table;
  int max_pages, page_size, num_pages, hkv, d;
  int64_t capacity;
};

struct AppendArgs {
  const void* k_new;
  const void* v_new;
  const void* q;
  __nv_bfloat16* q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;
  const float* rope;
  void* k_cache;
  void* v_cache;
  float* k_scales;
  float* v_scales;
  __nv_bfloat16* bounds;
  const int32_t* cu;
  const int32_t* cur_pos;
  int32_t* seqlens;
  int batch, total, hq, rot, interleaved, rope_rows;
  int cache_dtype;
  // how the work is cut: rows per token (without keys that the page role
  // takes), rows per part; page role: the tokens a CTA looks at
  int token_rows, part_rows, window;
  PoolArgs pool;
  Watchdog wd;
};

// Where token t goes: its sequence b, slot and (page * hkv) * page_size + offset
// base row.  False: padding, or out of range (`bad`).
struct Place {
  int b;
  int64_t slot;
  int64_t row0;  // cache row of KV head 0; head g is g * page_size further
};
__device__ __forceinline__ bool seq_of_token(const int32_t* cu, int batch, int t, int& b, int& i) {
  if (cu == nullptr) {
    b = t;
    i = 0;
    return true;
  }
  int lo = 0, hi = batch;  // the last b with cu[b] <= t, so empty sequences are passed over
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  b = lo;
  i = t - cu[lo];
  return i >= 0 && t < cu[lo + 1];
}
__device__ __forceinline__ bool page_row(const PoolArgs& P, int b, int64_t slot, int64_t& row0) {
  if (slot < 0 || slot >= P.capacity) return false;
  const int s = static_cast<int>(slot);
  const int pg = P.block_table[static_cast<int64_t>(b) * P.max_pages + s / P.page_size];
  if (pg < 0 || pg >= P.num_pages) return false;
  row0 = static_cast<int64_t>(pg) * P.hkv * P.page_size + s % P.page_size;
  return true;
}
__device__ __forceinline__ bool place_token(const AppendArgs& A, int t, Place& p, bool& bad) {
  int i;
  bad = false;
  if (!seq_of_token(A.cu, A.batch, t, p.b, i)) return false;
  p.slot = static_cast<int64_t>(A.cur_pos[p.b]) + i;
  if (!page_row(A.pool, p.b, p.slot, p.row0) || (A.rot > 0 && p.slot >= A.rope_rows)) {
    bad = true;
    return false;
  }
  return true;
}

// Channel offsets of lane `l`'s two chunks.
__device__ __forceinline__ void chunk_offsets(const AppendArgs& A, int l, bool rotated, int& a, int& b) {
  if (rotated && !A.interleaved && 8 * l < A.rot) {
    a = 4 * l;
    b = A.rot / 2 + 4 * l;
  } else {
    a = 8 * l;
    b = a + 4;
  }
}

// A lane's eight channels: x[0], x[1] of chunk a, x[2], x[3] of chunk b.
template <typename T>
__device__ __forceinline__ void widen8(const typename Vec4<T>::Raw& u, const typename Vec4<T>::Raw& v, float2 (&x)[4]) {
  float y[4], z[4];
  Vec4<T>::widen(u, y);
  Vec4<T>::widen(v, z);
  x[0] = make_float2(y[0], y[1]);
  x[1] = make_float2(y[2], y[3]);
  x[2] = make_float2(z[0], z[1]);
  x[3] = make_float2(z[2], z[3]);
}

// The lane's four angles at a slot; no rotation for lanes past rot_dim.
struct Angles {
  float4 c, s;
  bool any;
};
__device__ __forceinline__ Angles angles_of(const AppendArgs& A, int l, int64_t slot) {
  Angles r;
  r.any = 8 * l < A.rot;
  r.c = r.s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r.any) {
    const float* row = A.rope + slot * A.rot;
    r.c = *reinterpret_cast<const float4*>(row + 4 * l);
    r.s = *reinterpret_cast<const float4*>(row + A.rot / 2 + 4 * l);
  }
  return r;
}
// (a, b) <- (a c - b s, b c + a s), every product and sum rounded.  In scalars:
// the compiler contracts a packed product and a packed sum into one packed FMA,
// although each asks for its rounding (20 of 64 rows' int8 scales were off).
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = a;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(x, s));
}
__device__ __forceinline__ void rotate_pairs(float2& a, float2& b, float2 c, float2 s) {
  rotate_pair(a.x, b.x, c.x, s.x);
  rotate_pair(a.y, b.y, c.y, s.y);
}
__device__ __forceinline__ void rotate8(const AppendArgs& A, const Angles& g, float2 (&x)[4]) {
  if (!g.any) return;
  const float2 c0 = make_float2(g.c.x, g.c.y), c1 = make_float2(g.c.z, g.c.w);
  const float2 s0 = make_float2(g.s.x, g.s.y), s1 = make_float2(g.s.z, g.s.w);
  if (A.interleaved) {
    float2 a0 = make_float2(x[0].x, x[1].x), b0 = make_float2(x[0].y, x[1].y);
    float2 a1 = make_float2(x[2].x, x[3].x), b1 = make_float2(x[2].y, x[3].y);
    rotate_pairs(a0, b0, c0, s0);
    rotate_pairs(a1, b1, c1, s1);
    x[0] = make_float2(a0.x, b0.x);
    x[1] = make_float2(a0.y, b0.y);
    x[2] = make_float2(a1.x, b1.x);
    x[3] = make_float2(a1.y, b1.y);
  } else {
    rotate_pairs(x[0], x[2], c0, s0);
    rotate_pairs(x[1], x[3], c1, s1);
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint2 pack4(float2 lo, float2 hi) { return make_uint2(bf16x2(lo.x, lo.y), bf16x2(hi.x, hi.y)); }
__device__ __forceinline__ void store8_bf16(__nv_bfloat16* row, int a, int b, const float2 (&x)[4]) {
  *reinterpret_cast<uint2*>(row + a) = pack4(x[0], x[1]);
  *reinterpret_cast<uint2*>(row + b) = pack4(x[2], x[3]);
}

// The quantisers below need correctly rounded quotients (codes and scales are
// defined by them, and rows of bf16 values are full of exact halves).  With y
// the rounded reciprocal of b, Markstein's step RN(q0 + RN(a - q0 b) y), q0 =
// RN(a y), is that quotient as long as nothing leaves the normal range (see
// quant.cu; checked over all mantissas for the divisors 15 and 127).  Rows
// whose range or scale is outside [2^-60, 2^60] take the IEEE division, in a
// function of its own so that its code stays out of the loops.
__device__ __forceinline__ float divide_by(float a, float b, float y) {
  const float q0 = __fmul_rn(a, y);
  return __fmaf_rn(__fmaf_rn(-q0, b, a), y, q0);
}
__device__ __forceinline__ bool ordinary(float s) { return s >= 0x1p-60f && s <= 0x1p60f; }

// Four 4-bit codes, 4 bits each: round_half_even(15 (x - lo) / r).
__device__ __forceinline__ uint32_t codes4_fast(float2 x0, float2 x1, float lo, float r, float y) {
  const float2 nlo = make_float2(-lo, -lo), nr = make_float2(-r, -r), y2 = make_float2(y, y);
  const float2 fifteen = make_float2(15.0f, 15.0f), shift = make_float2(12582912.0f, 12582912.0f);  // 1.5 * 2^23
  uint32_t k[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 u = mul2(add2(h ? x1 : x0, nlo), fifteen);
    const float2 q0 = mul2(u, y2);
    const float2 z = add2(fma2(fma2(q0, nr, u), y2, q0), shift);
    k[2 * h] = __float_as_uint(z.x);
    k[2 * h + 1] = __float_as_uint(z.y);
  }
  // the low 16 bits of the shift's pattern are 0, so those of the sum are the four codes
  return (k[0] + (k[1] << 4) + (k[2] << 8) + (k[3] << 12)) & 0xffffu;
}
__device__ __noinline__ uint32_t codes4_any(float2 x0, float2 x1, float lo, float r) {
  const float x[4] = {x0.x, x0.y, x1.x, x1.y};
  uint32_t w = 0;
  for (int e = 0; e < 4; ++e) {
    const float q = r > 0.0f ? __fdiv_rn(__fmul_rn(__fsub_rn(x[e], lo), 15.0f), r) : 0.0f;
    w |= (static_cast<uint32_t>(__float2int_rn(q)) & 15u) << (4 * e);
  }
  return w;
}
__device__ __noinline__ uint32_t codes8_any(float2 x0, float2 x1, float s) {
  const float x[4] = {x0.x, x0.y, x1.x, x1.y};
  return quantise4_div(x, s);
}
__device__ __noinline__ float divide_any(float a, float b) { return __fdiv_rn(a, b); }

// Where rows go: the current one's codes or values and its scales, and the way
// to the next KV head's (or the next slot's).
template <int kCache>
struct Sink {
  uint8_t* dst;
  float* scale;
  static constexpr int kScales = kCache == FA_I4 ? 2 : kCache == FA_I8 ? 1 : 0;
  __device__ __forceinline__ static int row_bytes(int d) {
    return kCache == FA_BF16 ? 2 * d : kCache == FA_I8 ? d : d / 2;
  }
  __device__ __forceinline__ Sink(void* pool, float* scales, int64_t row, int d)
      : dst(static_cast<uint8_t*>(pool) + row * row_bytes(d)), scale(scales + row * kScales) {}
  __device__ __forceinline__ void advance(int rows, int d) {
    dst += static_cast<int64_t>(rows) * row_bytes(d);
    scale += static_cast<int64_t>(rows) * kScales;
  }
};

// One row into the cache by the W lanes that hold it (`own`: this lane holds
// channels).  Every lane of the group calls.
template <int W, int kCache>
__device__ __forceinline__ void store_row(const Sink<kCache>& to, int l, bool own, int a, int b, const float2 (&x)[4],
                                          unsigned mask) {
  if constexpr (kCache == FA_BF16) {
    if (own) store8_bf16(reinterpret_cast<__nv_bfloat16*>(to.dst), a, b, x);
  } else if constexpr (kCache == FA_I8) {
    float amax = 0.0f;
    if (own) {
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
    }
#pragma unroll
    for (int off = W >> 1; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, off));
    constexpr float k127 = 1.0f / 127.0f;
    const float s = ordinary(amax) ? divide_by(amax, 127.0f, k127) : divide_any(amax, 127.0f);
    if (own) {
      uint32_t u, v;
      if (ordinary(s)) {
        const float y = __frcp_rn(s);
        const float p[4] = {x[0].x, x[0].y, x[1].x, x[1].y}, q[4] = {x[2].x, x[2].y, x[3].x, x[3].y};
        u = quantise4_fast(p, s, y);
        v = quantise4_fast(q, s, y);
      } else {
        u = codes8_any(x[0], x[1], s);
        v = codes8_any(x[2], x[3], s);
      }
      *reinterpret_cast<uint32_t*>(to.dst + a) = u;
      *reinterpret_cast<uint32_t*>(to.dst + b) = v;
      if (l == 0) *to.scale = s;
    }
  } else {
    float lo = INFINITY, hi = -INFINITY;
    if (own) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo = min3f(lo, x[e].x, x[e].y);
        hi = max3f(hi, x[e].x, x[e].y);
      }
    }
#pragma unroll
    for (int off = W >> 1; off > 0; off >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(mask, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(mask, hi, off));
    }
    const float r = __fsub_rn(hi, lo);
    if (own) {
      uint32_t u, v;
      float step;
      if (ordinary(r)) {
        const float y = __frcp_rn(r);
        constexpr float k15 = 1.0f / 15.0f;
        step = divide_by(r, 15.0f, k15);
        u = codes4_fast(x[0], x[1], lo, r, y);
        v = codes4_fast(x[2], x[3], lo, r, y);
      } else {
        step = divide_any(r, 15.0f);
        u = codes4_any(x[0], x[1], lo, r);
        v = codes4_any(x[2], x[3], lo, r);
      }
      *reinterpret_cast<uint16_t*>(to.dst + a / 2) = static_cast<uint16_t>(u);
      *reinterpret_cast<uint16_t*>(to.dst + b / 2) = static_cast<uint16_t>(v);
      if (l == 0) *reinterpret_cast<float2*>(to.scale) = make_float2(step, lo);
    }
  }
}

// This thread's place in its group of W lanes.
template <int W>
struct Group {
  int l = threadIdx.x & (W - 1);
  unsigned mask = W == 32 ? 0xffffffffu : ((1u << (W & 31)) - 1u) << (threadIdx.x & 31 & ~(W - 1));
};

constexpr int kRows = 4;  // query rows a group has in flight (of K and V rows two: their arithmetic is longer)

// The rows [r0, r1) of one token: its hq queries, then its V rows, then (when
// the page role does not take them) its K rows.
template <typename T, int W, int kCache>
__device__ __forceinline__ void append_token(const AppendArgs& A, int t, int r0, int r1) {
  using V = Vec4<T>;
  const Group<W> G;
  const bool own = 8 * G.l < A.pool.d;
  Place p;
  bool bad;
  if (!place_token(A, t, p, bad)) {
    if (bad && G.l == 0) record_status(A.wd, kStatusRange);
    return;
  }
  int a, b;
  chunk_offsets(A, G.l, true, a, b);
  const Angles ang = angles_of(A, G.l, p.slot);
  const int hq = A.hq, hkv = A.pool.hkv;
  const int q1 = min(r1, hq);
  const T* q = static_cast<const T*>(A.q) + t * A.q_ts + r0 * A.q_hs;
  __nv_bfloat16* qo = A.q_out + t * A.qo_ts + r0 * A.qo_hs;
#pragma unroll 1
  for (int r = r0; r < q1; r += kRows, q += kRows * A.q_hs, qo += kRows * A.qo_hs) {
    typename V::Raw u[kRows], v[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (own && r + k < q1) {
        u[k] = V::load(q + k * A.q_hs + a);
        v[k] = V::load(q + k * A.q_hs + b);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (own && r + k < q1) {
        float2 x[4];
        widen8<T>(u[k], v[k], x);
        rotate8(A, ang, x);
        store8_bf16(qo + k * A.qo_hs, a, b, x);
      }
    }
  }
  // heads [g0, g1) of V or K
  auto cached = [&](auto rotated, const void* rows, int64_t ts, int64_t hs, void* pool, float* scales, int g0, int g1) {
    constexpr bool kRotated = decltype(rotated)::value;
    const int ra = kRotated ? a : 8 * G.l, rb = kRotated ? b : 8 * G.l + 4;
    const T* src = static_cast<const T*>(rows) + t * ts + g0 * hs;
    Sink<kCache> to(pool, scales, p.row0 + static_cast<int64_t>(g0) * A.pool.page_size, A.pool.d);
#pragma unroll 2
    for (int g = g0; g < g1; ++g, src += hs) {
      float2 x[4];
      if (own) {
        widen8<T>(V::load(src + ra), V::load(src + rb), x);
        if constexpr (kRotated) rotate8(A, ang, x);
      }
      store_row<W, kCache>(to, G.l, own, ra, rb, x, G.mask);
      to.advance(A.pool.page_size, A.pool.d);
    }
  };
  cached(std::false_type{}, A.v_new, A.v_ts, A.v_hs, A.v_cache, A.v_scales, max(r0 - hq, 0), min(r1 - hq, hkv));
  cached(std::true_type{}, A.k_new, A.k_ts, A.k_hs, A.k_cache, A.k_scales, max(r0 - hq - hkv, 0), r1 - hq - hkv);
}

__device__ __forceinline__ float2 min_of(float2 a, float2 b) { return make_float2(fminf(a.x, b.x), fminf(a.y, b.y)); }
__device__ __forceinline__ float2 max_of(float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)); }

// The new keys of the pages whose first new token is one of `window` tokens
// from t0 on, and those pages' bounds; the whole CTA together.
template <typename T, int W, int kCache>
__device__ __forceinline__ void append_pages(const AppendArgs& A, int t0, float2 (&s_lo)[4][kThreads],
                                             float2 (&s_hi)[4][kThreads]) {
  using V = Vec4<T>;
  constexpr int kGroups = kThreads / W;
  const Group<W> G;
  const bool own = 8 * G.l < A.pool.d;
  const int lane = threadIdx.x & 31, group = threadIdx.x / W;
  const int page = A.pool.page_size, hkv = A.pool.hkv;
  // lane j of every warp looks at token t0 + j
  int left = 0, off = 0;
  Place p;
  p.slot = p.row0 = 0;
  bool first = false;
  if (lane < A.window && t0 + lane < A.total) {
    bool bad;  // reported with the token's other rows
    first = place_token(A, t0 + lane, p, bad);
    if (first) {
      int b, i;
      seq_of_token(A.cu, A.batch, t0 + lane, b, i);
      off = static_cast<int>(p.slot % page);
      left = min(A.cu != nullptr ? min(A.cu[b + 1], A.total) - (t0 + lane) : 1, page - off);
      if (A.rot > 0) left = static_cast<int>(min(static_cast<int64_t>(left), A.rope_rows - p.slot));
      first = i == 0 || off == 0;  // else an earlier token's CTA has this page
    }
  }
  int ca, cb;
  chunk_offsets(A, G.l, true, ca, cb);
#pragma unroll 1
  for (unsigned todo = __ballot_sync(0xffffffffu, first); todo != 0; todo &= todo - 1) {
    const int j0 = __ffs(todo) - 1, t = t0 + j0;
    const int n = __shfl_sync(0xffffffffu, left, j0), at = __shfl_sync(0xffffffffu, off, j0);
    const int64_t slot = __shfl_sync(0xffffffffu, p.slot, j0), row0 = __shfl_sync(0xffffffffu, p.row0, j0);
    const int slices = n == 1 ? 1 : max(1, kGroups / hkv);
#pragma unroll 1
    for (int g0 = 0; g0 < hkv; g0 += kGroups) {
      const int g = g0 + (slices > 1 ? group % hkv : group), slice = slices > 1 ? group / hkv : 0;
      float2 lo[4], hi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = make_float2(INFINITY, INFINITY);
        hi[e] = make_float2(-INFINITY, -INFINITY);
      }
      if (g < hkv && slice < slices) {
        const T* src = static_cast<const T*>(A.k_new) + static_cast<int64_t>(t + slice) * A.k_ts + g * A.k_hs;
        Sink<kCache> to(A.k_cache, A.k_scales, row0 + slice + static_cast<int64_t>(g) * page, A.pool.d);
#pragma unroll 2
        for (int j = slice; j < n; j += slices, src += slices * A.k_ts) {
          float2 x[4];
          if (own) {
            widen8<T>(V::load(src + ca), V::load(src + cb), x);
            rotate8(A, angles_of(A, G.l, slot + j), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] = min_of(lo[e], x[e]);
              hi[e] = max_of(hi[e], x[e]);
            }
          }
          store_row<W, kCache>(to, G.l, own, ca, cb, x, G.mask);
          to.advance(slices, A.pool.d);
        }
      }
      if (slices > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s_lo[e][threadIdx.x] = lo[e];
          s_hi[e][threadIdx.x] = hi[e];
        }
        __syncthreads();
        if (slice == 0) {
#pragma unroll 1
          for (int o = 1; o < slices; ++o) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] = min_of(lo[e], s_lo[e][threadIdx.x + o * hkv * W]);
              hi[e] = max_of(hi[e], s_hi[e][threadIdx.x + o * hkv * W]);
            }
          }
        }
      }
      if (g < hkv && slice == 0 && own) {
        const int64_t plane = row0 / page + g;  // page * hkv + g
        __nv_bfloat16* dst = A.bounds + plane * 2 * A.pool.d;
        if (at > 0) {
          float2 x[4];
          widen8<__nv_bfloat16>(*reinterpret_cast<const uint2*>(dst + ca), *reinterpret_cast<const uint2*>(dst + cb), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) lo[e] = min_of(lo[e], x[e]);
          widen8<__nv_bfloat16>(*reinterpret_cast<const uint2*>(dst + A.pool.d + ca),
                                *reinterpret_cast<const uint2*>(dst + A.pool.d + cb), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) hi[e] = max_of(hi[e], x[e]);
        }
        store8_bf16(dst, ca, cb, lo);
        store8_bf16(dst + A.pool.d, ca, cb, hi);
      }
    }
  }
}

template <typename T, int W, int kCache>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendArgs A) {
  __shared__ float2 s_lo[4][kThreads], s_hi[4][kThreads];
  // grid row 0 is the page role (where bounds are kept), the others are the parts of the tokens' rows
  int part = static_cast<int>(blockIdx.y);
  if (A.bounds != nullptr) {
    if (part == 0) {
      if (static_cast<int64_t>(blockIdx.x) * A.window < A.total)
        append_pages<T, W, kCache>(A, static_cast<int>(blockIdx.x) * A.window, s_lo, s_hi);
      return;
    }
    --part;
  }
  if (A.seqlens != nullptr && blockIdx.x == 0 && part == 0) {
    for (int b = threadIdx.x; b < A.batch; b += kThreads) {
      const int64_t c0 = A.cu != nullptr ? A.cu[b] : b, c1 = A.cu != nullptr ? A.cu[b + 1] : b + 1;
      const int64_t end = static_cast<int64_t>(A.cur_pos[b]) + (c1 - c0);
      if (c0 < 0 || c1 < c0 || c1 > A.total || A.cur_pos[b] < 0 || end > A.pool.capacity) {
        record_status(A.wd, kStatusRange);
      } else {
        A.seqlens[b] = static_cast<int32_t>(end);
      }
    }
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  if (t >= A.total) return;
  const int r0 = part * A.part_rows;
  append_token<T, W, kCache>(A, static_cast<int>(t), r0, min(r0 + A.part_rows, A.token_rows));
}

// ---------------------------------------------------------------- read back
struct ReadArgs {
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;
  const float* v_scales;
  void* k_out;
  void* v_out;
  const int32_t* cu;
  const int32_t* start;
  int batch, total, cache_dtype, out_f32;
  int part_rows;  // of a token's rows, per grid row
  PoolArgs pool;
  Watchdog wd;
};

// A group of W lanes takes one token and `part_rows` of its 2 hkv rows (one
// part per grid row).
template <int W, int kCache>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs A) {
  const Group<W> G;
  const int d = A.pool.d, hkv = A.pool.hkv;
  const int64_t at_token = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  if (at_token >= A.total) return;
  const int t = static_cast<int>(at_token), part = blockIdx.y;  // neighbouring groups: neighbouring rows
  int b, i;
  int64_t row0;
  if (!seq_of_token(A.cu, A.batch, t, b, i)) return;
  if (!page_row(A.pool, b, static_cast<int64_t>(A.start != nullptr ? A.start[b] : 0) + i, row0)) {
    if (G.l == 0) record_status(A.wd, kStatusRange);
    return;
  }
  if (8 * G.l >= d) return;
  const int r1 = min((part + 1) * A.part_rows, 2 * hkv);
#pragma unroll 4
  for (int r = part * A.part_rows; r < r1; ++r) {
    const bool is_v = r >= hkv;
    const int g = is_v ? r - hkv : r;
    const int64_t row = row0 + static_cast<int64_t>(g) * A.pool.page_size;
    const void* pool = is_v ? A.v_cache : A.k_cache;
    const float* scales = is_v ? A.v_scales : A.k_scales;
    float2 x[4];
    if constexpr (kCache == FA_BF16) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pool) + row * d + 8 * G.l));
      widen8<__nv_bfloat16>(make_uint2(w.x, w.y), make_uint2(w.z, w.w), x);
    } else if constexpr (kCache == FA_I8) {
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(pool) + row * d + 8 * G.l));
      const float s = scales[row];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int u = static_cast<int>(e < 2 ? w.x : w.y) >> (16 * (e & 1));
        x[e] = mul2(make_float2(static_cast<float>(static_cast<int8_t>(u)), static_cast<float>(static_cast<int8_t>(u >> 8))),
                    make_float2(s, s));
      }
    } else {
      const uint32_t w =
          __ldcs(reinterpret_cast<const unsigned int*>(static_cast<const uint8_t*>(pool) + row * (d / 2) + 4 * G.l));
      const float2 s = *reinterpret_cast<const float2*>(scales + 2 * row);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // code + 2^23, exact, less 2^23
        const float2 c = make_float2(__uint_as_float(((w >> (8 * e)) & 15u) | 0x4b000000u),
                                     __uint_as_float(((w >> (8 * e + 4)) & 15u) | 0x4b000000u));
        const float2 code = add2(c, make_float2(-8388608.0f, -8388608.0f));
        // in scalars: a packed product and sum would become one operation
        x[e] = make_float2(__fadd_rn(__fmul_rn(code.x, s.x), s.y), __fadd_rn(__fmul_rn(code.y, s.x), s.y));
      }
    }
    const int64_t at = (static_cast<int64_t>(g) * A.total + t) * d + 8 * G.l;
    if (A.out_f32) {
      float* dst = static_cast<float*>(is_v ? A.v_out : A.k_out) + at;
      __stcs(reinterpret_cast<float4*>(dst), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
      __stcs(reinterpret_cast<float4*>(dst + 4), make_float4(x[2].x, x[2].y, x[3].x, x[3].y));
    } else {
      const uint2 u = pack4(x[0], x[1]), v = pack4(x[2], x[3]);
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? A.v_out : A.k_out) + at),
             make_uint4(u.x, u.y, v.x, v.y));
    }
  }
}

PoolArgs pool_args(const fa_kv_pages& pg, int hkv, int d) {
  PoolArgs P;
  P.block_table = pg.block_table;
  P.max_pages = pg.max_pages;
  P.page_size = pg.page_size;
  P.num_pages = pg.num_pages;
  P.hkv = hkv;
  P.d = d;
  P.capacity = static_cast<int64_t>(pg.max_pages) * pg.page_size;
  return P;
}

// Rows of a token per group: four, and twice that while the groups fill the
// device several times over (the lookups of a token are then spread over more rows).
int rows_per_item(int64_t total, int rows, int groups) {
  const int64_t enough = static_cast<int64_t>(device_sm_count()) * 8 * groups;
  int per = kRows;
  while (per < rows && total * ((rows + per - 1) / per) > enough) per *= 2;
  return per;
}

template <typename T, int W, int kCache>
fa_status launch_append_typed(AppendArgs& A, const LaunchCtx& ctx) {
  constexpr int kGroups = kThreads / W;
  A.token_rows = A.hq + (A.bounds != nullptr ? 1 : 2) * A.pool.hkv;
  A.part_rows = rows_per_item(A.total, A.token_rows, kGroups);
  const int parts = (A.token_rows + A.part_rows - 1) / A.part_rows;
  A.window = A.total <= 4 * device_sm_count() ? 1 : 8;
  int blocks = A.total / kGroups + 1;  // at least one, for cache_seqlens alone
  const int page_blocks = A.bounds != nullptr ? A.total / A.window + 1 : 0;
  if (blocks < page_blocks) blocks = page_blocks;
  if (parts >= 65535) return FA_ERR_UNSUPPORTED;
  note_variant(reinterpret_cast<const void*>(append_kernel<T, W, kCache>));
  append_kernel<T, W, kCache><<<dim3(blocks, parts + (A.bounds != nullptr ? 1 : 0)), kThreads, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
}
template <typename T, int W>
fa_status launch_append_width(AppendArgs& A, const LaunchCtx& ctx) {
  if (A.cache_dtype == FA_BF16) return launch_append_typed<T, W, FA_BF16>(A, ctx);
  if (A.cache_dtype == FA_I8) return launch_append_typed<T, W, FA_I8>(A, ctx);
  return launch_append_typed<T, W, FA_I4>(A, ctx);
}
template <typename T>
fa_status launch_append(AppendArgs& A, const LaunchCtx& ctx) {
  if (A.pool.d <= 16) return launch_append_width<T, 2>(A, ctx);
  if (A.pool.d <= 32) return launch_append_width<T, 4>(A, ctx);
  if (A.pool.d <= 64) return launch_append_width<T, 8>(A, ctx);
  if (A.pool.d <= 128) return launch_append_width<T, 16>(A, ctx);
  return launch_append_width<T, 32>(A, ctx);
}

template <int W, int kCache>
fa_status launch_read_typed(ReadArgs& A, const LaunchCtx& ctx) {
  constexpr int kGroups = kThreads / W;
  A.part_rows = rows_per_item(A.total, 2 * A.pool.hkv, kGroups);
  const int parts = (2 * A.pool.hkv + A.part_rows - 1) / A.part_rows;
  if (parts > 65535) return FA_ERR_UNSUPPORTED;
  note_variant(reinterpret_cast<const void*>(read_kernel<W, kCache>));
  read_kernel<W, kCache><<<dim3((A.total - 1) / kGroups + 1, parts), kThreads, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
}
template <int W>
fa_status launch_read(ReadArgs& A, const LaunchCtx& ctx) {
  if (A.cache_dtype == FA_BF16) return launch_read_typed<W, FA_BF16>(A, ctx);
  if (A.cache_dtype == FA_I8) return launch_read_typed<W, FA_I8>(A, ctx);
  return launch_read_typed<W, FA_I4>(A, ctx);
}

}  // namespace

fa_status launch_kv_append_rope(const fa_kv_append_rope_params& p, const fa_kv_pages& pages, const LaunchCtx& ctx) {
  if (p.total == 0 && p.cache_seqlens == nullptr) return FA_OK;
  AppendArgs A;
  A.k_new = p.k_new;
  A.v_new = p.v_new;
  A.q = p.q;
  A.q_out = static_cast<__nv_bfloat16*>(p.q_out);
  A.k_ts = p.k_token_stride;
  A.k_hs = p.k_head_stride;
  A.v_ts = p.v_token_stride;
  A.v_hs = p.v_head_stride;
  A.q_ts = p.q_token_stride;
  A.q_hs = p.q_head_stride;
  A.qo_ts = p.q_out_token_stride;
  A.qo_hs = p.q_out_head_stride;
  A.rope = p.rope_table;
  A.k_cache = p.k_cache;
  A.v_cache = p.v_cache;
  A.k_scales = p.k_scales;
  A.v_scales = p.v_scales;
  A.bounds = static_cast<__nv_bfloat16*>(p.key_bounds);
  A.cu = p.cu_seqlens;
  A.cur_pos = p.cur_pos;
  A.seqlens = p.cache_seqlens;
  A.batch = p.batch;
  A.total = p.total;
  A.hq = p.q != nullptr ? p.hq : 0;
  A.rot = p.rot_dim;
  A.interleaved = p.interleaved;
  A.rope_rows = p.rope_rows;
  A.cache_dtype = p.cache_dtype;
  A.pool = pool_args(pages, p.hkv, p.head_dim);
  A.wd = ctx.wd;
  if (p.x_dtype == FA_BF16) return launch_append<__nv_bfloat16>(A, ctx);
  return launch_append<float>(A, ctx);
}

fa_status launch_kv_read(const fa_kv_read_params& p, const fa_kv_pages& pages, const LaunchCtx& ctx) {
  if (p.total == 0) return FA_OK;
  ReadArgs A;
  A.k_cache = p.k_cache;
  A.v_cache = p.v_cache;
  A.k_scales = p.k_scales;
  A.v_scales = p.v_scales;
  A.k_out = p.k_out;
  A.v_out = p.v_out;
  A.cu = p.cu_seqlens;
  A.start = p.start;
  A.batch = p.batch;
  A.total = p.total;
  A.cache_dtype = p.cache_dtype;
  A.out_f32 = p.out_dtype == FA_F32 ? 1 : 0;
  A.pool = pool_args(pages, p.hkv, p.head_dim);
  A.wd = ctx.wd;
  if (p.head_dim <= 16) return launch_read<2>(A, ctx);
  if (p.head_dim <= 32) return launch_read<4>(A, ctx);
  if (p.head_dim <= 64) return launch_read<8>(A, ctx);
  if (p.head_dim <= 128) return launch_read<16>(A, ctx);
  return launch_read<32>(A, ctx);
}

}  // namespace fa
