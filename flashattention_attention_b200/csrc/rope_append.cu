// rope_append.cu -- append of any number of new tokens per sequence to a paged
// cache, keys and queries rotated to their positions on the way, and the
// read-back of cached rows (FlashRT QKV Cache RoPE, Kernels: rotation and
// cache write of the new K fused in one kernel).
//
// A row of d channels is held by W lanes (d / 16 rounded up to a power of two),
// 16 channels per lane in two chunks of eight (16-byte loads of bf16).  Rotating
// channel pairs (i, i + rot/2), lane i takes the chunks [8i, 8i+8) and [rot/2 +
// 8i, +8), so both members of a pair sit in one lane; rotating pairs (2i,
// 2i+1), and for channels past rot_dim, the two chunks are adjacent.  Either way
// lane i's eight pairs use angles 8i .. 8i+7.
//
// One launch does everything.  A group of W lanes takes one token and some of
// its rows: the token's sequence, slot, page and angles are found once and
// two rows' loads are in flight at a time.  Keys whose page bounds are kept
// go another way, since all new keys of a page have to meet: a CTA per page
// (of the first new token in it), its groups spread over KV heads and slices
// of the page's tokens, the slices' bounds joined in shared memory.  No page
// is touched by two CTAs, so there are no atomics and no order to depend on.
//
// Waits for memory at three CTAs an SM, two rows in flight a group: 16,384 tokens
// of 32 + 8 + 8 heads of 128 rotated, quantised to 4 bits and read back move 450
// MB in 107 us, 4.2 TB/s (64 % of a plain copy).  Both roles share one kernel and
// its 80 registers a thread, which do not hold all of it: 168 bytes a thread are
// spilled for bf16 rows into 4 bits at d = 128 (-Xptxas -v; 112 into int8, 56 into
// bf16, up to 188 for fp32 rows).  Two CTAs an SM: 125 us; four, with fewer
// registers: 110; four rows in flight: 108; roles in kernels of their own have not
// been tried.
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
  if (rotated && !A.interleaved && 16 * l < A.rot) {
    a = 8 * l;
    b = A.rot / 2 + 8 * l;
  } else {
    a = 16 * l;
    b = a + 8;
  }
}

// Eight consecutive elements as they are loaded, and their exact widening.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void widen(float2* x) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
};
template <>
struct Chunk<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = __ldcs(reinterpret_cast<const float4*>(p));
    hi = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void widen(float2* x) const {
    x[0] = make_float2(lo.x, lo.y);
    x[1] = make_float2(lo.z, lo.w);
    x[2] = make_float2(hi.x, hi.y);
    x[3] = make_float2(hi.z, hi.w);
  }
};

// A lane's 16 channels are x[0 .. 3] of chunk a and x[4 .. 7] of chunk b.

// The lane's eight angles at a slot; no rotation for lanes past rot_dim.
struct Angles {
  float2 c[4], s[4];
  bool any;
};
__device__ __forceinline__ Angles angles_of(const AppendArgs& A, int l, int64_t slot) {
  Angles r;
  r.any = 16 * l < A.rot;
#pragma unroll
  for (int e = 0; e < 4; ++e) r.c[e] = r.s[e] = make_float2(0.f, 0.f);
  if (r.any) {
    const float4* c = reinterpret_cast<const float4*>(A.rope + slot * A.rot + 8 * l);
    const float4* s = reinterpret_cast<const float4*>(A.rope + slot * A.rot + A.rot / 2 + 8 * l);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 u = c[e], v = s[e];
      r.c[2 * e] = make_float2(u.x, u.y);
      r.c[2 * e + 1] = make_float2(u.z, u.w);
      r.s[2 * e] = make_float2(v.x, v.y);
      r.s[2 * e + 1] = make_float2(v.z, v.w);
    }
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
__device__ __forceinline__ void rotate16(const AppendArgs& A, const Angles& g, float2 (&x)[8]) {
  if (!g.any) return;
  if (A.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rotate_pair(x[2 * e].x, x[2 * e].y, g.c[e].x, g.s[e].x);
      rotate_pair(x[2 * e + 1].x, x[2 * e + 1].y, g.c[e].y, g.s[e].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rotate_pair(x[e].x, x[4 + e].x, g.c[e].x, g.s[e].x);
      rotate_pair(x[e].y, x[4 + e].y, g.c[e].y, g.s[e].y);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(bf16x2(x[0].x, x[0].y), bf16x2(x[1].x, x[1].y), bf16x2(x[2].x, x[2].y), bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ void store16_bf16(__nv_bfloat16* row, int a, int b, const float2 (&x)[8]) {
  *reinterpret_cast<uint4*>(row + a) = pack8(x);
  *reinterpret_cast<uint4*>(row + b) = pack8(x + 4);
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
  // a power of two that keeps 15 (x - lo) finite and leaves the quotient as it is
  const float k = r > 0x1p60f ? 0x1p-8f : 1.0f, kr = __fmul_rn(r, k);
  for (int e = 0; e < 4; ++e) {
    const float q = r > 0.0f ? __fdiv_rn(__fmul_rn(__fmul_rn(__fsub_rn(x[e], lo), k), 15.0f), kr) : 0.0f;
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
__device__ __forceinline__ void store_row(const Sink<kCache>& to, int l, bool own, int a, int b, const float2 (&x)[8],
                                          unsigned mask) {
  if constexpr (kCache == FA_BF16) {
    if (own) store16_bf16(reinterpret_cast<__nv_bfloat16*>(to.dst), a, b, x);
  } else if constexpr (kCache == FA_I8) {
    float amax = 0.0f;
    if (own) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
    }
#pragma unroll
    for (int off = W >> 1; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, off));
    constexpr float k127 = 1.0f / 127.0f;
    const float s = ordinary(amax) ? divide_by(amax, 127.0f, k127) : divide_any(amax, 127.0f);
    if (own) {
      uint32_t w[4];
      if (ordinary(s)) {
        const float y = __frcp_rn(s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v[4] = {x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y};
          w[e] = quantise4_fast(v, s, y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = codes8_any(x[2 * e], x[2 * e + 1], s);
      }
      *reinterpret_cast<uint2*>(to.dst + a) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(to.dst + b) = make_uint2(w[2], w[3]);
      if (l == 0) *to.scale = s;
    }
  } else {
    float lo = INFINITY, hi = -INFINITY;
    if (own) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
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
      uint32_t w[4];
      float step;
      if (ordinary(r)) {
        const float y = __frcp_rn(r);
        constexpr float k15 = 1.0f / 15.0f;
        step = divide_by(r, 15.0f, k15);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = codes4_fast(x[2 * e], x[2 * e + 1], lo, r, y);
      } else {
        step = divide_any(r, 15.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = codes4_any(x[2 * e], x[2 * e + 1], lo, r);
      }
      *reinterpret_cast<uint32_t*>(to.dst + a / 2) = w[0] | (w[1] << 16);
      *reinterpret_cast<uint32_t*>(to.dst + b / 2) = w[2] | (w[3] << 16);
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

constexpr int kRows = 2;  // rows a group has in flight

// The rows [r0, r1) of one token: its hq queries, then its V rows, then (when
// the page role does not take them) its K rows.
template <typename T, int W, int kCache>
__device__ __forceinline__ void append_token(const AppendArgs& A, int t, int r0, int r1) {
  const Group<W> G;
  const bool own = 16 * G.l < A.pool.d;
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
    Chunk<T> u[kRows], v[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (own && r + k < q1) {
        u[k].load(q + k * A.q_hs + a);
        v[k].load(q + k * A.q_hs + b);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (own && r + k < q1) {
        float2 x[8];
        u[k].widen(x);
        v[k].widen(x + 4);
        rotate16(A, ang, x);
        store16_bf16(qo + k * A.qo_hs, a, b, x);
      }
    }
  }
  // heads [g0, g1) of V or K
  auto cached = [&](auto rotated, const void* rows, int64_t ts, int64_t hs, void* pool, float* scales, int g0, int g1) {
    constexpr bool kRotated = decltype(rotated)::value;
    const int ra = kRotated ? a : 16 * G.l, rb = kRotated ? b : 16 * G.l + 8;
    const T* src = static_cast<const T*>(rows) + t * ts + g0 * hs;
    Sink<kCache> to(pool, scales, p.row0 + static_cast<int64_t>(g0) * A.pool.page_size, A.pool.d);
#pragma unroll 2
    for (int g = g0; g < g1; ++g, src += hs) {
      float2 x[8];
      if (own) {
        Chunk<T> u, v;
        u.load(src + ra);
        v.load(src + rb);
        u.widen(x);
        v.widen(x + 4);
        if constexpr (kRotated) rotate16(A, ang, x);
      }
      store_row<W, kCache>(to, G.l, own, ra, rb, x, G.mask);
      to.advance(A.pool.page_size, A.pool.d);
    }
  };
  cached(std::false_type{}, A.v_new, A.v_ts, A.v_hs, A.v_cache, A.v_scales, max(r0 - hq, 0), min(r1 - hq, hkv));
  cached(std::true_type{}, A.k_new, A.k_ts, A.k_hs, A.k_cache, A.k_scales, max(r0 - hq - hkv, 0), r1 - hq - hkv);
}

// The new keys of the pages whose first new token is one of `window` tokens
// from t0 on, and those pages' bounds; the whole CTA together.
template <typename T, int W, int kCache>
__device__ __forceinline__ void append_pages(const AppendArgs& A, int t0, uint32_t (&s_lo)[8][kThreads],
                                             uint32_t (&s_hi)[8][kThreads]) {
  constexpr int kGroups = kThreads / W;
  const Group<W> G;
  const bool own = 16 * G.l < A.pool.d;
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
      // in bf16 pairs: rounding keeps the order, so the rounded bounds are the bounds of the rounded keys
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = 0x7f807f80u;  // +inf
        hi[e] = 0xff80ff80u;  // -inf
      }
      if (g < hkv && slice < slices) {
        const T* src = static_cast<const T*>(A.k_new) + static_cast<int64_t>(t + slice) * A.k_ts + g * A.k_hs;
        Sink<kCache> to(A.k_cache, A.k_scales, row0 + slice + static_cast<int64_t>(g) * page, A.pool.d);
#pragma unroll 2
        for (int j = slice; j < n; j += slices, src += slices * A.k_ts) {
          float2 x[8];
          if (own) {
            Chunk<T> u, v;
            u.load(src + ca);
            v.load(src + cb);
            u.widen(x);
            v.widen(x + 4);
            rotate16(A, angles_of(A, G.l, slot + j), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t k = bf16x2(x[e].x, x[e].y);
              lo[e] = bf16x2_min(lo[e], k);
              hi[e] = bf16x2_max(hi[e], k);
            }
          }
          store_row<W, kCache>(to, G.l, own, ca, cb, x, G.mask);
          to.advance(slices, A.pool.d);
        }
      }
      if (slices > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s_lo[e][threadIdx.x] = lo[e];
          s_hi[e][threadIdx.x] = hi[e];
        }
        __syncthreads();
        if (slice == 0) {
#pragma unroll 1
          for (int o = 1; o < slices; ++o) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              lo[e] = bf16x2_min(lo[e], s_lo[e][threadIdx.x + o * hkv * W]);
              hi[e] = bf16x2_max(hi[e], s_hi[e][threadIdx.x + o * hkv * W]);
            }
          }
        }
      }
      if (g < hkv && slice == 0 && own) {
        const int64_t plane = row0 / page + g;  // page * hkv + g
        uint4* row[4];  // the low row's two chunks, the high row's
        row[0] = reinterpret_cast<uint4*>(A.bounds + plane * 2 * A.pool.d + ca);
        row[1] = reinterpret_cast<uint4*>(A.bounds + plane * 2 * A.pool.d + cb);
        row[2] = reinterpret_cast<uint4*>(A.bounds + (plane * 2 + 1) * A.pool.d + ca);
        row[3] = reinterpret_cast<uint4*>(A.bounds + (plane * 2 + 1) * A.pool.d + cb);
        if (at > 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 u = *row[c], v = *row[2 + c];
            const uint32_t ul[4] = {u.x, u.y, u.z, u.w}, vl[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[4 * c + e] = bf16x2_min(lo[4 * c + e], ul[e]);
              hi[4 * c + e] = bf16x2_max(hi[4 * c + e], vl[e]);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          *row[c] = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
          *row[2 + c] = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
        }
      }
    }
  }
}

template <typename T, int W, int kCache>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const AppendArgs A) {
  __shared__ uint32_t s_lo[8][kThreads], s_hi[8][kThreads];
  griddep_launch_dependents();
  griddep_wait();
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
  if (blockIdx.x == 0 && part == 0) {  // offsets and lengths, once
    for (int b = threadIdx.x; b < A.batch; b += kThreads) {
      const int64_t c0 = A.cu != nullptr ? A.cu[b] : b, c1 = A.cu != nullptr ? A.cu[b + 1] : b + 1;
      const int64_t end = static_cast<int64_t>(A.cur_pos[b]) + (c1 - c0);
      const bool past_table = A.rot > 0 && c1 > c0 && end > A.rope_rows;  // its last tokens are not written
      if (c0 < 0 || c1 < c0 || c1 > A.total || A.cur_pos[b] < 0 || end > A.pool.capacity || past_table) {
        record_status(A.wd, kStatusRange);
      } else if (A.seqlens != nullptr) {
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

// A group of W lanes (d / 8 rounded up to a power of two, eight channels a
// lane) takes one token and `part_rows` of its 2 hkv rows (one part per grid row).
template <int W, int kCache>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs A) {
  griddep_launch_dependents();
  griddep_wait();
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
      Chunk<__nv_bfloat16> u;
      u.load(static_cast<const __nv_bfloat16*>(pool) + row * d + 8 * G.l);
      u.widen(x);
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
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? A.v_out : A.k_out) + at), pack8(x));
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
// device several times over (the lookups of a token are then spread over more
// rows).  One token of 32 + 8 + 8 heads: 4.2 us with four rows, 6.2 with eight; a
// 16384-token prompt: 124 us with four, 115 with eight, 107 with this rule.
int rows_per_item(int64_t total, int rows, int groups) {
  const int64_t enough = static_cast<int64_t>(device_sm_count()) * 8 * groups;
  int per = 4;
  while (per < rows && total * ((rows + per - 1) / per) > enough) per *= 2;
  return per;
}

template <typename T, int W, int kCache>
fa_status launch_append_typed(AppendArgs& A, const LaunchCtx& ctx) {
  constexpr int kGroups = kThreads / W;
  A.token_rows = A.hq + (A.bounds != nullptr ? 1 : 2) * A.pool.hkv;
  A.part_rows = rows_per_item(A.total, A.token_rows, kGroups);
  const int parts = (A.token_rows + A.part_rows - 1) / A.part_rows;
  // page role: a CTA per token where there are few, else per eight tokens.
  // One and eight a CTA, us, 32 + 8 + 8 heads of 128 into 4 bits: 148 sequences
  // of one token 8.3 and 16.5, 592 (the border on 148 SMs) 16.5 and 16.5, 740:
  // 18.5 and 18.5, 1184: 26.7 and 20.5; a prompt of 592 tokens 22.2 and 20.5, of
  // 2368: 37 and 24.7, of 16,384, most of which open no page, 164 and 107 with
  // the read-back
  A.window = A.total <= 4 * device_sm_count() ? 1 : 8;
  int blocks = A.total / kGroups + 1;  // at least one, for the lengths alone
  const int page_blocks = A.bounds != nullptr ? A.total / A.window + 1 : 0;
  if (blocks < page_blocks) blocks = page_blocks;
  if (parts >= 65535) return FA_ERR_UNSUPPORTED;
  return launch_dependent(append_kernel<T, W, kCache>, dim3(blocks, parts + (A.bounds != nullptr ? 1 : 0)), kThreads, 0, 0,
                          ctx.stream, A);
}
template <typename T, int W>
fa_status launch_append_width(AppendArgs& A, const LaunchCtx& ctx) {
  if (A.cache_dtype == FA_BF16) return launch_append_typed<T, W, FA_BF16>(A, ctx);
  if (A.cache_dtype == FA_I8) return launch_append_typed<T, W, FA_I8>(A, ctx);
  return launch_append_typed<T, W, FA_I4>(A, ctx);
}
template <typename T>
fa_status launch_append(AppendArgs& A, const LaunchCtx& ctx) {
  if (A.pool.d <= 16) return launch_append_width<T, 1>(A, ctx);
  if (A.pool.d <= 32) return launch_append_width<T, 2>(A, ctx);
  if (A.pool.d <= 64) return launch_append_width<T, 4>(A, ctx);
  if (A.pool.d <= 128) return launch_append_width<T, 8>(A, ctx);
  return launch_append_width<T, 16>(A, ctx);
}

template <int W, int kCache>
fa_status launch_read_typed(ReadArgs& A, const LaunchCtx& ctx) {
  constexpr int kGroups = kThreads / W;
  A.part_rows = rows_per_item(A.total, 2 * A.pool.hkv, kGroups);
  const int parts = (2 * A.pool.hkv + A.part_rows - 1) / A.part_rows;
  if (parts > 65535) return FA_ERR_UNSUPPORTED;
  return launch_dependent(read_kernel<W, kCache>, dim3((A.total - 1) / kGroups + 1, parts), kThreads, 0, 0, ctx.stream, A);
}
template <int W>
fa_status launch_read(ReadArgs& A, const LaunchCtx& ctx) {
  if (A.cache_dtype == FA_BF16) return launch_read_typed<W, FA_BF16>(A, ctx);
  if (A.cache_dtype == FA_I8) return launch_read_typed<W, FA_I8>(A, ctx);
  return launch_read_typed<W, FA_I4>(A, ctx);
}

}  // namespace

fa_status launch_kv_append_rope(const fa_kv_append_rope_params& p, const fa_kv_pages& pages, const LaunchCtx& ctx) {
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
