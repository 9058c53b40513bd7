// rope_append.cu -- append of any number of new tokens per sequence to a paged
// cache, keys and queries rotated to their positions on the way, and the
// read-back of cached rows (FlashRT QKV Cache RoPE, Kernels: rotation and
// cache write of the new K fused in one kernel).
//
// A row of d channels is held by d / 8 lanes, eight channels per lane in two
// chunks of four.  Rotating channel pairs (i, i + rot/2), lane i takes the
// chunks [4i, 4i+4) and [rot/2 + 4i, +4), so both members of a pair sit in
// one lane; rotating pairs (2i, 2i+1), and for channels past rot_dim, the two
// chunks are adjacent.  Either way lane i's four pairs use angles 4i .. 4i+3.
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

template <typename T>
__device__ __forceinline__ void load8(const T* row, int a, int b, float (&x)[8]) {
  float u[4], v[4];
  Vec4<T>::widen(Vec4<T>::load(row + a), u);
  Vec4<T>::widen(Vec4<T>::load(row + b), v);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = u[e];
    x[4 + e] = v[e];
  }
}

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}
__device__ __forceinline__ void rotate8(const AppendArgs& A, int l, int64_t slot, float (&x)[8]) {
  if (8 * l >= A.rot) return;
  const float* row = A.rope + slot * A.rot;
  const float4 c = *reinterpret_cast<const float4*>(row + 4 * l);
  const float4 s = *reinterpret_cast<const float4*>(row + A.rot / 2 + 4 * l);
  if (A.interleaved) {
    rotate_pair(x[0], x[1], c.x, s.x);
    rotate_pair(x[2], x[3], c.y, s.y);
    rotate_pair(x[4], x[5], c.z, s.z);
    rotate_pair(x[6], x[7], c.w, s.w);
  } else {
    rotate_pair(x[0], x[4], c.x, s.x);
    rotate_pair(x[1], x[5], c.y, s.y);
    rotate_pair(x[2], x[6], c.z, s.z);
    rotate_pair(x[3], x[7], c.w, s.w);
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void store8_bf16(__nv_bfloat16* row, int a, int b, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(row + a) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + b) = make_uint2(bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// Code of one channel of a 4-bit row: round_half_even(15 (x - lo) / r); the
// quotient is the correctly rounded one (Markstein's step as in quant.cu where
// r and 1 / r are normal, the IEEE division elsewhere), so the exact halves
// that rows of bf16 values are full of stay exact.
__device__ __forceinline__ uint32_t code4(float x, float lo, float r, float y, bool fast) {
  const float u = __fmul_rn(__fsub_rn(x, lo), 15.0f);
  float q;
  if (fast) {
    const float q0 = __fmul_rn(u, y);
    q = __fmaf_rn(__fmaf_rn(-q0, r, u), y, q0);
  } else {
    q = r > 0.0f ? __fdiv_rn(u, r) : 0.0f;
  }
  return static_cast<uint32_t>(__float2int_rn(q)) & 15u;
}

// One row into the cache by the `width` lanes that hold it (`own`: this lane
// holds channels).  Every lane of the group calls.
__device__ __forceinline__ void store_row(const AppendArgs& A, bool is_v, int64_t row, int l, int width, bool own,
                                          int a, int b, const float (&x)[8], unsigned mask) {
  void* pool = is_v ? A.v_cache : A.k_cache;
  const int d = A.pool.d;
  if (A.cache_dtype == FA_BF16) {
    if (own) store8_bf16(static_cast<__nv_bfloat16*>(pool) + row * d, a, b, x);
    return;
  }
  float* scales = is_v ? A.v_scales : A.k_scales;
  if (A.cache_dtype == FA_I8) {
    float amax = 0.0f;
    if (own) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
    }
    for (int off = width >> 1; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, off));
    const float s = __fdiv_rn(amax, 127.0f);
    const bool fast = s >= 0x1p-60f && s <= 0x1p60f;
    const float y = fast ? __frcp_rn(s) : 0.0f;
    if (own) {
      int8_t* dst = static_cast<int8_t*>(pool) + row * d;
      const float u[4] = {x[0], x[1], x[2], x[3]}, v[4] = {x[4], x[5], x[6], x[7]};
      *reinterpret_cast<uint32_t*>(dst + a) = fast ? quantise4_fast(u, s, y) : quantise4_div(u, s);
      *reinterpret_cast<uint32_t*>(dst + b) = fast ? quantise4_fast(v, s, y) : quantise4_div(v, s);
    }
    if (l == 0) scales[row] = s;
    return;
  }
  float lo = INFINITY, hi = -INFINITY;
  if (own) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
    }
  }
  for (int off = width >> 1; off > 0; off >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, off));
  }
  const float r = __fsub_rn(hi, lo);
  const bool fast = r >= 0x1p-60f && r <= 0x1p60f;
  const float y = fast ? __frcp_rn(r) : 0.0f;
  if (own) {
    uint8_t* dst = static_cast<uint8_t*>(pool) + row * (d / 2);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= code4(x[e], lo, r, y, fast) << (4 * (e & 3));
    *reinterpret_cast<uint16_t*>(dst + a / 2) = static_cast<uint16_t>(w[0]);
    *reinterpret_cast<uint16_t*>(dst + b / 2) = static_cast<uint16_t>(w[1]);
  }
  if (l == 0) *reinterpret_cast<float2*>(scales + 2 * row) = make_float2(__fdiv_rn(r, 15.0f), lo);
}

// The lane group of this thread: `width` lanes (a power of two) per row.
struct Group {
  int width, l;
  unsigned mask;
  bool own;
};
__device__ __forceinline__ Group lane_group(int d) {
  Group g;
  g.width = 2;
  while (g.width * 8 < d) g.width <<= 1;
  const int lane = threadIdx.x & 31;
  g.l = lane & (g.width - 1);
  g.mask = g.width == 32 ? 0xffffffffu : ((1u << g.width) - 1u) << (lane & ~(g.width - 1));
  g.own = 8 * g.l < d;
  return g;
}

// Rows of every new token: Q, K (unless the bounds kernel takes them) and V.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const AppendArgs A) {
  const Group G = lane_group(A.pool.d);
  if (A.seqlens != nullptr && blockIdx.x == 0) {
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
  const int per_token = A.hq + (A.bounds != nullptr ? 1 : 2) * A.pool.hkv;
  const int64_t items = static_cast<int64_t>(A.total) * per_token;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / G.width);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / G.width) + threadIdx.x / G.width; it < items;
       it += groups) {
    const int t = static_cast<int>(it / per_token);
    int h = static_cast<int>(it % per_token);
    Place p;
    bool bad;
    if (!place_token(A, t, p, bad)) {
      if (bad && G.l == 0) record_status(A.wd, kStatusRange);
      continue;
    }
    float x[8];
    int a, b;
    if (h < A.hq) {
      chunk_offsets(A, G.l, true, a, b);
      if (G.own) {
        load8(static_cast<const T*>(A.q) + t * A.q_ts + h * A.q_hs, a, b, x);
        rotate8(A, G.l, p.slot, x);
        store8_bf16(A.q_out + t * A.qo_ts + h * A.qo_hs, a, b, x);
      }
      continue;
    }
    h -= A.hq;
    const bool is_v = h < A.pool.hkv;
    if (!is_v) h -= A.pool.hkv;
    chunk_offsets(A, G.l, !is_v, a, b);
    if (G.own) {
      load8(is_v ? static_cast<const T*>(A.v_new) + t * A.v_ts + h * A.v_hs
                 : static_cast<const T*>(A.k_new) + t * A.k_ts + h * A.k_hs, a, b, x);
      if (!is_v) rotate8(A, G.l, p.slot, x);
    }
    store_row(A, is_v, p.row0 + static_cast<int64_t>(h) * A.pool.page_size, G.l, G.width, G.own, a, b, x, G.mask);
  }
}

// Keys with bounds: the CTA of a page's first new token writes all of the
// page's new keys and folds them into the page's bounds, one lane group per
// KV head, so no two groups touch one page's bounds.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_keys_kernel(const AppendArgs A) {
  const Group G = lane_group(A.pool.d);
  const int t0 = blockIdx.x;
  Place p;
  bool bad;
  if (!place_token(A, t0, p, bad)) return;  // reported by the rows kernel
  int b, i;
  seq_of_token(A.cu, A.batch, t0, b, i);
  const int off = static_cast<int>(p.slot % A.pool.page_size);
  if (i > 0 && off > 0) return;  // an earlier token's CTA has this page
  const int left = A.cu != nullptr ? min(A.cu[b + 1], A.total) - t0 : 1;
  const int n = min(left, A.pool.page_size - off);
  int ca, cb;
  chunk_offsets(A, G.l, true, ca, cb);
  for (int g = threadIdx.x / G.width; g < A.pool.hkv; g += kThreads / G.width) {
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = INFINITY;
      hi[e] = -INFINITY;
    }
    for (int j = 0; j < n; ++j) {
      float x[8];
      if (A.rot > 0 && p.slot + j >= A.rope_rows) break;
      if (G.own) {
        load8(static_cast<const T*>(A.k_new) + (t0 + j) * A.k_ts + g * A.k_hs, ca, cb, x);
        rotate8(A, G.l, p.slot + j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = fminf(lo[e], x[e]);
          hi[e] = fmaxf(hi[e], x[e]);
        }
      }
      store_row(A, false, p.row0 + j + static_cast<int64_t>(g) * A.pool.page_size, G.l, G.width, G.own, ca, cb, x,
                G.mask);
    }
    if (G.own) {
      const int64_t plane = p.row0 / A.pool.page_size + g;  // page * hkv + g
      __nv_bfloat16* dst = A.bounds + plane * 2 * A.pool.d;
      if (off > 0) {
        float olo[8], ohi[8];
        load8<__nv_bfloat16>(dst, ca, cb, olo);
        load8<__nv_bfloat16>(dst + A.pool.d, ca, cb, ohi);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = fminf(lo[e], olo[e]);
          hi[e] = fmaxf(hi[e], ohi[e]);
        }
      }
      store8_bf16(dst, ca, cb, lo);
      store8_bf16(dst + A.pool.d, ca, cb, hi);
    }
  }
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
  PoolArgs pool;
  Watchdog wd;
};

__global__ void __launch_bounds__(kThreads) read_rows_kernel(const ReadArgs A) {
  const Group G = lane_group(A.pool.d);
  const int d = A.pool.d, hkv = A.pool.hkv;
  const int64_t items = static_cast<int64_t>(A.total) * 2 * hkv;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / G.width);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / G.width) + threadIdx.x / G.width; it < items;
       it += groups) {
    const int t = static_cast<int>(it % A.total);  // neighbours read neighbouring rows
    const int h = static_cast<int>(it / A.total);
    const bool is_v = h >= hkv;
    const int g = is_v ? h - hkv : h;
    int b, i;
    if (!seq_of_token(A.cu, A.batch, t, b, i)) continue;
    int64_t row;
    if (!page_row(A.pool, b, static_cast<int64_t>(A.start != nullptr ? A.start[b] : 0) + i, row)) {
      if (G.l == 0) record_status(A.wd, kStatusRange);
      continue;
    }
    if (!G.own) continue;
    row += static_cast<int64_t>(g) * A.pool.page_size;
    const void* pool = is_v ? A.v_cache : A.k_cache;
    const float* scales = is_v ? A.v_scales : A.k_scales;
    float x[8];
    if (A.cache_dtype == FA_BF16) {
      load8<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(pool) + row * d, 8 * G.l, 8 * G.l + 4, x);
    } else if (A.cache_dtype == FA_I8) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(pool) + row * d + 8 * G.l);
      const float s = scales[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = e < 4 ? w.x : w.y;
        x[e] = __fmul_rn(static_cast<float>(static_cast<int8_t>(u >> (8 * (e & 3)))), s);
      }
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pool) + row * (d / 2) + 4 * G.l);
      const float2 s = *reinterpret_cast<const float2*>(scales + 2 * row);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(__fmul_rn(static_cast<float>((w >> (4 * e)) & 15u), s.x), s.y);
    }
    const int64_t at = (static_cast<int64_t>(g) * A.total + t) * d + 8 * G.l;
    if (A.out_f32) {
      float* dst = static_cast<float*>(is_v ? A.v_out : A.k_out) + at;
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? A.v_out : A.k_out) + at;
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
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

unsigned blocks_for(int64_t items, int d) {
  int width = 2;
  while (width * 8 < d) width <<= 1;
  const int64_t per = kThreads / width;
  const int64_t n = (items + per - 1) / per;
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
  return static_cast<unsigned>(n < 1 ? 1 : (n < most ? n : most));
}

template <typename T>
fa_status launch_append_typed(const AppendArgs& A, const LaunchCtx& ctx) {
  const int64_t items = static_cast<int64_t>(A.total) * (A.hq + (A.bounds != nullptr ? 1 : 2) * A.pool.hkv);
  note_variant(reinterpret_cast<const void*>(append_rows_kernel<T>));
  append_rows_kernel<T><<<blocks_for(items, A.pool.d), kThreads, 0, ctx.stream>>>(A);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (A.bounds == nullptr || A.total == 0) return FA_OK;
  note_variant(reinterpret_cast<const void*>(append_keys_kernel<T>));
  append_keys_kernel<T><<<static_cast<unsigned>(A.total), kThreads, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
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
  if (p.x_dtype == FA_BF16) return launch_append_typed<__nv_bfloat16>(A, ctx);
  return launch_append_typed<float>(A, ctx);
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
  note_variant(reinterpret_cast<const void*>(read_rows_kernel));
  read_rows_kernel<<<blocks_for(static_cast<int64_t>(p.total) * 2 * p.hkv, p.head_dim), kThreads, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
}

}  // namespace fa
