// decode_pages.cu -- single-query attention over page pools: every page of a
// 4-bit cache, or the chosen pages of a bf16, int8 or 4-bit one.
//
// One warp takes every 4th key of a split of one (sequence, KV head), a lane
// holding D / 32 channels of the key and of each query head's output; the
// warps' and splits' softmax states (m, l, O) are merged by a second kernel.
#include "internal.h"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

struct PageDecodeArgs {
  const __nv_bfloat16* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* seqlens;
  const int32_t* selected;  // null: every page
  int top_k;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  int64_t capacity;
  float* part;  // [batch*hq][splits][D + 2]
  __nv_bfloat16* out;
  int batch, hq, hkv, group, hkv_real, kv_split, splits, window;
  float scale_log2;
  Epilogue epi;
  Watchdog wd;
};

template <int D, int kKind>
__device__ __forceinline__ void load_key(const void* pool, const float* scales, int64_t row, int lane,
                                         float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if constexpr (kKind == FA_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(pool) + row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __bfloat162float(p[e]);
  } else if constexpr (kKind == FA_I8) {
    const int8_t* p = static_cast<const int8_t*>(pool) + row * D + lane * E;
    const float s = scales[row];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = static_cast<float>(p[e]) * s;
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(pool) + row * (D / 2);
    const float s = scales[2 * row], o = scales[2 * row + 1];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane * E + e;
      x[e] = static_cast<float>((p[c >> 1] >> (4 * (c & 1))) & 15) * s + o;
    }
  }
}

template <int D, int kKind>
__global__ void __launch_bounds__(kWarps * 32) decode_pages_kernel(const PageDecodeArgs A) {
  constexpr int E = D / 32, kG = 8;
  __shared__ float s_o[kWarps][kG][D];
  __shared__ float s_ml[kWarps][kG][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = blockIdx.x, split = blockIdx.y, b = seg / A.hkv, g = seg % A.hkv, gr = g / A.kv_split;
  const int64_t Lr = A.seqlens[b];
  const int64_t L = Lr < 0 ? 0 : (Lr > A.capacity ? A.capacity : Lr);
  if (L != Lr && threadIdx.x == 0) record_status(A.wd, kStatusRange);
  const int n_pages = static_cast<int>((L + A.page_size - 1) / A.page_size);
  const int64_t lo = A.window > 0 && L > A.window ? L - A.window : 0;
  const int64_t first = A.selected != nullptr ? 0 : lo;
  const int64_t last =
      A.selected != nullptr ? static_cast<int64_t>(min(A.top_k, n_pages)) * A.page_size : L;
  const int64_t n = last - first;
  const int64_t k0 = first + n * split / A.splits, k1 = first + n * (split + 1) / A.splits;
  float q[kG][E], o[kG][E], m[kG], l[kG];
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[h][e] = 0.f;
      q[h][e] = h < A.group ? __bfloat162float(A.q[(static_cast<int64_t>(b) * A.hq + g * A.group + h) * D + lane * E + e])
                            : 0.f;
    }
  }
  for (int64_t v = k0 + warp; v < k1; v += kWarps) {
    int64_t key = v;
    if (A.selected != nullptr) {
      const int lp = A.selected[(static_cast<int64_t>(b) * A.hkv_real + gr) * A.top_k + v / A.page_size];
      if (lp < 0 || lp >= n_pages) continue;
      key = static_cast<int64_t>(lp) * A.page_size + v % A.page_size;
      if (key >= L) continue;
    }
    int pg = A.block_table[static_cast<int64_t>(b) * A.max_pages + key / A.page_size];
    if (pg < 0 || pg >= A.num_pages) {
      if (lane == 0) record_status(A.wd, kStatusRange);
      pg = 0;
    }
    const int64_t row = (static_cast<int64_t>(pg) * A.hkv_real + gr) * A.page_size + key % A.page_size;
    float kx[E], vx[E];
    load_key<D, kKind>(A.k_cache, A.k_scales, row, lane, kx);
    load_key<D, kKind>(A.v_cache, A.v_scales, row, lane, vx);
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      if (h >= A.group) break;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[h][e], kx[e], s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= A.scale_log2;
      const float mn = fmaxf(m[h], s);
      const float a = exp2f(m[h] - mn), p = exp2f(s - mn);
      m[h] = mn;
      l[h] = l[h] * a + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[h][e] = o[h][e] * a + p * vx[e];
    }
  }
#pragma unroll
  for (int h = 0; h < kG; ++h) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][h][lane * E + e] = o[h][e];
    if (lane == 0) {
      s_ml[warp][h][0] = m[h];
      s_ml[warp][h][1] = l[h];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < A.group * D; i += kWarps * 32) {
    const int h = i / D, c = i % D;
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][h][0]);
    const float ref = M == -INFINITY ? 0.f : M;
    float sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float a = exp2f(s_ml[w][h][0] - ref);
      sum += a * s_ml[w][h][1];
      acc += a * s_o[w][h][c];
    }
    float* rec = A.part + ((static_cast<int64_t>(b) * A.hq + g * A.group + h) * A.splits + split) * (D + 2);
    rec[c] = acc;
    if (c == 0) {
      rec[D] = M;
      rec[D + 1] = sum;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(D) decode_pages_merge_kernel(const PageDecodeArgs A) {
  const float* rec = A.part + static_cast<int64_t>(blockIdx.x) * A.splits * (D + 2);
  float M = -INFINITY;
  for (int s = 0; s < A.splits; ++s) M = fmaxf(M, rec[s * (D + 2) + D]);
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f, acc = 0.f;
  for (int s = 0; s < A.splits; ++s) {
    const float a = exp2f(rec[s * (D + 2) + D] - ref);
    sum += a * rec[s * (D + 2) + D + 1];
    acc += a * rec[s * (D + 2) + threadIdx.x];
  }
  const float y = apply_epilogue(sum > 0.f ? acc / sum : 0.f, A.epi);
  A.out[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = __float2bfloat16_rn(y);
}

template <int D, int kKind>
fa_status launch_typed(PageDecodeArgs& A, const LaunchCtx& ctx) {
  note_variant(reinterpret_cast<const void*>(decode_pages_kernel<D, kKind>));
  decode_pages_kernel<D, kKind><<<dim3(A.batch * A.hkv, A.splits), kWarps * 32, 0, ctx.stream>>>(A);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  note_variant(reinterpret_cast<const void*>(decode_pages_merge_kernel<D>));
  decode_pages_merge_kernel<D><<<A.batch * A.hq, D, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
}
template <int D>
fa_status launch_dim(PageDecodeArgs& A, int kind, const LaunchCtx& ctx) {
  if (kind == FA_I4) return launch_typed<D, FA_I4>(A, ctx);
  if (kind == FA_I8) return launch_typed<D, FA_I8>(A, ctx);
  return launch_typed<D, FA_BF16>(A, ctx);
}

}  // namespace

fa_status launch_decode_pages(const fa_decode_params& p, const fa_kv_pages& pages, const int32_t* selected, int top_k,
                              const LaunchCtx& ctx) {
  PageDecodeArgs A;
  A.q = static_cast<const __nv_bfloat16*>(p.q);
  A.k_cache = p.k_cache;
  A.v_cache = p.v_cache;
  A.k_scales = p.k_scales;
  A.v_scales = p.v_scales;
  A.seqlens = p.cache_seqlens;
  A.selected = selected;
  A.top_k = top_k;
  A.block_table = pages.block_table;
  A.max_pages = pages.max_pages;
  A.page_size = pages.page_size;
  A.num_pages = pages.num_pages;
  A.capacity = p.capacity;
  A.part = static_cast<float*>(p.workspace);
  A.out = static_cast<__nv_bfloat16*>(p.out);
  const int full_group = p.hq / p.hkv;
  int split = (full_group + 7) / 8;  // a group of more than 8 heads runs in passes
  while (full_group % split != 0) ++split;
  A.batch = p.batch;
  A.hq = p.hq;
  A.hkv_real = p.hkv;
  A.kv_split = split;
  A.hkv = p.hkv * split;
  A.group = full_group / split;
  A.window = p.window;
  A.scale_log2 = p.softmax_scale * kLog2e;
  A.epi = make_epilogue(p.epilogue, p.n_epilogue);
  A.wd = ctx.wd;
  const int segs = A.batch * A.hkv;
  A.splits = 1 + device_sm_count() * 4 / segs;
  switch (p.head_dim) {
    case 32: return launch_dim<32>(A, p.kv_dtype, ctx);
    case 64: return launch_dim<64>(A, p.kv_dtype, ctx);
    case 96: return launch_dim<96>(A, p.kv_dtype, ctx);
    case 128: return launch_dim<128>(A, p.kv_dtype, ctx);
    case 256: return launch_dim<256>(A, p.kv_dtype, ctx);
  }
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
