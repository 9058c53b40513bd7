// page_select.cu -- the cache pages worth attending to, by an upper bound of
// the scores that each page's per-channel key bounds give.
//
//   score(b, g, p) = max_h sum_d max(q_hd lo_d, q_hd hi_d)
//
// Two kernels: the scores of every (sequence, KV head, page), as unsigned keys
// of the same order, and per (sequence, KV head) the top_k of them.  A product
// of two bf16 numbers is exact in fp32 (16 bits), and the sum is taken in
// fp64, so which of two near pages is better does not depend on rounding.
#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;

struct SelectArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  const int32_t* seqlens;
  int32_t* selected;
  uint32_t* keys;  // [batch*hkv][max_pages]
  int batch, hq, hkv, group, d, top_k, n_first, n_recent;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  int64_t capacity;
  Watchdog wd;
};

__device__ __forceinline__ int pages_of(const SelectArgs& A, int b, bool& bad) {
  const int64_t L = A.seqlens[b];
  const int64_t c = L < 0 ? 0 : (L > A.capacity ? A.capacity : L);
  bad = c != L;
  return static_cast<int>((c + A.page_size - 1) / A.page_size);
}

// Unsigned key with the order of the float (-0 and +0 equal).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) page_score_kernel(const SelectArgs A) {
  const int lane = threadIdx.x & 31;
  const int u = blockIdx.x;  // b * hkv + g
  const int b = u / A.hkv, g = u % A.hkv;
  bool bad;
  const int n = pages_of(A, b, bad);
  if (bad && threadIdx.x == 0) record_status(A.wd, kStatusRange);
  const int warps = gridDim.y * (kThreads / 32);
  for (int p = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); p < n; p += warps) {
    uint32_t key = 0xffffffffu;
    if (p >= A.n_first && p < n - A.n_recent) {
      int pg = A.block_table[static_cast<int64_t>(b) * A.max_pages + p];
      if (pg < 0 || pg >= A.num_pages) {
        if (lane == 0) record_status(A.wd, kStatusRange);
        pg = 0;
      }
      const __nv_bfloat16* row = A.bounds + (static_cast<int64_t>(pg) * A.hkv + g) * 2 * A.d;
      float best = -INFINITY;
      for (int h = 0; h < A.group; ++h) {
        const __nv_bfloat16* q = A.q + (static_cast<int64_t>(b) * A.hq + g * A.group + h) * A.d;
        double sum = 0.0;
        for (int c = lane; c < A.d; c += 32) {
          const float qv = __bfloat162float(q[c]);
          sum += fmaxf(qv * __bfloat162float(row[c]), qv * __bfloat162float(row[A.d + c]));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        best = fmaxf(best, static_cast<float>(sum));
      }
      key = order_key(best);
    }
    if (lane == 0) A.keys[static_cast<int64_t>(u) * A.max_pages + p] = key;
  }
}

// The top_k keys of one (sequence, KV head): radix selection of the k-th
// largest key, eight bits a pass, then the pages above it and the first of
// those equal to it, in page order.
__global__ void __launch_bounds__(kThreads) page_pick_kernel(const SelectArgs A) {
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int s_above[kThreads / 32], s_equal[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x;
  bool bad;
  const int n = pages_of(A, u / A.hkv, bad);
  const uint32_t* keys = A.keys + static_cast<int64_t>(u) * A.max_pages;
  int32_t* out = A.selected + static_cast<int64_t>(u) * A.top_k;
  if (n <= A.top_k) {
    for (int i = tid; i < A.top_k; i += kThreads) out[i] = i < n ? i : -1;
    return;
  }
  if (tid == 0) {
    s_prefix = 0;
    s_need = A.top_k;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t k = keys[i];
      if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, bin = 255;
      while (bin > 0 && hist[bin] < need) need -= hist[bin--];
      s_need = need;
      s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
    }
    __syncthreads();
  }
  const uint32_t kth = s_prefix;
  const int ties = s_need;  // pages equal to the k-th key that are kept
  int written = 0, tied = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? keys[i] : 0u;
    const bool above = i < n && k > kth, equal = i < n && k == kth;
    const unsigned ma = __ballot_sync(0xffffffffu, above), me = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) {
      s_above[warp] = __popc(ma);
      s_equal[warp] = __popc(me);
    }
    __syncthreads();
    int na = 0, ne = 0, ta = 0, te = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        na += s_above[w];
        ne += s_equal[w];
      }
      ta += s_above[w];
      te += s_equal[w];
    }
    const unsigned below = (1u << lane) - 1u;
    na += __popc(ma & below);
    ne += __popc(me & below);
    const int room = ties - tied;  // ties still kept before this block
    const int at = written + na + min(ne, room);
    if (above || (equal && ne < room)) out[at] = i;
    written += ta + min(te, room);
    tied += min(te, room);
    __syncthreads();
  }
}

}  // namespace

size_t page_select_workspace_bytes(int batch, int hkv, int max_pages) {
  return (static_cast<size_t>(batch) * hkv * max_pages * sizeof(uint32_t) + 15) / 16 * 16;
}

fa_status launch_page_select(const fa_page_select_params& p, const fa_kv_pages& pages, const LaunchCtx& ctx) {
  SelectArgs A;
  A.q = static_cast<const __nv_bfloat16*>(p.q);
  A.bounds = static_cast<const __nv_bfloat16*>(p.key_bounds);
  A.seqlens = p.cache_seqlens;
  A.selected = p.selected;
  A.keys = static_cast<uint32_t*>(p.workspace);
  A.batch = p.batch;
  A.hq = p.hq;
  A.hkv = p.hkv;
  A.group = p.hq / p.hkv;
  A.d = p.head_dim;
  A.top_k = p.top_k;
  A.n_first = p.n_first;
  A.n_recent = p.n_recent;
  A.block_table = pages.block_table;
  A.max_pages = pages.max_pages;
  A.page_size = pages.page_size;
  A.num_pages = pages.num_pages;
  A.capacity = static_cast<int64_t>(pages.max_pages) * pages.page_size;
  A.wd = ctx.wd;
  const int units = p.batch * p.hkv;
  int chunks = (pages.max_pages + kThreads / 32 - 1) / (kThreads / 32);
  const int most = (device_sm_count() * 16 + units - 1) / units;
  if (chunks > most) chunks = most;
  note_variant(reinterpret_cast<const void*>(page_score_kernel));
  page_score_kernel<<<dim3(units, chunks), kThreads, 0, ctx.stream>>>(A);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  note_variant(reinterpret_cast<const void*>(page_pick_kernel));
  page_pick_kernel<<<units, kThreads, 0, ctx.stream>>>(A);
  return cuda_status(cudaGetLastError());
}

}  // namespace fa
