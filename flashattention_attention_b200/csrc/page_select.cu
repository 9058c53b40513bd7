// page_select.cu -- the cache pages worth attending to, by an upper bound of
// the scores that each page's per-channel key bounds give.
//
//   score(b, g, p) = max_h sum_d max(q_hd lo_d, q_hd hi_d)
//                  = max_h (q_h+ . hi + q_h- . lo),   q+ = max(q, 0), q- = min(q, 0)
//
// Which of two near pages is better must not depend on rounding, so the sum is
// defined far more exactly than fp32; but only pages next to the k-th best need
// that:
//   1. every warp scores 16 pages at a time on mma.sync m16n8k16 (pages on M,
//      query heads on N, bf16 operands, fp32 sums) together with
//      A = |q| . max(|lo|, |hi|), which bounds the terms' absolute sum;
//   2. one block per (sequence, KV head) finds a narrow range [t0, t1] that
//      holds the k-th largest score.  With e = error_share max A every score is
//      within e of the exact one, so pages above t1 + 2e are in, pages below
//      t0 - 2e are out, and the few between are summed again in fp64 (products
//      of two bf16 numbers are exact) and rounded to fp32 once;
//   3. the rest of the k is taken from those, the lower page first where
//      rounded sums are equal, and the pages are written in order.
// Where the tables are short for the number of (sequence, KV head) pairs, a
// cluster per pair does all of it in one launch, the scores going straight into
// the choosing block's shared memory.  Else the pages of all pairs are dealt
// evenly to the device's warps and a second kernel chooses, since a pair's own
// cluster would go over its pages in rounds that each wait for memory (128
// pairs of up to 1021 pages: 22.6 us in clusters of two, 21.7 us dealt evenly,
// both before the choice became 2 us shorter).  Bound by latency: 37 MB of
// bounds are 6 us, the choosing block's steps (two reads of the scores, a
// histogram, the few pages between summed again, the list) about 5 us.
// One pass over the bounds, 4 d bytes a page; the choice works on 4 bytes a page.
#include "decode_mma.cuh"
#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kSelWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
// The error of a score, as a share of A: an fp32 sum on the tensor cores whose
// k-steps (d / 16 of hi and of lo) have 17 addends, each of which may lose
// 2^-22 of the largest partial sum (at most A).
__device__ __forceinline__ float error_share(int d) { return static_cast<float>(d / 8 * 17) * 0x1p-22f; }
// And what they may lose below fp32's normal range: 2^-126 for each addend (d <= 256).
constexpr float kErrorFloor = 0x1p-116f;

constexpr int kHeld = 4096;    // scores a block holds in shared memory (more stay in L2)
constexpr int kBetween = 256;  // pages next to the border that are ranked directly

struct PickShared {
  alignas(16) int hist[kBins];
  float scores[kHeld];
  float part[kMaxCluster][3];  // of each block's (or warp's) pages: largest A, least and greatest score
  int between[kBetween];
  uint32_t exact[kBetween];
  int warp_sum[kSelWarps];
  int bin, above, inside, n_in, n_between;
};

struct SelectArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  const int32_t* seqlens;
  int32_t* selected;
  // dealt evenly: the scores [batch*hkv][max_pages], and per 16 pages their
  // largest A, least and greatest score [batch*hkv][max_pages / 16 rounded up]
  float* scores;
  float4* parts;
  int batch, hq, hkv, group, d, top_k, n_first, n_recent;
  const int32_t* block_table;
  int max_pages, page_size, num_pages;
  int64_t capacity;
  Watchdog wd;
};

// Unsigned key with the order of the float (-0 and +0 equal).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A page id outside the pool is reported and read as page 0.
__device__ __forceinline__ int checked(const SelectArgs& A, int pg) {
  if (pg >= 0 && pg < A.num_pages) return pg;
  record_status(A.wd, kStatusRange);
  return 0;
}
__device__ __forceinline__ int page_id(const SelectArgs& A, int b, int p) {
  return checked(A, A.block_table[static_cast<int64_t>(b) * A.max_pages + p]);
}

// Scores of 16 pages of one unit by one warp: best[i] of page row gq + 8 i (in
// every lane quarter), and the largest A seen; pg: the lane's two page ids, -1
// for none.  kJ = ceil(d / 32): quarter qq holds channels [8 qq + 32 j, +8).
template <int kJ>
__device__ __forceinline__ void score_group(const SelectArgs& A, int b, int g, const int (&pg)[2], float (&best)[2],
                                            float& most) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, qq = lane & 3;
  const __nv_bfloat16* q_unit = A.q + (static_cast<int64_t>(b) * A.hq + static_cast<int64_t>(g) * A.group) * A.d;
  uint4 lo[2][kJ], hi[2][kJ];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4* row = reinterpret_cast<const uint4*>(A.bounds + (static_cast<int64_t>(pg[i]) * A.hkv + g) * 2 * A.d);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int chunk = qq + 4 * j;
      const bool ok = 8 * chunk < A.d && pg[i] >= 0;
      lo[i][j] = ok ? __ldcs(row + chunk) : make_uint4(0, 0, 0, 0);
      hi[i][j] = ok ? __ldcs(row + A.d / 8 + chunk) : make_uint4(0, 0, 0, 0);
    }
  }
  best[0] = best[1] = -INFINITY;
  for (int h0 = 0; h0 < A.group; h0 += 8) {  // eight query heads at a time
    float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
    const bool head_ok = h0 + gq < A.group;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int chunk = qq + 4 * j;
      uint4 qv = make_uint4(0, 0, 0, 0);
      if (head_ok && 8 * chunk < A.d)
        qv = *(reinterpret_cast<const uint4*>(q_unit + static_cast<int64_t>(h0 + gq) * A.d) + chunk);
      const uint32_t qr[4] = {qv.x, qv.y, qv.z, qv.w};
      const uint32_t lr[2][4] = {{lo[0][j].x, lo[0][j].y, lo[0][j].z, lo[0][j].w},
                                 {lo[1][j].x, lo[1][j].y, lo[1][j].z, lo[1][j].w}};
      const uint32_t hr[2][4] = {{hi[0][j].x, hi[0][j].y, hi[0][j].z, hi[0][j].w},
                                 {hi[1][j].x, hi[1][j].y, hi[1][j].z, hi[1][j].w}};
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t h4[4] = {hr[0][e], hr[1][e], hr[0][e + 1], hr[1][e + 1]};
        const uint32_t l4[4] = {lr[0][e], lr[1][e], lr[0][e + 1], lr[1][e + 1]};
        mma16816_bf16(s, h4, bf16x2_max(qr[e], 0u), bf16x2_max(qr[e + 1], 0u));
        mma16816_bf16(s, l4, bf16x2_min(qr[e], 0u), bf16x2_min(qr[e + 1], 0u));
        uint32_t a4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) a4[x] = bf16x2_max(h4[x] & 0x7fff7fffu, l4[x] & 0x7fff7fffu);
        mma16816_bf16(t, a4, qr[e] & 0x7fff7fffu, qr[e + 1] & 0x7fff7fffu);
      }
    }
    // rows gq, gq + 8; heads h0 + 2 qq, + 1
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (h0 + 2 * qq + (x & 1) < A.group) best[x >> 1] = fmaxf(best[x >> 1], s[x]);
      most = fmaxf(most, t[x]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 1));
    best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 2));
  }
}

// A warp's largest A, least and greatest score, the same in every lane.
__device__ __forceinline__ void warp_stats(float& most, float& least, float& greatest) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, off));
    greatest = fmaxf(greatest, __shfl_xor_sync(0xffffffffu, greatest, off));
  }
}

// A cluster's share of pages [lo_page, hi_page) of its unit, at most 16 pages
// per warp, into block 0's shared memory.
template <int kJ>
__device__ __forceinline__ void score_pages(const SelectArgs& A, PickShared& S, int b, int g, int lo_page, int hi_page,
                                            const int (&first_pg)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, qq = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t remote = mapa_shared(smem_u32(S.scores), 0);
  float most = 0.f, least = INFINITY, greatest = -INFINITY;
  const int p0 = lo_page + 16 * (rank * kSelWarps + warp);
  if (p0 < hi_page) {
    int pg[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) pg[i] = p0 + gq + 8 * i < hi_page ? checked(A, first_pg[i]) : -1;
    float best[2];
    score_group<kJ>(A, b, g, pg, best, most);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = p0 + gq + 8 * i;
      if (p >= hi_page) continue;
      least = fminf(least, best[i]);
      greatest = fmaxf(greatest, best[i]);
      if (qq == 0) st_cluster_f32(remote + 4 * (p - lo_page), best[i]);
    }
  }
  warp_stats(most, least, greatest);
  __shared__ float s_part[kSelWarps][3];
  if (lane == 0) {
    s_part[warp][0] = most;
    s_part[warp][1] = least;
    s_part[warp][2] = greatest;
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    const int x = threadIdx.x;
    float v = s_part[0][x];
    for (int w = 1; w < kSelWarps; ++w) v = x == 1 ? fminf(v, s_part[w][x]) : fmaxf(v, s_part[w][x]);
    st_cluster_f32(mapa_shared(smem_u32(&S.part[rank][x]), 0), v);
  }
}

// Pages of sequence b; whether they have to be chosen from is n > top_k.
__device__ __forceinline__ int pages_of(const SelectArgs& A, int b, bool report) {
  const int64_t Lr = A.seqlens[b];
  const int64_t L = Lr < 0 ? 0 : (Lr > A.capacity ? A.capacity : Lr);
  if (report && L != Lr) record_status(A.wd, kStatusRange);
  return static_cast<int>((L + A.page_size - 1) / A.page_size);
}

// Dealt evenly: groups of 16 pages of all units, warp after warp, the KV heads
// of the same pages next to each other (as their bounds are in memory).
constexpr int kMaxBatch = 1024;  // sequences per launch
template <int kJ>
__global__ void __launch_bounds__(kThreads, kJ == 8 ? 1 : 2) page_score_kernel(const SelectArgs A) {
  __shared__ int s_pre[kMaxBatch + 1];
  __shared__ int s_sum[kSelWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, qq = lane & 3;
  // groups before each sequence
  const int per = (A.batch + kThreads - 1) / kThreads;
  const int b0 = min(A.batch, static_cast<int>(threadIdx.x) * per), b1 = min(A.batch, b0 + per);
  auto groups = [&](int b, bool report) {
    const int n = pages_of(A, b, report);
    return n > A.top_k ? (n - A.n_first - A.n_recent + 15) / 16 * A.hkv : 0;
  };
  int own = 0;
  for (int b = b0; b < b1; ++b) own += groups(b, blockIdx.x == 0);
  int incl = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int at = incl - own, total = 0;
  for (int w = 0; w < kSelWarps; ++w) {
    if (w < warp) at += s_sum[w];
    total += s_sum[w];
  }
  for (int b = b0; b < b1; ++b) {
    s_pre[b] = at;
    at += groups(b, false);
  }
  if (threadIdx.x == 0) s_pre[A.batch] = total;
  __syncthreads();
  const int per_unit = (A.max_pages + 15) / 16;
  for (int x = blockIdx.x * kSelWarps + warp; x < total; x += gridDim.x * kSelWarps) {
    int b = 0, end = A.batch - 1;  // the last b with s_pre[b] <= x
    while (b < end) {
      const int mid = (b + end + 1) >> 1;
      if (s_pre[mid] <= x) b = mid; else end = mid - 1;
    }
    const int y = x - s_pre[b], group = y / A.hkv, g = y - group * A.hkv;
    const int hi_page = pages_of(A, b, false) - A.n_recent, p0 = A.n_first + 16 * group;
    int pg[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) pg[i] = p0 + gq + 8 * i < hi_page ? page_id(A, b, p0 + gq + 8 * i) : -1;
    float best[2], most = 0.f, least = INFINITY, greatest = -INFINITY;
    score_group<kJ>(A, b, g, pg, best, most);
    const int64_t u = static_cast<int64_t>(b) * A.hkv + g;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = p0 + gq + 8 * i;
      if (p >= hi_page) continue;
      least = fminf(least, best[i]);
      greatest = fmaxf(greatest, best[i]);
      if (qq == 0) A.scores[u * A.max_pages + p] = best[i];
    }
    warp_stats(most, least, greatest);
    if (lane == 0) A.parts[u * per_unit + group] = make_float4(most, least, greatest, 0.f);
  }
}

// Two consecutive bf16 values.
__device__ __forceinline__ float2 pair_at(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The exact score of page p by one warp: fp64 sums of exact products (in fp32
// they might pass its range at either end), rounded once; four heads' sums at a
// time.
__device__ float exact_score(const SelectArgs& A, int b, int g, int p) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* row = A.bounds + (static_cast<int64_t>(page_id(A, b, p)) * A.hkv + g) * 2 * A.d;
  const __nv_bfloat16* q = A.q + (static_cast<int64_t>(b) * A.hq + static_cast<int64_t>(g) * A.group) * A.d;
  float best = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < A.group; h += 4, q += 4 * A.d) {
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 2
    for (int c = 2 * lane; c < A.d; c += 64) {
      const float2 lo = pair_at(row + c), hi = pair_at(row + A.d + c);
      const double lx = lo.x, ly = lo.y, hx = hi.x, hy = hi.y;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 qv = h + k < A.group ? pair_at(q + k * A.d + c) : make_float2(0.f, 0.f);
        sum[k] = fma(static_cast<double>(qv.x), qv.x > 0.f ? hx : lx, sum[k]);
        sum[k] = fma(static_cast<double>(qv.y), qv.y > 0.f ? hy : ly, sum[k]);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], off);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (h + k < A.group) best = fmaxf(best, static_cast<float>(sum[k]));
  }
  return best;
}

// Exclusive sum over the block's threads, and the total.
__device__ __forceinline__ int block_scan(PickShared& S, int v, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  __syncthreads();
  if (lane == 31) S.warp_sum[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    if (w < warp) before += S.warp_sum[w];
    total += S.warp_sum[w];
  }
  return before + incl - v;
}

// Narrows [lo, hi], which holds all m keys key(i), to a range that holds the
// need-th largest (1-based) of them, with the number of keys above it: rounds
// of a histogram over the range found so far, 2048 bins each, the whole block
// together, until at most `few` keys are left in it or it is one key wide (at
// most three rounds).  S.hist is zero and the block in step on entry.
template <typename K>
__device__ __forceinline__ void kth_range(PickShared& S, int m, int need, int few, K key, uint32_t& lo, uint32_t& hi,
                                          int& above) {
  const int tid = threadIdx.x;
  above = 0;
  while (true) {
    const int bits = 32 - __clz(hi - lo);
    const int shift = bits > 11 ? bits - 11 : 0;
    for (int i = tid; i < m; i += kThreads) {
      const uint32_t k = key(i);
      if (k >= lo && k <= hi) atomicAdd(&S.hist[(k - lo) >> shift], 1);
    }
    __syncthreads();
    // the bin of the need-th key, counted from the top: thread t has bins
    // [kBins - 8 (t + 1), kBins - 8 t)
    static_assert(kBins == 8 * kThreads, "eight bins a thread");
    const int first = kBins - 8 * (tid + 1);
    const int4 u = *reinterpret_cast<const int4*>(&S.hist[first]), v = *reinterpret_cast<const int4*>(&S.hist[first + 4]);
    const int bins[8] = {v.w, v.z, v.y, v.x, u.w, u.z, u.y, u.x};  // from the top
    const int own = ((v.w + v.z) + (v.y + v.x)) + ((u.w + u.z) + (u.y + u.x));
    int total, before = above + block_scan(S, own, total);
    if (before < need && before + own >= need) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (before < need && before + bins[j] >= need) {
          S.bin = first + 7 - j;
          S.above = before;
          S.inside = bins[j];
        }
        before += bins[j];
      }
    }
    __syncthreads();
    above = S.above;
    lo += static_cast<uint32_t>(S.bin) << shift;
    const uint32_t width = (1u << shift) - 1u;
    if (hi - lo > width) hi = lo + width;
    if (shift == 0 || S.inside <= few) return;
    for (int i = tid; i < kBins; i += kThreads) S.hist[i] = 0;
    __syncthreads();
  }
}

__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// One block: the top_k of pages 0 .. n - 1, of which [lo, hi) have scores (sc, by
// page - lo; overwritten), with the stats of `parts` shares of them in S.part.
__device__ __forceinline__ void pick_pages(const SelectArgs& A, PickShared& S, float* sc, int parts, int u, int b, int g,
                                           int n, int lo, int hi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = hi - lo, need = A.top_k - (n - m);  // of the pages with scores
  int32_t* out = A.selected + static_cast<int64_t>(u) * A.top_k;
  uint32_t kth = 0xffffffffu;  // pages above this key are taken, and the first `ties` equal to it
  int ties = 0;
  if (need > 0) {
    float e = 0.f, least = INFINITY, greatest = -INFINITY;
    for (int r = 0; r < parts; ++r) {
      e = fmaxf(e, S.part[r][0]);
      least = fminf(least, S.part[r][1]);
      greatest = fmaxf(greatest, S.part[r][2]);
    }
    e = 2.f * (error_share(A.d) * e + kErrorFloor);
    uint32_t k0 = order_key(least), k1 = order_key(greatest);
    int above;
    kth_range(S, m, need, 4, [&](int i) { return order_key(sc[i]); }, k0, k1, above);
    // in: +inf, out: -inf, between: to be summed exactly
    const float in_from = key_float(k1) + e, out_to = key_float(k0) - e;
    int in = 0;
    for (int i = tid; i < m; i += kThreads) {
      const float v = sc[i];
      if (v > in_from) {
        ++in;
        sc[i] = INFINITY;
      } else if (v < out_to) {
        sc[i] = -INFINITY;
      } else {
        const int at = atomicAdd(&S.n_between, 1);
        if (at < kBetween) S.between[at] = i;
      }
    }
    in = __reduce_add_sync(0xffffffffu, in);
    if (lane == 0 && in > 0) atomicAdd(&S.n_in, in);
    __syncthreads();
    const int taken = S.n_in, n_between = S.n_between;
    if (n_between == need - taken && out_to > -INFINITY) {  // no choice to make: what is not out is in
      kth = order_key(-INFINITY);
    } else if (n_between <= kBetween) {
      for (int c = warp; c < n_between; c += kSelWarps) {
        const float x = exact_score(A, b, g, lo + S.between[c]);
        if (lane == 0) S.exact[c] = order_key(x);
      }
      __syncthreads();
      for (int c = tid; c < n_between; c += kThreads) {
        const uint32_t k = S.exact[c];
        const int i = S.between[c];
        int better = 0;
        for (int o = 0; o < n_between; ++o) better += S.exact[o] > k || (S.exact[o] == k && S.between[o] < i);
        sc[i] = better < need - taken ? INFINITY : -INFINITY;
      }
      kth = order_key(0.f);
    } else {
      // many equal or nearly equal pages: all exactly, then a second selection
      for (int i0 = 32 * warp; i0 < m; i0 += kThreads) {
        // (where sums passed fp32's range, e with them, nothing is in or out yet)
        const bool open = i0 + lane < m && (fabsf(sc[i0 + lane]) != INFINITY || !(e < INFINITY));
        for (unsigned left = __ballot_sync(0xffffffffu, open); left != 0; left &= left - 1) {
          const int i = i0 + __ffs(left) - 1;
          const float x = exact_score(A, b, g, lo + i);
          if (lane == 0) sc[i] = x;
        }
      }
      for (int i = tid; i < kBins; i += kThreads) S.hist[i] = 0;
      __syncthreads();
      k0 = order_key(-INFINITY);
      k1 = order_key(INFINITY);
      kth_range(S, m, need, 0, [&](int i) { return order_key(sc[i]); }, k0, k1, above);
      kth = k0;
      ties = need - above;
    }
    __syncthreads();
  }
  // in page order: the pages without scores, those above the k-th, and the first `ties` equal to it
  const int per = (n + kThreads - 1) / kThreads;
  const int p0 = min(n, tid * per), p1 = min(n, p0 + per);
  int above = 0, equal = 0, total;
  uint32_t taken_bits = 0;  // of a thread's first 32 pages
  for (int p = p0; p < p1; ++p) {
    bool take = p < lo || p >= hi;
    if (!take && need > 0) {
      const uint32_t k = order_key(sc[p - lo]);
      take = k > kth;
      equal += k == kth;
    }
    above += take;
    if (p - p0 < 32) taken_bits |= static_cast<uint32_t>(take) << (p - p0);
  }
  int at = block_scan(S, above, total), tied = 0;
  if (ties > 0) {  // the same for the whole block
    tied = block_scan(S, equal, total);
    at += min(tied, ties);
  } else if (per <= 32) {
    for (; taken_bits != 0; taken_bits &= taken_bits - 1) out[at++] = p0 + __ffs(taken_bits) - 1;
    return;
  }
  for (int p = p0; p < p1; ++p) {
    bool take = p < lo || p >= hi;
    if (!take && need > 0) {
      const uint32_t k = order_key(sc[p - lo]);
      take = k > kth || (k == kth && tied++ < ties);
    }
    if (take) out[at++] = p;
  }
}

// A sequence of no more pages than top_k: all of them.
__device__ __forceinline__ void all_pages(const SelectArgs& A, int u, int n) {
  int32_t* out = A.selected + static_cast<int64_t>(u) * A.top_k;
  for (int i = threadIdx.x; i < A.top_k; i += kThreads) out[i] = i < n ? i : -1;
}

template <int kJ>
__global__ void __launch_bounds__(kThreads, kJ == 8 ? 1 : 2) page_select_kernel(const SelectArgs A) {
  __shared__ PickShared S;
  griddep_launch_dependents();
  cluster_arrive_relaxed();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first = cluster_ctarank() == 0;
  const int u = blockIdx.x / cluster_size(), b = u / A.hkv, g = u % A.hkv;
  if (first) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) S.hist[i] = 0;
    if (threadIdx.x == 0) S.n_in = S.n_between = 0;
  }
  griddep_wait();
  // the first round's pages, looked up together with the length
  int pg[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = A.n_first + 16 * (static_cast<int>(cluster_ctarank()) * kSelWarps + warp) + (lane >> 2) + 8 * i;
    pg[i] = p < A.max_pages ? A.block_table[static_cast<int64_t>(b) * A.max_pages + p] : 0;
  }
  const int n = pages_of(A, b, first && threadIdx.x == 0);
  const int lo = A.n_first, hi = n - A.n_recent;
  cluster_wait();  // every block of the cluster has started: CTA 0's shared memory may be written
  const bool choose = n > A.top_k;  // the same for the whole cluster; then lo < hi
  if (choose) score_pages<kJ>(A, S, b, g, lo, hi, pg);
  cluster_sync_all();  // the cluster's scores are visible to block 0
  if (!first) return;
  if (choose) {
    pick_pages(A, S, S.scores, static_cast<int>(cluster_size()), u, b, g, n, lo, hi);
  } else {
    all_pages(A, u, n);
  }
}

// Dealt evenly: the choice of one unit.
__global__ void __launch_bounds__(kThreads) page_pick_kernel(const SelectArgs A) {
  __shared__ PickShared S;
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = blockIdx.x, b = u / A.hkv, g = u % A.hkv;
  for (int i = threadIdx.x; i < kBins; i += kThreads) S.hist[i] = 0;
  if (threadIdx.x == 0) S.n_in = S.n_between = 0;
  griddep_wait();
  const int n = pages_of(A, b, false);
  if (n <= A.top_k) {
    all_pages(A, u, n);
    return;
  }
  const int lo = A.n_first, hi = n - A.n_recent, m = hi - lo, groups = (m + 15) / 16;
  const float4* parts = A.parts + static_cast<int64_t>(u) * ((A.max_pages + 15) / 16);
  float* stored = A.scores + static_cast<int64_t>(u) * A.max_pages + lo;
  float* sc = m <= kHeld ? S.scores : stored;
  float first[4];  // on their way with the statistics
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = threadIdx.x + k * kThreads;
    first[k] = i < m ? __ldcg(stored + i) : 0.f;
  }
  float most = 0.f, least = INFINITY, greatest = -INFINITY;
  for (int i = threadIdx.x; i < groups; i += kThreads) {
    const float4 v = __ldcg(parts + i);
    most = fmaxf(most, v.x);
    least = fminf(least, v.y);
    greatest = fmaxf(greatest, v.z);
  }
  if (m <= kHeld) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (threadIdx.x + k * kThreads < m) sc[threadIdx.x + k * kThreads] = first[k];
    for (int i = threadIdx.x + 4 * kThreads; i < m; i += kThreads) sc[i] = __ldcg(stored + i);
  }
  warp_stats(most, least, greatest);
  if (lane == 0) {
    S.part[warp][0] = most;
    S.part[warp][1] = least;
    S.part[warp][2] = greatest;
  }
  __syncthreads();
  pick_pages(A, S, sc, kSelWarps, u, b, g, n, lo, hi);
}

// Blocks per cluster: as many as the device holds at once (two per SM).
int cluster_of(int64_t units) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 2;
  int cluster = 1;
  while (cluster < kMaxCluster && units * cluster * 2 <= most) cluster *= 2;
  return cluster;
}
// Whether a cluster per unit scores its pages in one round of 16 per warp (with
// the attention that follows, one sequence of 8 KV heads and 513 pages: 17.2 us,
// dealt evenly 20.6; 4 sequences of up to 1024 pages: 29.4 and 34.9).
bool one_round(int64_t units, int max_pages) { return cluster_of(units) * kSelWarps * 16 >= max_pages; }

template <int kJ>
fa_status launch_width(const SelectArgs& all, const LaunchCtx& ctx) {
  const int64_t units = static_cast<int64_t>(all.batch) * all.hkv;
  if (one_round(units, all.max_pages)) {
    const int cluster = cluster_of(units);
    return launch_dependent(page_select_kernel<kJ>, dim3(static_cast<unsigned>(units * cluster)), kThreads, 0, cluster,
                            ctx.stream, all);
  }
  const int blocks = device_sm_count() * (kJ == 8 ? 1 : 2);
  for (int b0 = 0; b0 < all.batch; b0 += kMaxBatch) {
    SelectArgs A = all;
    A.batch = all.batch - b0 < kMaxBatch ? all.batch - b0 : kMaxBatch;
    A.q += static_cast<int64_t>(b0) * A.hq * A.d;
    A.seqlens += b0;
    A.block_table += static_cast<int64_t>(b0) * A.max_pages;
    A.selected += static_cast<int64_t>(b0) * A.hkv * A.top_k;
    A.scores += static_cast<int64_t>(b0) * A.hkv * A.max_pages;
    A.parts += static_cast<int64_t>(b0) * A.hkv * ((A.max_pages + 15) / 16);
    fa_status st = launch_dependent(page_score_kernel<kJ>, dim3(blocks), kThreads, 0, 0, ctx.stream, A);
    if (st == FA_OK)
      st = launch_dependent(page_pick_kernel, dim3(static_cast<unsigned>(A.batch * A.hkv)), kThreads, 0, 0, ctx.stream, A);
    if (st != FA_OK) return st;
  }
  return FA_OK;
}

size_t parts_bytes(int64_t units, int max_pages) { return static_cast<size_t>(units) * ((max_pages + 15) / 16) * 16; }
}  // namespace

bool page_select_fits(int batch, int hkv, int max_pages) {
  // a launch's groups of 16 pages, and one round of the device's warps past them, are counted in an int
  const int64_t groups = static_cast<int64_t>(batch < kMaxBatch ? batch : kMaxBatch) * hkv * ((max_pages + 15) / 16);
  return one_round(static_cast<int64_t>(batch) * hkv, max_pages) || groups < (int64_t(1) << 31) - (1 << 16);
}

size_t page_select_workspace_bytes(int batch, int hkv, int max_pages) {
  const int64_t units = static_cast<int64_t>(batch) * hkv;
  if (one_round(units, max_pages)) return 0;
  return parts_bytes(units, max_pages) + static_cast<size_t>(units) * max_pages * sizeof(float);
}

fa_status launch_page_select(const fa_page_select_params& p, const fa_kv_pages& pages, const LaunchCtx& ctx) {
  if (static_cast<int64_t>(p.batch) * p.hkv >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  SelectArgs A;
  A.q = static_cast<const __nv_bfloat16*>(p.q);
  A.bounds = static_cast<const __nv_bfloat16*>(p.key_bounds);
  A.seqlens = p.cache_seqlens;
  A.selected = p.selected;
  A.parts = static_cast<float4*>(p.workspace);
  A.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) +
                                      parts_bytes(static_cast<int64_t>(p.batch) * p.hkv, pages.max_pages));
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
  if (p.head_dim <= 32) return launch_width<1>(A, ctx);
  if (p.head_dim <= 64) return launch_width<2>(A, ctx);
  if (p.head_dim <= 128) return launch_width<4>(A, ctx);
  return launch_width<8>(A, ctx);
}

}  // namespace fa
