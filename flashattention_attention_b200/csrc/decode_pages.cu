// decode_pages.cu -- single-query attention over page pools: every page of a
// 4-bit cache, or the chosen pages of a bf16, int8 or 4-bit one.
//
// The tiles (64 keys of a 4-bit cache up to D = 128, else 32) of all (sequence,
// KV head) segments are laid end to end and a grid of P warps ("workers") takes
// equal contiguous ranges of them.  A worker looks up its next 32 tiles at a
// time, one lane a tile (page list, block table), and keeps a ring of tiles in
// flight in its own shared memory.  Where that is faster, a cluster serves each
// segment instead (see cluster_of).
// Per tile, keys on the M side of mma.sync m16n8k16 and heads on N:
//   S^T[keys x 8 heads] = K[keys x d] . Q^T,  online softmax per head in fp32,
//   O^T[d x 8 heads] += V^T[d x keys] . P'
// A segment that lies within one worker's range is normalised and stored at
// once; one that is split leaves a record (m, l, O) per worker, which a second
// kernel merges (launched early, it waits for the first one's end; a worker that
// gave up waiting leaves no record, and its rows are meaningless, as reported).
//
// 4-bit rows (value = code * step + offset): codes enter the MMA exactly, as
// subnormal fp16 numbers (one AND for two of them), and
//   q . k = step (q . code) + offset sum(q),
//   sum_j p_j v_j = sum_j (p_j step_j) code_j + sum_j p_j offset_j
// where the second terms stay in fp32.  p_j step_j is rounded to fp16 after
// multiplication by a power of two, the head's unit, that follows the largest
// products up and down (softmax below), so that no step or weight is too small
// or too large for fp16 beside what came before it.
// int8 rows: the same without offsets.  A word of eight codes holds channels
// 0 .. 7 of its four bytes: the low halves of bytes 0 and 2 are channels 0 and
// 4, in an order that Q's fragments (and the output's addresses) follow.
// Codes are not centred (0 .. 15), so
//   sum_j w_j code_j + sum_j p_j offset_j  with w_j the rounded p_j step_j
// would multiply the roundings of w by numbers about three times as large as the
// values' spread, and the tensor core's additions to a large number would lose
// bits to one side.  So the second sum takes p_j (offset_j + 7.5 step_j), one
// more MMA with ones adds up w_j, and every 8 tiles (and at the end) 7.5 times
// that leaves the accumulators, which then hold sums of w_j (code_j - 7.5).
//
// A 4-bit row of 128 is 72 bytes and as much arithmetic as 256 bytes of bf16, so
// the kernel is bound by its instructions and their latencies: about 450 per 32
// keys and 8 head columns (128 of them the ANDs), ALU pipe 55 % and issue slots
// 50 % busy at the 12 warps an SM that 152 registers and 72 KB a CTA leave room
// for.  16 sequences, 274,568 keys, 32 query heads on 8: 67.6 us, 4.7 TB/s (72 %
// of a plain copy); one of 131,071 keys, 64 heads on 8: 44.3 us, 3.4 TB/s (its
// records leave room for eight warps an SM; twelve, with larger ones, were as
// fast).  Weights in two fp16 terms, as bf16 caches have them, would double the
// 16 MMAs of the second product to take the 1 % that their rounding adds to the
// error of the bf16 result.
#include <atomic>
#include <type_traits>

#include "decode_mma.cuh"
#include "internal.h"

namespace fa {
namespace {

constexpr int kThreads = kWarps * 32;
constexpr float kSlack = 8.f;    // binary orders a weight may pass its reference by
constexpr uint32_t kOnes = 0x3c003c00u;  // fp16 1, twice
constexpr float kTop = 32768.f;  // no weight as large as this enters fp16
constexpr int kMaxBatch = 256;  // sequences per launch (their tile prefix is in shared memory)

// Division of 0 <= x < 2^31 by a number known on the host, by multiplication
// (Granlund and Montgomery, division by invariant integers): x / d =
// (x * mul) >> (32 + shift) with mul = ceil(2^(32 + shift) / d), 2^shift >= d
// (mul has up to 33 bits; its low 32 are kept and x is added back).
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv of(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((uint64_t(1) << f.shift) < d) ++f.shift;
    f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
    return f;
  }
  __device__ __forceinline__ int div(int x) const {
    const uint32_t u = static_cast<uint32_t>(x);
    return static_cast<int>((static_cast<uint64_t>(__umulhi(u, mul)) + u) >> shift);
  }
};

struct PageArgs {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;  // 4-bit pools (the others come through tensor maps)
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* seqlens;
  const int32_t* selected;  // [batch][hkv_real][top_k]
  int top_k;
  const int32_t* block_table;
  int max_pages, page_size, num_pages, capacity;
  // for the merge kernel: tile prefix [batch + 1], and per segment with tiles
  // its first worker << 16 | its number of workers
  int32_t* prefix;
  uint32_t* range;
  float* rec_o;     // [batch*hkv + P][group][D]
  float* rec_ml;    // [batch*hkv + P][group][2]
  __nv_bfloat16* out;
  // a group of more than 8 query heads runs as kv_split passes over its KV
  // head: hkv counts these virtual heads, each serving `group` query heads
  int batch, hq, hkv, group, hkv_real, kv_split, window;
  int n_workers;
  FastDiv by_hkv, by_split, by_page, by_page_runs, by_group;
  float scale_log2;
  Epilogue epi;
  Watchdog wd;
};

template <int D, int kKind>
struct Tile {
  using G = Geom<D, kKind == FA_BF16>;
  static constexpr bool kI4 = kKind == FA_I4;
  // A tile is one or two runs of 32 keys, each within one page.  A 4-bit run is
  // small, and what a tile costs beside its keys' arithmetic is spread over two
  // -- but not at D = 256, where two stages of 64 keys leave room for one CTA an
  // SM (12 sequences of up to 1056 keys in 8 heads: 18.5 us, with 32 keys 16.4).
  static constexpr int kRuns = kI4 && D < 256 ? 2 : 1;
  static constexpr int kKeys = kTile * kRuns;
  static constexpr int kBytes = kI4 ? kKeys * D / 2 : G::kTileBytes;  // of K, and of V
  static constexpr int kScaleBytes = kI4 ? kKeys * 8 : kKind == FA_I8 ? kTile * 4 : 0;
  static constexpr int kScaleOff = 2 * kBytes;
  static constexpr int kStageBytes = kI4 ? kScaleOff + 2 * kScaleBytes : G::kStageBytes;
  static constexpr int kStages = kKind == FA_BF16 && D == 256 ? 1 : kI4 ? 2 : 3;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRing + (kI4 ? 128 : 1024) /*align*/ + kWarps * kStages * 8;
  static constexpr int kFit = 233472 / (kSmem + (kMaxBatch + 1) * 4 + 1024);
  // up to three CTAs per SM (168 registers a thread), two at D = 256
  static constexpr int kMost = D == 256 ? 2 : 3;
  static constexpr int kCtas = kFit < 1 ? 1 : (kFit < kMost ? kFit : kMost);
};

__device__ __forceinline__ int pages_in(const PageArgs& A, int L) { return L > 0 ? A.by_page.div(L - 1) + 1 : 0; }

// T tiles over P <= T workers: the first T % P take one more than the others.
struct Split {
  int each, more;
  __device__ __forceinline__ Split(int T, int P) : each(T / P), more(T - T / P * P) {}
  __device__ __forceinline__ int begin(int w) const { return w * each + min(w, more); }
  __device__ __forceinline__ int worker_of(int x) const {
    const int y = x - more * (each + 1);
    return y < 0 ? x / (each + 1) : more + y / each;
  }
};
// First key a sequence of length L attends to.
template <bool kSel>
__device__ __forceinline__ int first_key(const PageArgs& A, int L) {
  return !kSel && A.window > 0 ? max(0, L - A.window) : 0;
}
// Tiles of a segment of sequence length L.
template <int kKeys, bool kSel>
__device__ __forceinline__ int tiles_in(const PageArgs& A, int L) {
  if constexpr (kSel)
    return (min(A.top_k, pages_in(A, L)) * static_cast<int>(A.by_page_runs.d) + kKeys / kTile - 1) / (kKeys / kTile);
  return L > 0 ? (L - 1) / kKeys + 1 - first_key<kSel>(A, L) / kKeys : 0;  // (L + kKeys may not be an int)
}
__device__ __forceinline__ int length_of(const PageArgs& A, int b) { return max(0, min(A.seqlens[b], A.capacity)); }

constexpr int kNoKey = 0x7fffffff;
template <int kRuns>
struct TileInfo {
  int seg = 0;  // b * hkv + g
  int key0[kRuns], row[kRuns];  // each run's first position and its pool row; kNoKey, -1: nothing there counts
  __device__ __forceinline__ TileInfo() {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      key0[r] = kNoKey;
      row[r] = -1;
    }
  }
};

// Tile t of segment (b, g).
template <int kRuns, bool kSel>
__device__ __forceinline__ TileInfo<kRuns> tile_at(const PageArgs& A, int b, int g, int t) {
  const int gr = A.by_split.div(g);
  const int L = length_of(A, b), n_pages = pages_in(A, L);
  TileInfo<kRuns> info;
  info.seg = b * A.hkv + g;
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    int lp, off, key0;
    if constexpr (kSel) {
      const int run = kRuns * t + r, i = A.by_page_runs.div(run);
      off = (run - i * static_cast<int>(A.by_page_runs.d)) * kTile;
      if (i >= A.top_k || i >= n_pages) continue;
      lp = A.selected[(static_cast<int64_t>(b) * A.hkv_real + gr) * A.top_k + i];
      if (lp < 0 || lp >= n_pages) continue;
      key0 = lp * A.page_size + off;
    } else {
      key0 = (first_key<kSel>(A, L) / (kRuns * kTile) + t) * (kRuns * kTile) + r * kTile;
      lp = A.by_page.div(key0);
      off = key0 - lp * A.page_size;
      // behind the last key, or before the window, perhaps in a page that is gone
      if (key0 >= L || key0 + kTile <= first_key<kSel>(A, L)) continue;
    }
    if (key0 >= L) continue;
    int pg = A.block_table[static_cast<int64_t>(b) * A.max_pages + lp];
    if (pg < 0 || pg >= A.num_pages) {  // reported; page 0 keeps the loads inside the pool
      record_status(A.wd, kStatusRange);
      pg = 0;
    }
    info.key0[r] = key0;
    info.row[r] = (pg * A.hkv_real + gr) * A.page_size + off;
  }
  return info;
}
// Tile x of all segments' tiles, by their prefix over the sequences.
template <int kRuns, bool kSel>
__device__ __forceinline__ TileInfo<kRuns> tile_info(const PageArgs& A, const int32_t* pre, int x) {
  int lo = 0, hi = A.batch - 1;  // the last b with pre[b] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  const int Tb = A.by_hkv.div(pre[lo + 1] - pre[lo]), y = x - pre[lo], g = y / Tb;
  return tile_at<kRuns, kSel>(A, lo, g, y - g * Tb);
}

// S row r of a 16-key half is key key_of(r) of it: for packed rows of 64 bytes
// the K loads of rows (2i, 2i + 1) then fall on different banks, and so do half
// of the V loads of a thread quad.
template <int kKind>
__device__ __forceinline__ int key_of(int r) {
  return kKind == FA_I4 ? r ^ ((r >> 1) & 1) : r;
}

// kCluster: the CTAs of a cluster serve one segment, its tiles dealt evenly to
// their warps, and merge their states through distributed shared memory.
// Else: the tiles of all segments are dealt evenly to all warps.
template <int D, int kKind, bool kSel, bool kCluster>
__global__ void __launch_bounds__(kThreads, Tile<D, kKind>::kCtas)
    decode_pages_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k32, const __grid_constant__ CUtensorMap tm_v32,
                        const PageArgs A) {
  using TL = Tile<D, kKind>;
  using G = Geom<D, kKind == FA_BF16>;
  constexpr bool kBF = kKind == FA_BF16, kI4 = kKind == FA_I4, kI8 = kKind == FA_I8;
  constexpr int kStages = TL::kStages;
  constexpr int kSteps = D / 16;  // k-steps of S
  constexpr int kMT = D / 16;     // m-tiles of O^T
  constexpr bool kQuarter = D == 64 || D == 128;  // int8: see decode.cu
  extern __shared__ uint8_t page_smem_raw[];
  constexpr uintptr_t kAlign = kI4 ? 128 : 1024;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(page_smem_raw) + kAlign - 1) & ~(kAlign - 1));
  uint64_t* all_bars = reinterpret_cast<uint64_t*>(smem + TL::kRing);
  int32_t* pre = reinterpret_cast<int32_t*>(all_bars + kWarps * kStages);
  __shared__ int32_t warp_sums[kWarps];
  __shared__ float2 s_ml[kWarps][8];  // cluster: each warp's (m, l) per head

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, qq = lane & 3;
  uint64_t* bars = all_bars + warp * kStages;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  griddep_wait();
  // this warp's tiles: [t_first, t_first + my_tiles) of all, or of the cluster's segment
  int w = 0, T = 0, P = 1, t_first, my_tiles, the_seg = 0, the_b = 0, the_g = 0;
  if constexpr (kCluster) {
    const int c = static_cast<int>(cluster_size());
    the_seg = static_cast<int>(blockIdx.x) / c;
    the_b = A.by_hkv.div(the_seg);
    the_g = the_seg - the_b * A.hkv;
    const int L = A.seqlens[the_b];
    if ((L < 0 || L > A.capacity) && threadIdx.x == 0) record_status(A.wd, kStatusRange);
    const int64_t Tb = tiles_in<TL::kKeys, kSel>(A, length_of(A, the_b));
    const int workers = c * kWarps, v = static_cast<int>(cluster_ctarank()) * kWarps + warp;
    t_first = static_cast<int>(Tb * v / workers);
    my_tiles = static_cast<int>(Tb * (v + 1) / workers) - t_first;
    if (lane < 8) s_ml[warp][lane] = make_float2(-INFINITY, 0.f);
    __syncwarp();
  } else {
    // tile prefix over the sequences
    {
      const int per = (A.batch + kThreads - 1) / kThreads;
      const int b0 = min(A.batch, static_cast<int>(threadIdx.x) * per), b1 = min(A.batch, b0 + per);
      int own = 0;
      for (int b = b0; b < b1; ++b) {
        const int L = A.seqlens[b];
        if ((L < 0 || L > A.capacity) && blockIdx.x == 0) record_status(A.wd, kStatusRange);
        own += tiles_in<TL::kKeys, kSel>(A, length_of(A, b)) * A.hkv;
      }
      int incl = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      if (lane == 31) warp_sums[warp] = incl;
      __syncthreads();
      int at = incl - own;
      for (int v = 0; v < warp; ++v) at += warp_sums[v];
      for (int b = b0; b < b1; ++b) {
        pre[b] = at;
        if (blockIdx.x == 0) A.prefix[b] = at;
        at += tiles_in<TL::kKeys, kSel>(A, length_of(A, b)) * A.hkv;
      }
      if (threadIdx.x == 0) {
        int total = 0;
        for (int v = 0; v < kWarps; ++v) total += warp_sums[v];
        pre[A.batch] = total;
        if (blockIdx.x == 0) A.prefix[A.batch] = total;
      }
      __syncthreads();
    }
    T = pre[A.batch];
    P = min(A.n_workers, T);
    w = static_cast<int>(blockIdx.x) * kWarps + warp;
    if (w >= P) return;
    const Split split(T, P);
    t_first = split.begin(w);
    my_tiles = split.begin(w + 1) - t_first;
  }

  auto stage_ptr = [&](int s) { return smem + (warp * kStages + s) * TL::kStageBytes; };
  auto info_of = [&](int block) {
    const int x = block * 32 + lane;
    if (x >= my_tiles) return TileInfo<TL::kRuns>();
    if constexpr (kCluster) return tile_at<TL::kRuns, kSel>(A, the_b, the_g, t_first + x);
    return tile_info<TL::kRuns, kSel>(A, pre, t_first + x);
  };
  TileInfo<TL::kRuns> cur = info_of(0), nxt;
  auto cur_key0 = [&](int r) {
    if constexpr (TL::kRuns == 1) return cur.key0[0];
    return r ? cur.key0[TL::kRuns - 1] : cur.key0[0];
  };
  // tile i's loads into its stage s; i is less than 32 past the block `block`
  auto issue = [&](int i, int s, int block) {
    if (i >= my_tiles) return;
    int row[TL::kRuns];
#pragma unroll
    for (int r = 0; r < TL::kRuns; ++r)
      row[r] = __shfl_sync(0xffffffffu, (i >> 5) == block ? cur.row[r] : nxt.row[r], i & 31);
    if (!elect_one()) return;
    uint64_t* bar = &bars[s];
    uint8_t* st = stage_ptr(s);
    if constexpr (kI4) {
      // the runs of one page are copied as one
      const bool one = TL::kRuns == 2 && row[TL::kRuns - 1] == row[0] + kTile && row[0] >= 0;
      const int n = one ? 2 : (row[0] >= 0) + (TL::kRuns == 2 && row[TL::kRuns - 1] >= 0);
      if (n == 0) {
        mbar_arrive(bar);
        return;
      }
      mbar_expect_tx(bar, n * ((2 * TL::kBytes + 2 * TL::kScaleBytes) / TL::kRuns));
#pragma unroll 1
      for (int r = 0; r < TL::kRuns; ++r) {
        const int from = r ? row[TL::kRuns - 1] : row[0];
        if (from < 0 || (r == 1 && one)) continue;
        const uint32_t parts = one ? 1 : TL::kRuns, bytes = TL::kBytes / parts, scale_bytes = TL::kScaleBytes / parts;
        uint8_t* codes = st + r * (TL::kBytes / TL::kRuns);
        uint8_t* steps = st + TL::kScaleOff + r * (TL::kScaleBytes / TL::kRuns);
        const int64_t at = static_cast<int64_t>(from);
        bulk_load(codes, A.k_cache + at * (D / 2), bytes, bar);
        bulk_load(steps, A.k_scales + at * 2, scale_bytes, bar);
        bulk_load(codes + TL::kBytes, A.v_cache + at * (D / 2), bytes, bar);
        bulk_load(steps + TL::kScaleBytes, A.v_scales + at * 2, scale_bytes, bar);
      }
      return;
    }
    if (row[0] < 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_expect_tx(bar, 2 * TL::kBytes + 2 * TL::kScaleBytes);
    if constexpr (kI8) {
#pragma unroll
      for (int h = 0; h < G::kHalves; ++h) {
        tma_load_2d(st + h * kTile * G::kRowBytes, &tm_k, bar, G::kRowBytes * h, row[0]);
        tma_load_2d(st + TL::kBytes + h * kTile * G::kRowBytes, &tm_v, bar, G::kRowBytes * h, row[0]);
      }
      bulk_load(st + TL::kScaleOff, A.k_scales + row[0], TL::kScaleBytes, bar);
      bulk_load(st + TL::kScaleOff + TL::kScaleBytes, A.v_scales + row[0], TL::kScaleBytes, bar);
    } else if constexpr (kBF) {
#pragma unroll
      for (int c = 0; c < G::kNFull; ++c) {
        tma_load_2d(st + c * G::kChunkBytes, &tm_k, bar, 64 * c, row[0]);
        tma_load_2d(st + TL::kBytes + c * G::kChunkBytes, &tm_v, bar, 64 * c, row[0]);
      }
      if constexpr (G::kTail) {
        tma_load_2d(st + G::kNFull * G::kChunkBytes, &tm_k32, bar, 64 * G::kNFull, row[0]);
        tma_load_2d(st + TL::kBytes + G::kNFull * G::kChunkBytes, &tm_v32, bar, 64 * G::kNFull, row[0]);
      }
    }
  };
  for (int i = 0; i < kStages; ++i) issue(i, i, 0);
  nxt = info_of(1);

  // ---- per-segment state
  uint32_t qb0[kSteps], qb1[kSteps];
  float qs0 = 0.f, qs1 = 0.f;  // logit multipliers of heads 2qq, 2qq + 1
  float qm0 = 0.f, qm1 = 0.f;  // 4 bits: scale * sum of q
  float o[kMT][4];
  float m_run[2];                         // reference of each head's weights
  float2 nref = make_float2(0.f, 0.f);  // its negative, 0 where there is none
  float2 l_run;
  float2 om;    // 4 bits: sum of p * (offset + 7.5 step) (heads 2qq, 2qq + 1)
  float2 unit;  // quantised: power of two by which p * step enters the MMA
  [[maybe_unused]] float2 seen;  // quantised: this thread's largest p * step * unit since the units were looked at
  [[maybe_unused]] float sw[4];  // 4 bits: sum of the rounded p * step (rows gq and gq + 8 alike)
  auto reset = [&]() {
#pragma unroll
    for (int m = 0; m < kMT; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    m_run[0] = m_run[1] = -INFINITY;
    nref = make_float2(0.f, 0.f);
    l_run = om = seen = make_float2(0.f, 0.f);
    unit = make_float2(0x1p118f, 0x1p118f);  // the largest: any ordinary tile sets it
    sw[0] = sw[1] = sw[2] = sw[3] = 0.f;
  };
  // 4 bits: the accumulators' sums of code become sums of code - 7.5
  auto centre = [&]() {
    const float2 c = mul2(make_float2(sw[0], sw[1]), make_float2(-7.5f / kLowUnit, -7.5f / kLowUnit));
#pragma unroll
    for (int mi = 0; mi < kMT; ++mi) {
      o[mi][0] += c.x;
      o[mi][1] += c.y;
      o[mi][2] = fmaf(16.f, c.x, o[mi][2]);
      o[mi][3] = fmaf(16.f, c.y, o[mi][3]);
    }
    sw[0] = sw[1] = sw[2] = sw[3] = 0.f;
  };
  // Head j's unit so that `top` (any thread's, in the present unit) comes to [2^7,
  // 2^8) if it is not in [1, 2^15), and the head's accumulators in that unit:
  // powers of two, so nothing is rounded.  A unit that grows stops where the
  // accumulators would pass 2^100.
  auto refit = [&](int j, float top) {
    float& u = j ? unit.y : unit.x;
    float most = 0.f;
#pragma unroll
    for (int m = 0; m < kMT; ++m) most = fmaxf(most, fmaxf(fabsf(o[m][j]), fabsf(o[m][j + 2])));
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    }
    if (top == 0.f || (top >= 1.f && top < kTop)) return;
    // exponent bits: u's are 1 .. 245, so 1 / u is a normal number too
    const int had = static_cast<int>(__float_as_uint(u) >> 23);
    int to = had + 134 - static_cast<int>(__float_as_uint(top) >> 23);
    to = min(to, had + min(120, 227 - static_cast<int>(__float_as_uint(most) >> 23)));
    to = max(1, min(to, 245));
    u = __uint_as_float(static_cast<uint32_t>(to) << 23);
    const float ratio = u * __uint_as_float(static_cast<uint32_t>(254 - had) << 23);
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      o[m][j] *= ratio;
      o[m][j + 2] *= ratio;
    }
  };
  auto load_q = [&](int b, int g) {
    const bool head_ok = gq < A.group;
    const __nv_bfloat16* row = A.q + (static_cast<int64_t>(b) * A.hq + g * A.group + gq) * D;
    if constexpr (kBF) {
      const uint32_t* qw = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        qb0[ks] = head_ok ? qw[8 * ks + qq] : 0u;
        qb1[ks] = head_ok ? qw[8 * ks + 4 + qq] : 0u;
      }
      qs0 = qs1 = A.scale_log2;
      return;
    }
    // thread (head gq, quarter qq): a quarter of the channels, in the order of
    // its K words, as fp16 after a power of two that brings the largest |q| to
    // [2^14, 2^15) (exact for all that fp32 sums could tell apart)
    float qv[D / 4];
    float amax = 0.f, sum = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      const int dim0 = kI4 || kQuarter ? qq * (D / 4) + 8 * c : 32 * c + 8 * qq;
      if (head_ok) raw = *reinterpret_cast<const uint4*>(row + dim0);
      const uint32_t wv[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qv[8 * c + 2 * e] = __uint_as_float(wv[e] << 16);
        qv[8 * c + 2 * e + 1] = __uint_as_float(wv[e] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int e = 0; e < D / 4; ++e) {
      amax = fmaxf(amax, fabsf(qv[e]));
      sum += qv[e];
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    // the power of two from amax's exponent bits, kept where it and its inverse are normal
    const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 15), 254);
    const float up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);  // 2^(14 - (ex - 127))
    float qs_own = A.scale_log2 * __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
    if constexpr (kI4) qs_own *= kLowUnit;
    const float qm_own = A.scale_log2 * sum;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      // channels of the k-step's fragments: see i4x2_* and i8x2_*
      const int c0 = kI4 ? 8 * (ks / 2) + 2 * (ks % 2) : 4 * ks, far = kI4 ? 4 : 2;
      // (4 bits: odd channels are the high codes, 16 times as large as the low ones)
      const float up1 = kI4 ? up * (1.f / 16.f) : up;
      qb0[ks] = pack_f16x2(qv[c0] * up, qv[c0 + far] * up);
      qb1[ks] = pack_f16x2(qv[c0 + 1] * up1, qv[c0 + far + 1] * up1);
    }
    qs0 = __shfl_sync(0xffffffffu, qs_own, (2 * qq) * 4);
    qs1 = __shfl_sync(0xffffffffu, qs_own, (2 * qq + 1) * 4);
    qm0 = __shfl_sync(0xffffffffu, qm_own, (2 * qq) * 4);
    qm1 = __shfl_sync(0xffffffffu, qm_own, (2 * qq + 1) * 4);
  };
  // First channel of the run of consecutive ones that o[mi][j], o[mi][j + 2]
  // (and, for 4 bits, the same of m-tile mi + 1) hold.
  auto dim_of = [&](int mi) {
    if constexpr (kBF) return 16 * mi + gq;
    if constexpr (kI8) return 4 * (8 * (mi / 2) + gq) + 2 * (mi % 2);
    return 4 * (gq * (D / 32) + mi / 2) + 2 * (mi % 2);
  };
  // The segment's state: the output rows where this worker saw all of it, else
  // its record (segment + worker; cluster: in this warp's ring, [group][D]).
  float* held = reinterpret_cast<float*>(stage_ptr(0));
  auto finish = [&](int seg, bool whole) {
    if constexpr (kI4) centre();
    float l0 = l_run.x, l1 = l_run.y, m0 = om.x, m1 = om.y;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
      if constexpr (kI4) {
        m0 += __shfl_xor_sync(0xffffffffu, m0, off);
        m1 += __shfl_xor_sync(0xffffffffu, m1, off);
      }
    }
    const int64_t rec = static_cast<int64_t>(seg) + w;
    const int b = A.by_hkv.div(seg), g = seg - b * A.hkv;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      const int h = 2 * qq + j;
      if (h >= A.group) break;
      const float add = j ? m1 : m0, l = j ? l1 : l0;
      [[maybe_unused]] const float back = 1.f / (j ? unit.y : unit.x);
      float y[2 * kMT];
#pragma unroll
      for (int mi = 0; mi < kMT; ++mi) {
        const float lo = j ? o[mi][1] : o[mi][0], hi = j ? o[mi][3] : o[mi][2];
        if constexpr (kI4) {
          y[2 * mi] = fmaf(lo * kLowUnit, back, add);
          y[2 * mi + 1] = fmaf(hi * kHighUnit, back, add);
        } else {
          y[2 * mi] = kI8 ? lo * back : lo;
          y[2 * mi + 1] = kI8 ? hi * back : hi;
        }
      }
      if (!whole) {
        const float2 ml = make_float2(j ? m_run[1] : m_run[0], l);
        if (gq == 0) {
          if constexpr (kCluster) {
            s_ml[warp][h] = ml;
          } else {
            *reinterpret_cast<float2*>(A.rec_ml + (rec * A.group + h) * 2) = ml;
          }
        }
        float* ro = kCluster ? held + h * D : A.rec_o + (rec * A.group + h) * D;
#pragma unroll
        for (int mi = 0; mi < kMT; ++mi) {
          if constexpr (kBF) {
            ro[dim_of(mi)] = y[2 * mi];
            ro[dim_of(mi) + 8] = y[2 * mi + 1];
          } else {
            *reinterpret_cast<float2*>(ro + dim_of(mi)) = make_float2(y[2 * mi], y[2 * mi + 1]);
          }
        }
      } else {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int mi = 0; mi < 2 * kMT; ++mi) y[mi] *= inv;
        apply_epilogue_vec(y, A.epi);
        __nv_bfloat16* oo = A.out + (static_cast<int64_t>(b) * A.hq + g * A.group + h) * D;
#pragma unroll
        for (int mi = 0; mi < kMT; ++mi) {
          if constexpr (kBF) {
            oo[dim_of(mi)] = __float2bfloat16_rn(y[2 * mi]);
            oo[dim_of(mi) + 8] = __float2bfloat16_rn(y[2 * mi + 1]);
          } else {
            *reinterpret_cast<uint32_t*>(oo + dim_of(mi)) = pack_bf16x2(y[2 * mi], y[2 * mi + 1]);
          }
        }
      }
    }
  };

  int seg = 0, left = 0, key_end = 0, k_lo = 0;  // left: tiles until this worker leaves the segment
  bool whole = false;
  [[maybe_unused]] int tile_key = 0;  // every page: first key of the tile
  int s = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int i = 0; i < my_tiles; ++i) {
    if ((i & 31) == 0 && i > 0) {
      cur = nxt;
      nxt = info_of((i >> 5) + 1);
    }
    if (kCluster && i == 0) {
      seg = the_seg;
      reset();
      load_q(the_b, the_g);
      left = my_tiles;
      key_end = length_of(A, the_b);
      k_lo = first_key<kSel>(A, key_end);
      tile_key = (k_lo / TL::kKeys + t_first) * TL::kKeys;
    }
    if (!kCluster && left == 0) {
      seg = __shfl_sync(0xffffffffu, cur.seg, i & 31);
      const int b = A.by_hkv.div(seg), g = seg - b * A.hkv, Tb = A.by_hkv.div(pre[b + 1] - pre[b]);
      reset();
      load_q(b, g);
      const int done = t_first + i - (pre[b] + g * Tb);  // tiles of the segment before this worker's first
      left = min(Tb - done, my_tiles - i);
      whole = left == Tb;
      if (done == 0 && lane == 0) {
        const int n = Split(T, P).worker_of(pre[b] + g * Tb + Tb - 1) - w + 1;
        A.range[seg] = static_cast<uint32_t>(w) << 16 | static_cast<uint32_t>(n);
      }
      key_end = length_of(A, b);
      k_lo = first_key<kSel>(A, key_end);
      tile_key = (k_lo / TL::kKeys + done) * TL::kKeys;
    }
    // every lane polls; whether to go on is a decision of the whole warp
    const bool ready = wait_parity(&bars[s], parity, A.wd);
    if (!__all_sync(0xffffffffu, ready)) {
      // gave up (reported): no state; the copies still on their way get one more bounded wait
      for (int j = 1; j < min(kStages, my_tiles - i); ++j)
        wait_parity(&bars[(s + j) % kStages], s + j < kStages ? parity : parity ^ 1, A.wd);
      break;
    }
#pragma unroll 1
    for (int r = 0; r < TL::kRuns; ++r) {
      const int key0 = kSel ? __shfl_sync(0xffffffffu, cur_key0(r), i & 31) : tile_key + r * kTile;
      if (kSel ? key0 == kNoKey : key0 >= key_end || key0 + kTile <= k_lo) continue;
      const uint32_t kt = smem_u32(stage_ptr(s)) + r * (TL::kBytes / TL::kRuns);
      const uint32_t vt = kt + TL::kBytes;
      const uint32_t ksc = smem_u32(stage_ptr(s)) + TL::kScaleOff + r * (TL::kScaleBytes / TL::kRuns);
      const uint32_t vsc = ksc + TL::kScaleBytes;

      // ---- S^T = K . Q^T
      float sc[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float(&acc)[4] = sc[mt];
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
        if constexpr (kBF) {
          const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
            uint32_t a[4];
            ldsm_x4(bf_addr<D>(kt, 16 * mt + 8 * (mi % 2) + mr, 16 * ks + 8 * (mi / 2)), a);
            mma16816_bf16(acc, a, qb0[ks], qb1[ks]);
          }
        } else {
          const int r0 = 16 * mt + key_of<kKind>(gq), r1 = r0 + 8;
          constexpr int kWords = kI4 ? D / 32 : D / 16;  // of 4 bytes per thread and row
          uint32_t wa[kWords], wb[kWords];
          if constexpr (kI4) {
            const uint32_t a0 = kt + r0 * (D / 2) + qq * (D / 8), a1 = a0 + 8 * (D / 2);
            if constexpr (kWords % 4 == 0) {
#pragma unroll
              for (int c = 0; c < kWords / 4; ++c) {
                const uint4 x = lds128(a0 + 16 * c), y = lds128(a1 + 16 * c);
                wa[4 * c] = x.x; wa[4 * c + 1] = x.y; wa[4 * c + 2] = x.z; wa[4 * c + 3] = x.w;
                wb[4 * c] = y.x; wb[4 * c + 1] = y.y; wb[4 * c + 2] = y.z; wb[4 * c + 3] = y.w;
              }
            } else if constexpr (kWords == 2) {
              const uint2 x = lds64(a0), y = lds64(a1);
              wa[0] = x.x; wa[1] = x.y;
              wb[0] = y.x; wb[1] = y.y;
            } else {
#pragma unroll
              for (int c = 0; c < kWords; ++c) {
                wa[c] = lds32(a0 + 4 * c);
                wb[c] = lds32(a1 + 4 * c);
              }
            }
#pragma unroll
            for (int c = 0; c < kWords; ++c) {
              const uint32_t x = wa[c], y = wb[c];
              mma16816(acc, i4x2_low(x), i4x2_low(y), i4x2_high(x), i4x2_high(y), qb0[2 * c], qb1[2 * c]);
              mma16816(acc, i4x2_low(x >> 8), i4x2_low(y >> 8), i4x2_high(x >> 8), i4x2_high(y >> 8), qb0[2 * c + 1],
                       qb1[2 * c + 1]);
            }
          } else {
            if constexpr (kQuarter) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                const uint32_t off = (qq * (D / 64) + c) * 16;
                const uint4 x = lds128(kt + swz<D, false>(r0 * D + off)), y = lds128(kt + swz<D, false>(r1 * D + off));
                wa[4 * c] = x.x; wa[4 * c + 1] = x.y; wa[4 * c + 2] = x.z; wa[4 * c + 3] = x.w;
                wb[4 * c] = y.x; wb[4 * c + 1] = y.y; wb[4 * c + 2] = y.z; wb[4 * c + 3] = y.w;
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                const uint2 x = lds64(kt + i8_off<D>(r0, 32 * c + 8 * qq)), y = lds64(kt + i8_off<D>(r1, 32 * c + 8 * qq));
                wa[2 * c] = x.x; wa[2 * c + 1] = x.y;
                wb[2 * c] = y.x; wb[2 * c + 1] = y.y;
              }
            }
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks)
              mma16816(acc, i8x2_to_f16x2_even(wa[ks]), i8x2_to_f16x2_even(wb[ks]), i8x2_to_f16x2_odd(wa[ks]),
                       i8x2_to_f16x2_odd(wb[ks]), qb0[ks], qb1[ks]);
          }
        }
      }

      // ---- online softmax per head; positions are looked at only in tiles
      // that reach past [k_lo, key_end)
      uint32_t pb[2][2];
      // bf16: what rounding to bf16 took from the weights, for a second product
      // (eight bits of a weight are fewer than the result's own rounding keeps)
      [[maybe_unused]] uint32_t pl[2][2];
      auto softmax = [&](auto masked_tag) {
        constexpr bool kMasked = decltype(masked_tag)::value;
        float2 x[2][2];                             // [mt][key half], heads 2qq and 2qq + 1
        [[maybe_unused]] float vs[2][2], vo[2][2];  // quantised: V step, 4 bits: V offset
        float mx0 = -INFINITY, mx1 = -INFINITY;
        const float2 qs = make_float2(qs0, qs1);
        [[maybe_unused]] const float2 qm = make_float2(qm0, qm1);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int kl = 16 * mt + 8 * hf + key_of<kKind>(gq);
            const bool ok = !kMasked || (key0 + kl >= k_lo && key0 + kl < key_end);
            float2 v = mul2(make_float2(sc[mt][2 * hf], sc[mt][2 * hf + 1]), qs);
            if constexpr (kI4) {
              const uint2 sk = lds64(ksc + 8 * kl), sv = lds64(vsc + 8 * kl);
              const float step = __uint_as_float(sk.x), off = __uint_as_float(sk.y);
              v = fma2(v, make_float2(step, step), mul2(make_float2(off, off), qm));
              vs[mt][hf] = ok ? __uint_as_float(sv.x) : 0.f;
              vo[mt][hf] = ok ? fmaf(7.5f, __uint_as_float(sv.x), __uint_as_float(sv.y)) : 0.f;  // of code 7.5
            } else if constexpr (kI8) {
              const float step = __uint_as_float(lds32(ksc + 4 * kl));
              v = mul2(v, make_float2(step, step));
              vs[mt][hf] = ok ? __uint_as_float(lds32(vsc + 4 * kl)) : 0.f;
            }
            if (kMasked && !ok) v = make_float2(-INFINITY, -INFINITY);
            x[mt][hf] = v;
            mx0 = fmaxf(mx0, v.x);
            mx1 = fmaxf(mx1, v.y);
          }
        }
        // A head's reference moves, and O is rescaled, only when a logit passes
        // it by more than 8 (weights then reach 2^8, exact as factors), so most
        // tiles need no maximum across lanes.
        const bool up = mx0 > m_run[0] + kSlack || mx1 > m_run[1] + kSlack;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
          }
          const float mn0 = fmaxf(m_run[0], mx0), mn1 = fmaxf(m_run[1], mx1);
          nref = make_float2(mn0 == -INFINITY ? 0.f : -mn0, mn1 == -INFINITY ? 0.f : -mn1);
          const float2 al = make_float2(ex2_approx(m_run[0] + nref.x), ex2_approx(m_run[1] + nref.y));
          m_run[0] = mn0;
          m_run[1] = mn1;
          l_run = mul2(l_run, al);
          if constexpr (kI4) {
            om = mul2(om, al);
            sw[0] *= al.x;
            sw[1] *= al.y;
          }
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            o[m][0] *= al.x; o[m][2] *= al.x;
            o[m][1] *= al.y; o[m][3] *= al.y;
          }
        }
        float2 p[2][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float2 y = add2(x[mt][hf], nref);
            p[mt][hf] = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            l_run = add2(l_run, p[mt][hf]);
            if constexpr (kI4) om = fma2(p[mt][hf], make_float2(vo[mt][hf], vo[mt][hf]), om);
          }
        }
        // pb: S rows 2qq, 2qq + 1 and 8 + 2qq, 9 + 2qq of head gq
        if constexpr (kBF) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float2 v = p[mt][hf];
              const uint32_t packed = pack_bf16x2(v.x, v.y);
              pb[mt][hf] = transpose8x8(packed);
              pl[mt][hf] = transpose8x8(pack_bf16x2(v.x - __uint_as_float(packed << 16),
                                                    v.y - __uint_as_float(packed & 0xffff0000u)));
            }
          }
        } else {
          // p * step enters the MMA as fp16 (half a step of it, 2^-11 of a
          // weight; what 4-bit codes share is added in fp32, so it falls on
          // code - 7.5) after multiplication by the head's unit.  The unit is
          // set anew, and O rescaled with it, when a weight reaches 2^15, and
          // every 8 tiles where none of their weights reached 1: so what fp16
          // drops or rounds by its smallest step, 2^-25 of a unit, is small
          // beside a weight at most 16 tiles before it, however large those of
          // other tiles are.
          auto weigh = [&]() {
            float2 w[2][2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                w[mt][hf] = mul2(p[mt][hf], mul2(unit, make_float2(vs[mt][hf], vs[mt][hf])));
                pb[mt][hf] = transpose8x8(pack_f16x2(w[mt][hf].x, w[mt][hf].y));
              }
            }
            seen.x = max3f(seen.x, w[0][0].x, max3f(w[0][1].x, w[1][0].x, w[1][1].x));
            seen.y = max3f(seen.y, w[0][0].y, max3f(w[0][1].y, w[1][0].y, w[1][1].y));
          };
          weigh();
          // once; up to three times where a product with the old unit is infinite (four: a step is)
#pragma unroll 1
          for (int tries = 0; tries < 4 && __any_sync(0xffffffffu, fmaxf(seen.x, seen.y) >= kTop); ++tries) {
            if constexpr (kI4) centre();
            refit(0, seen.x);
            refit(1, seen.y);
            seen = make_float2(0.f, 0.f);
            weigh();
          }
        }
      };
      const bool inside = key0 >= k_lo && key0 + kTile <= key_end;
      if (inside) {
        softmax(std::false_type{});
      } else {
        softmax(std::true_type{});
      }

      // ---- O^T += V^T . P'
      if constexpr (kBF) {
        if (!inside) {
          // rows outside may hold NaN or Inf: zero them (P is 0 there)
          const int key = key0 + lane;
          if (key < k_lo || key >= key_end) {
#pragma unroll
            for (int c = 0; c < D; c += 8)
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(bf_addr<D>(vt, lane, c)), "r"(0u) : "memory");
            fence_proxy_async_smem();  // ordered before the copy that refills this stage
          }
          __syncwarp();
        }
        const int mi4 = lane >> 3, mr = lane & 7;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int mi = 0; mi < kMT; ++mi) {
            uint32_t a[4];
            ldsm_x4_trans(bf_addr<D>(vt, 16 * mt + 8 * (mi4 / 2) + mr, 16 * mi + 8 * (mi4 % 2)), a);
            mma16816_bf16(o[mi], a, pb[mt][0], pb[mt][1]);
            mma16816_bf16(o[mi], a, pl[mt][0], pl[mt][1]);
          }
        }
      } else if constexpr (kI8) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int kk0 = 16 * mt + 2 * qq;
#pragma unroll
          for (int pr = 0; pr < D / 32; ++pr) {
            const uint32_t xw = (8 * pr + gq) * 4;
            const uint32_t w0 = lds32(vt + i8_off<D>(kk0 + 0, xw)), w1 = lds32(vt + i8_off<D>(kk0 + 1, xw));
            const uint32_t w2 = lds32(vt + i8_off<D>(kk0 + 8, xw)), w3 = lds32(vt + i8_off<D>(kk0 + 9, xw));
            const uint32_t t01l = prmt(w0, w1, 0x5410), t01h = prmt(w0, w1, 0x7632);
            const uint32_t t23l = prmt(w2, w3, 0x5410), t23h = prmt(w2, w3, 0x7632);
            mma16816(o[2 * pr], i8x2_to_f16x2_even(t01l), i8x2_to_f16x2_odd(t01l), i8x2_to_f16x2_even(t23l),
                     i8x2_to_f16x2_odd(t23l), pb[mt][0], pb[mt][1]);
            mma16816(o[2 * pr + 1], i8x2_to_f16x2_even(t01h), i8x2_to_f16x2_odd(t01h), i8x2_to_f16x2_even(t23h),
                     i8x2_to_f16x2_odd(t23h), pb[mt][0], pb[mt][1]);
          }
        }
      } else {
        // thread (gq, qq): channels [gq D/8, (gq+1) D/8) of four keys a half
        // tile; `half` holds four channels of a key pair in its two 16-bit halves
        constexpr int kH = D / 32;
        auto four = [&](float (&lo)[4], float (&hi)[4], uint32_t t01, uint32_t t23, const uint32_t (&p)[2]) {
          mma16816(lo, i4x2_low(t01), i4x2_high(t01), i4x2_low(t23), i4x2_high(t23), p[0], p[1]);
          mma16816(hi, i4x2_low(t01 >> 8), i4x2_high(t01 >> 8), i4x2_low(t23 >> 8), i4x2_high(t23 >> 8), p[0], p[1]);
        };
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          mma16816(sw, kOnes, kOnes, kOnes, kOnes, pb[mt][0], pb[mt][1]);
          const uint32_t a0 = vt + gq * (D / 16) + 16 * mt * (D / 2);
          uint32_t at[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            at[e] = a0 + (key_of<kKind>(2 * qq + (e & 1)) + 8 * (e >> 1)) * (D / 2);
          if constexpr (kH % 2 == 0) {
            uint32_t wv[4][kH / 2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (kH == 8) {
                const uint4 x = lds128(at[e]);
                wv[e][0] = x.x; wv[e][1] = x.y; wv[e][2] = x.z; wv[e][3] = x.w;
              } else if constexpr (kH == 4) {
                const uint2 x = lds64(at[e]);
                wv[e][0] = x.x; wv[e][1] = x.y;
              } else {
                wv[e][0] = lds32(at[e]);
              }
            }
#pragma unroll
            for (int c = 0; c < kH / 2; ++c) {
              four(o[4 * c], o[4 * c + 1], prmt(wv[0][c], wv[1][c], 0x5410), prmt(wv[2][c], wv[3][c], 0x5410), pb[mt]);
              four(o[4 * c + 2], o[4 * c + 3], prmt(wv[0][c], wv[1][c], 0x7632), prmt(wv[2][c], wv[3][c], 0x7632), pb[mt]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kH; ++c) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint16_t hw;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hw) : "r"(at[e] + 2 * c));
                v[e] = hw;
              }
              four(o[2 * c], o[2 * c + 1], v[0] | (v[1] << 16), v[2] | (v[3] << 16), pb[mt]);
            }
          }
        }
      }
    }
    if constexpr (!kBF) {
      if ((i & 7) == 7) {
        if constexpr (kI4) centre();
        const unsigned same = 0x11111111u << qq;  // the lanes of this thread's heads
        const unsigned x = __ballot_sync(0xffffffffu, seen.x >= 1.f), y = __ballot_sync(0xffffffffu, seen.y >= 1.f);
        if (__any_sync(0xffffffffu, (x & same) == 0 || (y & same) == 0)) {
          refit(0, seen.x);
          refit(1, seen.y);
        }
        seen = make_float2(0.f, 0.f);
      }
    }
    // the stage is free: the tile kStages on goes there
    __syncwarp();
    fence_proxy_async_smem();
    issue(i + kStages, s, i >> 5);
    if (++s == kStages) {
      s = 0;
      parity ^= 1;
    }
    if (left > 1) tile_key += TL::kKeys;
    if (--left == 0) finish(seg, whole);
  }
  if constexpr (kCluster) {
    // every warp's state is in its CTA's shared memory: a thread takes two
    // channels of a head from all of them
    cluster_sync_all();
    const int c = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
    const uint32_t ml0 = smem_u32(&s_ml[0][0]), rec0 = smem_u32(smem);
    for (int x = rank * kThreads + static_cast<int>(threadIdx.x); x < A.group * (D / 2); x += c * kThreads) {
      const int h = x / (D / 2), dim = 2 * (x - h * (D / 2));
      float m = -INFINITY;
      for (int r = 0; r < c; ++r) {
#pragma unroll
        for (int v = 0; v < kWarps; ++v) m = fmaxf(m, ld_cluster_f2(mapa_shared(ml0 + (v * 8 + h) * 8, r)).x);
      }
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f;
      float y[2] = {0.f, 0.f};
      for (int r = 0; r < c; ++r) {
        float2 ml[kWarps], part[kWarps];
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          ml[v] = ld_cluster_f2(mapa_shared(ml0 + (v * 8 + h) * 8, r));
          part[v] = ld_cluster_f2(mapa_shared(rec0 + v * kStages * TL::kStageBytes + (h * D + dim) * 4, r));
        }
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          if (ml[v].x == -INFINITY) continue;  // no key there (and perhaps no record)
          const float wt = ex2_approx(ml[v].x - ref);
          l = fmaf(wt, ml[v].y, l);
          y[0] = fmaf(wt, part[v].x, y[0]);
          y[1] = fmaf(wt, part[v].y, y[1]);
        }
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
      y[0] *= inv;
      y[1] *= inv;
      apply_epilogue_vec(y, A.epi);
      *reinterpret_cast<uint32_t*>(A.out + (static_cast<int64_t>(the_b) * A.hq + the_g * A.group + h) * D + dim) =
          pack_bf16x2(y[0], y[1]);
    }
    cluster_sync_all();  // nobody leaves while its shared memory is read
  }
}

// One query head's split records into its output row; the rows of segments
// without a tile.  A warp takes every eighth record, a lane D / 32 consecutive
// channels of it; the weights of up to 1024 records are held at a time.
constexpr int kMergeThreads = 256;
constexpr int kMergeRecords = 1024;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_pages_merge_kernel(const PageArgs A) {
  constexpr int E = D / 32, kMergeWarps = kMergeThreads / 32;
  __shared__ float2 s_ml[kMergeRecords];
  __shared__ float s_red[2][kMergeWarps];
  __shared__ float s_o[kMergeWarps][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = A.by_group.div(blockIdx.x), h = blockIdx.x - seg * A.group;
  const int b = A.by_hkv.div(seg), g = seg - b * A.hkv;
  griddep_launch_dependents();
  griddep_wait();
  const int p0 = __ldcg(A.prefix + b), p1 = __ldcg(A.prefix + b + 1);
  const uint32_t range = __ldcg(A.range + seg);
  __nv_bfloat16* out = A.out + (static_cast<int64_t>(b) * A.hq + g * A.group + h) * D;
  if (p0 == p1) {  // no tile: nobody wrote the range
    const __nv_bfloat16 zero = __float2bfloat16_rn(apply_epilogue(0.f, A.epi));
    for (int c = tid; c < D; c += kMergeThreads) out[c] = zero;
    return;
  }
  const int n = range & 0xffffu;
  if (n == 1) return;  // stored by its worker
  // A range that no worker wrote, since one gave up waiting (reported), is
  // whatever the workspace held: past the workers it is not followed, and any
  // other leads to records inside the workspace and a meaningless row.
  if (n + static_cast<int>(range >> 16) > A.n_workers) return;
  const int64_t rec0 = static_cast<int64_t>(seg) + (range >> 16);
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int r0 = 0; r0 < n; r0 += kMergeRecords) {
    const int count = min(kMergeRecords, n - r0);
    float mine = -INFINITY;
    for (int r = tid; r < count; r += kMergeThreads) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(A.rec_ml) + (rec0 + r0 + r) * A.group + h);
      s_ml[r] = v;
      mine = fmaxf(mine, v.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, off));
    if (lane == 0) s_red[0][warp] = mine;
    __syncthreads();
    float top = m;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, s_red[0][w]);
    const float ref = top == -INFINITY ? 0.f : top;
    if (r0 > 0) {
      const float a = ex2_approx(m - ref);
      l *= a;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= a;
    }
    m = top;
#pragma unroll 8
    for (int r = warp; r < count; r += kMergeWarps) {
      const float2 v = s_ml[r];
      const float wt = ex2_approx(v.x - ref);
      l = fmaf(wt, v.y, l);  // the same in every lane
      const float* src = A.rec_o + ((rec0 + r0 + r) * A.group + h) * D + lane * E;
      float y[E];
      if constexpr (E % 4 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(y + e) = __ldcg(reinterpret_cast<const float4*>(src + e));
      } else if constexpr (E == 2) {
        *reinterpret_cast<float2*>(y) = __ldcg(reinterpret_cast<const float2*>(src));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = __ldcg(src + e);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, y[e], acc[e]);
    }
    __syncthreads();
  }
  if (lane == 0) s_red[1][warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) l += s_red[1][w];
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = tid; c < D; c += kMergeThreads) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) y += s_o[w][c];
    out[c] = __float2bfloat16_rn(apply_epilogue(y * inv, A.epi));
  }
}

struct Maps {
  CUtensorMap k, v, k32, v32;
};

// Tensor maps of the bf16 or int8 pools, as the contiguous decode's.
template <int D, bool kBF>
fa_status encode_maps(const fa_decode_params& p, const fa_kv_pages& pg, Maps* m) {
  using G = Geom<D, kBF>;
  const uint64_t dims[2] = {static_cast<uint64_t>(D), static_cast<uint64_t>(pg.num_pages) * p.hkv * pg.page_size};
  const uint64_t strides[1] = {static_cast<uint64_t>(D) * (kBF ? 2 : 1)};
  const uint32_t box[2] = {static_cast<uint32_t>(kBF ? 64 : G::kRowBytes), static_cast<uint32_t>(kTile)};
  const CUtensorMapSwizzle sw = G::kSwzMask == 0x70   ? CU_TENSOR_MAP_SWIZZLE_128B
                                : G::kSwzMask == 0x30 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_NONE;
  const CUtensorMapDataType dt = kBF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  fa_status st = encode_tensor_map(&m->k, dt, 2, p.k_cache, dims, strides, box, sw);
  if (st == FA_OK) st = encode_tensor_map(&m->v, dt, 2, p.v_cache, dims, strides, box, sw);
  if (st != FA_OK) return st;
  if constexpr (G::kTail) {
    const uint32_t box32[2] = {32, static_cast<uint32_t>(kTile)};
    st = encode_tensor_map(&m->k32, dt, 2, p.k_cache, dims, strides, box32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (st == FA_OK) st = encode_tensor_map(&m->v32, dt, 2, p.v_cache, dims, strides, box32, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  return st;
}

// Lets one kernel use this much shared memory; set once per device (`done` is
// that kernel's own).
fa_status allow_smem(const void* kern, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  if (done[dev].load(std::memory_order_acquire)) return FA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return FA_ERR_CUDA;
  done[dev].store(true, std::memory_order_release);
  return FA_OK;
}

// Tiles that a segment has at most.
template <int D, int kKind, bool kSel>
int64_t most_tiles(const PageArgs& A) {
  constexpr int kKeys = Tile<D, kKind>::kKeys;
  int64_t keys = A.capacity;
  if (kSel) {
    const int64_t chosen = static_cast<int64_t>(A.top_k) * A.page_size;
    keys = chosen < keys ? chosen : keys;
  } else if (A.window > 0 && static_cast<int64_t>(A.window) + kKeys < keys) {
    keys = static_cast<int64_t>(A.window) + kKeys;  // the window may start inside a tile
  }
  return (keys + kKeys - 1) / kKeys;
}

// One cluster per segment: as many CTAs as the device holds at once and the
// tiles are worth; 0 where spreading all tiles evenly over the device, and a
// second kernel's merge, is faster.  Counted in tiles one after the other: a
// cluster's warps take seg_tiles / (4 c) each, in turns where the clusters do
// not fit at once; an even split the device's share of all tiles, and about
// four tiles' time for the records, the second launch and its reads.
// Clustered and split, us, 4 bits, 8 KV heads of 128: one sequence of 257 keys
// 8.3 and 10.3, 8192: 14.4 and 12.6, 10,240: 15.1 and 16.4, 12,288 (split from
// here on): 16.5 and 15.1, 16,384: 20.5 and 18.4, 32,768: 32 and 21; 16 of 4096:
// 22.6 and 26.7, of 8192: 41.0 and 41.7; 128 pairs of 2048 chosen keys: 16.4 and
// 22.  Powers of two only: clusters of three made the selection before them wait
// (43 -> 48 us).
template <int D, int kKind>
int cluster_of(int64_t segs, int64_t seg_tiles) {
  const int64_t resident = static_cast<int64_t>(device_sm_count()) * Tile<D, kKind>::kCtas;
  int64_t c = 1;
  while (c < 8 && segs * c * 2 <= resident && c * kWarps < seg_tiles) c *= 2;
  const int64_t turns = (segs * c + resident - 1) / resident;
  const int64_t clustered = (seg_tiles + c * kWarps - 1) / (c * kWarps) * turns;
  const int64_t even = (segs * seg_tiles + resident * kWarps - 1) / (resident * kWarps) + 4;
  return clustered <= even && segs * c < (int64_t(1) << 31) ? static_cast<int>(c) : 0;
}

template <int D, int kKind, bool kSel>
fa_status launch_clustered(const PageArgs& A, const Maps& maps, int cluster, const LaunchCtx& ctx) {
  using TL = Tile<D, kKind>;
  auto kern = decode_pages_kernel<D, kKind, kSel, true>;
  static_assert(TL::kStages * TL::kStageBytes >= 8 * D * 4, "a warp's record in its ring");
  static std::atomic<bool> allowed[64];
  const fa_status st = allow_smem(reinterpret_cast<const void*>(kern), TL::kSmem, allowed);
  if (st != FA_OK) return st;
  return launch_dependent(kern, dim3(static_cast<unsigned>(static_cast<int64_t>(A.batch) * A.hkv * cluster)), kThreads,
                          TL::kSmem, cluster, ctx.stream, maps.k, maps.v, maps.k32, maps.v32, A);
}

template <int D, int kKind, bool kSel>
fa_status launch_typed(const fa_decode_params& p, const fa_kv_pages& pg, PageArgs A, const LaunchCtx& ctx) {
  using TL = Tile<D, kKind>;
  auto kern = decode_pages_kernel<D, kKind, kSel, false>;
  auto merge = decode_pages_merge_kernel<D>;
  Maps maps = {};
  fa_status st = FA_OK;
  if constexpr (kKind != FA_I4) {
    st = encode_maps<D, kKind == FA_BF16>(p, pg, &maps);
    if (st != FA_OK) return st;
  }
  const int64_t seg_tiles = most_tiles<D, kKind, kSel>(A);
  if (const int cluster = cluster_of<D, kKind>(static_cast<int64_t>(p.batch) * A.hkv, seg_tiles))
    return launch_clustered<D, kKind, kSel>(A, maps, cluster, ctx);
  static std::atomic<bool> allowed[64];
  static_assert(TL::kSmem + (kMaxBatch + 1) * 4 <= 232448, "shared memory of a CTA");
  st = allow_smem(reinterpret_cast<const void*>(kern), TL::kSmem + (kMaxBatch + 1) * 4, allowed);
  if (st != FA_OK) return st;
  // Workers: four per CTA, as many CTAs as fit, as far as the caller's
  // workspace holds their records (it is sized for eight workers per SM that
  // serve min(hq, 8) heads each).
  const int sms = device_sm_count();
  const int room = sms * 8 * (p.hq < 8 ? p.hq : 8) / A.group;
  int workers = sms * TL::kCtas * kWarps;
  if (workers > room) workers = room / kWarps * kWarps;
  const size_t plan = (static_cast<size_t>(p.batch + 1 + static_cast<size_t>(p.batch) * p.hq) * 4 + 255) / 256 * 256;
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  A.prefix = reinterpret_cast<int32_t*>(ws);
  A.range = reinterpret_cast<uint32_t*>(ws) + (p.batch < kMaxBatch ? p.batch : kMaxBatch) + 1;
  const PageArgs all = A;
  for (int b0 = 0; b0 < p.batch; b0 += kMaxBatch) {
    A.batch = p.batch - b0 < kMaxBatch ? p.batch - b0 : kMaxBatch;
    A.q = all.q + static_cast<int64_t>(b0) * A.hq * D;
    A.out = all.out + static_cast<int64_t>(b0) * A.hq * D;
    A.seqlens = all.seqlens + b0;
    A.block_table = all.block_table + static_cast<int64_t>(b0) * A.max_pages;
    if (kSel) A.selected = all.selected + static_cast<int64_t>(b0) * A.hkv_real * A.top_k;
    // no more workers than there can be tiles
    const int64_t most = seg_tiles * A.batch * A.hkv;
    if (most >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
    A.n_workers = most < workers ? static_cast<int>((most + kWarps - 1) / kWarps * kWarps) : workers;
    A.rec_o = reinterpret_cast<float*>(ws + plan);
    A.rec_ml = A.rec_o + (static_cast<size_t>(A.batch) * A.hkv + A.n_workers) * A.group * D;
    // an ordinary launch: blocks that came while an earlier kernel still held
    // its places would lie unevenly on the SMs (44 -> 51 us with one sequence
    // of 131071 keys, called back to back)
    note_variant(reinterpret_cast<const void*>(kern));
    kern<<<A.n_workers / kWarps, kThreads, TL::kSmem + (A.batch + 1) * 4, ctx.stream>>>(maps.k, maps.v, maps.k32, maps.v32,
                                                                                        A);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    st = launch_dependent(merge, dim3(static_cast<unsigned>(A.batch * A.hkv * A.group)), kMergeThreads, 0, 0, ctx.stream, A);
    if (st != FA_OK) return st;
  }
  return FA_OK;
}

// Calls f(dimension, kind, selected?) with the call's head size, cache type and
// form as types; FA_ERR_UNSUPPORTED for a head size without kernels.
template <int D, typename F>
fa_status dispatch_kind(int kind, bool selected, const F& f) {
  using Dim = std::integral_constant<int, D>;
  using I4 = std::integral_constant<int, FA_I4>;
  if (!selected) return f(Dim{}, I4{}, std::false_type{});
  if (kind == FA_I4) return f(Dim{}, I4{}, std::true_type{});
  if (kind == FA_I8) return f(Dim{}, std::integral_constant<int, FA_I8>{}, std::true_type{});
  return f(Dim{}, std::integral_constant<int, FA_BF16>{}, std::true_type{});
}
template <typename F>
fa_status dispatch(const fa_decode_params& p, bool selected, const F& f) {
  switch (p.head_dim) {
    case 32: return dispatch_kind<32>(p.kv_dtype, selected, f);
    case 64: return dispatch_kind<64>(p.kv_dtype, selected, f);
    case 96: return dispatch_kind<96>(p.kv_dtype, selected, f);
    case 128: return dispatch_kind<128>(p.kv_dtype, selected, f);
    case 256: return dispatch_kind<256>(p.kv_dtype, selected, f);
  }
  return FA_ERR_UNSUPPORTED;
}

PageArgs page_args(const fa_decode_params& p, const fa_kv_pages& pages, const int32_t* selected, int top_k) {
  PageArgs A = {};
  A.q = static_cast<const __nv_bfloat16*>(p.q);
  A.k_cache = static_cast<const uint8_t*>(p.k_cache);
  A.v_cache = static_cast<const uint8_t*>(p.v_cache);
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
  A.out = static_cast<__nv_bfloat16*>(p.out);
  const int full_group = p.hq / p.hkv;
  int split = (full_group + 7) / 8;
  while (full_group % split != 0) ++split;
  A.hq = p.hq;
  A.hkv_real = p.hkv;
  A.kv_split = split;
  A.hkv = p.hkv * split;
  A.group = full_group / split;
  A.window = p.window;
  A.by_hkv = FastDiv::of(A.hkv);
  A.by_split = FastDiv::of(A.kv_split);
  A.by_page = FastDiv::of(A.page_size);
  A.by_page_runs = FastDiv::of(A.page_size / kTile);
  A.by_group = FastDiv::of(A.group);
  A.scale_log2 = p.softmax_scale * kLog2e;
  A.epi = make_epilogue(p.epilogue, p.n_epilogue);
  A.batch = p.batch;
  return A;
}

}  // namespace

bool decode_pages_needs_workspace(const fa_decode_params& p, const fa_kv_pages& pages, int top_k) {
  const PageArgs A = page_args(p, pages, nullptr, top_k);
  int cluster = 0;
  dispatch(p, top_k > 0, [&](auto d, auto kind, auto sel) {
    cluster = cluster_of<d, kind>(static_cast<int64_t>(p.batch) * A.hkv, most_tiles<d, kind, sel>(A));
    return FA_OK;
  });
  return cluster == 0;
}

fa_status launch_decode_pages(const fa_decode_params& p, const fa_kv_pages& pages, const int32_t* selected, int top_k,
                              const LaunchCtx& ctx) {
  PageArgs A = page_args(p, pages, selected, top_k);
  A.wd = ctx.wd;
  return dispatch(p, selected != nullptr,
                  [&](auto d, auto kind, auto sel) { return launch_typed<d, kind, sel>(p, pages, A, ctx); });
}

}  // namespace fa
