// decode_mma.cuh -- what the single-query attention kernels share: geometry of
// bf16 and int8 cache tiles in shared memory, shared-memory and mma.sync
// wrappers, and exact widening of codes.
#pragma once

#include "device.cuh"

namespace fa {

constexpr int kWarps = 4;    // compute warps (workers) per CTA
constexpr int kTile = 32;    // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool kBF>
struct Geom {
  static constexpr int kTileBytes = kTile * D * (kBF ? 2 : 1);  // int8 codes or bf16
  static constexpr int kScaleBytes = kBF ? 0 : 2 * kTile * 4;    // K and V scales (int8)
  static constexpr int kScaleOff = 2 * kTileBytes;
  static constexpr int kStageBytes = ((2 * kTileBytes + kScaleBytes) + 1023) / 1024 * 1024;
  // bf16: 128-byte swizzle of 64-dim chunks [32 rows x 128 B], then for D =
  // 32 or 96 a 32-dim tail chunk [32 rows x 64 B] with the 64-byte swizzle.
  // int8 rows: D = 64 and 128 fill one TMA box with the 64- / 128-byte
  // swizzle; D = 256 is two 128-byte halves (two boxes, 4 KB apart in the
  // tile); D = 32 and 96 are plain rows
  static constexpr int kSwzMask = (kBF || D == 128 || D == 256) ? 0x70 : (D == 64 ? 0x30 : 0);
  static constexpr int kRowBytes = kBF ? 128 : (D > 128 ? 128 : D);  // bytes per row of one box
  static constexpr int kHalves = (!kBF && D > 128) ? D / 128 : 1;   // int8 boxes per tile row
  static constexpr int kChunkBytes = kTile * 128;
  static constexpr int kNFull = D / 64;                 // bf16: full 64-dim chunks
  static constexpr bool kTail = kBF && (D % 64) == 32;  // bf16: a 32-dim tail chunk
  // stages per worker ring (a bf16 tile at D = 256 is 32 KB: one stage,
  // the producer refilling it as soon as its worker releases it)
  static constexpr int kStages = (kBF && D == 256) ? 1 : 3;
  static constexpr int kCtas = ((kBF && (D == 128 || D == 96)) || D == 256) ? 1 : 2;
  static constexpr int kSmem = kWarps * kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
  // sequences whose tile prefix fits in the shared memory the CTAs per SM
  // leave over (228 KB per SM, 1 KB reserved per CTA, 256 B margin)
  static constexpr int kPrefixCap = ((233472 / kCtas) - 1024 - kSmem - 256) / 4 - 1;
};
// TMA swizzle of a byte offset inside a tile whose base is aligned to the
// swizzle period: bits [4,7) (128B) or [4,6) (64B) ^= bits [7,10) / [7,9).
template <int D, bool kBF>
__device__ __forceinline__ uint32_t swz(uint32_t lin) {
  return lin ^ ((lin >> 3) & Geom<D, kBF>::kSwzMask);
}
// Offset of byte b of int8 row r inside a tile (the box halves of D = 256).
template <int D>
__device__ __forceinline__ uint32_t i8_off(int r, int b) {
  using G = Geom<D, false>;
  return (b / G::kRowBytes) * (kTile * G::kRowBytes) + swz<D, false>(r * G::kRowBytes + b % G::kRowBytes);
}
// Shared address of element (key r, dim c) of a bf16 tile at `tile`.
template <int D>
__device__ __forceinline__ uint32_t bf_addr(uint32_t tile, int r, int c) {
  using G = Geom<D, true>;
  if (G::kTail && c / 64 == G::kNFull) {  // the 32-dim tail: 64-byte rows, 64-byte swizzle
    const uint32_t lin = r * 64 + (c % 64) * 2;
    return tile + G::kNFull * G::kChunkBytes + (lin ^ ((lin >> 3) & 0x30));
  }
  return tile + (c / 64) * G::kChunkBytes + swz<D, true>(r * 128 + (c % 64) * 2);
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// fp16x2 of the signed bytes 0 and 2 of w (exact).
__device__ __forceinline__ uint32_t i8x2_to_f16x2_even(uint32_t w) {
  uint32_t t, r;
  asm("lop3.b32 %0, %1, 0x00ff00ff, 0x64806480, 0x6a;" : "=r"(t) : "r"(w));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0x64806480u));
  return r;
}
// fp16x2 of the signed bytes 1 and 3 of w (exact).
__device__ __forceinline__ uint32_t i8x2_to_f16x2_odd(uint32_t w) { return i8x2_to_f16x2_even(w >> 8); }

// fp16x2 pairs 1152 + c of the signed bytes of w: bytes 0, 2 -> even and
// 1, 3 -> odd (exact; the caller removes the bias).  byte ^ 0x80 = c + 128
// becomes the low mantissa byte of 1024 (fp16 0x6400).
__device__ __forceinline__ void i8x4_to_f16x2_biased(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t x = w ^ 0x80808080u;
  even = prmt(x, 0x64646464u, 0x4240);
  odd = prmt(x, 0x64646464u, 0x4341);
}
constexpr float kCodeBias = 1152.0f;

// fp16x2 of 4-bit codes as subnormal numbers: a code in mantissa bits 0-3 of
// an otherwise empty half is exactly code * 2^-24, one in bits 4-7 is
// code * 2^-20, and the MMA multiplies subnormal inputs exactly.  So one AND
// widens two codes: those in the low halves of bytes 0 and 2 of w, and those
// in the high halves.
__device__ __forceinline__ uint32_t i4x2_low(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t i4x2_high(uint32_t w) { return w & 0x00f000f0u; }
constexpr float kLowUnit = 16777216.f;  // 2^24
constexpr float kHighUnit = 1048576.f;  // 2^20

// Four 8x8 b16 matrices; lane l gives the row address of matrix l / 8, row l % 8.
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}


__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

}  // namespace fa
