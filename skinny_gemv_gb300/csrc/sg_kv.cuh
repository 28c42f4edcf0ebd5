// The paged NVFP4 KV cache: byte layout, quantisation and decoding, shared by the
// kernels that append to it, read it back and attend over it.
//
// A key or value row (head dimension 128) is 8 blocks of 16 elements; element x
// is held as an E2M1 code and the block's E4M3 scale, x ~ e2m1(code) * scale * g
// with one power of two g per cache (k_scale, v_scale).  A page holds page_size
// tokens (a multiple of 16) as [kv head][token tile of 16][2304 bytes]; a tile is
// K codes (1024), K scales (128), V codes (1024), V scales (128).  The orders
// inside a tile are those in which a warp's m16n8k16 fragments want them (lane
// 4 g + t): keys g and g + 8 are the rows of a score product, so K codes are plain
// rows; keys 2t, 2t + 1, 2t + 8, 2t + 9 are the summed axis of a value product, so
// the V codes of such a key pair and one block of 16 dims share a 16-byte word.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace sg {

constexpr int kKvDim = 128;        // head dimension
constexpr int kKvBlock = 16;       // elements per scale
constexpr int kKvBlocks = kKvDim / kKvBlock;
constexpr int kKvTile = 16;        // tokens per tile
constexpr int kKvKScaleOff = 1024;
constexpr int kKvVCodeOff = 1152;
constexpr int kKvVScaleOff = 2176;
constexpr int kKvTileBytes = 2304;

// Byte offsets inside a tile: token r (0-15), block q (0-7).
__host__ __device__ constexpr int kv_k_code(int r, int q) { return 64 * r + 8 * q; }
__host__ __device__ constexpr int kv_k_scale(int r, int q) {
  return kKvKScaleOff + ((r & 7) * 4 + (q >> 1)) * 4 + (r >> 3) * 2 + (q & 1);
}
__host__ __device__ constexpr int kv_v_code(int r, int q) {
  return kKvVCodeOff + (r >> 3) * 512 + (q * 4 + ((r & 7) >> 1)) * 16 + (r & 1) * 8;
}
__host__ __device__ constexpr int kv_v_scale(int r, int q) {
  return kKvVScaleOff + (q * 4 + ((r & 7) >> 1)) * 4 + (r >> 3) * 2 + (r & 1);
}

// Where a cache lives: page p at base + p * pitch bytes.
struct KvCache {
  uint8_t* base;
  int64_t pitch;
  int32_t num_pages;
  int32_t page_size;  // a multiple of 16
};

// The tile of (page, kv head, token offset inside the page).
__device__ __forceinline__ uint8_t* kv_tile(const KvCache& c, int32_t page, int head, int offset) {
  return c.base + page * c.pitch + (static_cast<int64_t>(head) * (c.page_size / kKvTile) + offset / kKvTile) * kKvTileBytes;
}

// Two E4M3 bytes to half2 (exact; 0x7f is NaN).
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return *reinterpret_cast<const __half2*>(&r);
}

// Two E2M1 codes (a byte, low nibble first) to half2 (exact).
__device__ __forceinline__ __half2 e2m1x2_half2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, u, v, w;\n\tmov.b32 {t, u, v, w}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
  return *reinterpret_cast<const __half2*>(&r);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Eight E2M1 codes (a word, low nibble first) to four half2 times a scale (exact: 2 + 4
// significant bits).
__device__ __forceinline__ void e2m1x8_times(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  uint32_t c[4];
  asm("{\n\t.reg .b8 t, u, v, w;\n\tmov.b32 {t, u, v, w}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\tcvt.rn.f16x2.e2m1x2 %1, u;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, v;\n\tcvt.rn.f16x2.e2m1x2 %3, w;\n\t}"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&c[i]), s));
}

// Eight floats to a word of E2M1 codes, the first in the low nibble (nearest, ties to
// even, magnitudes past 6 to 6).
__device__ __forceinline__ uint32_t e2m1x8_from(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, u, v, w;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 u, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 v, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 w, %8, %7;\n\t"
      "mov.b32 %0, {t, u, v, w};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// A float to E4M3 (nearest, ties to even, past 448 to 448, NaN to 0x7f).
__device__ __forceinline__ uint32_t e4m3_from(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x), "f"(0.f));
  return r & 0xFFu;
}

// 1 / x to about 2^-23 (rcp.approx).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// |x| with the sign of the bits `s` (a small negative rounds to code -0, not +0).
__device__ __forceinline__ float signed_as(float x, uint32_t s) {
  return __uint_as_float((__float_as_uint(x) & 0x7FFFFFFFu) | (s & 0x80000000u));
}

// Quantises half a block: 8 bf16 values (4 words, low half first) of this lane, the
// other 8 in the neighbouring lane (lane ^ 1), divided by the power of two 1 / inv_g.
// `codes` receives 4 bytes of E2M1 pairs; returns the block's scale byte e4m3(amax /
// 6).  A NaN anywhere makes the scale NaN (the maximum is taken over the bit patterns,
// where NaN sorts above infinity); an infinity saturates.  The codes are those of
// exact arithmetic: x / s is either a midpoint of two codes or at least 2^-9
// (relative), so 2^-11, away from every midpoint, since x has 8 significant bits, s 4
// and a midpoint 3; so x * (1 / s), off by 2^-22 (relative), is rounded to a multiple
// of 2^-13 first (by adding and taking away 1.5 * 2^10), which restores the midpoints
// and moves nothing else across one.  amax / 6 against the midpoints of E4M3 likewise
// (5 significant bits), rounded to 12 bits first.  Every lane of the pair takes part.
__device__ __forceinline__ uint32_t kv_quantise(const uint4& v, float inv_g, uint32_t* codes) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t top2 = 0;  // two 16-bit maxima
#pragma unroll
  for (int i = 0; i < 4; ++i) top2 = __vmaxu2(top2, x[i] & 0x7FFF7FFFu);
  top2 = __vmaxu2(top2, __shfl_xor_sync(0xFFFFFFFFu, top2, 1));
  const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
  const uint32_t sixth = __float_as_uint(__uint_as_float(top << 16) * inv_g * (1.f / 6.f));
  // (a NaN must not carry into the sign)
  const uint32_t scale = e4m3_from(__uint_as_float((sixth + (sixth < 0x7F800000u ? 0x800u : 0u)) & 0xFFFFF000u));
  const float s = __low2float(e4m3x2_half2(scale));
  const float r = s > 0.f ? reciprocal(s) * inv_g : 0.f;
  constexpr float kGrid = 1536.f;  // 1.5 * 2^10: sums keep multiples of 2^-13
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = signed_as(fmaf(__uint_as_float(x[i] << 16), r, kGrid) - kGrid, x[i] << 16);
    y[2 * i + 1] = signed_as(fmaf(__uint_as_float(x[i] & 0xFFFF0000u), r, kGrid) - kGrid, x[i]);
  }
  *codes = e2m1x8_from(y);
  return scale;
}

}  // namespace sg
