// kv4.cuh — the 4-bit paged KV cache's layout and number formats.
//
// A row is the 128 channels of one token's K or V in one KV head: 8 blocks of
// 16 channels.  A block holds one scale byte and sixteen 4-bit codes.
//   code   sign bit, then e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6
//   scale  unsigned, 5 exponent and 3 mantissa bits: byte b stands for the
//          fp16 number with bits b << 7, so it decodes with one shift.
//          Bytes 0 .. 0xE2 (10240) are scales; 0xFF (a NaN) marks a block
//          that held a NaN or an infinity.
// code * scale has at most 6 significant bits and is below 65504: exact in
// fp16 and in bf16, and the decode kernel multiplies in fp16 without rounding.
//
// A tile is 16 tokens of one KV head (2304 bytes), the rows of one
// m16n8k16 matrix instruction, laid out so that lane (g, q) = (lane / 4,
// lane % 4) of a warp finds what its fragments need in 16-byte pieces at
// lane * 16 and its scales in one word at lane * 4:
//   [0, 1024)     K codes: token t at t * 64, channel c in byte c / 2
//                 (even channels in the low nibble)
//   [1024, 2048)  V codes: 512 * (t / 8) + 64 * (c / 16) + 16 * ((t % 8) / 2)
//                 + 8 * (t % 2) + (c % 16) / 2
//   [2048, 2176)  K scales: 16 * (t % 8) + 4 * (b / 2) + 2 * (t / 8) + b % 2
//   [2176, 2304)  V scales: 16 * b + 4 * ((t % 8) / 2) + 2 * (t / 8) + t % 2
// Every byte belongs to one token, so tokens are appended independently.
// A page of one head is page_size / 16 tiles in a row, a page its KV heads in
// a row, so a run of tokens of one head is one contiguous piece.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace da {

constexpr int kKv4Row = 128;
constexpr int kKv4Tile = 16;
constexpr int kKv4TileBytes = 2304;
constexpr int kKv4VCodes = 1024;
constexpr int kKv4KScales = 2048;
constexpr int kKv4VScales = 2176;
constexpr int kKv4MaxScale = 0xE2;
constexpr int kKv4BadScale = 0xFF;

// Page sizes are powers of two of at least one tile.
inline bool kv4_page_size_ok(int ps) {
  return ps >= kKv4Tile && ps <= 1024 && (ps & (ps - 1)) == 0;
}
inline int kv4_shift(int ps) {
  int s = 0;
  while ((1 << s) < ps) ++s;
  return s;
}

// Two e2m1 codes (low nibble first) of each byte of w as fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c,
                                                uint32_t& d) {
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "mov.b32 {x0, x1, x2, x3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, x1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, x3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}

// Eight floats to a word of codes, the first in the low four bits (round to
// nearest even, saturating at 6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x3, %8, %7;\n\t"
      "mov.b32 %0, {x0, x1, x2, x3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Scale byte to the value it stands for.
__device__ __forceinline__ float kv4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

}  // namespace da
