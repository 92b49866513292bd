// paged4.cuh -- the strips of the 4-bit latent cache: 16 tokens in kStrip bytes.
//
// With stored exponent e (a byte, e + 127) and group offsets d, a token's latent
// channel c of group g = c / 16 is E2M1(code) * 2^(e + 6 - d[g]) and its rope channel
// E4M3(code) * 2^e.  In a strip (r = token % 16):
//   [0, 4096)     row r at 256 r: group g at 16 (g % 16) + 8 (g / 16), two little-
//                 endian words of 8 channels.  Channel j of a word: magnitude code at
//                 bits 4j .. 4j + 2, sign at bit 8j + 7 (j < 4) or 8(j - 4) + 3 (j >= 4)
//   [4096, 5120)  rope codes, row r at 64 r
//   [5120, 5376)  offsets, row r at 16 r: byte u = d[u] | d[u + 16] << 4
//   [5376, 5392)  exponents
// A nibble's lower three bits look its magnitude up (a byte permutation takes four at
// once), and the signs of channels 0-3 and, four bits up, 4-7 of a word then lie where
// four looked-up bytes have theirs: 7 operations for 8 channels.  Groups g and g + 16
// lie side by side so that the 16-byte loads of eight threads of a row fill 16-byte
// units of one 128-channel chunk.
#pragma once

#include "cpmla_internal.cuh"

namespace cpmla {

constexpr int kStrip = CPMLA_PAGED4_STRIP_BYTES;
constexpr int kStripRope = 4096, kStripOff = 5120, kStripExp = 5376;
constexpr int kP4ExpMin = -64, kP4ExpMax = 119, kP4OffMax = 11;
constexpr int kP4Nan = 255;  // stored exponent of a token that holds a NaN

#ifdef __CUDACC__

// The stored exponent as it is read: 63 .. 246, or NaN.
__device__ __forceinline__ float p4_scale(int stored) {
  const int s = max(kP4ExpMin + 127, min(stored, kP4ExpMax + 127));
  return __int_as_float(stored == kP4Nan ? 0x7FFFFFFF : s << 23);
}

// 16 channels of a group (two words of codes) as E4M3, for a token on the scale 2^e:
// E2M1 * 2^(6 - d).  Magnitude 1/2 at offset d is the E4M3 code 8 (12 - d), and all
// others lie above it by what they do at every d <= 11, so a group has one table.
__device__ __forceinline__ uint4 p4_e4m3x16(uint32_t w0, uint32_t w1, uint32_t d) {
  const uint32_t m = 8u * (12u - min(d, (uint32_t)kP4OffMax));
  const uint32_t lo = 0x0C080000u + m * 0x01010100u, hi = 0x1C181410u + m * 0x01010101u;
  const uint32_t s0 = w0 & 0x77777777u, s1 = w1 & 0x77777777u;
  return make_uint4(__byte_perm(lo, hi, s0) | (w0 & 0x80808080u),
                    __byte_perm(lo, hi, s0 >> 16) | (w0 << 4 & 0x80808080u),
                    __byte_perm(lo, hi, s1) | (w1 & 0x80808080u),
                    __byte_perm(lo, hi, s1 >> 16) | (w1 << 4 & 0x80808080u));
}

#endif  // __CUDACC__

}  // namespace cpmla
