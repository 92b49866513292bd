// paged4_cache.cu -- tokens into the paged 4-bit latent cache, and listed slots read
// back (mla_paged4_cache_insert, mla_paged4_cache_read).
//
// A token is coded by itself: e = the least exponent in [-64, 119] with |x| <= 448 2^e
// for its finite channels, a latent group's d = the largest in 0 .. 11 with |x| <= 7
// 2^(e + 6 - d) (7 is where E2M1 stops rounding to its largest, 6); scaling by a power
// of two is exact, so each code is the nearest one to the exact quotient.
//
// Bound by HBM: 1152 B in and 337 B out a token, and the other way.  A warp takes a few
// tokens, all their loads in flight first.  Writing, lane g has group g, so that a group's
// maximum needs no exchange and the token's is one reduction (131,072 tokens: 35 us,
// 5.6 TB/s; 37 with the lanes as when reading).  Reading, a lane has 8 channels of group
// lane / 2 and of group 16 + lane / 2, so that a row is stored 512 bytes at a time
// (34 us, 40 with 32 bytes a lane side by side; 65,536 slots in no order 18.6, 5.3 TB/s).
#include "attn_common.cuh"
#include "paged4.cuh"

namespace cpmla {
namespace {

constexpr int kThreads4 = 128;
constexpr int kTokIn = 4, kTokOut = 2;  // tokens of a warp

struct P4Args {
  const __nv_bfloat16 *kv;
  __nv_bfloat16 *out;
  int64_t stride;
  int n;
  const int64_t *slot;
  uint8_t *cache;
  int64_t n_slots;
  int *status;
};

__device__ __forceinline__ int64_t p4_slot(const P4Args &a, int64_t t, int lane) {
  if (t >= a.n) return -1;
  const int64_t s = a.slot[t];
  if (s >= 0 && s < a.n_slots) return s;
  if (s != -1 && lane == 0) record_status(a.status, CPMLA_ERR_INDEX);
  return -1;
}

// Least s with |x| <= 1.75 2^(s + up) for the bf16 magnitude bits m of x.
__device__ __forceinline__ int least_exp(uint32_t m, int up) {
  return (int)(m >> 7) - 127 - up + ((m & 0x7Fu) > 0x60u ? 1 : 0);
}

// Two words of 8 E2M1 codes of 8 bf16 pairs times mul.
__device__ __forceinline__ uint32_t e2m1x8(const uint4 &v, float mul) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16) * mul;
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * mul;
  }
  uint32_t c;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(c)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  // signs of codes 0-3 (bits 3, 7, 11, 15) to bits 7, 15, 23, 31; of 4-7 to 3, 11, 19, 27
  auto spread = [](uint32_t s) {
    s = (s | s << 8) & 0x00880088u;
    return (s | s << 4) & 0x08080808u;
  };
  return (c & 0x77777777u) | spread(c & 0x8888u) << 4 | spread(c >> 16 & 0x8888u);
}

__global__ void __launch_bounds__(kThreads4) paged4_insert_kernel(const P4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * (kThreads4 / 32) + (threadIdx.x >> 5)) * kTokIn;
  uint4 v[kTokIn][2];
  uint32_t rope[kTokIn];
  int64_t s[kTokIn];
#pragma unroll
  for (int u = 0; u < kTokIn; ++u) {
    s[u] = -1;
    v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
    rope[u] = 0;
    if (t0 + u < a.n) {
      const __nv_bfloat16 *src = a.kv + (t0 + u) * a.stride;
      v[u][0] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * lane);
      v[u][1] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * lane + 1);
      rope[u] = __ldg(reinterpret_cast<const uint32_t *>(src + CPMLA_DV) + lane);
      s[u] = p4_slot(a, t0 + u, lane);
    }
  }
#pragma unroll
  for (int u = 0; u < kTokIn; ++u) {
    if (s[u] < 0) continue;
    // bf16 magnitudes order like their bits, infinities and NaN above all finite ones
    const uint32_t w[9] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x,
                           v[u][1].y, v[u][1].z, v[u][1].w, rope[u]};
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
    uint32_t gm = max(m2 & 0xFFFFu, m2 >> 16);
    uint32_t rm = max(w[8] & 0x7FFFu, w[8] >> 16 & 0x7FFFu);
    bool nan = false;
    if (__any_sync(0xffffffffu, max(gm, rm) >= 0x7F80u)) {  // the rare case: finite ones only
      nan = max(gm, rm) > 0x7F80u;
      gm = rm = 0;
#pragma unroll
      for (int i = 0; i < 9; ++i)
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          const uint32_t x = w[i] >> h & 0x7FFFu;
          if (x < 0x7F80u) (i < 8 ? gm : rm) = max(i < 8 ? gm : rm, x);
        }
      nan = __any_sync(0xffffffffu, nan);
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(gm, rm));
    const int e = max(kP4ExpMin, min(least_exp(top, 8), kP4ExpMax));
    const int d = max(0, min(e + 6 - least_exp(gm, 2), kP4OffMax));
    const float mul = __int_as_float((127 - (e + 6 - d)) << 23);
    uint8_t *strip = a.cache + (s[u] >> 4) * kStrip;
    const int r = (int)(s[u] & 15);
    *reinterpret_cast<uint2 *>(strip + 256 * r + 16 * (lane & 15) + 8 * (lane >> 4)) =
        make_uint2(e2m1x8(v[u][0], mul), e2m1x8(v[u][1], mul));
    const float rmul = __int_as_float((127 - e) << 23);
    uint16_t rc;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(rc)
        : "f"(__uint_as_float(w[8] & 0xFFFF0000u) * rmul), "f"(__uint_as_float(w[8] << 16) * rmul));
    reinterpret_cast<uint16_t *>(strip + kStripRope + 64 * r)[lane] = rc;
    const int d2 = __shfl_down_sync(0xffffffffu, d, 16);
    if (lane < 16) strip[kStripOff + 16 * r + lane] = (uint8_t)(d | d2 << 4);
    if (lane == 0) strip[kStripExp + r] = (uint8_t)(nan ? kP4Nan : e + 127);
  }
}

// Four bf16 of the lower four magnitude codes of sel and the signs in the top bits of
// sign's bytes, times mul (both halves): values of at most 6 2^125, two bits long.
__device__ __forceinline__ uint2 bf16x4_of_e2m1(uint32_t sel, uint32_t sign, uint32_t mul) {
  const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | (sign & 0x80808080u);
  const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
  const uint32_t x = __byte_perm(lo, hi, 0x5140), y = __byte_perm(lo, hi, 0x7362);
  uint2 o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.x) : "r"(x), "r"(mul));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o.y) : "r"(y), "r"(mul));
  return o;
}
__device__ __forceinline__ uint4 bf16x8_of_e2m1(uint32_t w, uint32_t mul) {
  const uint32_t sel = w & 0x77777777u;
  const uint2 a = bf16x4_of_e2m1(sel, w, mul), b = bf16x4_of_e2m1(sel >> 16, w << 4, mul);
  return make_uint4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(kThreads4) paged4_read_kernel(const P4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * (kThreads4 / 32) + (threadIdx.x >> 5)) * kTokOut;
  uint4 c[kTokOut];
  uint32_t rope[kTokOut], off[kTokOut], ex[kTokOut];
  int64_t s[kTokOut];
#pragma unroll
  for (int u = 0; u < kTokOut; ++u) s[u] = p4_slot(a, t0 + u, lane);
#pragma unroll
  for (int u = 0; u < kTokOut; ++u) {
    c[u] = make_uint4(0, 0, 0, 0);
    rope[u] = off[u] = 0;
    ex[u] = 127;
    if (s[u] < 0) continue;  // zeros
    const uint8_t *strip = a.cache + (s[u] >> 4) * kStrip;
    const int r = (int)(s[u] & 15);
    c[u] = __ldg(reinterpret_cast<const uint4 *>(strip + 256 * r) + (lane >> 1));
    rope[u] = __ldg(reinterpret_cast<const uint16_t *>(strip + kStripRope + 64 * r) + lane);
    off[u] = __ldg(strip + kStripOff + 16 * r + (lane >> 1));
    ex[u] = __ldg(strip + kStripExp + r);
  }
#pragma unroll
  for (int u = 0; u < kTokOut; ++u) {
    if (t0 + u >= a.n) break;
    const float f = p4_scale((int)ex[u]);
    __nv_bfloat16 *dst = a.out + (t0 + u) * a.stride;
#pragma unroll
    for (int y = 0; y < 2; ++y) {  // groups lane / 2 and 16 + lane / 2
      const int d = min((int)(off[u] >> 4 * y & 15), kP4OffMax);
      // 2^(e + 6 - d), or NaN (whose exponent field the sum must not leave)
      const uint32_t mb = ex[u] == kP4Nan ? 0x7FFFu : (__float_as_uint(f) >> 16) + ((6 - d) << 7);
      const uint32_t w = y == 0 ? (lane & 1 ? c[u].y : c[u].x) : (lane & 1 ? c[u].w : c[u].z);
      reinterpret_cast<uint4 *>(dst)[32 * y + lane] = bf16x8_of_e2m1(w, mb | mb << 16);
    }
    const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)rope[u]);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
    reinterpret_cast<uint32_t *>(dst + CPMLA_DV)[lane] = pack_bf16x2(x.x * f, x.y * f);
  }
}

int p4_check(const char *fn, const void *rows, int64_t stride, int n, const int64_t *slot,
             const void *cache, int n_blocks, int block_size) {
  CPMLA_CHECK_ARG(n >= 0, "%s: n=%d < 0", fn, n);
  CPMLA_CHECK_ARG(stride >= CPMLA_DQK && stride % 8 == 0,
                  "%s: kv_token_stride=%lld must be >= 576 and a multiple of 8", fn,
                  (long long)stride);
  CPMLA_CHECK_ARG(paged_block_size_ok(block_size), "%s: block_size=%d is not 16, 32, 64 or 128",
                  fn, block_size);
  CPMLA_CHECK_ARG(n_blocks >= 1, "%s: n_blocks=%d < 1", fn, n_blocks);
  if (n == 0) return CPMLA_OK;
  CPMLA_CHECK_ARG(rows && slot && cache, "%s: a required pointer is NULL", fn);
  CPMLA_CHECK_ARG(((uintptr_t)rows & 15) == 0 && ((uintptr_t)cache & 15) == 0,
                  "%s: kv and cache must be 16-byte aligned", fn);
  return CPMLA_OK;
}

}  // namespace
}  // namespace cpmla

extern "C" int mla_paged4_cache_insert(const void *kv, int64_t kv_token_stride, int n,
                                       const int64_t *slot_mapping, void *cache, int n_blocks,
                                       int block_size, void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged4_cache_insert";
  const int rc = p4_check(fn, kv, kv_token_stride, n, slot_mapping, cache, n_blocks, block_size);
  if (rc != CPMLA_OK || n == 0) return rc;
  P4Args a{static_cast<const __nv_bfloat16 *>(kv), nullptr, kv_token_stride, n, slot_mapping,
           static_cast<uint8_t *>(cache), (int64_t)n_blocks * block_size, status_word()};
  if (!a.status) return fail(CPMLA_ERR_CUDA, "%s: status word unavailable", fn);
  const int per = kThreads4 / 32 * kTokIn;
  paged4_insert_kernel<<<(unsigned)(((int64_t)n + per - 1) / per), kThreads4, 0,
                         static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged4_cache_insert: launch");
  return CPMLA_OK;
}

extern "C" int mla_paged4_cache_read(const void *cache, int n_blocks, int block_size,
                                     const int64_t *slot_mapping, int n, void *kv,
                                     int64_t kv_token_stride, void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged4_cache_read";
  const int rc = p4_check(fn, kv, kv_token_stride, n, slot_mapping, cache, n_blocks, block_size);
  if (rc != CPMLA_OK || n == 0) return rc;
  P4Args a{nullptr, static_cast<__nv_bfloat16 *>(kv), kv_token_stride, n, slot_mapping,
           const_cast<uint8_t *>(static_cast<const uint8_t *>(cache)),
           (int64_t)n_blocks * block_size, status_word()};
  if (!a.status) return fail(CPMLA_ERR_CUDA, "%s: status word unavailable", fn);
  const int per = kThreads4 / 32 * kTokOut;
  paged4_read_kernel<<<(unsigned)(((int64_t)n + per - 1) / per), kThreads4, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged4_cache_read: launch");
  return CPMLA_OK;
}
