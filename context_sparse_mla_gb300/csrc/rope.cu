// rope.cu -- rotary positions of the 64 rope channels of queries and keys (mla_rope),
// and their frequencies (mla_rope_freqs).
//
// The angle pos * f has to be known modulo a turn, and pos is large: in units of 2^-64
// of a turn, with f as a whole number F of them, pos * F modulo 2^64 is exact, so one
// 64-bit product replaces a reduction in binary64 (of which a GB300 does few).  F is
// off by less than 5/4 units (f below 2^-9 has bits behind the last, which are cut):
// 2^-32 of a turn at the largest position.  The half turns that are left, in [-1, 1), are
// rounded to binary32: by 2^-26 of a turn, 1e-7, at most.
//
// A row is 128 B in a longer one.  8 lanes take a row, 4 rows a step of a warp; lane
// 8 i + c computes pair 4 c + i, and the lanes of a column c share theirs: each needs
// pairs 4 c .. 4 c + 3, of channels 8 c .. (pairs) or 4 c .. and 32 + 4 c .. (halves).
#include <cmath>

#include "attn_common.cuh"

namespace cpmla {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 20;  // of a warp: 16 heads and the key, 17, are one warp's
constexpr int kRopePairs = CPMLA_DROPE / 2;

struct RopeArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *qo, *ko;
  int64_t qt, qh, qot, qoh, kt, kot;
  int H, rows;  // heads of q; rows of a token (the heads, then the key)
  int n, parts, per;  // tokens; a token's parts, of so many rows, a warp's work each
  const int32_t *pos;
  float amp;
  int halves, inverse;
  uint64_t turns[kRopePairs];
};

struct RopeRow {
  uint2 a, b;  // first and second half, or channels 8 c .. + 3 and + 4 .. + 7
};

// A warp's work is per <= kRopeRows rows of a token, all loaded before the angle is known
// (and the next position beside them): bound by HBM, with the rows' 128 bytes apart
// (32,771 tokens of 16 heads and the key: 28 us, 5.1 TB/s; 43 with the angle first and the
// 17th row behind the others).  Eight blocks an SM and a loop: 28 us, 31 without the loop.
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kU = kRopeRows / 4;
  const int lane = threadIdx.x & 31, c = lane & 7, g = lane >> 3;
  const int64_t n_work = (int64_t)a.n * a.parts;
  const int64_t n_warps = (int64_t)gridDim.x * (kRopeThreads / 32);
  const uint64_t turn = a.turns[4 * c + g];
  const int x0 = a.halves ? 4 * c : 8 * c, x1 = a.halves ? x0 + 32 : x0 + 4;
  int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  int p = w < n_work ? a.pos[w / a.parts] : -1;
  while (w < n_work) {
    const int64_t t = w / a.parts, nxt = w + n_warps;
    const int r0 = (int)(w - t * a.parts) * a.per, r1 = min(r0 + a.per, a.rows);
    RopeRow v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + g + 4 * u;
      if (r >= r1) break;
      const __nv_bfloat16 *src = r < a.H ? a.q + t * a.qt + r * a.qh : a.k + t * a.kt;
      v[u].a = *reinterpret_cast<const uint2 *>(src + x0);
      v[u].b = *reinterpret_cast<const uint2 *>(src + x1);
    }
    const int p_nxt = nxt < n_work ? a.pos[nxt / a.parts] : -1;
    float s, co;
    sincospif((float)(int64_t)((uint64_t)p * turn) * 0x1p-63f, &s, &co);
    co *= a.amp;
    s *= a.inverse ? -a.amp : a.amp;
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, co, 8 * i + c);
      sn[i] = __shfl_sync(0xffffffffu, s, 8 * i + c);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + g + 4 * u;
      if (r >= r1 || p < 0) break;
      // the four pairs' first and second channels
      float x[4], y[4];
      const uint32_t wd[4] = {v[u].a.x, v[u].a.y, v[u].b.x, v[u].b.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(wd[i] << 16), hi = __uint_as_float(wd[i] & 0xFFFF0000u);
        if (a.halves) {
          (i < 2 ? x : y)[2 * i & 3] = lo;
          (i < 2 ? x : y)[(2 * i & 3) + 1] = hi;
        } else {
          x[i] = lo;
          y[i] = hi;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float nx = fmaf(x[i], cs[i], -(y[i] * sn[i]));
        y[i] = fmaf(x[i], sn[i], y[i] * cs[i]);
        x[i] = nx;
      }
      RopeRow o;
      if (a.halves) {
        o.a = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        o.b = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      } else {
        o.a = make_uint2(pack_bf16x2(x[0], y[0]), pack_bf16x2(x[1], y[1]));
        o.b = make_uint2(pack_bf16x2(x[2], y[2]), pack_bf16x2(x[3], y[3]));
      }
      __nv_bfloat16 *dst = r < a.H ? a.qo + t * a.qot + r * a.qoh : a.ko + t * a.kot;
      *reinterpret_cast<uint2 *>(dst + x0) = o.a;
      *reinterpret_cast<uint2 *>(dst + x1) = o.b;
    }
    w = nxt;
    p = p_nxt;
  }
}

// f / 2 pi in units of 2^-64 of a turn, modulo 2^64, for 0 <= f <= 6: 1 / 2 pi as the
// sum of two binary64, the product's rounding error by a fused multiply-add.
uint64_t turns_of(double f) {
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double t = f * hi, r = std::fma(f, hi, -t) + f * lo;
  return (uint64_t)std::ldexp(t, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(r, 64));
}

}  // namespace
}  // namespace cpmla

extern "C" int mla_rope_freqs(double base, double factor, int original_len, double beta_fast,
                              double beta_slow, double *inv_freq) {
  using namespace cpmla;
  const char *fn = "mla_rope_freqs";
  CPMLA_CHECK_ARG(std::isfinite(base) && base > 1, "%s: base=%g must be > 1", fn, base);
  CPMLA_CHECK_ARG(std::isfinite(factor) && factor >= 1, "%s: factor=%g must be >= 1", fn, factor);
  CPMLA_CHECK_ARG(factor == 1 || original_len >= 1, "%s: original_len=%d < 1", fn, original_len);
  CPMLA_CHECK_ARG(factor == 1 || (std::isfinite(beta_fast) && beta_slow > 0 && beta_fast > beta_slow),
                  "%s: beta_fast=%g, beta_slow=%g: 0 < slow < fast", fn, beta_fast, beta_slow);
  CPMLA_CHECK_ARG(inv_freq, "%s: inv_freq is NULL", fn);
  double low = 0, high = 0;
  if (factor != 1) {
    // the (fractional) pair whose wave makes this many turns over the trained length
    auto at = [&](double turns) {
      return CPMLA_DROPE * std::log(original_len / (turns * 6.283185307179586477)) /
             (2 * std::log(base));
    };
    low = std::fmax(0.0, std::floor(at(beta_fast)));
    high = std::fmin(CPMLA_DROPE - 1.0, std::ceil(at(beta_slow)));
  }
  for (int i = 0; i < kRopePairs; ++i) {
    const double f = std::pow(base, -2.0 * i / CPMLA_DROPE);
    const double ramp =
        factor == 1 ? 0
                    : std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 0.001)));
    inv_freq[i] = f * (1 - ramp) + f / factor * ramp;
  }
  return CPMLA_OK;
}

extern "C" int mla_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride, int H,
                        void *q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                        const void *k, int64_t k_token_stride, void *k_out,
                        int64_t ko_token_stride, int n, const int32_t *pos,
                        const double *inv_freq, float amplitude, int layout, int inverse,
                        void *stream) {
  using namespace cpmla;
  const char *fn = "mla_rope";
  CPMLA_CHECK_ARG(n >= 0, "%s: n=%d < 0", fn, n);
  CPMLA_CHECK_ARG(H >= 0 && H <= 1024, "%s: H=%d outside 0..1024", fn, H);
  CPMLA_CHECK_ARG(layout == CPMLA_ROPE_PAIRS || layout == CPMLA_ROPE_HALVES,
                  "%s: unknown layout %d", fn, layout);
  CPMLA_CHECK_ARG(std::isfinite(amplitude), "%s: amplitude must be finite", fn);
  CPMLA_CHECK_ARG(inv_freq, "%s: inv_freq is NULL", fn);
  for (int i = 0; i < kRopePairs; ++i)
    CPMLA_CHECK_ARG(inv_freq[i] >= 0 && inv_freq[i] <= 6, "%s: inv_freq[%d]=%g outside 0..6", fn, i,
                    inv_freq[i]);
  CPMLA_CHECK_ARG((((uintptr_t)q | (uintptr_t)q_out | (uintptr_t)k | (uintptr_t)k_out) & 7) == 0,
                  "%s: q, k and their outputs must be 8-byte aligned", fn);
  // (strides of a dimension of one entry are not used)
  const struct {
    int64_t stride;
    bool used, out;
  } st[6] = {{q_token_stride, H > 0 && n > 1, false}, {q_head_stride, H > 1, false},
             {qo_token_stride, H > 0 && n > 1, true}, {qo_head_stride, H > 1, true},
             {k_token_stride, k && n > 1, false},     {ko_token_stride, k && n > 1, true}};
  for (const auto &x : st)
    CPMLA_CHECK_ARG(!x.used || (x.stride % 4 == 0 && x.stride >= (x.out ? CPMLA_DROPE : 0)),
                    "%s: stride %lld: multiples of 4 elements, those of outputs >= 64", fn,
                    (long long)x.stride);
  if (n == 0) return CPMLA_OK;
  CPMLA_CHECK_ARG(H == 0 || (q && q_out), "%s: q and q_out are required with heads", fn);
  CPMLA_CHECK_ARG((k == nullptr) == (k_out == nullptr), "%s: k and k_out go together", fn);
  CPMLA_CHECK_ARG(H > 0 || k, "%s: neither q nor k", fn);
  CPMLA_CHECK_ARG(pos, "%s: pos is NULL", fn);
  RopeArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.qo = static_cast<__nv_bfloat16 *>(q_out);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.ko = static_cast<__nv_bfloat16 *>(k_out);
  a.qt = q_token_stride;
  a.qh = q_head_stride;
  a.qot = qo_token_stride;
  a.qoh = qo_head_stride;
  a.kt = k_token_stride;
  a.kot = ko_token_stride;
  a.H = H;
  a.rows = H + (k ? 1 : 0);
  a.n = n;
  a.pos = pos;
  a.amp = amplitude;
  a.halves = layout == CPMLA_ROPE_HALVES;
  a.inverse = inverse != 0;
  for (int i = 0; i < kRopePairs; ++i) a.turns[i] = turns_of(inv_freq[i]);
  a.parts = (a.rows + kRopeRows - 1) / kRopeRows;
  a.per = (a.rows + a.parts - 1) / a.parts;
  const int64_t warps = (int64_t)n * a.parts;
  const int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  rope_kernel<<<(unsigned)(grid < 152 * 8 ? grid : 152 * 8), kRopeThreads, 0,
                static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_rope: launch");
  return CPMLA_OK;
}
