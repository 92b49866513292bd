// paged4_attn.cu -- attention of listed tokens over the paged 4-bit latent cache
// (mla_paged4_attn).
//
// A warp takes an entry and a head and goes over the row's keys one by one with the
// running maximum and sum of a softmax: lane g has group g of the latent (16 channels)
// and two rope channels; scores and sums are binary32.
#include <cmath>

#include "attn_common.cuh"
#include "paged4.cuh"

namespace cpmla {
namespace {

struct P4AttnArgs {
  const __nv_bfloat16 *q;
  int64_t q_stride;
  int H;
  const uint8_t *cache;
  int n_blocks, shift, B, T;
  const int32_t *table;
  int64_t stride;
  const int32_t *tokens, *pos, *req;
  int n;
  const int32_t *kv_lo, *kv_hi;
  float scale_log2;
  const float *sink;
  __nv_bfloat16 *o;
  float *lse;
  int *status;
};

__device__ __forceinline__ float p4_e2m1(uint32_t w, int j) {
  const uint32_t m = w >> (4 * j) & 7, neg = w >> (j < 4 ? 8 * j + 7 : 8 * (j - 4) + 3) & 1;
  const float v = m < 4 ? 0.5f * m : (m < 6 ? m - 2.f : 2.f * m - 8.f);
  return neg ? -v : v;
}

__global__ void __launch_bounds__(128) paged4_attn_simple(const P4AttnArgs a) {
  const int lane = threadIdx.x & 31, i = blockIdx.x;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int b = a.req[i], p = a.pos[i], t = a.tokens ? a.tokens[i] : i;
  if (b == -1 || h >= a.H) return;
  if (b < 0 || b >= a.B || t < 0 || t >= a.T || p < 0 || p >= (1 << 30) ||
      (p >> a.shift) >= a.stride) {
    if (lane == 0) record_status(a.status, CPMLA_ERR_INDEX);
    return;
  }
  const __nv_bfloat16 *qr = a.q + t * a.q_stride + (int64_t)h * CPMLA_DQK;
  float q[18], o[16];
  for (int c = 0; c < 16; ++c) q[c] = __bfloat162float(qr[16 * lane + c]) * a.scale_log2;
  for (int c = 0; c < 2; ++c) q[16 + c] = __bfloat162float(qr[CPMLA_DV + 2 * lane + c]) * a.scale_log2;
  for (int c = 0; c < 16; ++c) o[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int lo = a.kv_lo ? max(a.kv_lo[i], 0) : 0, hi = a.kv_hi ? min(a.kv_hi[i], p) : p;
  for (int x = lo; x <= hi; ++x) {
    const int blk = a.table[b * a.stride + (x >> a.shift)];
    if (blk < 0 || blk >= a.n_blocks) {
      if (lane == 0) record_status(a.status, CPMLA_ERR_INDEX);
      continue;
    }
    const int64_t slot = ((int64_t)blk << a.shift) + (x & ((1 << a.shift) - 1));
    const uint8_t *strip = a.cache + (slot >> 4) * kStrip;
    const int r = (int)(slot & 15);
    const uint2 w = *reinterpret_cast<const uint2 *>(strip + 256 * r + 16 * (lane & 15) + 8 * (lane >> 4));
    const int d = min(strip[kStripOff + 16 * r + (lane & 15)] >> (lane >> 4) * 4 & 15, kP4OffMax);
    const float f = p4_scale(strip[kStripExp + r]);
    float s = 0.f, v[16];
    for (int c = 0; c < 16; ++c) {
      v[c] = p4_e2m1(c < 8 ? w.x : w.y, c & 7) * exp2f(6.f - d);
      s = fmaf(q[c], v[c], s);
    }
    const uint32_t h2 =
        e4m3x2_to_f16x2(reinterpret_cast<const uint16_t *>(strip + kStripRope + 64 * r)[lane]);
    const float2 rp = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
    s = fmaf(q[16], rp.x, fmaf(q[17], rp.y, s));
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= f;
    const float mn = fmaxf(m, s), c0 = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float e = s != s ? s : exp2f(s - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l = fmaf(l, c0, e);
    for (int c = 0; c < 16; ++c) o[c] = fmaf(o[c], c0, e * f * v[c]);
  }
  const bool empty = m == -INFINITY && l == 0.f;
  const float L = empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  const float g = empty ? 0.f : sink_factor(a.sink, h, L) / l;
  const int64_t row = (int64_t)t * a.H + h;
  if (lane == 0) a.lse[row] = L;
  for (int c = 0; c < 16; ++c) a.o[row * CPMLA_DV + 16 * lane + c] = __float2bfloat16_rn(o[c] * g);
}

}  // namespace
}  // namespace cpmla

extern "C" int mla_paged4_attn(const void *q, int64_t q_token_stride, int H, const void *cache,
                               int n_blocks, int block_size, const int32_t *block_table, int B,
                               int64_t table_stride, const int32_t *tokens, const int32_t *pos,
                               const int32_t *req, int n_tokens, const int32_t *kv_lo,
                               const int32_t *kv_hi, float softmax_scale, const float *sink, int T,
                               void *o_out, float *lse_out, void *workspace,
                               size_t workspace_bytes, void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged4_attn";
  CPMLA_CHECK_ARG(n_tokens >= 0, "%s: n_tokens=%d < 0", fn, n_tokens);
  CPMLA_CHECK_ARG(H >= 1 && H <= 128, "%s: H=%d outside 1..128", fn, H);
  if (H > 64 && H % 64 != 0)
    return fail(CPMLA_ERR_UNSUPPORTED, "%s: H=%d above 64 must be a multiple of 64", fn, H);
  CPMLA_CHECK_ARG(q_token_stride >= (int64_t)H * CPMLA_DQK && q_token_stride % 8 == 0,
                  "%s: q_token_stride=%lld must be >= H*576 and a multiple of 8", fn,
                  (long long)q_token_stride);
  CPMLA_CHECK_ARG(paged_block_size_ok(block_size), "%s: block_size=%d is not 16, 32, 64 or 128",
                  fn, block_size);
  CPMLA_CHECK_ARG(n_blocks >= 1 && (int64_t)n_blocks * block_size <= INT32_MAX,
                  "%s: n_blocks=%d: at least 1, and fewer than 2^31 slots", fn, n_blocks);
  CPMLA_CHECK_ARG(B >= 1 && table_stride >= 1, "%s: B=%d, table_stride=%lld", fn, B,
                  (long long)table_stride);
  CPMLA_CHECK_ARG(std::isfinite(softmax_scale) && softmax_scale > 0.f,
                  "%s: softmax_scale must be finite and > 0", fn);
  CPMLA_CHECK_ARG(T >= 1 || n_tokens == 0, "%s: T=%d", fn, T);
  if (n_tokens == 0) return CPMLA_OK;
  CPMLA_CHECK_ARG(q && cache && block_table && pos && req && o_out && lse_out,
                  "%s: a required pointer is NULL", fn);
  CPMLA_CHECK_ARG(((uintptr_t)q & 15) == 0 && ((uintptr_t)cache & 15) == 0 &&
                      ((uintptr_t)o_out & 15) == 0,
                  "%s: q, cache and o_out must be 16-byte aligned", fn);
  CPMLA_CHECK_ARG(workspace != nullptr && ((uintptr_t)workspace & 255) == 0,
                  "%s: workspace must be non-NULL and 256-byte aligned", fn);
  CPMLA_CHECK_ARG(workspace_bytes >= mla_paged_attn_workspace_size(H, n_tokens),
                  "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes,
                  mla_paged_attn_workspace_size(H, n_tokens));
  int *status = status_word();
  if (!status) return fail(CPMLA_ERR_CUDA, "%s: status word unavailable", fn);
  P4AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_token_stride;
  a.H = H;
  a.cache = static_cast<const uint8_t *>(cache);
  a.n_blocks = n_blocks;
  a.shift = paged_block_shift(block_size);
  a.B = B;
  a.T = T;
  a.table = block_table;
  a.stride = table_stride;
  a.tokens = tokens;
  a.pos = pos;
  a.req = req;
  a.n = n_tokens;
  a.kv_lo = kv_lo;
  a.kv_hi = kv_hi;
  a.scale_log2 = softmax_scale * 1.44269504088896340736f;
  a.sink = sink;
  a.o = static_cast<__nv_bfloat16 *>(o_out);
  a.lse = lse_out;
  a.status = status;
  paged4_attn_simple<<<dim3(n_tokens, (H + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged4_attn: launch");
  return CPMLA_OK;
}
