// paged_attn.cu -- attention of listed tokens over the paged 8-bit latent
// cache (mla_paged_attn).
//
// One CTA per (entry, head): for 128 keys at a time thread i scores key i,
// then owns value channels 4 i .. 4 i + 3; the running maximum and sum of the
// softmax are carried over the tiles.  Everything in binary32.
#include <cmath>

#include "attn_common.cuh"

namespace cpmla {
namespace {

struct PagedArgs {
  const __nv_bfloat16 *q;
  int64_t q_stride;
  int H;
  const uint8_t *cache;
  const uint8_t *exp;
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

__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedArgs a) {
  __shared__ float sq[CPMLA_DQK];
  __shared__ float sp[128];
  __shared__ int64_t srow[128];
  __shared__ float red[4];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int i = blockIdx.x, h = blockIdx.y;
  const int b = a.req[i];
  if (b == -1) return;
  const int g = a.tokens ? a.tokens[i] : i;
  const int64_t p = a.pos[i];
  if (b < -1 || b >= a.B || g < 0 || g >= a.T || p < 0 || (p >> a.shift) >= a.stride) {
    if (t == 0) record_status(a.status, CPMLA_ERR_INDEX);
    return;
  }
  int64_t lo = a.kv_lo && a.kv_lo[i] > 0 ? a.kv_lo[i] : 0;
  int64_t hi = a.kv_hi && a.kv_hi[i] < p ? a.kv_hi[i] : p;
  for (int d = t; d < CPMLA_DQK; d += 128)
    sq[d] = __bfloat162float(a.q[(int64_t)g * a.q_stride + (int64_t)h * CPMLA_DQK + d]);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = lo; k0 <= hi; k0 += 128) {
    __syncthreads();
    float s = -INFINITY;
    srow[t] = -1;
    if (k0 + t <= hi) {
      const int blk = a.table[(int64_t)b * a.stride + ((k0 + t) >> a.shift)];
      if (blk < 0 || blk >= a.n_blocks) {
        record_status(a.status, CPMLA_ERR_INDEX);
      } else {
        const int64_t row = ((int64_t)blk << a.shift) + ((k0 + t) & ((1 << a.shift) - 1));
        srow[t] = row;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.cache + row * CPMLA_DQK);
        float acc = 0.f;
        for (int c = 0; c < CPMLA_DQK / 16; ++c) {
          const uint4 w = __ldg(src + c);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(u[x >> 1] >> (16 * (x & 1))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            acc += f.x * sq[16 * c + 2 * x] + f.y * sq[16 * c + 2 * x + 1];
          }
        }
        s = ldexpf(acc, (int)a.exp[blk] - 127) * a.scale_log2;
      }
    }
    float tm = s;
#pragma unroll
    for (int off = 16; off; off >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, off));
    if (lane == 0) red[warp] = tm;
    __syncthreads();
    tm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, tm), mr = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(m - mr);
    const float e = srow[t] >= 0 ? exp2f(s - mr) : 0.f;
    const float f = srow[t] >= 0 ? ldexpf(e, (int)a.exp[srow[t] >> a.shift] - 127) : 0.f;
    sp[t] = f;
    float sum = e;
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    l = l * al + (red[0] + red[1]) + (red[2] + red[3]);
    m = mn;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= al;
    for (int j = 0; j < 128; ++j) {
      if (srow[j] < 0) continue;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(a.cache + srow[j] * CPMLA_DQK) + t);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(w >> (16 * x)));
        const float2 f2 = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        o[2 * x] += sp[j] * f2.x;
        o[2 * x + 1] += sp[j] * f2.y;
      }
    }
  }
  const bool empty = m == -INFINITY;
  const float L = empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  const float f = empty ? 0.f : sink_factor(a.sink, h, L) / l;
  uint2 w = make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
  reinterpret_cast<uint2 *>(a.o + ((int64_t)g * a.H + h) * CPMLA_DV)[t] = w;
  if (t == 0) a.lse[(int64_t)g * a.H + h] = L;
}

}  // namespace
}  // namespace cpmla

extern "C" size_t mla_paged_attn_workspace_size(int H, int n_tokens) {
  if (H < 1 || H > 128 || n_tokens < 0) return 0;
  return 256;
}

extern "C" int mla_paged_attn(const void *q, int64_t q_token_stride, int H, const void *cache,
                              const uint8_t *cache_exp, int n_blocks, int block_size,
                              const int32_t *block_table, int B, int64_t table_stride,
                              const int32_t *tokens, const int32_t *pos, const int32_t *req,
                              int n_tokens, const int32_t *kv_lo, const int32_t *kv_hi,
                              float softmax_scale, const float *sink, int T, void *o_out,
                              float *lse_out, void *workspace, size_t workspace_bytes,
                              void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged_attn";
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
  CPMLA_CHECK_ARG(q && cache && cache_exp && block_table && pos && req && o_out && lse_out,
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
  PagedArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_token_stride;
  a.H = H;
  a.cache = static_cast<const uint8_t *>(cache);
  a.exp = cache_exp;
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
  paged_attn_kernel<<<dim3(n_tokens, H), 128, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_attn: launch");
  return CPMLA_OK;
}
