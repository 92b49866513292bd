// paged4_attn.cu -- attention over the paged 4-bit latent cache (mla_paged4_attn).
#include "paged_attn.cuh"

extern "C" int mla_paged4_attn(const void *q, int64_t q_token_stride, int H, const void *cache,
                               int n_blocks, int block_size, const int32_t *block_table, int B,
                               int64_t table_stride, const int32_t *tokens, const int32_t *pos,
                               const int32_t *req, int n_tokens, const int32_t *kv_lo,
                               const int32_t *kv_hi, float softmax_scale, const float *sink, int T,
                               void *o_out, float *lse_out, void *workspace,
                               size_t workspace_bytes, void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged4_attn";
  PagedArgs a{};
  int R = 0;
  const int rc = paged_attn_args<true>(fn, q, q_token_stride, H, cache, nullptr, n_blocks, block_size,
                                 block_table, B, table_stride, tokens, pos, req, n_tokens, kv_lo,
                                 kv_hi, softmax_scale, sink, T, o_out, lse_out, workspace,
                                 workspace_bytes, a, &R);
  if (rc != CPMLA_OK || R == 0) return rc;
  // (no tensor maps: strips are copied as they lie)
  CUtensorMap tm[2];
  memset(tm, 0, sizeof tm);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return R == 64 ? launch_paged<64, true>(fn, a, tm, st) : launch_paged<16, true>(fn, a, tm, st);
}
