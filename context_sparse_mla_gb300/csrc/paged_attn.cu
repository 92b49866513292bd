// paged_attn.cu -- attention over the paged 8-bit latent cache (mla_paged_attn).
#include "paged_attn.cuh"

extern "C" size_t mla_paged_attn_workspace_size(int H, int n_tokens) {
  if (H < 1 || H > 128 || n_tokens < 0) return 0;
  return cpmla::pg_layout(n_tokens, 64).total;
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
  PagedArgs a{};
  int R = 0;
  const int rc = paged_attn_args<false>(fn, q, q_token_stride, H, cache, cache_exp, n_blocks, block_size,
                                 block_table, B, table_stride, tokens, pos, req, n_tokens, kv_lo,
                                 kv_hi, softmax_scale, sink, T, o_out, lse_out, workspace,
                                 workspace_bytes, a, &R);
  if (rc != CPMLA_OK || R == 0) return rc;
  // the cache as [slots, 576] bytes in boxes of one block (of at most a tile's rows)
  // x 128 latent or the 64 rope channels, swizzled as the MMA reads them
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(CPMLA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {
    memset(&tm[i], 0, sizeof tm[i]);
    cuuint64_t dims[2] = {CPMLA_DQK, (cuuint64_t)n_blocks * block_size};
    cuuint64_t strides[1] = {CPMLA_DQK};
    cuuint32_t box[2] = {i == 0 ? 128u : 64u,
                         (cuuint32_t)(block_size < kPgTile ? block_size : kPgTile)};
    cuuint32_t estr[2] = {1, 1};
    const CUresult cr =
        enc(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(cache), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            i == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS)
      return fail(CPMLA_ERR_CUDA, "%s: tensor map encode failed (%d)", fn, (int)cr);
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return R == 64 ? launch_paged<64, false>(fn, a, tm, st) : launch_paged<16, false>(fn, a, tm, st);
}
