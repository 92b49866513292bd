// paged_maps.cu -- a serving step's block tables and slot maps, built on the
// GPU from the request lengths (mla_paged_maps).
//
// With h_b = ceil(ctx_b / bs) blocks held and t_b = ceil((ctx_b + new_b) / bs)
// - h_b taken, two exclusive prefix sums over the requests give each request's
// first token entry and its first place in the free list; everything else is
// local to a token: its request is found by bisection in the token sums, its
// block comes from the table (index < h_b) or straight from the free list, so
// no token waits for a table write, and the token that opens a taken block
// writes that block's table entry.  A block counts as taken also where the token
// that opens it has no entry (more tokens than n_slots): the last CTA writes the
// table entries of those.
//
// Bound by latency: the arrays of a decode step are kilobytes.  So one launch,
// and every CTA computes the sums over the requests itself (1024 lengths per
// round, read from L2) instead of waiting for another CTA.
#include "cpmla_internal.cuh"

namespace cpmla {
namespace {

constexpr int kMapsThreads = 1024;
constexpr int kMapsTokens = 2048;  // token entries per CTA

struct MapsArgs {
  const int32_t *ctx, *nw, *free_blocks, *head;
  int32_t *table, *cu, *pos, *req, *head_out;
  int64_t *slot;
  int64_t stride;
  int B, shift, n_blocks, n_free, n_slots;
  int *status;
};

__global__ void __launch_bounds__(kMapsThreads) paged_maps_kernel(const MapsArgs a) {
  // sums before each of a round's requests: tokens and taken blocks
  __shared__ int64_t s_tok[kMapsThreads + 1], s_blk[kMapsThreads + 1];
  __shared__ int s_ctx[kMapsThreads];
  __shared__ int64_t s_wt[32], s_wb[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << a.shift;
  const int64_t i0 = (int64_t)blockIdx.x * kMapsTokens;
  const int64_t i1 = i0 + kMapsTokens < a.n_slots ? i0 + kMapsTokens : a.n_slots;
  int64_t tok0 = 0, blk0 = a.head ? a.head[0] : 0;
  bool bad = blk0 < 0;
  for (int r0 = 0; r0 < a.B; r0 += kMapsThreads) {
    const int b = r0 + tid;
    int64_t n = 0, take = 0;
    int c = 0;
    if (b < a.B) {
      c = a.ctx[b];
      n = a.nw[b];
      if (c < 0 || n < 0) bad = true;
      c = c < 0 ? 0 : c;
      n = n < 0 ? 0 : n;
      take = ((c + n + bs - 1) >> a.shift) - (((int64_t)c + bs - 1) >> a.shift);
    }
    const int64_t st = warp_scan_add(n, lane), sb = warp_scan_add(take, lane);
    if (lane == 31) {
      s_wt[warp] = st;
      s_wb[warp] = sb;
    }
    s_ctx[tid] = c;
    __syncthreads();
    if (warp == 0) {
      s_wt[lane] = warp_scan_add(s_wt[lane], lane);
      s_wb[lane] = warp_scan_add(s_wb[lane], lane);
    }
    __syncthreads();
    const int64_t end_t = tok0 + (warp ? s_wt[warp - 1] : 0) + st;
    const int64_t end_b = blk0 + (warp ? s_wb[warp - 1] : 0) + sb;
    s_tok[tid + 1] = end_t;
    s_blk[tid + 1] = end_b;
    if (tid == 0) {
      s_tok[0] = tok0;
      s_blk[0] = blk0;
    }
    if (blockIdx.x == 0 && b < a.B) {
      a.cu[b + 1] = (int32_t)(end_t < INT32_MAX ? end_t : INT32_MAX);
      if (b == 0) a.cu[0] = 0;
    }
    __syncthreads();
    tok0 = s_tok[kMapsThreads];
    blk0 = s_blk[kMapsThreads];
    // this CTA's entries that belong to these requests
    const int64_t lo = s_tok[0] > i0 ? s_tok[0] : i0, hi = tok0 < i1 ? tok0 : i1;
    for (int64_t i = lo + tid; i < hi; i += kMapsThreads) {
      int x = 0, y = kMapsThreads;  // s_tok[x] <= i < s_tok[y]
      while (y - x > 1) {
        const int m = (x + y) >> 1;
        if (s_tok[m] <= i)
          x = m;
        else
          y = m;
      }
      const int64_t p = s_ctx[x] + (i - s_tok[x]);
      const int64_t bi = p >> a.shift;
      const int64_t held = ((int64_t)s_ctx[x] + bs - 1) >> a.shift;
      int blk = -1;
      if (bi >= a.stride) {
        bad = true;
      } else if (bi < held) {
        blk = a.table[(int64_t)(r0 + x) * a.stride + bi];
      } else {
        const int64_t k = s_blk[x] + bi - held;
        if (k >= 0 && k < a.n_free) blk = a.free_blocks[k];
      }
      if (blk < 0 || blk >= a.n_blocks) {
        bad = true;
        blk = -1;
      }
      if (bi >= held && bi < a.stride && (p & (bs - 1)) == 0)
        a.table[(int64_t)(r0 + x) * a.stride + bi] = blk;
      a.slot[i] = blk < 0 ? -1 : ((int64_t)blk << a.shift) + (p & (bs - 1));
      a.pos[i] = (int32_t)(p < INT32_MAX ? p : INT32_MAX);
      a.req[i] = r0 + x;
    }
    // blocks that tokens behind n_slots open: a warp a request
    if (tok0 > a.n_slots && blockIdx.x == gridDim.x - 1) {
      for (int x = warp; x < kMapsThreads && r0 + x < a.B; x += kMapsThreads / 32) {
        if (s_tok[x + 1] <= a.n_slots) continue;
        const int64_t c = s_ctx[x], held = (c + bs - 1) >> a.shift;
        // the first column that opens at an entry >= n_slots, and the end of those taken
        const int64_t from = (c + a.n_slots - s_tok[x] + bs - 1) >> a.shift;
        const int64_t end = held + s_blk[x + 1] - s_blk[x];
        const int64_t last = end < a.stride ? end : a.stride;
        for (int64_t col = (from > held ? from : held) + lane; col < last; col += 32) {
          const int64_t k = s_blk[x] + col - held;
          const int blk = k >= 0 && k < a.n_free ? a.free_blocks[k] : -1;
          a.table[(int64_t)(r0 + x) * a.stride + col] = blk >= 0 && blk < a.n_blocks ? blk : -1;
        }
      }
    }
    __syncthreads();  // the sums are read
  }
  for (int64_t i = (tok0 > i0 ? tok0 : i0) + tid; i < i1; i += kMapsThreads) {
    a.slot[i] = -1;
    a.pos[i] = -1;
    a.req[i] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.head_out[0] = (int32_t)(blk0 < INT32_MAX ? blk0 : INT32_MAX);
    if (tok0 > a.n_slots) bad = true;
  }
  if (bad) record_status(a.status, CPMLA_ERR_INDEX);
}

}  // namespace
}  // namespace cpmla

extern "C" int mla_paged_maps(const int32_t *ctx_len, const int32_t *new_len, int B,
                              int block_size, int n_blocks, const int32_t *free_blocks, int n_free,
                              const int32_t *free_head, int32_t *block_table, int64_t table_stride,
                              int n_slots, int32_t *cu_seqlens, int64_t *slot_mapping,
                              int32_t *pos, int32_t *req, int32_t *free_head_out, void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged_maps";
  CPMLA_CHECK_ARG(B >= 1 && B <= 65536, "%s: B=%d outside 1..65536", fn, B);
  CPMLA_CHECK_ARG(paged_block_size_ok(block_size), "%s: block_size=%d is not 16, 32, 64 or 128",
                  fn, block_size);
  CPMLA_CHECK_ARG(n_blocks >= 1 && n_free >= 0 && n_slots >= 0,
                  "%s: n_blocks=%d, n_free=%d, n_slots=%d", fn, n_blocks, n_free, n_slots);
  CPMLA_CHECK_ARG(table_stride >= 1, "%s: table_stride=%lld < 1", fn, (long long)table_stride);
  CPMLA_CHECK_ARG(ctx_len && new_len && block_table && cu_seqlens && free_head_out,
                  "%s: a required pointer is NULL", fn);
  CPMLA_CHECK_ARG(free_blocks || n_free == 0, "%s: free_blocks is NULL", fn);
  CPMLA_CHECK_ARG((slot_mapping && pos && req) || n_slots == 0, "%s: a token array is NULL", fn);
  CPMLA_CHECK_ARG(free_head != free_head_out, "%s: free_head and free_head_out are one word", fn);
  int *status = status_word();
  if (!status) return fail(CPMLA_ERR_CUDA, "%s: status word unavailable", fn);
  MapsArgs a{};
  a.ctx = ctx_len;
  a.nw = new_len;
  a.free_blocks = free_blocks;
  a.head = free_head;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.pos = pos;
  a.req = req;
  a.head_out = free_head_out;
  a.slot = slot_mapping;
  a.stride = table_stride;
  a.B = B;
  a.shift = paged_block_shift(block_size);
  a.n_blocks = n_blocks;
  a.n_free = n_free;
  a.n_slots = n_slots;
  a.status = status;
  const int grid = n_slots > kMapsTokens ? (int)(((int64_t)n_slots + kMapsTokens - 1) / kMapsTokens)
                                         : 1;
  paged_maps_kernel<<<grid, kMapsThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_maps: launch");
  return CPMLA_OK;
}
