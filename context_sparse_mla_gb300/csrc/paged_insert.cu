// paged_insert.cu -- tokens into the paged 8-bit latent cache, one power-of-two
// scale per block (mla_paged_cache_insert).
//
// For the tokens N that a call puts into a block: e_N = the least e >= -64 with
// amax(N) <= 448 * 2^e; the block's exponent is e_N if N holds row 0 (the block
// starts anew), else max(old, e_N); a raised exponent re-codes the rows that
// stay as E4M3(code * 2^(old - e)).  x * 2^-e is exact in binary32, so every
// code is the E4M3 value nearest to the exact quotient.
//
// Bound by HBM: 1152 B read and 576 B written a token.  The scale depends on
// all tokens of a block, so a block is one CTA's work and its tokens stay in
// registers between the maximum and the coding: one read.  A CTA looks at
// kInsChunk list entries and takes the runs (tokens of one block, side by
// side) that start there: a run of up to kShortRun tokens -- a decode row --
// goes to the warp of its first token, a longer one to the whole CTA.
#include "cpmla_internal.cuh"

namespace cpmla {
namespace {

constexpr int kPinThreads = 256;
constexpr int kPinWarps = kPinThreads / 32;
constexpr int kInsChunk = kPinWarps;  // list entries per CTA: one per warp
constexpr int kShortRun = 4;
constexpr int kRowRegs = 8;           // rows of a long run that a warp holds at once
constexpr int kExpMin = -64, kExpMax = 120;
constexpr int kChunks = CPMLA_DQK / 4;  // 144 four-channel chunks a row

struct PinArgs {
  const __nv_bfloat16 *kv;
  int64_t stride;
  int64_t n;
  const int64_t *slot;
  uint8_t *cache;
  uint8_t *exp;
  int64_t n_slots;
  int shift;
  int *status;
};

// A token's row, four channels at a time: chunk lane + 32 i (i = 4: lanes 0-15).
struct Row {
  uint2 v[5];
};

__device__ __forceinline__ Row load_row(const PinArgs &a, int64_t t, int lane) {
  Row r;
  const uint2 *src = reinterpret_cast<const uint2 *>(a.kv + t * a.stride);
#pragma unroll
  for (int i = 0; i < 5; ++i)
    r.v[i] = (i < 4 || lane < kChunks - 128) ? __ldg(src + lane + 32 * i) : make_uint2(0, 0);
  return r;
}

// The larger of m and the bits of |x| over the finite bf16 of two words.
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, uint32_t w) {
  const uint32_t a = (w << 16) & 0x7FFF0000u, b = w & 0x7FFF0000u;
  m = a < 0x7F800000u && a > m ? a : m;
  return b < 0x7F800000u && b > m ? b : m;
}
__device__ __forceinline__ uint32_t row_amax(const Row &r, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 5; ++i) m = amax_bits(amax_bits(m, r.v[i].x), r.v[i].y);
  return m;
}

// The least e in [kExpMin, kExpMax] with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int exp_of(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - ((bits & 0x7FFFFFu) > 0x600000u ? 7 : 8);
  return e < kExpMin ? kExpMin : e;
}
// 2^-d for 0 <= d; 0 below the normal range (every E4M3 product is then 0)
__device__ __forceinline__ float pow2_neg(int d) {
  return d > 126 ? 0.f : __int_as_float((127 - d) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void store_row(const PinArgs &a, int64_t slot, const Row &r, float inv,
                                          int lane) {
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.cache + slot * CPMLA_DQK);
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    if (i < 4 || lane < kChunks - 128)
      dst[lane + 32 * i] = e4m3x4(__uint_as_float(r.v[i].x << 16) * inv,
                                  __uint_as_float(r.v[i].x & 0xFFFF0000u) * inv,
                                  __uint_as_float(r.v[i].y << 16) * inv,
                                  __uint_as_float(r.v[i].y & 0xFFFF0000u) * inv);
  }
}

// Four codes times f.
__device__ __forceinline__ uint32_t recode(uint32_t w, float f) {
  float x[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w >> (16 * h))));
    const float2 f2 = __half22float2(*reinterpret_cast<__half2 *>(&h2));
    x[2 * h] = f2.x * f;
    x[2 * h + 1] = f2.y * f;
  }
  return e4m3x4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ int old_exp(const PinArgs &a, int64_t blk) {
  const int e = (int)a.exp[blk] - 127;
  return e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);
}

// A block id no run has: a skipped entry.
__device__ __forceinline__ int64_t block_of(const PinArgs &a, int64_t i, bool record) {
  const int64_t s = a.slot[i];
  if (s < 0 || s >= a.n_slots) {
    if (record && s != -1) record_status(a.status, CPMLA_ERR_INDEX);
    return -1;
  }
  return s >> a.shift;
}

__global__ void __launch_bounds__(kPinThreads) paged_insert_kernel(const PinArgs a) {
  __shared__ int64_t s_blk[kInsChunk];
  __shared__ int64_t s_len[kInsChunk];  // tokens of the long run that starts at an entry, else 0
  __shared__ int64_t s_owner[128];      // long run: last token of each row of the block, or -1
  __shared__ uint32_t s_amax;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t i0 = (int64_t)blockIdx.x * kInsChunk;
  const int bs = 1 << a.shift;

  // ---- the run that starts at this warp's entry, if one does
  const int64_t t = i0 + warp;
  int64_t blk = -1, len = 0;
  if (t < a.n) {
    blk = block_of(a, t, lane == 0);
    if (blk >= 0 && t > 0 && block_of(a, t - 1, false) == blk) blk = -1;
  }
  if (blk >= 0) {
    len = 1;
    for (;;) {
      const int64_t i = t + len + lane;
      const bool same = i < a.n && block_of(a, i, false) == blk;
      const uint32_t b = __ballot_sync(0xffffffffu, same);
      if (b == 0xffffffffu) {
        len += 32;
        continue;
      }
      len += __ffs(~b) - 1;
      break;
    }
  }
  if (lane == 0) {
    s_blk[warp] = blk;
    s_len[warp] = len > kShortRun ? len : 0;
  }
  if (len > 0 && len <= kShortRun) {
    Row r[kShortRun];
    int64_t s[kShortRun];
    uint32_t m = 0;
    bool starts = false;
#pragma unroll
    for (int u = 0; u < kShortRun; ++u) {
      s[u] = -1;
      if (u < len) {
        s[u] = a.slot[t + u];
        r[u] = load_row(a, t + u, lane);
      }
    }
    // of tokens with one slot the last is kept
#pragma unroll
    for (int u = 0; u < kShortRun; ++u)
#pragma unroll
      for (int w = u + 1; w < kShortRun; ++w)
        if (s[w] == s[u]) s[u] = -1;
#pragma unroll
    for (int u = 0; u < kShortRun; ++u) {
      if (s[u] < 0) continue;
      m = row_amax(r[u], m);
      starts |= (s[u] & (bs - 1)) == 0;
    }
    m = __reduce_max_sync(0xffffffffu, m);
    int e = exp_of(m);
    if (!starts) {
      const int eo = old_exp(a, blk);
      if (eo >= e) {
        e = eo;
      } else {
        const float f = pow2_neg(e - eo);
        for (int row = 0; row < bs; ++row) {
          const int64_t sl = (blk << a.shift) + row;
          bool mine = false;
#pragma unroll
          for (int u = 0; u < kShortRun; ++u) mine |= s[u] == sl;
          if (mine) continue;
          uint32_t *p = reinterpret_cast<uint32_t *>(a.cache + sl * CPMLA_DQK);
#pragma unroll
          for (int i = 0; i < 5; ++i)
            if (i < 4 || lane < kChunks - 128) p[lane + 32 * i] = recode(p[lane + 32 * i], f);
        }
      }
    }
    const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
    for (int u = 0; u < kShortRun; ++u)
      if (s[u] >= 0) store_row(a, s[u], r[u], inv, lane);
    __syncwarp();  // every lane has read the old exponent
    if (lane == 0) a.exp[blk] = (uint8_t)(e + 127);
  }
  __syncthreads();

  // ---- longer runs, one after another by the whole CTA
  for (int w = 0; w < kInsChunk; ++w) {
    const int64_t L = s_len[w];
    if (L == 0) continue;
    const int64_t b = s_blk[w], t0 = i0 + w;
    if (tid < bs) s_owner[tid] = -1;
    if (tid == 0) s_amax = 0;
    __syncthreads();
    for (int64_t i = tid; i < L; i += kPinThreads)
      atomicMax(reinterpret_cast<long long *>(&s_owner[a.slot[t0 + i] & (bs - 1)]), (long long)i);
    __syncthreads();
    const bool starts = s_owner[0] >= 0;
    // rows of the block in turn: row warp + 8 j is this warp's (coalesced, and
    // at most 16 rows a warp, duplicates or not)
    Row r[kRowRegs];
    uint32_t m = 0;
    const int per = bs / kPinWarps;  // 2 .. 16 rows a warp
    for (int j0 = 0; j0 < per; j0 += kRowRegs) {
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) {
        const int row = warp + kPinWarps * (j0 + j);
        if (j0 + j < per && s_owner[row] >= 0) r[j] = load_row(a, t0 + s_owner[row], lane);
      }
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) {
        const int row = warp + kPinWarps * (j0 + j);
        if (j0 + j < per && s_owner[row] >= 0) m = row_amax(r[j], m);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(&s_amax, m);
    __syncthreads();
    int e = exp_of(s_amax);
    float f = 1.f;
    if (!starts) {
      const int eo = old_exp(a, b);
      if (eo >= e)
        e = eo;
      else
        f = pow2_neg(e - eo);
    }
    const float inv = __int_as_float((127 - e) << 23);
    // blocks of 128: the registers hold the last 8 rows, the first 8 are read again
    for (int j0 = per > kRowRegs ? per - kRowRegs : 0; j0 >= 0; j0 -= kRowRegs) {
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) {
        const int row = warp + kPinWarps * (j0 + j);
        if (j0 + j >= per) continue;
        const int64_t sl = (b << a.shift) + row;
        if (s_owner[row] >= 0) {
          if (j0 + kRowRegs < per) r[j] = load_row(a, t0 + s_owner[row], lane);
          store_row(a, sl, r[j], inv, lane);
        } else if (f != 1.f) {
          uint32_t *p = reinterpret_cast<uint32_t *>(a.cache + sl * CPMLA_DQK);
#pragma unroll
          for (int i = 0; i < 5; ++i)
            if (i < 4 || lane < kChunks - 128) p[lane + 32 * i] = recode(p[lane + 32 * i], f);
        }
      }
    }
    __syncthreads();  // every thread has read the old exponent and s_owner
    if (tid == 0) a.exp[b] = (uint8_t)(e + 127);
  }
}

}  // namespace
}  // namespace cpmla

extern "C" int mla_paged_cache_insert(const void *kv, int64_t kv_token_stride, int n,
                                      const int64_t *slot_mapping, void *cache,
                                      uint8_t *cache_exp, int n_blocks, int block_size,
                                      void *stream) {
  using namespace cpmla;
  const char *fn = "mla_paged_cache_insert";
  CPMLA_CHECK_ARG(n >= 0, "%s: n=%d < 0", fn, n);
  CPMLA_CHECK_ARG(kv_token_stride >= CPMLA_DQK && kv_token_stride % 8 == 0,
                  "%s: kv_token_stride=%lld must be >= 576 and a multiple of 8", fn,
                  (long long)kv_token_stride);
  CPMLA_CHECK_ARG(paged_block_size_ok(block_size), "%s: block_size=%d is not 16, 32, 64 or 128",
                  fn, block_size);
  CPMLA_CHECK_ARG(n_blocks >= 1, "%s: n_blocks=%d < 1", fn, n_blocks);
  if (n == 0) return CPMLA_OK;
  CPMLA_CHECK_ARG(kv && slot_mapping && cache && cache_exp, "%s: a required pointer is NULL", fn);
  CPMLA_CHECK_ARG(((uintptr_t)kv & 15) == 0 && ((uintptr_t)cache & 15) == 0,
                  "%s: kv and cache must be 16-byte aligned", fn);
  int *status = status_word();
  if (!status) return fail(CPMLA_ERR_CUDA, "%s: status word unavailable", fn);
  PinArgs a{};
  a.kv = static_cast<const __nv_bfloat16 *>(kv);
  a.stride = kv_token_stride;
  a.n = n;
  a.slot = slot_mapping;
  a.cache = static_cast<uint8_t *>(cache);
  a.exp = cache_exp;
  a.n_slots = (int64_t)n_blocks * block_size;
  a.shift = paged_block_shift(block_size);
  a.status = status;
  const int64_t grid = ((int64_t)n + kInsChunk - 1) / kInsChunk;
  paged_insert_kernel<<<(unsigned)grid, kPinThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_cache_insert: launch");
  return CPMLA_OK;
}
