// paged_insert.cu -- tokens into the paged 8-bit latent cache, one power-of-two
// scale per block (mla_paged_cache_insert).
//
// For the tokens N that a call puts into a block: e_N = the least e >= -64 with
// amax(N) <= 448 * 2^e; the block's exponent is e_N if N holds row 0 (the block
// starts anew), else max(old, e_N); a raised exponent re-codes the rows that
// stay as E4M3(code * 2^(old - e)).  x * 2^-e is exact (in bf16 too, but for what
// rounds to 0), so every
// code is the E4M3 value nearest to the exact quotient.
//
// Bound by HBM: 1152 B read and 576 B written a token, and for few tokens by the
// chain slots -> rows -> maximum -> codes.  The scale depends on all tokens of a
// block, so they stay in registers between the maximum and the coding: one read.
// A CTA takes the runs (tokens of one block, side by side but for skipped entries
// between them) that start at its list entries: one read of the slots around tells
// starts and ends, where skipped entries do not fill all of it; then the CTA looks
// further, 1,024 entries at a time.  A run of up to kShortRun entries -- a decode row --
// goes to one warp, longer ones, and those that raise their block's scale, to the CTA,
// 64 rows (one block, or several of 16 or 32 rows) at a time.  A row costs a warp about
// 150 instructions in all: maxima and scaling work on pairs of bf16 (340 with a
// comparison, a product and a test for infinities a channel).
// Measured (a call alone, with the cache cold unless named): 131,072 tokens of one
// prompt 55 us (4.1 TB/s of bytes it must move) in blocks of 64 or 128, 59 us in blocks
// of 16; in a graph 32 single tokens 2.8 us, 8,192 prompt tokens 6.3 us from L2.  Single
// tokens that all raise their block's scale: 32 of them 10 us, 500 18 us (156 and 160
// when a warp re-coded its block's rows one after another).  32 single tokens before
// 4,000 skipped entries 6.6 us, before 130,000 61 us: the CTA of the last token looks
// through them.  Runs that ended at a skipped entry, so that one between two tokens of
// a block made two runs of it, took 53 us for the prompt and 2.2 us for the 32 tokens.
// What is left is latency: two CTAs of 8 rows a warp fill an SM's registers (512
// threads of 4 rows took 57 us and spilled).
#include "cpmla_internal.cuh"

namespace cpmla {
namespace {

constexpr int kPinThreads = 256;
constexpr int kPinWarps = kPinThreads / 32;
constexpr int kPinWave = 304;         // CTAs that run at once
constexpr int kMaxChunk = 64;         // list entries a CTA takes the runs of, at most
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
  int chunk;  // list entries per CTA
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

// Maximum of |x| of a row's bf16, as two halves of 16 bits: the bits of |x| order
// like |x|, infinities and NaN above all finite values.
__device__ __forceinline__ uint32_t row_amax(const Row &r, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 5; ++i)
    m = __vmaxu2(__vmaxu2(m, r.v[i].x & 0x7FFF7FFFu), r.v[i].y & 0x7FFF7FFFu);
  return m;
}
// One half's maximum over the warp, as binary32 bits.
__device__ __forceinline__ uint32_t warp_amax(uint32_t m) {
  return __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)) << 16;
}
constexpr uint32_t kInfBits = 0x7F800000u;
// The maximum over the finite entries of a row, the rare case (bits for max).
__device__ __noinline__ uint32_t finite_amax(const PinArgs &a, int64_t t, int lane, uint32_t m) {
  const uint16_t *src = reinterpret_cast<const uint16_t *>(a.kv + t * a.stride);
#pragma unroll 1
  for (int i = lane; i < CPMLA_DQK; i += 32) {
    const uint32_t x = src[i] & 0x7FFFu;
    m = x < 0x7F80u && x > m ? x : m;
  }
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

// x * inv of two bf16, inv a power of two: exact, but for results too small
// for any E4M3 value but 0.
__device__ __forceinline__ uint32_t scale2(uint32_t x, uint32_t inv) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(inv));
  return y;
}
__device__ __forceinline__ uint32_t inv_scale(int e) {
  const uint32_t b = (uint32_t)(127 - e) << 7;
  return b | (b << 16);
}

__device__ __forceinline__ void store_row(const PinArgs &a, int64_t slot, const Row &r,
                                          uint32_t inv, int lane) {
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.cache + slot * CPMLA_DQK) + lane;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const uint32_t x = scale2(r.v[i].x, inv), y = scale2(r.v[i].y, inv);
    if (i < 4 || lane < kChunks - 128)
      dst[32 * i] = e4m3x4(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u),
                           __uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u));
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

// A row's codes, as they lie in the cache, and written back times f.
__device__ __forceinline__ Row load_codes(const PinArgs &a, int64_t slot, int lane) {
  Row r;
  const uint32_t *src = reinterpret_cast<const uint32_t *>(a.cache + slot * CPMLA_DQK) + lane;
#pragma unroll
  for (int i = 0; i < 5; ++i)
    r.v[i].x = (i < 4 || lane < kChunks - 128) ? src[32 * i] : 0;
  return r;
}
__device__ __forceinline__ void recode_row(const PinArgs &a, int64_t slot, const Row &r, float f,
                                           int lane) {
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.cache + slot * CPMLA_DQK) + lane;
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (i < 4 || lane < kChunks - 128) dst[32 * i] = recode(r.v[i].x, f);
}

__device__ __forceinline__ int old_exp(const PinArgs &a, int64_t blk) {
  const int e = (int)a.exp[blk] - 127;
  return e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);
}

// Slot of an entry; -1 (skipped) when it lies outside the cache or the list.
__device__ __forceinline__ int64_t slot_of(const PinArgs &a, int64_t i, bool record) {
  if (i < 0 || i >= a.n) return -1;
  const int64_t s = a.slot[i];
  if (s >= 0 && s < a.n_slots) return s;
  if (record && s != -1) record_status(a.status, CPMLA_ERR_INDEX);
  return -1;
}

__global__ void __launch_bounds__(kPinThreads) paged_insert_kernel(const PinArgs a) {
  __shared__ int64_t s_slot[kPinThreads];  // slots from the entry before the CTA's first
  __shared__ uint32_t s_val[kPinWarps + 1];  // bit i: s_slot[i] is not skipped
  __shared__ uint32_t s_new[kPinWarps];      // bit i: ... and a run starts with it
  __shared__ int s_far, s_stop, s_last;      // entries beyond s_slot, by their place in the list
  __shared__ int s_start[kMaxChunk], s_len[kMaxChunk];  // the long ones among them
  __shared__ int s_owner[128];  // long runs: last token of each row of the block, or -1
  __shared__ int s_n_long;
  __shared__ uint32_t s_amax[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t i0 = (int64_t)blockIdx.x * a.chunk;
  const int bs = 1 << a.shift;

  // ---- one read of the slots around: they tell where runs start and end
  const int64_t here = slot_of(a, i0 - 1 + tid, tid >= 1 && tid <= a.chunk);
  s_slot[tid] = here;
  const uint32_t val = __ballot_sync(0xffffffffu, here >= 0);
  if (lane == 0) s_val[warp] = val;
  if (tid == 0) {
    s_val[kPinWarps] = 0;
    s_n_long = 0;
    s_far = s_last = -1;
    s_stop = INT32_MAX;
  }
  __syncthreads();
  // the last entry below k of s_slot that is not skipped, or -1
  auto valid_below = [&](int k) {
    int w = k >> 5;
    uint32_t b = s_val[w] & ((1u << (k & 31)) - 1);
    while (b == 0 && w > 0) b = s_val[--w];
    return b ? 32 * w + 31 - __clz(b) : -1;
  };
  const uint64_t first = ~0ull >> (64 - a.chunk);  // the CTA's entries
  auto own_bits = [&](const uint32_t *m) {          // ... bits 1 .. chunk of a mask
    return (m[0] >> 1 | (uint64_t)m[1] << 31 | (uint64_t)m[2] << 63) & first;
  };
  // the block of the last entry before s_slot, where an entry of the CTA needs it
  int64_t before = -1;
  if ((s_val[0] & 1) == 0 && i0 > 1 && own_bits(s_val) != 0) {
    bool hit = false;
    for (int64_t top = i0 - 2; top >= 0 && !hit; top -= 4 * kPinThreads) {
      int at = -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = top - tid - u * kPinThreads;
        if (slot_of(a, i, false) >= 0) at = max(at, (int)i);
      }
      if (at >= 0) atomicMax(&s_far, at);
      hit = __syncthreads_or(at >= 0);
    }
    if (hit) before = a.slot[s_far] >> a.shift;
  }
  bool starts = false;
  if (here >= 0 && tid >= 1) {
    const uint32_t b = val & ((1u << lane) - 1);
    const int p = b ? tid - lane + 31 - __clz(b) : valid_below(tid - lane);
    starts = (p >= 0 ? s_slot[p] >> a.shift : before) != here >> a.shift;
  }
  {
    const uint32_t g = __ballot_sync(0xffffffffu, starts);
    if (lane == 0) s_new[warp] = g;
  }
  const bool ends = __syncthreads_or(starts && tid > a.chunk);  // all within s_slot
  uint64_t go = own_bits(s_new);
  // the first start above k of s_slot, or kPinThreads
  auto start_above = [&](int k) {
    int w = (k + 1) >> 5;
    uint32_t b = w < kPinWarps ? s_new[w] & ~0u << ((k + 1) & 31) : 0;
    while (b == 0 && ++w < kPinWarps) b = s_new[w];
    return b ? 32 * w + __ffs(b) - 1 : kPinThreads;
  };
  // where the last run ends, if not within s_slot
  if (go != 0 && !ends && i0 - 1 + kPinThreads < a.n) {
    const int64_t blk = s_slot[64 - __clzll(go)] >> a.shift;
    int last = -1;
    bool stop = false;
    for (int64_t top = i0 - 1 + kPinThreads; top < a.n && !stop; top += 4 * kPinThreads) {
      int64_t x[4];
      int other = INT32_MAX;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = top + tid + u * kPinThreads;
        x[u] = slot_of(a, i, false);
        if (x[u] >= 0 && x[u] >> a.shift != blk) other = min(other, (int)i);
      }
      if (other != INT32_MAX) atomicMin(&s_stop, other);
      stop = __syncthreads_or(other != INT32_MAX);
      const int end = *(volatile int *)&s_stop;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = top + tid + u * kPinThreads;
        if (x[u] >= 0 && i < end) last = max(last, (int)i);
      }
    }
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
  }
  // the runs in turn to the warps
  for (int k = 0; go != 0; ++k) {
    const int c = __ffsll(go) - 1;
    go &= go - 1;
    if (k % kPinWarps != warp) continue;
    const int64_t t = i0 + c, blk = s_slot[c + 1] >> a.shift;
    const int end = start_above(c + 1);
    int len = valid_below(end) - c;
    if (end == kPinThreads && s_last >= 0) len = s_last - (int)t + 1;
    auto leave = [&] {  // to the whole CTA
      if (lane == 0) {
        const int i = atomicAdd(&s_n_long, 1);
        s_start[i] = c;
        s_len[i] = len;
      }
    };
    if (len > kShortRun) {
      leave();
      continue;
    }
    const int eo = old_exp(a, blk);
    Row r[kShortRun];
    int64_t s[kShortRun];
    uint32_t m = 0;
    bool starts = false;
#pragma unroll
    for (int u = 0; u < kShortRun; ++u) {
      s[u] = -1;
      if (u < len) s[u] = s_slot[c + 1 + u];
      if (s[u] >= 0) r[u] = load_row(a, t + u, lane);
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
    m = warp_amax(m);
    if (m >= kInfBits) {
      m = 0;
      for (int u = 0; u < len; ++u) {
        bool kept = s_slot[c + 1 + u] >= 0;  // s[u], without an index known at run time
        for (int w = u + 1; w < len; ++w) kept &= s_slot[c + 1 + w] != s_slot[c + 1 + u];
        if (kept) m = finite_amax(a, t + u, lane, m);
      }
      m = warp_amax(m);
    }
    int e = exp_of(m);
    if (!starts) {
      if (eo < e) {  // the block's other rows are re-coded
        leave();
        continue;
      }
      e = eo;
    }
    const uint32_t inv = inv_scale(e);
#pragma unroll
    for (int u = 0; u < kShortRun; ++u)
      if (s[u] >= 0) store_row(a, s[u], r[u], inv, lane);
    __syncwarp();  // every lane has read the old exponent
    if (lane == 0) a.exp[blk] = (uint8_t)(e + 127);
  }
  __syncthreads();

  // ---- longer runs: 64 rows at a time, of one block or of several small ones
  const int groups = bs < 64 ? 64 / bs : 1, n_warps = kPinWarps / groups;
  const int g = warp / n_warps, gw = warp % n_warps, gt = tid - g * n_warps * 32;
  int *owner = s_owner + g * bs;
  for (int k0 = 0; k0 < s_n_long; k0 += groups) {
    const bool mine = k0 + g < s_n_long;
    const int w = mine ? s_start[k0 + g] : 0, L = mine ? s_len[k0 + g] : 0;
    const int64_t b = s_slot[w + 1] >> a.shift, t0 = i0 + w;
    const int eo = mine ? old_exp(a, b) : 0;
    for (int i = gt; i < bs; i += n_warps * 32) owner[i] = -1;
    if (gt == 0) s_amax[g] = 0;
    __syncthreads();
    for (int i = gt; i < L; i += n_warps * 32) {
      const int64_t x = w + 1 + i < kPinThreads ? s_slot[w + 1 + i] : slot_of(a, t0 + i, false);
      if (x >= 0) atomicMax(&owner[x & (bs - 1)], i);
    }
    __syncthreads();
    // row gw + n_warps j of the block is this warp's, 8 of them at once
    Row r[kRowRegs];
    uint32_t m = 0;
    const int per = bs / n_warps;  // 8, or 16 in blocks of 128
    for (int j0 = 0; j0 < per; j0 += kRowRegs) {
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) {
        const int o = owner[gw + n_warps * (j0 + j)];
        r[j] = Row{};
        if (o >= 0) r[j] = load_row(a, t0 + o, lane);
      }
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) m = row_amax(r[j], m);
    }
    m = warp_amax(m);
    if (m >= kInfBits) {
      m = 0;
      for (int row = gw; row < bs; row += n_warps)
        if (owner[row] >= 0) m = finite_amax(a, t0 + owner[row], lane, m);
      m = warp_amax(m);
    }
    if (lane == 0) atomicMax(&s_amax[g], m);
    __syncthreads();
    int e = exp_of(s_amax[g]);
    float f = 1.f;
    if (owner[0] < 0) {  // the block goes on
      if (eo >= e)
        e = eo;
      else
        f = pow2_neg(e - eo);
    }
    const uint32_t inv = inv_scale(e);
    // blocks of 128: the registers hold the last 8 rows, the first 8 are read again
    for (int j0 = per - kRowRegs; j0 >= 0 && mine; j0 -= kRowRegs) {
      if (j0 + kRowRegs < per || f != 1.f) {
#pragma unroll
        for (int j = 0; j < kRowRegs; ++j) {
          const int row = gw + n_warps * (j0 + j), o = owner[row];
          if (o >= 0) {
            if (j0 + kRowRegs < per) r[j] = load_row(a, t0 + o, lane);
          } else if (f != 1.f) {
            r[j] = load_codes(a, (b << a.shift) + row, lane);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kRowRegs; ++j) {
        const int row = gw + n_warps * (j0 + j);
        const int64_t sl = (b << a.shift) + row;
        if (owner[row] >= 0)
          store_row(a, sl, r[j], inv, lane);
        else if (f != 1.f)
          recode_row(a, sl, r[j], f, lane);
      }
    }
    if (mine && gt == 0) a.exp[b] = (uint8_t)(e + 127);
    __syncthreads();  // owner and s_amax are free again
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
  // Entries per CTA: one while the CTAs run at once (two on each of 152 SMs), so that
  // blocks whose scale rises are re-coded side by side (32 single tokens that all
  // raise theirs take 10 us, 35 with 8 a CTA); then up to 64, so that a prompt's long
  // runs need not wait for CTAs that find no start.  Measured with 8, 16, 32, 64:
  // 8,192 prompt tokens 9.7, 7.1, 6.2, 5.4 us; 131,072 of them 109, 76, 59, 55 us; and
  // the other way 4,000 single tokens 6.7, 7.9, 8.3, 14.5 us.
  a.chunk = 1;
  while (a.chunk < kMaxChunk && (int64_t)a.chunk * kPinWave < n) a.chunk *= 2;
  const int64_t grid = ((int64_t)n + a.chunk - 1) / a.chunk;
  paged_insert_kernel<<<(unsigned)grid, kPinThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_cache_insert: launch");
  return CPMLA_OK;
}
