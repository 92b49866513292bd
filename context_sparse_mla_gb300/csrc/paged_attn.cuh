// paged_attn.cuh -- what the attentions over the paged 8-bit and 4-bit caches share: the
// list of entries, the plan that cuts it into pieces for the SMs, the walk over a CTA's
// pieces, the split of q, the join of cut rows, the workspace and the checks.
#pragma once

#include <atomic>
#include <cmath>
#include <cstring>

#include "attn_common.cuh"

namespace cpmla {
namespace {

constexpr int kPgMaxCtas = 160;   // at most one CTA per SM
constexpr int kPgTileLog = 6;     // 64 keys a tile
// The plan's units are tiles: what a piece costs beside its tiles (8, 12 and 16 were
// measured: 8,192 prompt tokens 1,270, 1,163 and 1,160 us, 64-head chunks 459, 442 and
// 436), and what is worth a CTA of its own (one token of 8,192 keys: 28 us with 8, 24
// with 4, where more parts cost the join more).
constexpr int kPgUnitTail = 16;
constexpr int kPgMinUnits = 4;
// Parts up to which a row's join is a warp's (8 tokens of 4,096 keys x 16 heads: 23 us
// with 8, 27 with 16; 32 tokens of 16,384 keys x 64 heads: 97 with 8, 110 with 4).
constexpr int kPgLongJoin = 8;
constexpr int kPgPlanThreads = 1024;
constexpr int kPgEarly = 4096;    // entries up to which the attention is launched early

struct PagedArgs {
  const __nv_bfloat16 *q;
  int64_t q_stride;
  int H;
  const uint8_t *exp;     // 8 bits: a block's exponent
  const uint8_t *strips;  // 4 bits: the cache
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
  int hc, g, n_hg;  // heads per group, tokens per group, head groups
  int n_cta;
  struct PgGroup *groups;
  int4 *start;      // [kPgMaxCtas + 1]: (group, head group, tile) a CTA starts at
  int4 *joins;      // counts of short and long ones, then two words for each group that is
                    // cut: (group, head group, first CTA, parts), (first entry, rows, -, -);
                    // short ones from the front, those of many parts from the back
  float *o_part;    // [2 kPgMaxCtas][R][512]
  // [2 kPgMaxCtas][R]: a part's LSE, base 2, as a reference (-inf: no key) and what lies
  // above it (4 bits: log2 of the sum, which a reference of 2^24 and more would swallow)
  float2 *lse_part;
  int *status;
};

// Entries first .. first + count - 1: one request's tokens.
struct PgGroup {
  int first, count, req, t_lo;         // t_lo: first tile
  int n_tiles, lo_min, hi_max, lo_max; // bounds over the rows that see a key
  int hi_min, pad;
  long long u0;                        // tile units before this group
};

// An entry as it is listed (its loads wait for nothing), and what it says.
struct PgListed {
  int b, p, t, lo, hi;
};
__device__ __forceinline__ PgListed pg_listed(const PagedArgs &a, int i) {
  if (i < 0 || i >= a.n) return PgListed{-1, 0, 0, 0, 0};
  return PgListed{a.req[i], a.pos[i], a.tokens ? a.tokens[i] : i, a.kv_lo ? a.kv_lo[i] : 0,
                  a.kv_hi ? a.kv_hi[i] : INT32_MAX};
}
struct PgEntry {
  bool ok, bad;
  int b, lo, hi;
};
__device__ __forceinline__ PgEntry pg_entry(const PagedArgs &a, const PgListed &x) {
  PgEntry e{false, false, x.b, max(x.lo, 0), min(x.hi, x.p)};
  if (x.b == -1) return e;
  e.bad = x.b < 0 || x.b >= a.B || x.t < 0 || x.t >= a.T || x.p < 0 || x.p >= (1 << 30) ||
          (x.p >> a.shift) >= a.stride;
  e.ok = !e.bad;
  return e;
}

// ------------------------------------------------------------------ the plan
// Groups are runs of up to g entries of one request, cut at multiples of g.
// A group's length in tile units is its tiles plus kPgUnitTail for each head
// group; CTA c starts at unit floor(total c / n).  One CTA: the entries go by in
// rounds through shared memory, and thread c looks up CTA c's start.
__global__ void __launch_bounds__(kPgPlanThreads) paged_plan_kernel(const PagedArgs a) {
  grid_launch_dependents();
  __shared__ int s_b[kPgPlanThreads], s_lo[kPgPlanThreads], s_hi[kPgPlanThreads];
  __shared__ long long s_u0[kPgPlanThreads];
  __shared__ int s_nt[kPgPlanThreads];
  __shared__ long long s_u[32];
  __shared__ int s_n[32];
  __shared__ int4 s_start[kPgMaxCtas + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int round = kPgPlanThreads / a.g * a.g;  // entries a round: no group crosses
  long long u_base = 0;
  int n_base = 0;
  PgListed nxt = pg_listed(a, tid < round ? tid : -1);
  for (int r0 = 0; r0 < a.n; r0 += round) {
    const int i = r0 + tid;
    const PgEntry e = pg_entry(a, nxt);
    if (r0 + round < a.n) nxt = pg_listed(a, tid < round ? i + round : -1);
    if (e.bad) record_status(a.status, CPMLA_ERR_INDEX);
    s_b[tid] = e.ok ? e.b : -1;
    s_lo[tid] = e.lo;
    s_hi[tid] = e.hi;
    __syncthreads();
    PgGroup m{};
    const bool start = e.ok && (tid % a.g == 0 || s_b[tid - 1] != e.b);
    if (start) {
      m.first = i;
      m.req = e.b;
      m.lo_min = INT32_MAX;
      m.hi_max = -1;
      m.lo_max = -1;
      m.hi_min = INT32_MAX;
      do {
        const int lo = s_lo[tid + m.count], hi = s_hi[tid + m.count];
        if (lo <= hi) {
          m.lo_min = min(m.lo_min, lo);
          m.hi_max = max(m.hi_max, hi);
        }
        m.lo_max = max(m.lo_max, lo);
        m.hi_min = min(m.hi_min, hi);
        ++m.count;
      } while ((tid + m.count) % a.g != 0 && s_b[tid + m.count] == e.b);
      if (m.hi_max >= 0) {
        m.t_lo = m.lo_min >> kPgTileLog;
        m.n_tiles = (m.hi_max >> kPgTileLog) - m.t_lo + 1;
      }
    }
    const long long units = start ? (long long)a.n_hg * (m.n_tiles + kPgUnitTail) : 0;
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    const long long su = warp_scan_add(units, lane);
    if (lane == 31) {
      s_u[warp] = su;
      s_n[warp] = __popc(starts);
    }
    __syncthreads();
    if (warp == 0) {
      s_u[lane] = warp_scan_add(s_u[lane], lane);
      s_n[lane] = (int)warp_scan_add(s_n[lane], lane);
    }
    __syncthreads();
    if (start) {
      const int k = (warp ? s_n[warp - 1] : 0) + __popc(starts & ((1u << lane) - 1));
      m.u0 = u_base + (warp ? s_u[warp - 1] : 0) + su - units;
      a.groups[n_base + k] = m;
      s_u0[k] = m.u0;
      s_nt[k] = m.n_tiles;
    }
    u_base += s_u[31];
    n_base += s_n[31];
    __syncthreads();
  }
  // CTA c's start: the last group with u0 <= u
  const long long total = u_base;
  const int n = total == 0 ? 0 : (int)max(1ll, min((long long)a.n_cta, total / kPgMinUnits));
  const bool one_round = a.n <= round;
  if (tid <= kPgMaxCtas) {
    int4 st = make_int4(n_base, 0, 0, 0);
    if (tid < n) {
      const long long u = total * tid / n;
      int x = 0, y = n_base;
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if ((one_round ? s_u0[mid] : a.groups[mid].u0) <= u)
          x = mid;
        else
          y = mid;
      }
      const int tiles = one_round ? s_nt[x] : a.groups[x].n_tiles, len = tiles + kPgUnitTail;
      const int rel = (int)(u - (one_round ? s_u0[x] : a.groups[x].u0));
      int hg = rel / len, off = rel - hg * len;
      if (off > 0 && off >= tiles) {  // in the group's tail: the next one
        off = 0;
        if (++hg == a.n_hg) {
          hg = 0;
          ++x;
        }
      }
      st = make_int4(x, hg, off, 0);
    }
    s_start[tid] = st;
    a.start[tid] = st;
  }
  __syncthreads();
  // what is cut, by the first boundary inside it: CTAs c - 1, c, ... have parts
  static_assert(kPgMaxCtas <= 5 * 32, "five warps look for cuts");
  if (warp < 5) {
    const int c = tid + 1;
    const int4 st = s_start[c], p = s_start[c - 1];
    const bool in = st.z > 0, cont = in && p.z > 0 && p.x == st.x && p.y == st.y;
    const uint32_t b = __ballot_sync(0xffffffffu, cont);
    if (lane == 0) s_n[warp] = (int)b;
    named_bar_sync(1, 160);
    int parts = 0;
    if (in && !cont) {  // boundaries tid + 1 .. behind it in the same piece
      int e = tid + 1;
      for (int x = e >> 5; x < 5; ++x) {
        const uint32_t gone = ~(uint32_t)s_n[x] & (x == e >> 5 ? ~0u << (e & 31) : ~0u);
        e = gone ? 32 * x + __ffs(gone) - 1 : 32 * (x + 1);
        if (gone) break;
      }
      parts = e - tid + 1;
    }
    const bool lng = parts > kPgLongJoin;
    const uint32_t bs = __ballot_sync(0xffffffffu, parts > 0 && !lng);
    const uint32_t bl = __ballot_sync(0xffffffffu, lng);
    if (lane == 0) s_n[8 + warp] = __popc(bs) | __popc(bl) << 16;
    named_bar_sync(1, 160);
    int at = 0;
    for (int x = 0; x < warp; ++x) at += s_n[8 + x];
    const uint32_t below = (1u << lane) - 1;
    if (parts > 0) {
      const int k = lng ? kPgMaxCtas - 1 - (at >> 16) - __popc(bl & below)
                        : (at & 0xFFFF) + __popc(bs & below);
      const PgGroup &m = a.groups[st.x];
      a.joins[1 + 2 * k] = make_int4(st.x, st.y, c - 1, parts);
      a.joins[2 + 2 * k] = make_int4(m.first, m.count * a.hc, 0, 0);
    }
    if (tid == 159) {
      at += __popc(bs) | __popc(bl) << 16;
      a.joins[0] = make_int4(at & 0xFFFF, at >> 16, 0, 0);
    }
  }
}

// The pieces of a CTA: (group, head group) and a range of its tiles.
struct PgWalk {
  int4 s, e;
  int g, hg, t0, t1;  // the current piece
  PgGroup m;
  bool first;
  __device__ __forceinline__ PgWalk(const PagedArgs &a, int cta)
      : s(a.start[cta]), e(a.start[cta + 1]), first(true) {}
  __device__ __forceinline__ bool next(const PagedArgs &a) {
    if (!first) {
      s.z = 0;
      if (++s.y == a.n_hg) {
        s.y = 0;
        ++s.x;
      }
    }
    const bool last = s.x == e.x && s.y == e.y;
    if (s.x > e.x || (s.x == e.x && s.y > e.y) || (last && s.z >= e.z)) return false;
    if (first || s.y == 0) m = a.groups[s.x];
    first = false;
    g = s.x;
    hg = s.y;
    t0 = s.z;
    t1 = last ? e.z : m.n_tiles;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == m.n_tiles; }
};

constexpr int kPgTile = 1 << kPgTileLog;
constexpr int kPgSlot = kPgTile * 128;  // a latent chunk: [64 keys x 128 channels]
constexpr int kPgRope = kPgTile * 64;   // [64 keys x 64]
constexpr uint32_t kPgTmemCols = 512;

constexpr unsigned long long kPgDrainNs = 20ull * 1000 * 1000;
__device__ __forceinline__ void pg_drain(uint64_t *bar, uint32_t parity,
                                         unsigned long long limit_ns) {
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < limit_ns) {
  }
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
// {h, l} of two channels x down (bf16 pairs): h = E4M3(x), l = E4M3(16 (x - h)), two
// codes each.  fp16 holds x down to 2^-24, and x - h exactly; l ends at 2^-13.
__device__ __forceinline__ uint2 split_q(uint32_t w, uint32_t down) {
  uint32_t x, f;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w), "r"(down));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;"
      : "=r"(f)
      : "f"(__uint_as_float(x & 0xFFFF0000u)), "f"(__uint_as_float(x << 16)));
  const uint32_t h = e4m3x2_of_f16x2(f);
  uint32_t d = f16x2_sub(f, e4m3x2_to_f16x2((uint16_t)h));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(d), "r"(0x4C004C00u));  // 16
  return make_uint2(h, e4m3x2_of_f16x2(d));
}
// The same of four channels.
__device__ __forceinline__ uint2 split_q4(uint32_t w0, uint32_t w1, uint32_t down) {
  const uint2 a = split_q(w0, down), b = split_q(w1, down);
  return make_uint2(a.x | (b.x << 16), a.y | (b.y << 16));
}
// x 2^d for d of any size: 2^d itself may lie outside binary32 where the product does not.
__device__ __forceinline__ float pg_scale(float x, float d) {
  const float h = fast_exp2(0.5f * d);
  return x == 0.f ? 0.f : x * h * h;
}

// ------------------------------------------------------------------ the join
// A row of a join (group, head group, first CTA, parts) from its parts, in an order
// that the plan alone decides, each weighted by 2^(its LSE - the largest); lane t has
// channels 128 k + 4 t .. + 3.  The parts were just written and lie in L2, so what
// takes time is the chain of loads: kAhead parts are on their way at once, the first
// beside the LSE.  Of nw warps warp w sums parts w, w + nw, ...
template <int R>
struct PgJoin {
  static constexpr int kL = (kPgMaxCtas + 31) / 32, kAhead = 2;
  float4 o[4];
  float mx, above, l;  // the row's LSE is mx + above + log2 l
  int h;
  int64_t orow;  // the row of the output
  __device__ __forceinline__ PgJoin(const PagedArgs &a, const int4 &jn, const int4 &jg, int r,
                                    int w, int nw, int lane) {
    const int n = jn.w;
    // part 0 is CTA jn.z's second, part i the first of CTA jn.z + i
    auto at = [&](int i) { return (int64_t)(2 * (jn.z + i) + (i == 0 ? 1 : 0)) * R + r; };
    float4 v[kAhead][4];
    auto fetch = [&](int i, float4 *d) {
      const float4 *src = reinterpret_cast<const float4 *>(a.o_part + at(i) * CPMLA_DV) + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = __ldcg(src + 32 * k);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(min(w + nw * i, n - 1), v[i]);
    const int e = jg.x + r / a.hc;
    h = jn.y * a.hc + r % a.hc;
    orow = (int64_t)(a.tokens ? a.tokens[e] : e) * a.H + h;
    float2 s[kL];
    float p[kL];
    mx = above = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < kL; ++k) {
      s[k] = lane + 32 * k < n ? __ldcg(a.lse_part + at(lane + 32 * k))
                               : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, s[k].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
    for (int k = 0; k < kL; ++k) {
      p[k] = s[k].x == -INFINITY ? -INFINITY : s[k].x - mx + s[k].y;
      above = fmaxf(above, p[k]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
      above = fmaxf(above, __shfl_xor_sync(0xffffffffu, above, off));
#pragma unroll
    for (int k = 0; k < kL; ++k) {
      p[k] = p[k] == -INFINITY ? 0.f : exp2f(p[k] - above);  // NaN stays
      l += p[k];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = w; i0 < n; i0 += nw * kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int ii = i0 + nw * u;
        float wt = p[0];
#pragma unroll
        for (int k = 1; k < kL; ++k) wt = ii >> 5 == k ? p[k] : wt;
        wt = __shfl_sync(0xffffffffu, wt, ii & 31);
        if (ii >= n) wt = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[k].x = fmaf(wt, v[u][k].x, o[k].x);
          o[k].y = fmaf(wt, v[u][k].y, o[k].y);
          o[k].z = fmaf(wt, v[u][k].z, o[k].z);
          o[k].w = fmaf(wt, v[u][k].w, o[k].w);
        }
        if (ii + nw * kAhead < n) fetch(ii + nw * kAhead, v[u]);
      }
    }
  }
  // Factor of the row's output; the first thread writes L.
  __device__ __forceinline__ float finish(const PagedArgs &a, bool first) const {
    const bool empty = mx == -INFINITY && l == 0.f;  // l may be NaN
    const float L = empty ? -INFINITY : (mx + (above + log2f(l))) * 0.69314718055994530942f;
    if (first) a.lse[orow] = L;
    return empty ? 0.f : sink_factor(a.sink, h, L) / l;
  }
};
__device__ __forceinline__ uint2 pack_bf16x4(float4 v, float f) {
  return make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}

// Every row of every group in the plan's joins: by a warp, or, of more than kPgLongJoin
// parts, by a CTA.  (One token of 131,072 keys has 152 parts: 39 us a call instead of
// 78 with a warp for each row.)
constexpr int kPgJoinThreads = 256, kPgJoinCtas = 152 * 8;
template <int R>
__global__ void __launch_bounds__(kPgJoinThreads) paged_join_kernel(const PagedArgs a) {
  constexpr int kWarps = kPgJoinThreads / 32;
  __shared__ float4 s_o[kWarps][CPMLA_DV / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  const int4 counts = a.joins[0];
  const int n_long = counts.y * R * kWarps;  // one code for both: it comes from L2
  for (int x = blockIdx.x * kWarps + warp; x < n_long + counts.x * R; x += gridDim.x * kWarps) {
    const bool lng = x < n_long;  // of all of the CTA's warps
    const int y = lng ? x / kWarps : x - n_long, r = y % R;
    const int k = lng ? kPgMaxCtas - 1 - y / R : y / R;
    const int4 jn = a.joins[1 + 2 * k], jg = a.joins[2 + 2 * k];
    if (r >= jg.y) continue;
    PgJoin<R> j(a, jn, jg, r, lng ? warp : 0, lng ? kWarps : 1, lane);
    int c = lane;  // channels 4 c .., and three times 128 further
    if (lng) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s_o[warp][32 * i + lane] = j.o[i];
      __syncthreads();
      c = threadIdx.x % (CPMLA_DV / 4);
      j.o[0] = s_o[0][c];
      for (int w = 1; w < kWarps; ++w) {
        const float4 v = s_o[w][c];
        j.o[0] = make_float4(j.o[0].x + v.x, j.o[0].y + v.y, j.o[0].z + v.z, j.o[0].w + v.w);
      }
      __syncthreads();
    }
    const float f = j.finish(a, lane == 0);
    uint2 *dst = reinterpret_cast<uint2 *>(a.o + j.orow * CPMLA_DV) + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == 0 || !lng) dst[32 * i] = pack_bf16x4(j.o[i], f);
  }
}

// Workspace sections, each 256-byte aligned.
struct PgLayout {
  size_t start, joins, groups, o, lse, total;
};
PgLayout pg_layout(int n, int R) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PgLayout L{};
  L.joins = up((kPgMaxCtas + 1) * sizeof(int4));
  L.groups = L.joins + up((2 * kPgMaxCtas + 1) * sizeof(int4));
  L.lse = L.groups + up((size_t)n * sizeof(PgGroup));
  L.o = L.lse + up((size_t)2 * kPgMaxCtas * R * sizeof(float2));
  L.total = L.o + (size_t)2 * kPgMaxCtas * R * CPMLA_DV * 4;
  return L;
}

// Rows of a piece: 16 for single tokens of up to 16 heads, else 64.  The lengths lie
// on the device, so single tokens are told from the list's length and the table's
// (and an eighth more, for padding and the odd longer one).  Measured, 32 requests of
// 16,384 keys and 16 heads: with one token each 80 us in 16 rows and 91 in 64 (of
// which 16 are used), with two 132 and 94; a prompt of 4,096 tokens 1,402 and 410.
// 32 rows were never the best: 99, 101 and 890 us, and 101 for single tokens of 32
// heads, 95 in 64 rows.  B is the table's height and not the number of requests that are
// there: one prompt in a table of as many rows as it has tokens is in 16 rows too (1,000
// tokens of 16 heads 165 us, 64 in 64 rows; 200 of 8 heads 25 and 44).
int pg_rows(int hc, int n_tokens, int B) {
  return hc <= 16 && n_tokens <= B + (int64_t)B / 8 ? 16 : 64;
}

// SMs of the current device, at most kPgMaxCtas (-1 on failure), with the kernels for R =
// 16 and 64 rows allowed their shared memory there; asked once a device and R (known:
// the caller's own).
constexpr int kPgMaxDevices = 64;
using PgKnown = std::atomic<int>[2][kPgMaxDevices];
template <class Kernel>
int pg_device(const char *fn, PgKnown &known, int R, Kernel kernel, int smem) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const bool keep = e == cudaSuccess && dev >= 0 && dev < kPgMaxDevices;
  std::atomic<int> &slot = known[R == 64 ? 1 : 0][keep ? dev : 0];
  if (keep && (sms = slot.load(std::memory_order_acquire)) > 0) return sms;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) {
    fail(CPMLA_ERR_CUDA, "%s: device: %s", fn, cudaGetErrorString(e));
    return -1;
  }
  sms = sms < kPgMaxCtas ? sms : kPgMaxCtas;
  if (keep) slot.store(sms, std::memory_order_release);
  return sms;
}

// The plan, the attention kernel (of R rows a piece; x: its further arguments), the join.
template <int R, class Kernel, class... X>
int launch_paged(const char *fn, const PagedArgs &a, Kernel kernel, int threads, int smem,
                 cudaStream_t st, const X &...x) {
  auto failed = [fn](cudaError_t e, const char *what) {
    return fail(CPMLA_ERR_CUDA, "%s: %s: %s", fn, what, cudaGetErrorString(e));
  };
  cudaError_t e;
  paged_plan_kernel<<<1, kPgPlanThreads, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return failed(e, "plan launch");
  // The other two may start while the kernel ahead of them still runs (their setup
  // beside its end) and wait for its end before they read what it wrote.  The
  // attention does so for up to kPgEarly entries: with 2,500 it takes 470 us
  // instead of 487; with 8,192, where the plan takes 26 us, 1,338 instead of 1,217.
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.attrs = &at;
  cfg.numAttrs = a.n <= kPgEarly ? 1 : 0;
  cfg.stream = st;
  cfg.gridDim = dim3(a.n_cta);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kernel, a, x...);
  if (e != cudaSuccess) return failed(e, "launch");
  if (a.n_cta > 1) {
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(kPgJoinCtas);
    cfg.blockDim = dim3(kPgJoinThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, paged_join_kernel<R>, a);
    if (e != cudaSuccess) return failed(e, "join launch");
  }
  return CPMLA_OK;
}

// Argument checks of both entry points, and what the kernels take.  *R_out: rows of a
// piece, 0 when there is nothing to do.  (n_cta is the caller's.)
int paged_attn_args(const char *fn, bool four, const void *q, int64_t q_token_stride, int H,
                    const void *cache, const uint8_t *cache_exp, int n_blocks, int block_size,
                    const int32_t *block_table, int B, int64_t table_stride, const int32_t *tokens,
                    const int32_t *pos, const int32_t *req, int n_tokens, const int32_t *kv_lo,
                    const int32_t *kv_hi, float softmax_scale, const float *sink, int T,
                    void *o_out, float *lse_out, void *workspace, size_t workspace_bytes, PagedArgs &a,
                    int *R_out) {
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
  if (n_tokens == 0) {
    *R_out = 0;
    return CPMLA_OK;
  }
  CPMLA_CHECK_ARG(q && cache && (four || cache_exp) && block_table && pos && req && o_out && lse_out,
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
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_token_stride;
  a.H = H;
  a.exp = cache_exp;
  a.strips = static_cast<const uint8_t *>(cache);
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
  a.hc = H <= 64 ? H : 64;
  const int R = pg_rows(a.hc, n_tokens, B);
  a.g = R / a.hc;
  a.n_hg = H / a.hc;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const PgLayout L = pg_layout(n_tokens, R);
  a.start = reinterpret_cast<int4 *>(ws + L.start);
  a.joins = reinterpret_cast<int4 *>(ws + L.joins);
  a.groups = reinterpret_cast<PgGroup *>(ws + L.groups);
  a.lse_part = reinterpret_cast<float2 *>(ws + L.lse);
  a.o_part = reinterpret_cast<float *>(ws + L.o);
  *R_out = R;
  return CPMLA_OK;
}

}  // namespace
}  // namespace cpmla
