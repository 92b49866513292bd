// paged_attn.cu -- attention of listed tokens over the paged 8-bit latent
// cache (mla_paged_attn): prompt chunks and single tokens in one list.
//
// With codes c_j (E4M3), block exponents e_j and q = 2^a (h + l / 16), h and l
// E4M3 vectors, a score in base 2 is
//   t_j = scale log2(e) 2^(a + e_j) (h . c_j + l . c_j / 16)
// and, with u_j = t_j + e_j, o = sum 2^(u_j - m) c_j / sum 2^(t_j - m): the
// block's scale of the value rides in the exponent of its weight.  So both
// GEMMs read the cache's bytes as they lie in memory:
//   * q's bf16 has 8 significant bits, an E4M3 has 4: h = E4M3(q 2^-a) and l =
//     E4M3(16 (q 2^-a - h)) hold it exactly down to 2^-13 of the row's unit
//     (2^-22 of its largest channel).
//   * p_j = 2^(u_j - m), as fp16, is the sum of three E5M2: 9 significant bits
//     (a bf16 has 8) where p >= 2^-8, and at worst 2^-17 off below.  m follows
//     each tile's maximum both ways: it moves when the tile's largest p leaves
//     [2^4, 2^15.75], to make it 2^10, so weights keep their 9 bits down to
//     2^-12 of a tile's own largest one at least, whatever the other tiles
//     hold.  (A first token with almost all of the weight and next to no value
//     is common; two E4M3 terms, which need a third fewer MMAs, reach 2^-9 and
//     lose the tokens beside it.)  m stays within 2^60 of its highest value,
//     beyond which a tile adds nothing.
//
// One CTA works on R = 64 rows (G tokens of one request x Hc heads) and 128
// keys at a time, as the dense kernel does:
//   S^T = C . [h | l]^T   M = 128 keys, N = 128, K = 576 (kind::f8f6f4), into
//                         one of two TMEM buffers
//   O^T += C^T . P^T      M = 128 channels x 4, N = 64, K = 128 keys, for the
//                         three parts of p; 256 TMEM columns
// The value is the latent itself: a chunk [128 keys x 128 channels] stays in
// its 16 KB ring slot from the score GEMM to the PV GEMM, so a tile costs 72
// KB of loads (the bf16 kernel's: 288 KB).
//
// The work is cut by tiles, not by rows: a first launch (one CTA) groups the
// entries, counts tiles and gives every SM the same number of tile units; a
// group that is cut leaves normalised fp32 parts in the workspace, at most two
// for each SM, and a third launch joins them in a fixed order.
//
// Warps: 0 issues the score GEMMs, 1 and 2 the PV GEMMs (chunks 0, 2 and 1,
// 3), 3 loads (lane p: page p of a tile), 4-19 are four softmax warpgroups of
// 16 rows (thread = key of the tile / channel of an O^T chunk).  Every wait is
// bounded; on expiry the CTA records CPMLA_ERR_TIMEOUT, drains its copies and
// MMAs, frees TMEM and exits.
#include <cmath>
#include <cstring>

#include "attn_common.cuh"

namespace cpmla {
namespace {

constexpr int kPgMaxCtas = 160;   // at most one CTA per SM
constexpr int kPgUnitTail = 2;    // a group's fixed cost, in tiles (plan)
constexpr int kPgMinUnits = 4;    // tile units worth a CTA of its own
constexpr int kPgPlanThreads = 1024;

struct PagedArgs {
  const __nv_bfloat16 *q;
  int64_t q_stride;
  int H;
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
  int hc, g, n_hg;  // heads per group, tokens per group, head groups
  int n_cta;
  struct PgGroup *groups;
  int4 *start;      // [kPgMaxCtas + 1]: (group, head group, tile) a CTA starts at
  float *o_part;    // [2 kPgMaxCtas][R][512]
  float *lse_part;  // [2 kPgMaxCtas][R], base 2
  int *status;
};

// Entries first .. first + count - 1: one request's tokens.
struct PgGroup {
  int first, count, req, t_lo;         // t_lo: first 128-key tile
  int n_tiles, lo_min, hi_max, lo_max; // bounds over the rows that see a key
  int hi_min, pad;
  long long u0;                        // tile units before this group
};

struct PgEntry {
  bool ok, bad;
  int b, lo, hi;
};
__device__ __forceinline__ PgEntry pg_entry(const PagedArgs &a, int i) {
  PgEntry e{false, false, -1, 1, 0};
  if (i < 0 || i >= a.n) return e;
  e.b = a.req[i];
  if (e.b == -1) return e;
  const int p = a.pos[i], t = a.tokens ? a.tokens[i] : i;
  e.bad = e.b < 0 || e.b >= a.B || t < 0 || t >= a.T || p < 0 || p >= (1 << 30) ||
          (p >> a.shift) >= a.stride;
  e.ok = !e.bad;
  e.lo = a.kv_lo ? max(a.kv_lo[i], 0) : 0;
  e.hi = a.kv_hi ? min(a.kv_hi[i], p) : p;
  return e;
}

// ------------------------------------------------------------------ the plan
__device__ __forceinline__ long long pg_scan(long long v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += up;
  }
  return v;
}

// Groups are runs of up to g entries of one request, cut at multiples of g.
// A group's length in tile units is its tiles plus kPgUnitTail for each head
// group; CTA c starts at unit floor(total c / n).
__global__ void __launch_bounds__(kPgPlanThreads) paged_plan_kernel(const PagedArgs a) {
  __shared__ long long s_u[32], s_n[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long u_base = 0;
  int n_base = 0;
  for (int r0 = 0; r0 < a.n; r0 += kPgPlanThreads) {
    const int i = r0 + tid;
    const PgEntry e = pg_entry(a, i);
    if (e.bad) record_status(a.status, CPMLA_ERR_INDEX);
    bool start = e.ok;
    if (start && i % a.g != 0) {
      const PgEntry p = pg_entry(a, i - 1);
      start = !p.ok || p.b != e.b;
    }
    PgGroup m{};
    if (start) {
      m.first = i;
      m.req = e.b;
      m.lo_min = INT32_MAX;
      m.hi_max = -1;
      m.lo_max = -1;
      m.hi_min = INT32_MAX;
      PgEntry x = e;
      for (;;) {
        if (x.lo <= x.hi) {
          m.lo_min = min(m.lo_min, x.lo);
          m.hi_max = max(m.hi_max, x.hi);
        }
        m.lo_max = max(m.lo_max, x.lo);
        m.hi_min = min(m.hi_min, x.hi);
        const int nx = i + ++m.count;
        if (nx % a.g == 0) break;
        x = pg_entry(a, nx);
        if (!x.ok || x.b != e.b) break;
      }
      if (m.hi_max >= 0) {
        m.t_lo = m.lo_min >> 7;
        m.n_tiles = (m.hi_max >> 7) - m.t_lo + 1;
      }
    }
    const long long units = start ? (long long)a.n_hg * (m.n_tiles + kPgUnitTail) : 0;
    const long long su = pg_scan(units, lane), sn = pg_scan(start ? 1 : 0, lane);
    __syncthreads();
    if (lane == 31) {
      s_u[warp] = su;
      s_n[warp] = sn;
    }
    __syncthreads();
    if (warp == 0) {
      s_u[lane] = pg_scan(s_u[lane], lane);
      s_n[lane] = pg_scan(s_n[lane], lane);
    }
    __syncthreads();
    if (start) {
      m.u0 = u_base + (warp ? s_u[warp - 1] : 0) + su - units;
      a.groups[n_base + (int)((warp ? s_n[warp - 1] : 0) + sn) - 1] = m;
    }
    u_base += s_u[31];
    n_base += (int)s_n[31];
  }
  __syncthreads();
  // starts: the CTA boundaries that fall into each group
  const long long total = u_base;
  long long want = total / kPgMinUnits;
  const int n = total == 0 ? 0 : (int)(want < 1 ? 1 : (want < a.n_cta ? want : a.n_cta));
  for (int g = tid; g < n_base; g += kPgPlanThreads) {
    const PgGroup m = a.groups[g];
    const int len = m.n_tiles + kPgUnitTail;
    const long long u1 = m.u0 + (long long)a.n_hg * len;
    for (long long c = (m.u0 * n + total - 1) / total; c < n; ++c) {
      const long long u = total * c / n;
      if (u >= u1) break;
      int hg = (int)((u - m.u0) / len), off = (int)((u - m.u0) % len), gg = g;
      if (off > 0 && off >= m.n_tiles) {  // in the group's tail: the next one
        off = 0;
        if (++hg == a.n_hg) {
          hg = 0;
          ++gg;
        }
      }
      a.start[c] = make_int4(gg, hg, off, 0);
    }
  }
  for (int c = n + tid; c <= kPgMaxCtas; c += kPgPlanThreads)
    a.start[c] = make_int4(n_base, 0, 0, 0);
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

// ------------------------------------------------------------- the attention
constexpr int kPR = 64;                       // rows per CTA
constexpr int kPWG = 4;                       // softmax warpgroups
constexpr int kPRW = kPR / kPWG;              // rows per warpgroup
constexpr int kPCtl = 4;                      // control warps
constexpr int kPThreads = 32 * kPCtl + 128 * kPWG;
constexpr int kPSlots = 7;                    // ring slots
constexpr int kPSlot = 128 * 128;             // [128 keys x 128 channels]
constexpr int kPRope = 128 * 64;
constexpr int kPQBlock = 2 * kPR * 128;       // one 128-channel block of [h; l]
constexpr int kPQBytes = 4 * kPQBlock + 2 * kPR * 64;
constexpr int kPPBytes = 128 * kPR;           // one part of P^T
constexpr int kPParts = 3;
constexpr uint32_t kPTmemCols = 512;          // S^T 2 x 128, O^T 256

struct PgCtrl {
  uint64_t full[kPSlots], empty[kPSlots];
  uint64_t rope_full, rope_empty;
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, p_free;
  uint64_t q_full, q_free;
  uint64_t o_full, o_free;
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort;
  int bflag[kPWG][2];
  int move[kPWG];        // tile + 1 of the last move of a reference
  int rlo[kPR], rhi[kPR];
  int tok[kPR];          // global token of a row, or -1
  alignas(16) float qf[kPR];
  alignas(16) float m_ref[kPR];
  alignas(16) float alpha[kPR];
  alignas(16) float inv[kPR];
  float m_hi[kPR];
  float red[kPWG][4][kPRW];
};
constexpr int kPSmem = 1024 + kPQBytes + kPParts * kPPBytes + kPRope + kPSlots * kPSlot +
                       (int)sizeof(PgCtrl);
static_assert(kPSmem <= 232448, "shared memory budget");

__device__ __forceinline__ void pg_drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
  }
}

// Two fp16 less their upper bytes (an E5M2 each, cut): exact.
__device__ __forceinline__ uint32_t f16x2_minus_upper(uint32_t h2) {
  const uint32_t up = h2 & 0xFF00FF00u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h2),
                            *reinterpret_cast<const __half2 *>(&up));
  return *reinterpret_cast<const uint32_t *>(&d);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// {h, l} of two channels: h = E4M3(x), l = E4M3(16 (x - h)), two codes each
__device__ __forceinline__ uint2 split_q(float x0, float x1) {
  const uint32_t h = e4m3x2(x0, x1);
  const uint32_t b = e4m3x2_to_f16x2((uint16_t)h);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&b));
  return make_uint2(h, e4m3x2(16.f * (x0 - f.x), 16.f * (x1 - f.y)));
}
// 2^e for the stored exponent e + 127
__device__ __forceinline__ float pg_pow2(int stored) {
  return stored == 0 ? 5.877471754e-39f : __int_as_float(stored << 23);
}

__global__ void __launch_bounds__(kPThreads, 1)
    paged_attn_kernel(const __grid_constant__ PagedArgs a,
                      const __grid_constant__ CUtensorMap tm_lat,
                      const __grid_constant__ CUtensorMap tm_rope) {
  if (a.start[blockIdx.x].x == a.start[blockIdx.x + 1].x &&
      a.start[blockIdx.x].y == a.start[blockIdx.x + 1].y &&
      a.start[blockIdx.x].z == a.start[blockIdx.x + 1].z)
    return;  // no tiles for this CTA
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sQ = smem;                       // 4 blocks [128 rows x 128], rope [128 rows x 64]
  uint8_t *sP = sQ + kPQBytes;              // three parts of P^T: [128 keys x 64 rows]
  uint8_t *sRope = sP + kPParts * kPPBytes;  // [128 keys x 64]
  uint8_t *sRing = sRope + kPRope;
  PgCtrl &c = *reinterpret_cast<PgCtrl *>(sRing + kPSlots * kPSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kPSlots; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.s_free[s], 128 * kPWG);
    }
    mbar_init(&c.rope_full, 1);
    mbar_init(&c.rope_empty, 1);
    mbar_init(&c.p_full, 128 * kPWG);
    mbar_init(&c.p_free, 2);
    mbar_init(&c.q_full, 128 * kPWG);
    mbar_init(&c.q_free, 1);
    mbar_init(&c.o_full, 2);
    mbar_init(&c.o_free, 128 * kPWG);
    for (int s = 0; s < 3; ++s) mbar_init(&c.drain[s], 1);
    c.abort = 0;
    for (int g = 0; g < kPWG; ++g) c.move[g] = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&c.tmem_base, kPTmemCols);
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&tm_lat);
    tma_prefetch_desc(&tm_rope);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  const uint32_t tO = tmem + 4 * kPR;  // S^T buffer b at tmem + 2 R b; O^T chunk ch at tO + R ch
  volatile int *abort = &c.abort;
  PgWalk w(a, blockIdx.x);

  if (warp == 0) {
    // ------------------------------------------------------ score-GEMM issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_e4m3(128, 2 * kPR, 0, 0);
      const uint64_t dq = smem_desc(smem_u32(sQ), 16, 1024, kSwz128);
      const uint64_t dqr = smem_desc(smem_u32(sQ + 4 * kPQBlock), 16, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), 16, 1024, kSwz128);
      const uint64_t drr = smem_desc(smem_u32(sRope), 16, 512, kSwz64);
      bool ok = true;
      uint32_t j = 0, piece = 0, slot = 0, par = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        if (!mbar_wait(&c.q_full, piece & 1, abort, a.status)) {
          ok = false;
          break;
        }
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          const uint32_t b = j & 1;
          if ((j >= 2 && !mbar_wait(&c.s_free[b], ((j >> 1) - 1) & 1, abort, a.status)) ||
              !mbar_wait(&c.rope_full, j & 1, abort, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dS = tmem + b * 2 * kPR;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma_f8_ss(dS, drr + ((k * 32) >> 4), dqr + ((k * 32) >> 4), id, k);
          mma_commit(&c.rope_empty);
          for (int ch = 0; ch < 4; ++ch) {
            if (!mbar_wait(&c.full[slot], par, abort, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = dr + ((slot * kPSlot) >> 4), db = dq + ((ch * kPQBlock) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_ss(dS, da + ((k * 32) >> 4), db + ((k * 32) >> 4), id, 1u);
            if (++slot == kPSlots) {
              slot = 0;
              par ^= 1;
            }
          }
          if (!ok) break;
          mma_commit(&c.s_full[b]);
        }
        if (ok) mma_commit(&c.q_free);
        ++piece;
      }
      if (!ok) {
        mma_commit(&c.drain[0]);
        pg_drain(&c.drain[0], 0);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------ PV-GEMM issuers
    if (lane == 0) {
      const int me = warp - 1;
      constexpr uint32_t id = idesc_e4m3_e5m2(128, kPR, 1, 1);
      const uint64_t dp = smem_desc(smem_u32(sP), kPPBytes, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), kPSlot, 1024, kSwz128);
      bool ok = true;
      uint32_t j = 0, piece = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        if (piece > 0 && !mbar_wait(&c.o_free, (piece - 1) & 1, abort, a.status)) {
          ok = false;
          break;
        }
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          if (!mbar_wait(&c.p_full, j & 1, abort, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ch = me + 2 * i;
            const uint32_t slot = (4 * j + ch) % kPSlots;
            const uint64_t da = dr + ((slot * kPSlot) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int y = 0; y < kPParts; ++y)
                mma_f8_ss(tO + ch * kPR, da + ((k * 4096) >> 4),
                          dp + ((y * kPPBytes + k * 32 * kPR) >> 4), id,
                          (t > w.t0 || k > 0 || y > 0) ? 1u : 0u);
            }
            mma_commit(&c.empty[slot]);
          }
          mma_commit(&c.p_free);
        }
        if (ok) mma_commit(&c.o_full);
        ++piece;
      }
      if (!ok) {
        mma_commit(&c.drain[1 + me]);
        pg_drain(&c.drain[1 + me], 0);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------ loads
    // lane p < 128 / block_size: page p of the tile
    const int bs = 1 << a.shift, ppt = 128 >> a.shift;
    bool ok = true;
    uint32_t j = 0, slot = 0, use = 0, ropes = 0;
    while (ok && w.next(a)) {
      const int32_t *row = a.table + (int64_t)w.m.req * a.stride;
      auto page = [&](int t) {
        const int p0 = (w.m.t_lo + t) * 128 + lane * bs;
        if (lane >= ppt || t >= w.t1 || p0 > w.m.hi_max || p0 + bs <= w.m.lo_min) return -1;
        const int blk = row[p0 >> a.shift];
        return blk >= 0 && blk < a.n_blocks ? blk : -1;
      };
      int nxt = page(w.t0);
      for (int t = w.t0; t < w.t1 && ok; ++t, ++j) {
        const int blk = nxt;
        nxt = page(t + 1);
        const int np = __popc(__ballot_sync(0xffffffffu, blk >= 0));
        const int y = blk << a.shift;
        for (int ch = -1; ch < 4; ++ch) {
          uint64_t *fb = ch < 0 ? &c.rope_full : &c.full[slot];
          int good = 1;
          if (lane == 0) {
            if (ch < 0)
              good = j < 1 || mbar_wait(&c.rope_empty, (j - 1) & 1, abort, a.status);
            else
              good = use == 0 || mbar_wait(&c.empty[slot], (use - 1) & 1, abort, a.status);
            if (good) mbar_arrive_expect_tx(fb, (uint32_t)(np * bs * (ch < 0 ? 64 : 128)));
          }
          good = __shfl_sync(0xffffffffu, good, 0);
          if (!good) {
            ok = false;
            break;
          }
          if (blk >= 0) {
            if (ch < 0)
              tma_load_2d(sRope + lane * bs * 64, &tm_rope, CPMLA_DV, y, fb);
            else
              tma_load_2d(sRing + slot * kPSlot + lane * bs * 128, &tm_lat, ch * 128, y, fb);
          }
          __syncwarp();
          if (ch < 0) ++ropes;
          if (ch >= 0 && ++slot == kPSlots) {
            slot = 0;
            ++use;
          }
        }
      }
    }
    // the copies of the last uses have landed before the CTA exits
    if (!ok && lane == 0) {
      const uint32_t n = use * kPSlots + slot;
      for (uint32_t i = n > kPSlots ? n - kPSlots : 0; i < n; ++i)
        pg_drain(&c.full[i % kPSlots], (i / kPSlots) & 1);
      if (ropes > 0) pg_drain(&c.rope_full, (ropes - 1) & 1);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ softmax, output
    const int sw = warp - kPCtl, wg = sw >> 2, q4 = warp & 3;
    const int t = q4 * 32 + lane;  // key of a tile, channel of an O^T chunk
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int cb = wg * kPRW;
    const int bar = 1 + wg;
    int seq = 0;
    bool ok = true;
    uint32_t j = 0, piece = 0;
    while (ok && w.next(a)) {
      const int r_valid = w.m.count * a.hc, h0 = w.hg * a.hc;
      const int32_t *row = a.table + (int64_t)w.m.req * a.stride;
      const bool some = w.t1 > w.t0;
      // this warpgroup's threads are done with the previous piece's rows (a
      // warpgroup keeps to its own rows, so no barrier spans two of them)
      named_bar_sync(bar, 128);
      if (some && piece > 0 &&
          !group_wait(&c.q_free, (piece - 1) & 1, t, bar, c.bflag[wg], seq, abort, a.status)) {
        ok = false;
      }
      // Q: warp sw takes rows 4 sw .. 4 sw + 3; channels 4 (lane + 32 i) ..
      if (ok) {
#pragma unroll 1
        for (int rr = 0; rr < kPR / (4 * kPWG); ++rr) {
          const int r = sw * (kPR / (4 * kPWG)) + rr;
          const int l = r / a.hc, hh = r - l * a.hc;
          const bool there = r < r_valid;
          uint2 v[5];
          int tok = -1;
          if (there) {
            const int i = w.m.first + l;
            tok = a.tokens ? a.tokens[i] : i;
            if (lane == 0) {
              c.rlo[r] = a.kv_lo ? max(a.kv_lo[i], 0) : 0;
              c.rhi[r] = a.kv_hi ? min(a.kv_hi[i], a.pos[i]) : a.pos[i];
            }
          } else if (lane == 0) {
            c.rlo[r] = 1;
            c.rhi[r] = 0;
          }
          const uint2 *src = reinterpret_cast<const uint2 *>(
              a.q + (int64_t)(there ? tok : 0) * a.q_stride + (int64_t)(h0 + hh) * CPMLA_DQK);
          uint32_t mx = 0;
          bool fin = true;
#pragma unroll
          for (int i = 0; i < 5; ++i) {
            v[i] = make_uint2(0, 0);
            if (there && some && (i < 4 || lane < 16)) v[i] = __ldg(src + lane + 32 * i);
            const uint32_t x[4] = {v[i].x << 16, v[i].x & 0xFFFF0000u, v[i].y << 16,
                                   v[i].y & 0xFFFF0000u};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ab = x[k] & 0x7FFFFFFFu;
              if (ab >= 0x7F800000u)
                fin = false;
              else
                mx = max(mx, ab);
            }
          }
          mx = __reduce_max_sync(0xffffffffu, mx);
          fin = __all_sync(0xffffffffu, fin);
          // 2^ae: the largest channel in (224, 448] (ae >= -100: smaller rows
          // keep fewer bits)
          int ae = (int)(mx >> 23) - 127 - ((mx & 0x7FFFFFu) > 0x600000u ? 7 : 8);
          ae = ae < -100 ? -100 : ae;
          const float down = __int_as_float((127 - ae) << 23);
          if (lane == 0) {
            // a row with an infinite or NaN channel is NaN throughout
            c.qf[r] = there ? (fin ? __int_as_float((127 + ae) << 23) * a.scale_log2 : NAN) : 0.f;
            c.tok[r] = tok;
            c.m_ref[r] = there ? -INFINITY : 1e30f;  // rows of no token get weight 0
            c.m_hi[r] = -INFINITY;
            c.alpha[r] = 1.f;
          }
          if (some) {
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              if (i == 4 && lane >= 16) break;
              const uint2 p0 = split_q(__uint_as_float(v[i].x << 16) * down,
                                       __uint_as_float(v[i].x & 0xFFFF0000u) * down);
              const uint2 p1 = split_q(__uint_as_float(v[i].y << 16) * down,
                                       __uint_as_float(v[i].y & 0xFFFF0000u) * down);
              const uint32_t hi = p0.x | (p1.x << 16), lo = p0.y | (p1.y << 16);
              if (i < 4) {
                // channels 128 i + 4 lane ..: block i, byte 4 lane of the row
                const int off = i * kPQBlock + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
                *reinterpret_cast<uint32_t *>(sQ + off + r * 128) = hi;
                *reinterpret_cast<uint32_t *>(sQ + off + (kPR + r) * 128) = lo;
              } else {
                const int off =
                    4 * kPQBlock + (((lane >> 2) ^ ((r >> 1) & 3)) << 4) + (lane & 3) * 4;
                *reinterpret_cast<uint32_t *>(sQ + off + r * 64) = hi;
                *reinterpret_cast<uint32_t *>(sQ + off + (kPR + r) * 64) = lo;
              }
            }
          }
        }
        fence_proxy_async_smem();
        if (some) mbar_arrive(&c.q_full);
      }
      named_bar_sync(bar, 128);
      if (!ok) break;

      // key t of tile x: its block's stored exponent, or -1 when no row of the
      // group may see it; the block of the next tile's key is fetched a tile
      // ahead of its exponent
      auto block_at = [&](int x) {
        const int p = (w.m.t_lo + x) * 128 + t;
        if (x >= w.t1 || p < w.m.lo_min || p > w.m.hi_max) return -1;
        const int blk = row[p >> a.shift];
        if (blk < 0 || blk >= a.n_blocks) {
          record_status(a.status, CPMLA_ERR_INDEX);
          return -1;
        }
        return blk;
      };
      auto exp_of_block = [&](int blk) { return blk >= 0 ? min((int)__ldg(a.exp + blk), 254) : -1; };
      float l_part[kPRW];
#pragma unroll
      for (int r = 0; r < kPRW; ++r) l_part[r] = 0.f;
      int e_cur = exp_of_block(block_at(w.t0));
      int b_nxt = block_at(w.t0 + 1);
      for (int x = w.t0; x < w.t1; ++x, ++j) {
        const int e_nxt = exp_of_block(b_nxt);
        b_nxt = block_at(x + 2);
        const uint32_t sb = j & 1;
        if (!group_wait(&c.s_full[sb], (j >> 1) & 1, t, bar, c.bflag[wg], seq, abort, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[kPRW];
        {
          float lo[kPRW];
          tmem_ld16(tmem + sb * 2 * kPR + lane_off + cb, s);
          tmem_ld16(tmem + sb * 2 * kPR + lane_off + kPR + cb, lo);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < kPRW; ++r) s[r] = fmaf(lo[r], 0.0625f, s[r]);
        }
        tc_fence_before();
        mbar_arrive(&c.s_free[sb]);
        const float kf = e_cur >= 0 ? pg_pow2(e_cur) : 0.f;
        const float ku = (float)(e_cur - 127);
        const int p = (w.m.t_lo + x) * 128 + t;
        const bool open = p - t >= w.m.lo_max && p - t + 127 <= w.m.hi_min &&
                          __all_sync(0xffffffffu, e_cur >= 0);
        bool nan = false;
        if (!open) {
#pragma unroll
          for (int r = 0; r < kPRW; ++r) nan |= s[r] != s[r];
        }
#pragma unroll
        for (int r = 0; r < kPRW; r += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(&c.qf[cb + r]);
          s[r] = fmaf(s[r] * kf, f.x, ku);
          s[r + 1] = fmaf(s[r + 1] * kf, f.y, ku);
          s[r + 2] = fmaf(s[r + 2] * kf, f.z, ku);
          s[r + 3] = fmaf(s[r + 3] * kf, f.w, ku);
        }
        if (!open) {
#pragma unroll
          for (int r = 0; r < kPRW; ++r)
            if (e_cur < 0 || p < c.rlo[cb + r] || p > c.rhi[cb + r]) s[r] = -INFINITY;
          if (nan) {
            // NaN codes in a key that not every row may see: weight zero times
            // NaN would reach the others, so the key's values become zero (a
            // row that does see it has a NaN weight)
            bool found = false;
            for (int ch = 0; ch < 4; ++ch) {
              const uint32_t *kr = reinterpret_cast<const uint32_t *>(
                  sRing + ((4 * j + ch) % kPSlots) * kPSlot + t * 128);
              for (int i = 0; i < 32; ++i) {
                const uint32_t v = ~kr[i] & 0x7F7F7F7Fu;  // a zero byte: a NaN code
                found |= ((v - 0x01010101u) & ~v & 0x80808080u) != 0;
              }
            }
            if (found)
              for (int ch = 0; ch < 4; ++ch)
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4 *>(sRing + ((4 * j + ch) % kPSlots) * kPSlot + t * 128 +
                                             i * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        {
          float v[kPRW];
#pragma unroll
          for (int r = 0; r < kPRW; ++r) v[r] = s[r];
          warp_transpose_reduce<kPRW, true>(v, lane);
          if ((lane & 1) == 0) c.red[wg][q4][lane >> 1] = v[0];
        }
        named_bar_sync(bar, 128);
        if (t < kPRW) {
          const int r = cb + t;
          const float tm = fmaxf(fmaxf(c.red[wg][0][t], c.red[wg][1][t]),
                                 fmaxf(c.red[wg][2][t], c.red[wg][3][t]));
          const float m_old = c.m_ref[r];
          float m_new = m_old;
          if (r < r_valid && tm > -INFINITY) {
            const float m_hi = fmaxf(c.m_hi[r], tm);
            c.m_hi[r] = m_hi;
            const float d = tm - m_old;  // +inf at a row's first key
            if (d > 15.75f)
              m_new = tm - 10.f;
            else if (d < 4.f)
              m_new = fminf(m_old, fmaxf(tm, m_hi - 60.f) - 10.f);
          }
          c.alpha[r] = m_old == -INFINITY ? 0.f : fast_exp2(m_old - m_new);
          c.m_ref[r] = m_new;
          if (m_new != m_old) c.move[wg] = (int)j + 1;
        }
        named_bar_sync(bar, 128);
        const bool moved = c.move[wg] == (int)j + 1;
        if (moved) {
#pragma unroll
          for (int r = 0; r < kPRW; ++r)
            l_part[r] = l_part[r] == 0.f ? 0.f : l_part[r] * c.alpha[cb + r];
        }
        // p as fp16 bits, split by cutting: an E5M2 is the upper byte of an fp16,
        // so each part is the upper byte of what is left (nothing is negative);
        // the last part is rounded
        uint32_t part[kPParts][kPRW / 4];
        const float kd = e_cur >= 0 ? pg_pow2(254 - e_cur) : 0.f;  // 2^-e
#pragma unroll
        for (int r = 0; r < kPRW; r += 4) {
          const float4 m4 = *reinterpret_cast<const float4 *>(&c.m_ref[cb + r]);
          const float m[4] = {m4.x, m4.y, m4.z, m4.w};
          float pv[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            pv[y] = fast_exp2(s[r + y] - (m[y] == -INFINITY ? 0.f : m[y]));
            l_part[r + y] = fmaf(pv[y], kd, l_part[r + y]);
          }
          uint32_t a0 = pack_f16x2(pv[0], pv[1]), a1 = pack_f16x2(pv[2], pv[3]);
#pragma unroll
          for (int y = 0; y < kPParts; ++y) {
            if (y == kPParts - 1) {
              a0 += 0x00800080u;
              a1 += 0x00800080u;
            }
            part[y][r / 4] = __byte_perm(a0, a1, 0x7531);
            if (y < kPParts - 1) {
              a0 = f16x2_minus_upper(a0);
              a1 = f16x2_minus_upper(a1);
            }
          }
        }
        // the PV GEMM of the tile before is done with P^T and O^T
        if (j >= 1 &&
            !group_wait(&c.p_free, (j - 1) & 1, t, bar, c.bflag[wg], seq, abort, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (moved && x > w.t0) {
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            float o[kPRW];
            const uint32_t col = tO + lane_off + ch * kPR + cb;
            tmem_ld16(col, o);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < kPRW; ++r) o[r] = o[r] == 0.f ? 0.f : o[r] * c.alpha[cb + r];
            tmem_st16(col, o);
          }
          tmem_st_wait();
        }
        uint8_t *pr = sP + t * kPR + ((wg ^ ((t >> 1) & 3)) << 4);
#pragma unroll
        for (int y = 0; y < kPParts; ++y)
          *reinterpret_cast<uint4 *>(pr + y * kPPBytes) =
              make_uint4(part[y][0], part[y][1], part[y][2], part[y][3]);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&c.p_full);
        e_cur = e_nxt;
      }
      if (!ok) break;
      // ---------------------------------------------- this piece's output
      const bool whole = w.whole();
      if (some && !group_wait(&c.o_full, piece & 1, t, bar, c.bflag[wg], seq, abort, a.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      warp_transpose_reduce<kPRW, false>(l_part, lane);
      if ((lane & 1) == 0) c.red[wg][q4][lane >> 1] = l_part[0];
      named_bar_sync(bar, 128);
      const int part = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      if (t < kPRW) {
        const int r = cb + t;
        const float l = (c.red[wg][0][t] + c.red[wg][1][t]) + (c.red[wg][2][t] + c.red[wg][3][t]);
        const float m = c.m_ref[r];
        const bool empty = m == -INFINITY && l == 0.f;  // l may be NaN
        const float l2 = empty ? -INFINITY : m + log2f(l);
        float f = empty ? 0.f : 1.f / l;
        if (r < r_valid) {
          if (whole) {
            const int hh = h0 + r % a.hc;
            const float L = l2 * 0.69314718055994530942f;
            f *= sink_factor(a.sink, hh, L);
            a.lse[(int64_t)c.tok[r] * a.H + hh] = L;
          } else {
            a.lse_part[(int64_t)part * kPR + r] = l2;
          }
        }
        c.inv[r] = f;
      }
      named_bar_sync(bar, 128);
      const bool odd = (lane & 1) != 0;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        float o[kPRW];
        if (some) {
          tmem_ld16(tO + lane_off + ch * kPR + cb, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int r = 0; r < kPRW; ++r) o[r] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kPRW; ++r) {
          const float f = c.inv[cb + r];
          o[r] = f == 0.f ? 0.f : o[r] * f;
        }
        if (whole) {
          // lane pairs trade one value: the even lane stores row r at channels
          // t, t + 1, the odd lane row r + 1 at t - 1, t
#pragma unroll
          for (int r = 0; r < kPRW; r += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? o[r] : o[r + 1], 1);
            const int y = cb + r + (odd ? 1 : 0);
            if (y < r_valid)
              *reinterpret_cast<uint32_t *>(
                  a.o + ((int64_t)c.tok[y] * a.H + h0 + y % a.hc) * CPMLA_DV + ch * 128 +
                  (t & ~1)) = odd ? pack_bf16x2(got, o[r + 1]) : pack_bf16x2(o[r], got);
          }
        } else {
#pragma unroll
          for (int r = 0; r < kPRW; ++r)
            if (cb + r < r_valid)
              a.o_part[((int64_t)part * kPR + cb + r) * CPMLA_DV + ch * 128 + t] = o[r];
        }
      }
      tc_fence_before();
      if (some) {
        mbar_arrive(&c.o_free);
        ++piece;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kPTmemCols);
  }
}

// ------------------------------------------------------------------ the join
// Boundary c = blockIdx.x + 1 of the plan: if it is the first that cuts its
// group, rows 4 blockIdx.y .. + 3 of the group are joined from their parts, in
// CTA order.
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedArgs a) {
  const int c0 = blockIdx.x + 1, t = threadIdx.x;
  const int4 s = a.start[c0], p = a.start[c0 - 1];
  if (s.z == 0 || (p.x == s.x && p.y == s.y && p.z > 0)) return;
  const PgGroup m = a.groups[s.x];
  int n = 1;  // parts: 2 c0 - 1, then 2 c0, 2 (c0 + 1), ...
  while (c0 + n <= a.n_cta) {
    const int4 x = a.start[c0 + n];
    if (x.x != s.x || x.y != s.y || x.z == 0) break;
    ++n;
  }
  for (int rr = 0; rr < 4; ++rr) {
    const int r = blockIdx.y * 4 + rr;
    if (r >= m.count * a.hc) return;
    auto part = [&](int i) { return (int64_t)(i == 0 ? 2 * c0 - 1 : 2 * (c0 + i - 1)) * kPR + r; };
    float mx = -INFINITY;
    for (int i = 0; i <= n; ++i) mx = fmaxf(mx, a.lse_part[part(i)]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i <= n; ++i) {
      const float li = a.lse_part[part(i)];
      if (li == -INFINITY) continue;
      const float wt = exp2f(li - mx);
      l += wt;
      const float4 v = reinterpret_cast<const float4 *>(a.o_part + part(i) * CPMLA_DV)[t];
      o.x = fmaf(wt, v.x, o.x);
      o.y = fmaf(wt, v.y, o.y);
      o.z = fmaf(wt, v.z, o.z);
      o.w = fmaf(wt, v.w, o.w);
    }
    const int i = m.first + r / a.hc, h = s.y * a.hc + r % a.hc;
    const int64_t tok = a.tokens ? a.tokens[i] : i;
    const bool empty = mx == -INFINITY && l == 0.f;  // l may be NaN
    const float L = empty ? -INFINITY : (mx + log2f(l)) * 0.69314718055994530942f;
    const float f = empty ? 0.f : sink_factor(a.sink, h, L) / l;
    reinterpret_cast<uint2 *>(a.o + (tok * a.H + h) * CPMLA_DV)[t] =
        make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    if (t == 0) a.lse[tok * a.H + h] = L;
  }
}

// Workspace sections, each 256-byte aligned.
struct PgLayout {
  size_t start, groups, o, lse, total;
};
PgLayout pg_layout(int n) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PgLayout L{};
  L.groups = up((kPgMaxCtas + 1) * sizeof(int4));
  L.lse = L.groups + up((size_t)n * sizeof(PgGroup));
  L.o = L.lse + up((size_t)2 * kPgMaxCtas * kPR * 4);
  L.total = L.o + (size_t)2 * kPgMaxCtas * kPR * CPMLA_DV * 4;
  return L;
}

}  // namespace
}  // namespace cpmla

extern "C" size_t mla_paged_attn_workspace_size(int H, int n_tokens) {
  if (H < 1 || H > 128 || n_tokens < 0) return 0;
  return cpmla::pg_layout(n_tokens).total;
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
  a.hc = H <= 64 ? H : 64;
  a.g = kPR / a.hc;
  a.n_hg = H / a.hc;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_attn: device");
  a.n_cta = sms < kPgMaxCtas ? sms : kPgMaxCtas;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const PgLayout L = pg_layout(n_tokens);
  a.start = reinterpret_cast<int4 *>(ws + L.start);
  a.groups = reinterpret_cast<PgGroup *>(ws + L.groups);
  a.lse_part = reinterpret_cast<float *>(ws + L.lse);
  a.o_part = reinterpret_cast<float *>(ws + L.o);
  // the cache as [slots, 576] bytes in boxes of one block x 128 latent or the
  // 64 rope channels, swizzled as the MMA reads them
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(CPMLA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {
    memset(&tm[i], 0, sizeof tm[i]);
    cuuint64_t dims[2] = {CPMLA_DQK, (cuuint64_t)n_blocks * block_size};
    cuuint64_t strides[1] = {CPMLA_DQK};
    cuuint32_t box[2] = {i == 0 ? 128u : 64u, (cuuint32_t)block_size};
    cuuint32_t estr[2] = {1, 1};
    const CUresult cr =
        enc(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(cache), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            i == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (cr != CUDA_SUCCESS)
      return fail(CPMLA_ERR_CUDA, "%s: tensor map encode failed (%d)", fn, (int)cr);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
  if (e != cudaSuccess) return cuda_fail(e, "mla_paged_attn: set shared memory size");
  paged_plan_kernel<<<1, kPgPlanThreads, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "mla_paged_attn: plan launch");
  paged_attn_kernel<<<a.n_cta, kPThreads, kPSmem, st>>>(a, tm[0], tm[1]);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "mla_paged_attn: launch");
  if (a.n_cta > 1) {
    paged_join_kernel<<<dim3(a.n_cta - 1, kPR / 4), 128, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "mla_paged_attn: join launch");
  }
  return CPMLA_OK;
}
