// paged4_attn.cu -- attention of listed tokens over the paged 4-bit latent cache
// (mla_paged4_attn): prompt chunks and single tokens in one list.
//
// E2M1 x 2^(6 - d) with d <= 11 is an E4M3 without rounding, so a tile of 64 keys is
// expanded in shared memory into E4M3 codes c_j on the token's own scale 2^e_j, and the
// products are those of the 8-bit cache.  With q = 2^a (h + l / 16), h and l E4M3 vectors,
//   t_j = scale log2(e) 2^(a + e_j) (h . c_j + l . c_j / 16),  u_j = t_j + e_j
//   o = sum 2^(u_j - m) c_j / sum 2^(t_j - m)
//   S = [h; l] . C^T     q (2R lanes) in TMEM, N = 64 keys, K = 576 (kind::f8f6f4)
//   O^T += C^T . P^T     M = 128 channels x 4, N = R a part of P, K = 64 keys
//                        (kind::mxf8f6f4)
// A weight is two E4M3, p' = h + l with p' = 2^(u - sub) at most 2^8 for the largest of 32
// keys of a row, on a scale 2^(sub - m) that the MMA takes for each row and 32 keys: 8
// significant bits and 2^-17 of that largest, with 16 MMAs where the 8-bit kernel's three
// E5M2 (a range for a whole tile) take 24.
//
// A piece of work is R = 16 or 64 rows (tokens of one request x heads) and a range of their
// keys, as the plan cuts them.  Warps: 0 and 1 (R = 16: 2 too)
// issue the MMAs, 3 loads, 4-11 do the softmax and
// the output, 12-15 bring q in, 16-23 expand.  Every wait is bounded; on expiry the CTA
// records CPMLA_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
//
// What bounds it, measured (32 tokens of 4,096 to 131,072 keys).  R = 16: 185 us a call
// with 16 heads, 3.6 TB/s (the 8-bit cache's 222, 5.1 TB/s); R = 64: 266 us with 64 heads,
// 1.04 PFLOP/s of the exact products (271).  A tile takes 1,700 and 2,500 cycles.  Shared
// memory is busy for 1,300 and 1,900 of them, the tensor core for 800 and 1,300, and a
// scheduler issues 1,250 and 1,550 instructions, half of them of the pipe that takes one
// every two cycles (the expansion alone 730 cycles).  None of these fills the time: a tile
// keeps its place in the ring for the chain of its expansion, scores, softmax and PV, 8,300
// and 9,700 cycles, and there are places for 5 and 4.  8,192 prompt tokens of 16 heads
// 1,184 us (1,151).  On the way here: the roles' loops have to fit the instruction cache
// together (a softmax loop with 32 keys side by side instead of 16: 680 us for the 64
// heads); a wait by one lane leaves its warp apart, and what follows is issued twice (484,
// 398); a tile's MMAs behind one election (266, 325 with one for each); a reference that
// next to never moves (257, 394 with moves beyond 28); strips taken into registers at once,
// by two groups of warps in turn.
#include <type_traits>

#include "paged4.cuh"
#include "paged_attn.cuh"

namespace cpmla {
namespace {

constexpr int kP4Threads = 768;   // warpgroups: control, two softmax, q, two that expand
constexpr int kP4Tile = 4 * kPgSlot;              // ring slot: a tile's latent chunks
constexpr int kP4Pack = kPgTile / 16 * kStrip;    // a tile's strips
// Registers a thread by warpgroup, dealt out anew from the 80 that 768 threads are
// launched with: a tile's scores of a thread are 32, a strip's share 48.
constexpr int kP4Regs = 80, kP4RegsCtl = 48, kP4RegsSoftmax = 112, kP4RegsQ = 64, kP4RegsX = 72;
static_assert(kP4RegsCtl + 2 * kP4RegsSoftmax + kP4RegsQ + 2 * kP4RegsX <= 6 * kP4Regs,
              "shares of what the block is launched with");

template <int R>
struct P4Cfg {
  static constexpr int kPart = R * kPgTile;  // one part of P: [R rows x 64 keys]
  static constexpr int kP = 2 * kPart;
  // R = 16: both parts of P side by side in one PV MMA, with accumulators of their own
  static constexpr int kWide = R == 16 ? 2 : 1;
  static constexpr int kOW = R * kWide;  // columns of an O^T chunk
  // Issuers of the scores: with 16 rows two, for the even and the odd tiles (184 us for 32
  // tokens of 16 heads, 189 with one); with 64 rows one (260 us with 64 heads, 266 with two
  // for PV beside it).
  static constexpr int kQkW = R == 64 ? 1 : 2;
  // R = 16: q lies in each quarter of the lanes, so that any warp has the scores of all
  // rows: two of a softmax warpgroup take 32 of the tile's keys each, others than the
  // other warpgroup's, so that every scheduler has one (189 us for the 32 tokens of 16
  // heads; 191 with the same two, and with one warp a tile 276 where this was 228).
  static constexpr bool kSplit = R == 16;
  static constexpr int kLanes = kSplit ? 2 * R : R;  // rows and their copies
  static constexpr int kLive = kLanes / 16;          // warps of a warpgroup that have rows
  // q's steps of 32 channels in TMEM (64 rows leave columns for 15; an even number is less
  // code), and the rest in shared memory: [2R lanes x 64] a pair of steps
  static constexpr int kQSteps = R == 64 ? 14 : 18;
  static constexpr int kQPair = 2 * R * 64, kQRest = (18 - kQSteps) / 2 * kQPair;
  // TMEM columns behind q's: the scales of the values (1, four columns) and of the weights
  // (four for even and for odd tiles; rows 32 x .. 32 x + 31 in column x, in each quarter
  // of the lanes); two S buffers; O^T
  static constexpr int kColScale = 8 * kQSteps;
  static constexpr int kColS = (kColScale + 12 + 15) / 16 * 16;
  static constexpr int kColO = kColS + 2 * kPgTile;
  static_assert(kColO + 4 * kOW <= (int)kPgTmemCols, "TMEM columns");
  // places for tiles, for the strips that are expanded into them, and for the tiles' rope,
  // which the PV GEMM does not hold (with it a tile fewer has room)
  static constexpr int kSlots = R == 16 ? 5 : 4, kPacks = 2, kRopes = 3;
  static constexpr int kFixed = kQRest + 2 * kP + kSlots * kP4Tile + kRopes * kPgRope +
                                kPacks * kP4Pack;
};
// 2^e, e and 2^-e of a tile's keys (the upper half moved by 16 bytes: two threads' loads
// of 32 keys apart share no bank), and its groups of 16 keys that have a page.
constexpr int kP4High = 26;
__host__ __device__ constexpr int p4_key(int k) { return k + (k >> 5) * 4; }
struct P4KeyScale {
  float up[p4_key(kPgTile)], e[p4_key(kPgTile)], down[p4_key(kPgTile)];
  alignas(8) uint32_t there;
  uint8_t high[4];  // a strip has a token of e > kP4High
  uint32_t pad[2];
};

template <int R>
struct P4Ctrl {
  using Cfg = P4Cfg<R>;
  // the scales of a buffer's weights as they are copied to TMEM: [row % 32][row / 32][32 keys]
  alignas(128) uint8_t sf[2][32][4][4];
  alignas(16) P4KeyScale ks[Cfg::kSlots];
  uint64_t full[Cfg::kSlots], empty[Cfg::kSlots];  // ring slots
  uint64_t pack_full[Cfg::kPacks], pack_empty[Cfg::kPacks], rope_free[Cfg::kRopes];
  // S and P have a buffer for each softmax warpgroup: even and odd tiles
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], p_free[2];
  uint64_t ref[4];  // a live warp's references of a tile are decided
  // for even and odd pieces, as a waiter may be a piece behind: q is in place; the
  // softmax is done with a piece, its output written
  uint64_t q_full[2], o_free[2];
  uint64_t q_free, o_full;
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort;
  uint32_t there[Cfg::kPacks];  // as in P4KeyScale
  float qf[2][R];  // a piece's scale of q row r, times softmax scale and log2 e
  float m_ref[Cfg::kLanes];
  float stat_l[2][Cfg::kLanes], stat_m[2][Cfg::kLanes];  // sums of 2^t, and their references
  alignas(16) float alpha[2][R];
  uint32_t mv[2][4];  // a live warp has a row whose reference moved
  // per softmax warp: a row's output factor (inv times inv2) and its row of the output
  // (-1: none)
  alignas(16) float inv[8][R / 2], inv2[8][R / 2];
  int64_t orow[8][R / 2];
};
template <int R>
constexpr int p4_smem() {
  return 1024 + P4Cfg<R>::kFixed + 128 + (int)sizeof(P4Ctrl<R>);
}
static_assert(p4_smem<64>() <= 232448 && p4_smem<16>() <= 232448, "shared memory budget");

// Now and then within a wait: when it was first seen here (t0, 0 at
// first), or 0 when it is to be given up, as mbar_wait does.  Out of line: its roles'
// loops fill the instruction cache, and a wait's twenty copies were a third of their code.
__device__ __noinline__ unsigned long long p4_keep_waiting(unsigned long long t0,
                                                           volatile int *abort, int *status) {
  if (*abort || *reinterpret_cast<volatile int *>(status) == CPMLA_ERR_TIMEOUT) {
    *abort = 1;
    return 0;
  }
  const unsigned long long t = global_timer_ns();
  if (t0 == 0) return t;
  if (t - t0 <= kWaitLimitNs) return t0;
  *abort = 1;
  record_status(status, CPMLA_ERR_TIMEOUT);
  return 0;
}
// Bounded wait of a warp, of all lanes (which may wait for barriers of their own) and with
// one exit of the loop for all of them.  Lanes that leave a loop or a branch by
// themselves do not come together again (__activemask() has 31 lanes, behind a
// __syncwarp() or a shuffle too), and what follows is issued twice.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          int *status) {
  unsigned long long t0 = 0;
  for (uint32_t it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it)
    if ((it & 63u) == 0) {
      t0 = p4_keep_waiting(t0, abort, status);
      if (__any_sync(0xffffffffu, t0 == 0)) return false;
    }
  return true;
}
// Two E4M3 of each of four fp16 x (pairs): E4M3(x), and E4M3 of what it leaves.
__device__ __forceinline__ uint32_t e4m3x4_of_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}"
      : "=r"(r)
      : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint2 split_p4(uint32_t x, uint32_t y) {
  const uint32_t h = e4m3x4_of_f16x2(x, y);
  return make_uint2(h, e4m3x4_of_f16x2(f16x2_sub(x, e4m3x2_to_f16x2((uint16_t)h)),
                                       f16x2_sub(y, e4m3x2_to_f16x2((uint16_t)(h >> 16)))));
}
// Weights have scales of their own and the sum of 2^t has a reference of its own,
// so that only O^T limits m: a row's m starts kP4Over above its first tile's largest u and
// moves when a tile's largest lies kP4Up above it; a sum of 2^30 values stays below
// 2^(30 + 9 + 80).  A tile's weights lose bits where its largest u lies 72 below the first
// tile's, and are 0 at 89: in a channel that the heavier tokens have, binary32 holds
// nothing of them either; in one where those are all zero they are lost.  m never goes
// down.  (With m 6 below the first tile's largest and moves 28 above it each row moves now
// and then, and every eighth tile of 64 rows waits for the PV GEMM: 394 us where this
// takes 257.)
constexpr float kP4Over = 40.f, kP4Up = 80.f;
// What a thread's n keys need in the tiles that few are: those of an open end, with a page
// that is not there, or with a value of 2^26 and more.  Out of line, as the roles' loops
// fill the instruction cache.
// u: position p .. of the keys; those outside lo .. hi, or in a group of 16 without a bit of
// there, become -inf (a group that the row attends to and that is not there is a bad one:
// between the ranges of two rows of a piece a block may be anything).  Returns the largest
// u.  Behind the n: the largest t = u - e, the sum of 2^(t - max), and 1 if a key that is
// left has e > kP4High.
__device__ __noinline__ float p4_rare(float *u, const float *e, int n, int p, int lo, int hi,
                                      uint32_t there, int *status) {
  float top = -INFINITY, t_max = -INFINITY, t_sum = 0.f;
  bool wide = false;
#pragma unroll 1
  for (int g = 0; g < n; g += 16) {
    const bool gone = ((there >> (g >> 4)) & 1) == 0;
    if (gone && max(lo, p + g) <= min(hi, p + g + 15)) record_status(status, CPMLA_ERR_INDEX);
    const int from = gone ? 16 : lo - p - g, to = hi - p - g;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const float v = i < from || i > to ? -INFINITY : u[g + i];
      u[g + i] = v;
      top = fmaxf(top, v);
      t_max = fmaxf(t_max, v - e[g + i]);
      wide |= v > -INFINITY && e[g + i] > (float)kP4High;
    }
  }
  u[n + 2] = wide ? 1.f : 0.f;
  u[n] = t_max;  // (-inf, no reference at all, where nothing is left)
  if (t_max == -INFINITY) t_max = 0.f;
  if (__any_sync(0xffffffffu, wide))
#pragma unroll 4
    for (int i = 0; i < n; ++i) t_sum += fast_exp2(u[i] - e[i] - t_max);
  u[n + 1] = t_sum;
  return top;
}
// The sum of 2^t and its reference behind a tile with wide exponents: of what they were
// ahead of it (l.x on l.y) and p4_rare's sum; else what they have become (d).
__device__ __noinline__ float2 p4_wide(const float *rare, float2 l, float2 d) {
  if (rare[2] == 0.f) return d;
  const float m = fmaxf(l.y, rare[0]);
  return make_float2(pg_scale(l.x, l.y - m) + pg_scale(rare[1], rare[0] - m), m);
}

template <int R>
__global__ void __launch_bounds__(kP4Threads, 1)
    paged4_attn_kernel(const __grid_constant__ PagedArgs a) {
  using Cfg = P4Cfg<R>;
  constexpr int NS = Cfg::kSlots, NP = Cfg::kPacks, NR = Cfg::kRopes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sQr = smem;                   // q's last steps
  uint8_t *sP = sQr + Cfg::kQRest;       // two P of two parts
  uint8_t *sRing = sP + 2 * Cfg::kP;     // tiles: four latent chunks
  uint8_t *sRope = sRing + NS * kP4Tile;
  uint8_t *sPack = sRope + NR * kPgRope;  // strips as they lie in the cache
  P4Ctrl<R> &c = *reinterpret_cast<P4Ctrl<R> *>(
      ((uintptr_t)sPack + NP * kP4Pack + 127) & ~(uintptr_t)127);
  // (what a shuffle from one lane gives is known to be the same in all: roles' branches and
  // MMAs' operands in uniform registers)
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&c.full[s], 4);
      mbar_init(&c.empty[s], 1);
    }
    for (int s = 0; s < NP; ++s) {
      mbar_init(&c.pack_full[s], 1);
      mbar_init(&c.pack_empty[s], 4);
    }
    for (int s = 0; s < NR; ++s) mbar_init(&c.rope_free[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.s_free[s], Cfg::kLive);
      mbar_init(&c.p_full[s], Cfg::kLive);
      mbar_init(&c.p_free[s], 1);
      mbar_init(&c.q_full[s], 4);
      mbar_init(&c.o_free[s], 8);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&c.ref[s], 1);
    mbar_init(&c.q_free, Cfg::kQkW);
    mbar_init(&c.o_full, 1);
    for (int s = 0; s < 3; ++s) mbar_init(&c.drain[s], 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&c.tmem_base, kPgTmemCols);
  grid_launch_dependents();  // the join may be set up; it waits for this grid's end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();  // the plan is there
  const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem_base, 0);
  // S buffer b at tS + 64 b, O^T chunk ch at tO + kOW ch
  const uint32_t tS = tmem + Cfg::kColS, tO = tmem + Cfg::kColO;
  const uint32_t tSA = tmem + Cfg::kColScale, tSB = tSA + 4;
  volatile int *abort = &c.abort;
  PgWalk w(a, blockIdx.x);
  if (warp < 4) {
    reg_dealloc<kP4RegsCtl>();
    if (warp == 0 || (Cfg::kQkW == 2 && warp == 2)) {
      // ------------------------------------------------------ score-GEMM issuers
      // (two: one for the even tiles and one for the odd)
      const int me = warp >> 1;
      constexpr uint32_t id = idesc_e4m3(128, kPgTile, 0, 0);
      const uint64_t dqr = smem_desc(smem_u32(sQr), 16, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), 16, 1024, kSwz128);
      const uint64_t drr = smem_desc(smem_u32(sRope), 16, 512, kSwz64);
      bool ok = true;
      uint32_t j = 0, piece = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        ok = warp_wait(&c.q_full[piece & 1], (piece >> 1) & 1, abort, a.status);
        if (!ok) break;
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          if (Cfg::kQkW == 2 && (j & 1) != (uint32_t)me) continue;
          const uint32_t slot = j % NS, dS = tS + (j & 1) * kPgTile;
          if (j >= 2)
            ok = warp_wait(&c.s_free[j & 1], ((j >> 1) - 1) & 1, abort, a.status);
          if (ok) ok = warp_wait(&c.full[slot], (j / NS) & 1, abort, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = dr + ((slot * kP4Tile) >> 4);
          const uint64_t drb = drr + ((j % NR * kPgRope) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int n = 0; n < 18; ++n) {
              const uint64_t b = n < 16 ? db + ((n / 4 * kPgSlot + n % 4 * 32) >> 4)
                                        : drb + (((n - 16) * 32) >> 4);
              const int i = n - Cfg::kQSteps;  // behind q's in TMEM: pairs in shared memory
              if (i < 0)
                mma_f8_ts(dS, tmem + n * 8, b, id, n != 0 ? 1u : 0u);
              else
                mma_f8_ss(dS, dqr + ((i / 2 * Cfg::kQPair + i % 2 * 32) >> 4), b, id, 1u);
            }
            mma_commit(&c.s_full[j & 1]);
            mma_commit(&c.rope_free[j % NR]);
          }
          __syncwarp();
        }
        if (ok && elect_one()) mma_commit(&c.q_free);
        ++piece;
      }
      if (!ok) {
        if (elect_one()) mma_commit(&c.drain[warp]);
        pg_drain(&c.drain[warp], 0, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------ PV-GEMM issuer
      constexpr int W = Cfg::kWide;  // parts a MMA
      constexpr uint32_t id = idesc_mx_e4m3(128, R * W, 1, 0);
      const uint64_t dp = smem_desc(smem_u32(sP), 16, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), kPgSlot, 1024, kSwz128);
      const uint64_t df = smem_desc(smem_u32(c.sf), 128, 128, 0);
      bool ok = true;
      uint32_t j = 0, piece = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        if (piece > 0)
          ok = warp_wait(&c.o_free[(piece - 1) & 1], ((piece - 1) >> 1) & 1, abort,
                               a.status);
        for (int t = w.t0; ok && t < w.t1; ++t, ++j) {
          const uint32_t b = j & 1;
          ok = warp_wait(&c.p_full[b], (j >> 1) & 1, abort, a.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            // (a thread's MMAs are behind its copies, but a copy need not be behind MMAs: the
            // scales of the tile before have a place of their own, and those of the one ahead of
            // it are read, as this tile's weights are only there behind its PV GEMM)
            tmem_cp_32x128b(tSB + 4 * b, df + ((b * sizeof c.sf[0]) >> 4));
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              const uint64_t da = dr + ((j % NS * kP4Tile + ch * kPgSlot) >> 4);
              uint32_t acc = t > w.t0 ? 1u : 0u;
#pragma unroll
              for (uint32_t k = 0; k < kPgTile / 32; ++k)
#pragma unroll
                for (uint32_t y = 0; y < 2; y += W) {
                  const uint64_t db = dp + ((b * Cfg::kP + y * Cfg::kPart + k * 32) >> 4);
                  // (a byte of a row's scales for each 32 keys)
                  mma_mx_ss(tO + ch * Cfg::kOW, da + ((k * 4096) >> 4), db,
                            id | idesc_mx_b_scale(k), tSA, tSB + 4 * b, acc);
                  acc = 1;
                }
            }
            mma_commit(&c.empty[j % NS]);
            mma_commit(&c.p_free[b]);
          }
          __syncwarp();
        }
        if (ok && elect_one()) mma_commit(&c.o_full);
        ++piece;
      }
      if (!ok) {
        if (elect_one()) mma_commit(&c.drain[warp]);
        pg_drain(&c.drain[warp], 0, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------ loads
      // Lane p: page p of a tile (a tile is half of a block of 128), whose strips lie side
      // by side: one copy.
      const int bs = 1 << a.shift, rows = bs < kPgTile ? bs : kPgTile, ppt = kPgTile / rows;
      const uint32_t page_bytes = rows * (kStrip / 16);
      bool ok = true;
      uint32_t j = 0;
      while (ok && w.next(a)) {
        const int32_t *row = a.table + (int64_t)w.m.req * a.stride;
        // first row in the cache of this lane's page, or -1
        auto page = [&](int t) {
          const int p0 = ((w.m.t_lo + t) << kPgTileLog) + lane * rows;
          if (lane >= ppt || t >= w.t1 || p0 > w.m.hi_max || p0 + rows <= w.m.lo_min) return -1;
          const int blk = row[p0 >> a.shift];
          return blk >= 0 && blk < a.n_blocks ? (blk << a.shift) + (p0 & (bs - 1)) : -1;
        };
        int nxt = page(w.t0);
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          const int y = nxt;
          nxt = page(t + 1);
          const uint32_t slot = j % NP;
          // (groups of 16 keys that are there: a page is 1, 2 or 4 of them)
          uint32_t there = __ballot_sync(0xffffffffu, y >= 0);
          const uint32_t bytes = __popc(there) * page_bytes;
          if (rows >= 32) there = rows == 64 ? there * 15u : (there & 1u) * 3u + (there & 2u) * 6u;
          ok = warp_wait(&c.pack_empty[slot], (j / NP & 1) ^ 1, abort, a.status);
          if (!ok) break;
          if (lane == 0) {
            c.there[slot] = there;
            mbar_arrive_expect_tx(&c.pack_full[slot], bytes);
          }
          __syncwarp();
          if (y >= 0)
            bulk_load_g2s(sPack + slot * kP4Pack + lane * page_bytes,
                          a.strips + (int64_t)(y >> 4) * kStrip, page_bytes,
                          &c.pack_full[slot]);
          __syncwarp();
        }
      }
      // giving up: the copies in flight have landed before the CTA exits
      if (!ok && lane == 0) {
        for (uint32_t i = j > NP ? j - NP : 0; i < j; ++i)
          pg_drain(&c.pack_full[i % NP], (i / NP) & 1, kPgDrainNs);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    reg_alloc<kP4RegsSoftmax>();
    // ------------------------------------------------------ softmax
    // The two warpgroups take the tiles in turn, each with a score and a P buffer of its
    // own.  Of a warp's 32 lanes of the scores the first 16 are the h parts of 16 q rows,
    // the last 16 their l parts; threads r and r + 16 load both parts of row r, for half
    // of the warp's keys each (R = 64: all 64; R = 16: 32, of one of two live warps).
    // The references go from tile to tile in shared memory, from a warp of one warpgroup
    // to one of the other.  A warp that gives up goes on through the loop without waiting
    // or writing, so that the barriers stay matched.
    const int q4 = warp & 3, wg = (warp - 4) >> 2;
    constexpr bool kSplit = Cfg::kSplit;
    const int qi = kSplit ? q4 & 1 : q4;  // which of the live warps
    const int rc = qi * 16 + (lane & 15), r = kSplit ? lane & 15 : rc;  // a row('s copy)
    const int kb = kSplit ? qi * 32 + (lane >> 4) * 16 : (lane >> 4) * 32;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int bar_wg = 1 + wg;
    constexpr int kBarAll = 3;
    const bool live = kSplit ? q4 >> 1 == wg : q4 * 16 < R;  // the warp has rows
    bool ok = true;
    uint32_t j = 0, piece = 0;
    const float one = __uint_as_float(0x7F7F7F7Fu), ones[4] = {one, one, one, one};
    if (wg == 0) tmem_st4(tSA + lane_off, ones);
    tmem_st_wait();
    tc_fence_before();
    // a piece's bounds for this thread's row; asked for before the output of the piece ahead
    bool mine = false;
    int lo = 1, hi = 0, x = 0;
    auto begin = [&] {
      mine = r < w.m.count * a.hc;
      lo = 1;
      hi = 0;
      if (mine) {
        const int i = w.m.first + r / a.hc;
        lo = a.kv_lo ? max(a.kv_lo[i], 0) : 0;
        hi = a.kv_hi ? max(-1, min(a.kv_hi[i], a.pos[i])) : a.pos[i];  // (p4_rare subtracts)
      }
      x = w.t0 + ((j & 1) == (uint32_t)wg ? 0 : 1);  // this warpgroup's first tile
    };
    bool more = w.next(a);
    if (more) begin();
    while (more) {
      const bool some = w.t1 > w.t0;  // else a group that sees no key
      if (ok && some)
        ok = warp_wait(&c.q_full[piece & 1], (piece >> 1) & 1, abort, a.status);
      const float qf = ok && some && mine ? c.qf[piece & 1][r] : 0.f;
      float m_own = -INFINITY, l = 0.f;  // the sum l of 2^t is on reference m_own
      for (uint32_t jj = j + (x - w.t0); x < w.t1; x += 2, jj += 2) {
        // (warps that free the scores alone: for others the next ones may be there already)
        if (live && ok) ok = warp_wait(&c.s_full[wg], (jj >> 1) & 1, abort, a.status);
        tc_fence_after();
        // Steps of kK keys a thread, rolled: the roles' loops have to stay in the
        // instruction cache together (32 KB at an instruction a cycle).  Between the
        // passes u stays in registers, its steps in turn in the first kK.
        constexpr int kK = 16, kU = kSplit ? 16 : 32, kSteps = kU / kK;
        constexpr int kHalf = kSplit ? 16 : 32;  // columns from lane to lane + 16
        const P4KeyScale &ks = c.ks[jj % NS];
        float u[kU], bt = -INFINITY;
        float rare[kU + 3];  // (in local memory: out-of-line code alone uses it)
        auto turn = [&](const float *last) {  // the steps of u by one, with a new last one
#pragma unroll
          for (int n = 0; n + kK < kU; ++n) u[n] = u[n + kK];
#pragma unroll
          for (int n = 0; n < kK; ++n) u[kU - kK + n] = last[n];
        };
        if (live && ok) {
          const uint32_t col = tS + wg * kPgTile + lane_off + (kSplit ? 32 * qi : 0);
          const float4 *kx = reinterpret_cast<const float4 *>(ks.up + p4_key(kb));
          const float4 *ke = reinterpret_cast<const float4 *>(ks.e + p4_key(kb));
#pragma unroll 1
          for (int g = 0; g < kSteps; ++g) {
            float s[kK], v[kK];
            tmem_ld_16x32bx2_x16<kHalf>(col + kK * g, s);
            tmem_ld_16x32bx2_x16<kHalf>(col + kK * g + (16u << 16), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kK / 4; ++i) {
              const float4 f = kx[kK / 4 * g + i], e = ke[kK / 4 * g + i];
              const float ff[4] = {f.x, f.y, f.z, f.w}, ee[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int n = 4 * i + y;
                s[n] = fmaf(fmaf(v[n], 0.0625f, s[n]) * qf, ff[y], ee[y]);
              }
            }
#pragma unroll
            for (int n = 0; n < kK; ++n) bt = fmaxf(bt, s[n]);
            turn(s);
          }
          tc_fence_before();
          warp_arrive(&c.s_free[wg], lane);
          const int p0 = (w.m.t_lo + x) << kPgTileLog;
          const uint2 th = *reinterpret_cast<const uint2 *>(&ks.there);
          const uint32_t there = th.x;
          if (((there ^ 15u) | th.y) != 0 || p0 < w.m.lo_max || p0 + kPgTile - 1 > w.m.hi_min) {
#pragma unroll
            for (int n = 0; n < kU; ++n) rare[n] = u[n];
            bt = p4_rare(rare, ks.e + p4_key(kb), kU, p0 + kb, lo, hi, there >> (kb >> 4),
                         a.status);
#pragma unroll
            for (int n = 0; n < kU; ++n) u[n] = rare[n];
            if (kSplit) rare[kU + 2] += __shfl_xor_sync(0xffffffffu, rare[kU + 2], 16);
          }
        }
        // the largest u of the 32 keys that share a scale, and what the warp has of the row
        const float bo = __shfl_xor_sync(0xffffffffu, bt, 16);
        float um = fmaxf(bt, bo);
        if (kSplit) bt = um;
        float m_old = -INFINITY;
        if (live && x > w.t0) {
          if (ok) ok = warp_wait(&c.ref[qi], (jj - 1) & 1, abort, a.status);
          m_old = c.m_ref[rc];
        }
        float m_new = m_old;
        // (+inf at a row's first key)
        if (named_bar_or(bar_wg, 128, live && mine && um > -INFINITY && um - m_old > kP4Up)) {
          if constexpr (kSplit) {
            // (the maxima of the two warps' keys, where the piece's end has its sums)
            if (live && lane < 16) c.stat_l[wg][rc] = um;
            named_bar_sync(bar_wg, 128);
            um = fmaxf(c.stat_l[wg][r], c.stat_l[wg][16 + r]);
          }
          if (mine && um > -INFINITY && um - m_old > kP4Up) m_new = ceilf(um) + kP4Over;
          const bool moved = live && m_old > -INFINITY && m_new != m_old;
          const uint32_t mv = __ballot_sync(0xffffffffu, moved);
          // (half of the exponent, twice: m may rise by more than binary32's 126 where what O^T
          // holds is 2^-7 of what comes)
          if (live && lane < 16) c.alpha[wg][r] = moved ? fast_exp2(0.5f * (m_old - m_new)) : 1.f;
          if (lane == 0) c.mv[wg][q4] = mv;
          named_bar_sync(bar_wg, 128);
          if ((c.mv[wg][0] | c.mv[wg][1] | c.mv[wg][2] | c.mv[wg][3]) != 0) {
            // the PV GEMM of the tile before is done with O^T; behind that of the one ahead of
            // it, as a wait tells a phase from the next alone (jj - 3 may still run)
            if (ok && jj >= 2)
              ok = warp_wait(&c.p_free[wg], ((jj >> 1) - 1) & 1, abort, a.status);
            if (ok)
              ok = warp_wait(&c.p_free[wg ^ 1], ((jj - 1) >> 1) & 1, abort, a.status);
            tc_fence_after();
            if (ok) {
#pragma unroll 1
              for (int qr = 0; qr < R / 16; ++qr) {
                // only row quarters (16 columns of O^T) in which a row moved
                if (!kSplit && c.mv[wg][qr] == 0) continue;
#pragma unroll 1
                for (int cc = 0; cc < 4 * Cfg::kWide; ++cc) {
                  float o[16];
                  tmem_ld16(tO + lane_off + cc * R + qr * 16, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const float h = c.alpha[wg][qr * 16 + i];
                    o[i] = o[i] == 0.f ? 0.f : o[i] * h * h;
                  }
                  tmem_st16(tO + lane_off + cc * R + qr * 16, o);
                }
              }
              tmem_st_wait();
            }
            tc_fence_before();
            named_bar_sync(bar_wg, 128);  // all quarters of the lanes are done
          }
        }
        if (live) {
          if (lane < 16) c.m_ref[rc] = m_new;
          if (ok) warp_arrive(&c.ref[qi], lane);
          // p = 2^(u - m) of 32 keys is p' = 2^(u - sub), at most 2^8, times 2^(sub - m)
          const bool some_key = mine && bt > -INFINITY;
          // (from 2^27 on the difference is rounded, to 16 too, which an E4M3 does not hold)
          const float top = bt - (ceilf(bt) - 8.f) > 8.f ? bt : ceilf(bt) - 8.f;
          // (rounded up: to nearest it may be 128 below m, and the scale's byte that of NaN)
          const float sub = some_key ? fmaxf(top, __fadd_ru(m_new, -120.f)) : 0.f;
          // the PV GEMM of this buffer's last tile is done with it
          if (ok && jj >= 2)
            ok = warp_wait(&c.p_free[wg], ((jj >> 1) - 1) & 1, abort, a.status);
          if (ok) {
            const uint8_t se = (uint8_t)(some_key ? (int)(sub - m_new) + 127 : 127);
            if constexpr (kSplit) {
              if (lane < 16) {  // (rows of the two parts)
                c.sf[wg][r][0][qi] = se;
                c.sf[wg][16 + r][0][qi] = se;
              }
            } else {
              c.sf[wg][r & 31][r >> 5][lane >> 4] = se;
            }
            float sum[2] = {0.f, 0.f};
            uint8_t *pr = sP + wg * Cfg::kP + r * kPgTile;
            const float4 *kd = reinterpret_cast<const float4 *>(ks.down + p4_key(kb));
#pragma unroll 1
            for (int g = 0; g < kSteps; ++g) {
              // p' in two E4M3, as q
              uint32_t part[2][kK / 4];
#pragma unroll
              for (int i = 0; i < kK / 4; ++i) {
                const float4 f = kd[kK / 4 * g + i];
                const float ff[4] = {f.x, f.y, f.z, f.w};
                float pv[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  pv[y] = fast_exp2(u[4 * i + y] - sub);
                  sum[y & 1] = fmaf(pv[y], ff[y], sum[y & 1]);
                }
                const uint2 p2 = split_p4(pack_f16x2(pv[0], pv[1]), pack_f16x2(pv[2], pv[3]));
                part[0][i] = p2.x;
                part[1][i] = p2.y;
              }
#pragma unroll
              for (int y = 0; y < 2; ++y)
                *reinterpret_cast<uint4 *>(
                    pr + y * Cfg::kPart + ((((kb >> 4) + g) ^ ((r >> 1) & 3)) << 4)) =
                    make_uint4(part[y][0], part[y][1], part[y][2], part[y][3]);
#pragma unroll
              for (int n = 0; n + kK < kU; ++n) u[n] = u[n + kK];
            }
            const bool high = *reinterpret_cast<const uint32_t *>(ks.high) != 0;
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&c.p_full[wg], lane);
            // the sum of 2^t goes by a reference of its own (values and weights may lie
            // 183 binades apart)
            const float2 was = make_float2(l, m_own);
            const float lr = some_key ? fmaxf(m_own, sub) : m_own;
            if (lr != m_own) {
              l = pg_scale(l, m_own - lr);
              m_own = lr;
            }
            l += pg_scale(sum[0] + sum[1], sub - lr);
            // (2^t of the keys is p' 2^(sub - e), and p' keeps all of it where the exponents of
            // the 32 lie at most 90 apart: none is above kP4High)
            if (high) {
              const float2 x = p4_wide(rare + kU, was, make_float2(l, m_own));
              l = x.x;
              m_own = x.y;
            }
          }
        }
      }
      j += w.t1 - w.t0;
      const float lo_ = __shfl_xor_sync(0xffffffffu, l, 16);
      const float mo = __shfl_xor_sync(0xffffffffu, m_own, 16), mx = fmaxf(m_own, mo);
      l = pg_scale(l, m_own - mx) + pg_scale(lo_, mo - mx);
      m_own = mx;
      // ---------------------------------------------- this piece's O and LSE
      const int r_valid = w.m.count * a.hc, h0 = w.hg * a.hc, first = w.m.first, hc = a.hc;
      const int part = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      const bool whole = w.whole();
      more = w.next(a);
      if (more) begin();
      // A warp has a quarter of the channels (its TMEM lanes) and half of the rows.
      named_bar_sync(kBarAll, 256);  // both have decided their last references
      if (live && lane < 16) {
        c.stat_l[wg][rc] = l;
        c.stat_m[wg][rc] = m_own;
      }
      named_bar_sync(kBarAll, 256);
      if (ok && some) ok = warp_wait(&c.o_full, piece & 1, abort, a.status);
      tc_fence_after();
      if (ok) {
        constexpr int RH = R / 2, RS = RH < 16 ? RH : 16;
        const int sw = warp - 4;
        if (lane < RH) {
          const int rr = wg * RH + lane;
          // the sum of 2^t, on the reference ml
          float sl = 0.f, ml = -INFINITY;
#pragma unroll
          for (int y = 0; y < Cfg::kLanes; y += R)
            ml = fmaxf(ml, fmaxf(c.stat_m[0][rr + y], c.stat_m[1][rr + y]));
#pragma unroll
          for (int y = 0; y < Cfg::kLanes; y += R)
#pragma unroll
            for (int g = 0; g < 2; ++g)
              sl += pg_scale(c.stat_l[g][rr + y], c.stat_m[g][rr + y] - ml);
          const bool empty = ml == -INFINITY && sl == 0.f;  // l may be NaN
          const float l2 = empty ? -INFINITY : ml + log2f(sl);
          // 2^(m - ml) / sl in two factors, the first with half of its exponent: it may
          // lie outside binary32 where its products with O^T do not
          const int k = (int)(__float_as_uint(sl) >> 23) - 127;
          const float e = empty || sl != sl ? 0.f : c.m_ref[rr] - ml - (float)k;
          const float half = rintf(0.5f * e);
          c.inv2[sw][lane] = fast_exp2(e - half);
          float f = pg_scale(empty ? 0.f : 1.f / (sl * __int_as_float((127 - k) << 23)), half);
          int64_t orow = -1;
          if (rr < r_valid) {
            if (whole) {
              const int hh = h0 + rr % hc, i = first + rr / hc;
              const float L = l2 * 0.69314718055994530942f;
              f *= sink_factor(a.sink, hh, L);
              orow = (int64_t)(a.tokens ? a.tokens[i] : i) * a.H + hh;
              if (q4 == 0) a.lse[orow] = L;
            } else if (q4 == 0) {
              // (a sum that is NaN on no reference)
              a.lse_part[(int64_t)part * R + rr] =
                  make_float2(sl != sl ? 0.f : ml, empty ? 0.f : log2f(sl));
            }
          }
          c.inv[sw][lane] = f;
          c.orow[sw][lane] = orow;
        }
        __syncwarp();
        const int t = q4 * 32 + lane;
        // RS rows (columns of O^T) of a channel chunk at a time; a warp's 32 lanes
        // are 32 channels of a row side by side.  A part's rows lie behind one
        // another, and so do RS heads of a token where Hc is a multiple of RS:
        // one address and constant offsets.
        const bool dense = hc % RS == 0;
#pragma unroll 1
        for (int cb = 0; cb < RH && wg * RH + cb < r_valid; cb += RS) {
          float f[RS];
#pragma unroll
          for (int y = 0; y < RS; ++y) f[y] = c.inv[sw][cb + y];
          __nv_bfloat16 *po = a.o + c.orow[sw][cb] * CPMLA_DV + t;
          float *pp = a.o_part + ((int64_t)part * R + wg * RH + cb) * CPMLA_DV + t;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch, po += 128, pp += 128) {
            float o[RS];
            if (some) {
              float w3[Cfg::kWide][RS];
#pragma unroll
              for (int y = 0; y < Cfg::kWide; ++y) {
                const uint32_t col = tO + lane_off + ch * Cfg::kOW + y * R + wg * RH + cb;
                if (RS == 16)
                  tmem_ld16(col, w3[y]);
                else
                  tmem_ld8(col, w3[y]);
              }
              tmem_ld_wait();
#pragma unroll
              for (int z = 0; z < RS; ++z) {
                o[z] = w3[0][z];
#pragma unroll
                for (int y = 1; y < Cfg::kWide; ++y) o[z] += w3[y][z];
              }
            } else {
#pragma unroll
              for (int y = 0; y < RS; ++y) o[y] = 0.f;
            }
#pragma unroll
            for (int y = 0; y < RS; ++y)
              o[y] = o[y] * f[y] * c.inv2[sw][cb + y];
            if (!whole) {
#pragma unroll
              for (int y = 0; y < RS; ++y) pp[y * CPMLA_DV] = o[y];
            } else if (dense) {
#pragma unroll
              for (int y = 0; y < RS; ++y) po[y * CPMLA_DV] = __float2bfloat16_rn(o[y]);
            } else {
#pragma unroll 1
              for (int y = 0; y < RS; ++y) {
                // (o by a selected register: y is not a constant here)
                float v = o[0];
#pragma unroll
                for (int z = 1; z < RS; ++z) v = z == y ? o[z] : v;
                const int64_t orow = c.orow[sw][cb + y];
                if (orow >= 0) a.o[orow * CPMLA_DV + ch * 128 + t] = __float2bfloat16_rn(v);
              }
            }
          }
        }
      }
      tc_fence_before();
      if (some) {
        if (ok) warp_arrive(&c.o_free[piece & 1], lane);
        ++piece;
      }
      named_bar_sync(kBarAll, 256);  // the statistics are read
    }
  } else if (warp < 16) {
    reg_dealloc<kP4RegsQ>();
    // ------------------------------------------------------ q into TMEM
    const int q4 = warp & 3;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int rows0 = Cfg::kSplit ? 0 : q4 * 16;  // the warp's first row
    bool ok = true;
    // q of piece k.  TMEM lanes 0-15 of this warp's 32 are the h parts of 16 rows, lanes
    // 16-31 the l parts: thread 4 y + c reads 8 channels of rows y and y + 8, 32 channels a
    // step with its quad, and two 16-lane stores put the parts where they belong.
    // (The loops are kept short: code that runs once a piece comes from L2, at
    // about 8 cycles an instruction.)
    auto load_q = [&](const PgWalk &v, uint32_t k) {
      const int r_valid = v.m.count * a.hc, y8 = lane >> 2, c4 = lane & 3;
      const uint4 *src[2];
      uint32_t mx[2] = {0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // (rows of no token read the group's first one and are not used)
        const int rr = rows0 + 8 * x + y8 < r_valid ? rows0 + 8 * x + y8 : 0;
        const int n = v.m.first + rr / a.hc;
        src[x] = reinterpret_cast<const uint4 *>(
                     a.q + (int64_t)(a.tokens ? a.tokens[n] : n) * a.q_stride +
                     (int64_t)(v.hg * a.hc + rr % a.hc) * CPMLA_DQK) +
                 c4;
      }
      auto fetch = [&](int n, uint4 *w) {
#pragma unroll
        for (int x = 0; x < 2; ++x) w[x] = __ldg(src[x] + 4 * n);
      };
      {
#pragma unroll 1
        for (int n = 0; n < 18; n += 6) {
          uint4 w[6][2];
#pragma unroll
          for (int i = 0; i < 6; ++i) fetch(n + i, w[i]);
#pragma unroll
          for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // the larger of two bf16 magnitudes in each half (NaN above all)
              const uint32_t m01 = __vmaxu2(w[i][x].x & 0x7FFF7FFFu, w[i][x].y & 0x7FFF7FFFu);
              const uint32_t m23 = __vmaxu2(w[i][x].z & 0x7FFF7FFFu, w[i][x].w & 0x7FFF7FFFu);
              mx[x] = __vmaxu2(mx[x], __vmaxu2(m01, m23));
            }
        }
      }
      uint4 w[4][2];
      uint32_t down[2];
      float up[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t m = max(mx[x] & 0xFFFFu, mx[x] >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^ae brings the largest channel into (224, 448]; ae >= -60 (rows below
        // keep fewer bits)
        int ae = (int)(m >> 7) - 127 - ((m & 0x7Fu) > 0x60u ? 7 : 8);
        ae = ae < -60 ? -60 : (ae > 120 ? 120 : ae);
        down[x] = (uint32_t)(127 - ae) * 0x00800080u;
        // a row with an infinite or NaN channel is NaN throughout
        up[x] = m >= 0x7F80u ? NAN : __int_as_float((127 + ae) << 23) * a.scale_log2;
      }
      // a step's words for the two stores
      auto split = [&](const uint4 *v, uint32_t *p) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint2 p0 = split_q4(v[x].x, v[x].y, down[x]);
          const uint2 p1 = split_q4(v[x].z, v[x].w, down[x]);
          p[2 * x] = p0.x;
          p[2 * x + 1] = p1.x;
          p[4 + 2 * x] = p0.y;
          p[5 + 2 * x] = p1.y;
        }
      };
      auto put = [&](int n, const uint32_t *p) {
        const uint32_t at = tmem + lane_off + n * 8;
        tmem_st_16x256b_x1(at, p[0], p[1], p[2], p[3]);
        tmem_st_16x256b_x1(at + (16u << 16), p[4], p[5], p[6], p[7]);
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) fetch(i, w[i]);
      // the softmax is done with the piece two before (its scales' place is used
      // again, and it has seen that piece's q_full), the score GEMMs with q
      if (k > 1) ok = warp_wait(&c.o_free[k & 1], ((k >> 1) - 1) & 1, abort, a.status);
      if (k > 0 && ok) ok = warp_wait(&c.q_free, (k - 1) & 1, abort, a.status);
      if (!ok) return;
      tc_fence_after();
      {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (c4 == 0 && (!Cfg::kSplit || q4 == 0)) c.qf[k & 1][rows0 + 8 * x + y8] = up[x];
        // a step's words into its half of a pair in shared memory
        auto put_smem = [&](int n, const uint4 *v) {
          const int i = n - Cfg::kQSteps;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint2 p0 = split_q4(v[x].x, v[x].y, down[x]);
            const uint2 p1 = split_q4(v[x].z, v[x].w, down[x]);
            const int ln = q4 * 32 + 8 * x + y8, ck = (i & 1) * 2 + (c4 >> 1);
            uint8_t *d = sQr + (i >> 1) * Cfg::kQPair + ln * 64 +
                         ((ck ^ ((ln >> 1) & 3)) << 4) + (c4 & 1) * 8;
            *reinterpret_cast<uint2 *>(d) = make_uint2(p0.x, p1.x);
            *reinterpret_cast<uint2 *>(d + 1024) = make_uint2(p0.y, p1.y);  // lane + 16
          }
        };
        constexpr int kQLoop = Cfg::kQSteps / 4 * 4;  // 12 or 16
#pragma unroll 1
        for (int n = 0; n < kQLoop; n += 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[8];
            split(w[i], p);
            put(n + i, p);
            fetch(min(n + i + 4, 17), w[i]);
          }
        }
        if constexpr (kQLoop < 16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kQLoop + i < Cfg::kQSteps) {
              uint32_t p[8];
              split(w[i], p);
              put(kQLoop + i, p);
            } else {
              put_smem(kQLoop + i, w[i]);
            }
            if (i < 2) fetch(16 + i, w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (Cfg::kQSteps == 18) {
            uint32_t p[8];
            split(w[i], p);
            put(16 + i, p);
          } else {
            put_smem(16 + i, w[i]);
          }
        }
        tmem_st_wait();
        fence_proxy_async_smem();
      }
      tc_fence_before();
      warp_arrive(&c.q_full[k & 1], lane);
    };
    for (uint32_t k = 0; ok && w.next(a);)
      if (w.t1 > w.t0) load_q(w, k++);
  } else {
    reg_dealloc<kP4RegsX>();
    // ------------------------------------------------------ 4-bit codes to E4M3
    // Two groups of four warps take the tiles in turn, so that one's waits run beside the
    // other's arithmetic (a warp of each on every scheduler).  A warp takes a strip: a
    // thread 16 bytes of a token (groups u and u + 16) at a time, which become a 16-byte
    // unit of two chunks each.  All of it is in registers before anything else, so that the
    // group's next strips are on their way while these are worked on.
    const int xw = warp & 3, xg = (warp >> 2) & 1, u = lane & 15, half = lane >> 4;
    const int k0 = 16 * xw;
    bool ok = true;
    uint32_t j = 0;
    while (ok && w.next(a)) {
      for (int t = w.t0; t < w.t1; ++t, ++j) {
        if ((j & 1) != (uint32_t)xg) continue;
        const uint32_t ps = j % NP, es = j % NS;
        ok = warp_wait(&c.pack_full[ps], (j / NP) & 1, abort, a.status);
        if (!ok) break;
        const uint8_t *strip = sPack + ps * kP4Pack + xw * kStrip;
        uint4 v[8], rope[2];
        uint32_t off[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = *reinterpret_cast<const uint4 *>(strip + 512 * i + 256 * half + 16 * u);
          off[i] = strip[kStripOff + 32 * i + 16 * half + u];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rope[i] = *reinterpret_cast<const uint4 *>(strip + kStripRope + 512 * i + 16 * lane);
        const int e = strip[kStripExp + u];
        const uint32_t there = c.there[ps];
        warp_arrive(&c.pack_empty[ps], lane);
        // The PV GEMM is done with the tile's place, the scores with the rope's (a barrier's
        // phase before its first is complete).  The rope's phase ahead of this one, tile j -
        // 6's, has to be over before that wait: with one issuer, whose scores end in order,
        // this group's last one was for j - 5's, and the two are waited for at once; with two
        // issuers the tile's place tells it (j - 5's values are behind j - 6's scores).
        if constexpr (Cfg::kQkW == 1) {
          ok = warp_wait(half ? &c.rope_free[j % NR] : &c.empty[es],
                         ((half ? j / NR : j / NS) & 1) ^ 1, abort, a.status);
        } else {
          ok = warp_wait(&c.empty[es], (j / NS & 1) ^ 1, abort, a.status);
          if (ok) ok = warp_wait(&c.rope_free[j % NR], (j / NR & 1) ^ 1, abort, a.status);
        }
        if (!ok) break;
        uint8_t *dst = sRing + es * kP4Tile + (u >> 3) * kPgSlot + (k0 + half) * 128;
        // (four tokens a turn: 8,192 prompt tokens 1,197 us, 1,220 with all eight side by side)
#pragma unroll 1
        for (int h = 0; h < 2; ++h, dst += 1024) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint8_t *d = dst + i * 256 + (((u & 7) ^ (2 * i + half)) << 4);
            *reinterpret_cast<uint4 *>(d) = p4_e4m3x16(v[i].x, v[i].y, off[i] & 15);
            *reinterpret_cast<uint4 *>(d + 2 * kPgSlot) = p4_e4m3x16(v[i].z, v[i].w, off[i] >> 4);
            v[i] = v[i + 4];
            off[i] = off[i + 4];
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = k0 + (lane >> 2) + 8 * i;
          *reinterpret_cast<uint4 *>(sRope + j % NR * kPgRope + k * 64 +
                                     (((lane & 3) ^ ((k >> 1) & 3)) << 4)) = rope[i];
        }
        P4KeyScale &ks = c.ks[es];
        if (lane < 16) {
          const int k = p4_key(k0 + lane);
          const float up = p4_scale(e);
          ks.up[k] = up;
          ks.e[k] = (float)max(kP4ExpMin, min(e - 127, kP4ExpMax));
          // 2^-e: the exponent field mirrored about that of 1 (NaN: a finite value)
          ks.down[k] = __uint_as_float((254u << 23) - __float_as_uint(up));
          ks.there = there;
        }
        const bool high = __any_sync(0xffffffffu, e - 127 > kP4High);
        if (lane == 0) ks.high[xw] = high;
        fence_proxy_async_smem();
        warp_arrive(&c.full[es], lane);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kPgTmemCols);
  }
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
  PagedArgs a{};
  int R = 0;
  const int rc = paged_attn_args(fn, true, q, q_token_stride, H, cache, nullptr, n_blocks,
                                 block_size, block_table, B, table_stride, tokens, pos, req,
                                 n_tokens, kv_lo, kv_hi, softmax_scale, sink, T, o_out, lse_out,
                                 workspace, workspace_bytes, a, &R);
  if (rc != CPMLA_OK || R == 0) return rc;
  static PgKnown known;
  auto run = [&](auto kernel, auto rows, int smem) {
    a.n_cta = pg_device(fn, known, R, kernel, smem);
    if (a.n_cta < 0) return (int)CPMLA_ERR_CUDA;
    return launch_paged<decltype(rows)::value>(fn, a, kernel, kP4Threads, smem,
                                               static_cast<cudaStream_t>(stream));
  };
  return R == 64 ? run(paged4_attn_kernel<64>, std::integral_constant<int, 64>{}, p4_smem<64>())
                 : run(paged4_attn_kernel<16>, std::integral_constant<int, 16>{}, p4_smem<16>());
}
