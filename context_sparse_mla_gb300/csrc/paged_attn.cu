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
//     [2^-4, 2^15.75], so a weight is off by at most 2^-13 of its tile's own
//     largest one, whatever the other tiles hold.  (A first token with almost all of
//     the weight and next to no value is common; two E4M3 terms, which need a third
//     fewer MMAs, reach 2^-9 and lose the tokens beside it.)  A move rescales O^T and
//     waits for the PV GEMM before, about a tile's time, hence the wide window, and m
//     goes no further than it must (p to 2^-2 or 2^14; a row's first to 2^6): the window
//     comes to lie around the row's tiles.  Scores of standard deviation 4 (32 tokens
//     of 16,384 keys x 64 heads): 116 us, 138 with every move to 2^6, 96 without moves;
//     a move at every tile, 196, is the worst.  How far m may go down is bounded by the
//     sums that it takes along in binary32 (kPgFallU): a tile further below the row's
//     largest u adds nothing to O^T.
// A piece of work is R = 16 or 64 rows (G tokens of one request x Hc heads) and
// a range of their keys, 64 at a time:
//   S = [h; l] . C^T      q (2R lanes) in TMEM, the tile's keys as N = 64, K = 576
//                         (kind::f8f6f4; the rope's 64 from shared memory), into
//                         one of two S buffers
//   O^T += C^T . P^T      M = 128 channels x 4, N = R a part of p (parts side by
//                         side where TMEM has the columns), K = 64 keys
// The value is the latent itself: a tile's chunks [64 keys x 128 channels] stay in
// their ring slot from the score GEMM to the PV GEMM, so 64 keys cost 36 KB of
// loads, once for R rows (the bf16 kernel's: 144 KB), in a ring of 5 or 6 tiles.
// Two softmax warpgroups take the tiles in turn; S rows lie on TMEM lanes, so a
// row's threads read 32 keys each and one shuffle joins them.
//
// The work is cut by tiles, not by rows: a first launch (one CTA) groups the
// entries, counts tiles and gives every SM the same number of tile units; a
// group that is cut leaves normalised fp32 parts in the workspace, at most two
// for each SM, and a third launch joins them in a fixed order.  One request's
// token uses up to 152 SMs that way, and lists of any mix end together.
//
// Warps: 0-2 issue the MMAs (R = 64: 0 the scores, 1 and 2 PV; R = 16: 0 and 2
// the scores, 1 PV), 3 loads, 4-11 do the softmax and the output, 12-15 bring q
// in.  Every wait is bounded; on expiry the CTA records CPMLA_ERR_TIMEOUT, drains
// its copies and MMAs, frees TMEM and exits.
//
// What bounds it, measured.  R = 16 (32 tokens of 4,096 to 131,072 keys x 16 heads):
// HBM; 222 us a call, 5.1 TB/s over the whole call, 5.6 in the kernel.  R = 64: shared
// memory and the MMA issue.  A tile's 42 MMAs read 188 KB of it (each part of p
// reads the 4 KB of keys again: three parts side by side would need 768 TMEM
// columns) and the copies write 36 KB, about 1,800 cycles at 128 B a cycle; it
// takes 2,050.  Between two pieces the tensor core stands still for 10 to 13 tiles:
// the last softmax and PV, the output, and q's split do not overlap the next
// piece's.  8,192 tokens x 16 heads 1,171 us (1.00 PFLOP/s of the exact products).
#include <type_traits>

#include "paged_attn.cuh"

namespace cpmla {
namespace {

// ------------------------------------------------------------- the attention
constexpr int kPgThreads = 512;     // control, two softmax and one q warpgroup
constexpr int kPgParts = 3;         // E5M2 parts of a weight
constexpr int kPgTileBytes = 4 * kPgSlot + kPgRope;  // ring slot: a tile

template <int R>
struct PgCfg {
  static constexpr int kPart = R * kPgTile;  // one part of P: [R rows x 64 keys]
  static constexpr int kP = kPgParts * kPart;
  // Parts of P side by side in one PV MMA, each with accumulators of its own (TMEM
  // holds 4 R kWide + 256 columns): an MMA of N = 16 takes 40 cycles and one of N = 48
  // or 64 takes 48, most of them for the 4 KB of keys, which N = 48 reads once for three.
  static constexpr int kWide = R == 16 ? 3 : 1;
  static constexpr int kOW = R * kWide;  // columns of an O^T chunk
  // MMA issuers (warps 0-2): R = 64 has 24 PV MMAs a tile for two threads beside the
  // 18 of the scores, R = 16 has 8 for one, and the scores two
  static constexpr int kPvW = R == 64 ? 2 : 1, kQkW = 3 - kPvW;
  static constexpr int kQRope = 2 * R * 64;  // q's rope: [2R lanes x 64]
  static constexpr int kFixed = kQRope + 2 * kP;
  // Steps of q (of 16) split before the wait for q's place, at 8 registers each: between
  // the pieces of a prompt the split was 16,000 cycles of waiting (8,192 tokens of 16
  // heads: 1,215 us with none, 1,160 with 8).  R = 16 is slower with it (247, 222 us).
  static constexpr int kQAhead = R == 64 ? 8 : 0;
  static constexpr int kSlots = R == 16 ? 6 : 5;  // tiles in the ring
};

template <int R>
struct PgCtrl {
  uint64_t full[PgCfg<R>::kSlots], empty[PgCfg<R>::kSlots];  // ring slots
  // S and P have a buffer for each softmax warpgroup: even and odd tiles
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], p_free[2];
  uint64_t ref[4];     // row quarter's references of a tile are decided
  // for even and odd pieces, as a waiter may be a piece behind: q is in place; the
  // softmax is done with a piece, its output written
  uint64_t q_full[2], o_free[2];
  uint64_t q_free, o_full;
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort;
  float qf[2][R];      // a piece's scale of q row r, times softmax scale and log2 e
  float m_ref[R], m_low[R];  // the reference, and the least it may become
  float stat_l[2][R];
  alignas(16) float alpha[2][R];
  uint32_t mv[2][4];  // a row quarter has a row whose reference moved
  // per softmax warp: a row's output factor and its row of the output (-1: none)
  alignas(16) float inv[8][R / 2];
  int64_t orow[8][R / 2];
};
template <int R>
constexpr int pg_smem() {
  return 1024 + PgCfg<R>::kFixed + PgCfg<R>::kSlots * kPgTileBytes + (int)sizeof(PgCtrl<R>);
}
static_assert(pg_smem<64>() <= 232448 && pg_smem<16>() <= 232448, "shared memory budget");

// Bounded wait of a warp: lane 0 waits, the warp takes its result.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int lane,
                                          volatile int *abort, int *status) {
  int ok = 1;
  if (lane == 0) ok = mbar_wait(bar, parity, abort, status) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Two fp16 less their upper bytes (an E5M2 each, cut): exact.
__device__ __forceinline__ uint32_t f16x2_minus_upper(uint32_t h2) {
  const uint32_t up = h2 & 0xFF00FF00u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h2),
                            *reinterpret_cast<const __half2 *>(&up));
  return *reinterpret_cast<const uint32_t *>(&d);
}
// How far below the largest u and t = u - e of a row its reference m may lie: two sums
// over N <= 2^30 keys have to stay in binary32,
//   O^T  sum 2^(u - m) c   <= N 448 2^(max u - m): 2^117 with m >= max u - 80 + 2
//   l    sum 2^(u - m - e) <= N 2^(max t - m):     2^124 with m >= max t - 96 + 2
// (max t is far above max u where the heaviest keys lie in blocks of very small values:
// one of zeros has e = -64).
constexpr float kPgFallU = 80.f, kPgFallT = 96.f;
// 2^e for the stored exponent e + 127, 63 .. 247
__device__ __forceinline__ float pg_pow2(int stored) { return __int_as_float(stored << 23); }
template <int R>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_attn_kernel(const __grid_constant__ PagedArgs a,
                      const __grid_constant__ CUtensorMap tm_lat,
                      const __grid_constant__ CUtensorMap tm_rope) {
  using Cfg = PgCfg<R>;
  constexpr int NS = Cfg::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sQr = smem;                    // q's rope (the MMA reads 128 lanes; those behind
                                          // 2R are whatever follows, and not used)
  uint8_t *sP = sQr + Cfg::kQRope;        // two P of three parts
  uint8_t *sRing = sP + 2 * Cfg::kP;      // tiles: four latent chunks, the rope
  PgCtrl<R> &c = *reinterpret_cast<PgCtrl<R> *>(sRing + NS * kPgTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], Cfg::kPvW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.s_free[s], 4);
      mbar_init(&c.p_full[s], 4);
      mbar_init(&c.p_free[s], Cfg::kPvW);
      mbar_init(&c.q_full[s], 4);
      mbar_init(&c.o_free[s], 8);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&c.ref[s], 1);
    mbar_init(&c.q_free, Cfg::kQkW);
    mbar_init(&c.o_full, Cfg::kPvW);
    for (int s = 0; s < 3; ++s) mbar_init(&c.drain[s], 1);
    c.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&c.tmem_base, kPgTmemCols);
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&tm_lat);
    tma_prefetch_desc(&tm_rope);
  }
  grid_launch_dependents();  // the join may be set up; it waits for this grid's end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();  // the plan is there
  const uint32_t tmem = c.tmem_base;
  // columns: q [0, 128), S buffer b at tS + 64 b, O^T chunk ch at tO + kOW ch
  const uint32_t tS = tmem + 128, tO = tS + 2 * kPgTile;
  volatile int *abort = &c.abort;
  PgWalk w(a, blockIdx.x);

  if (warp == 0 || (Cfg::kQkW == 2 && warp == 2)) {
    // ------------------------------------------------------ score-GEMM issuers
    // (two: one for the even tiles and one for the odd)
    const int me = warp >> 1;
    if (lane == 0) {
      constexpr uint32_t id = idesc_e4m3(128, kPgTile, 0, 0);
      const uint64_t dqr = smem_desc(smem_u32(sQr), 16, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), 16, 1024, kSwz128);
      const uint64_t drr = smem_desc(smem_u32(sRing + 4 * kPgSlot), 16, 512, kSwz64);
      bool ok = true;
      uint32_t j = 0, piece = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        if (!mbar_wait(&c.q_full[piece & 1], (piece >> 1) & 1, abort, a.status)) {
          ok = false;
          break;
        }
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          if (Cfg::kQkW == 2 && (j & 1) != (uint32_t)me) continue;
          const uint32_t slot = j % NS, dS = tS + (j & 1) * kPgTile;
          if ((j >= 2 && !mbar_wait(&c.s_free[j & 1], ((j >> 1) - 1) & 1, abort, a.status)) ||
              !mbar_wait(&c.full[slot], (j / NS) & 1, abort, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t db = dr + ((slot * kPgTileBytes) >> 4);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_ts(dS, tmem + ch * 32 + k * 8, db + ((ch * kPgSlot + k * 32) >> 4), id,
                        (ch | k) != 0 ? 1u : 0u);
          const uint64_t drb = drr + ((slot * kPgTileBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma_f8_ss(dS, dqr + ((k * 32) >> 4), drb + ((k * 32) >> 4), id, 1u);
          mma_commit(&c.s_full[j & 1]);
        }
        if (ok) mma_commit(&c.q_free);
        ++piece;
      }
      if (!ok) {
        mma_commit(&c.drain[warp]);
        pg_drain(&c.drain[warp], 0, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------ PV-GEMM issuers
    // (a thread gets an MMA out every 75-100 cycles, the tensor core takes 48).
    // Loops here and at the edges stay rolled: all warps' code together is more
    // than the instruction cache holds beside the softmax, and straight code
    // that runs once a piece took 8 cycles an instruction.
    if (lane == 0) {
      const int me = warp - 1;
      constexpr int W = Cfg::kWide;  // parts a MMA
      static_assert(kPgParts % W == 0, "no part is left over");
      constexpr uint32_t id = idesc_e4m3_e5m2(128, R * W, 1, 0);
      const uint64_t dp = smem_desc(smem_u32(sP), 16, 512, kSwz64);
      const uint64_t dr = smem_desc(smem_u32(sRing), kPgSlot, 1024, kSwz128);
      bool ok = true;
      uint32_t j = 0, piece = 0;
      while (ok && w.next(a)) {
        if (w.t1 <= w.t0) continue;
        if (piece > 0 && !mbar_wait(&c.o_free[(piece - 1) & 1], ((piece - 1) >> 1) & 1, abort,
                                     a.status)) {
          ok = false;
          break;
        }
        for (int t = w.t0; t < w.t1; ++t, ++j) {
          const uint32_t b = j & 1;
          if (!mbar_wait(&c.p_full[b], (j >> 1) & 1, abort, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int ch = me; ch < 4; ch += Cfg::kPvW) {
            const uint64_t da = dr + ((j % NS * kPgTileBytes + ch * kPgSlot) >> 4);
            uint32_t acc = t > w.t0 ? 1u : 0u;
#pragma unroll 1
            for (uint32_t k = 0; k < kPgTile / 32; ++k)
#pragma unroll
              for (uint32_t y = 0; y < kPgParts; y += W) {
                mma_f8_ss(tO + ch * Cfg::kOW, da + ((k * 4096) >> 4),
                          dp + ((b * Cfg::kP + y * Cfg::kPart + k * 32) >> 4), id, acc);
                acc = 1;
              }
          }
          mma_commit(&c.empty[j % NS]);
          mma_commit(&c.p_free[b]);
        }
        if (ok) mma_commit(&c.o_full);
        ++piece;
      }
      if (!ok) {
        mma_commit(&c.drain[warp]);
        pg_drain(&c.drain[warp], 0, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------ loads
    // Lane 5 p + x: chunk x (4: the rope) of page p of a tile (a tile is half of a
    // block of 128).  One instruction issues the boxes of all lanes, about 80
    // cycles each; box after box, each behind its own wait, 128 keys took 4200
    // cycles and bounded the kernel.
    const int bs = 1 << a.shift, rows = bs < kPgTile ? bs : kPgTile, ppt = kPgTile / rows;
    const int pg = lane / 5, kd = lane - 5 * pg;
    const bool act = pg < ppt;
    const CUtensorMap *tm = kd == 4 ? &tm_rope : &tm_lat;
    bool ok = true;
    uint32_t j = 0;
    while (ok && w.next(a)) {
      const int32_t *row = a.table + (int64_t)w.m.req * a.stride;
      // first row in the cache of this lane's page, or -1
      auto page = [&](int t) {
        const int p0 = ((w.m.t_lo + t) << kPgTileLog) + pg * rows;
        if (!act || t >= w.t1 || p0 > w.m.hi_max || p0 + rows <= w.m.lo_min) return -1;
        const int blk = row[p0 >> a.shift];
        return blk >= 0 && blk < a.n_blocks ? (blk << a.shift) + (p0 & (bs - 1)) : -1;
      };
      int nxt = page(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++j) {
        const int y = nxt;
        nxt = page(t + 1);
        const int np = __popc(__ballot_sync(0xffffffffu, kd == 0 && y >= 0));
        const uint32_t slot = j % NS;
        uint64_t *fb = &c.full[slot];
        uint8_t *dst =
            sRing + slot * kPgTileBytes + kd * kPgSlot + pg * rows * (kd == 4 ? 64 : 128);
        bool good = true;
        if (lane == 0) {
          good = j < NS || mbar_wait(&c.empty[slot], (j / NS - 1) & 1, abort, a.status);
          if (good) mbar_arrive_expect_tx(fb, (uint32_t)(np * rows) * CPMLA_DQK);
        }
        if (!__all_sync(0xffffffffu, good)) {
          ok = false;
          break;
        }
        if (y >= 0) tma_load_2d(dst, tm, kd * 128, y, fb);
        __syncwarp();
      }
    }
    // giving up: the copies in flight have landed before the CTA exits
    if (!ok && lane == 0) {
      for (uint32_t i = j > NS ? j - NS : 0; i < j; ++i)
        pg_drain(&c.full[i % NS], (i / NS) & 1, kPgDrainNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------ softmax
    // The two warpgroups take the tiles in turn, each with a score and a P buffer of
    // its own, so that one's waits and shuffles run beside the other's arithmetic.
    // Of a warp's 32 lanes of the scores the first 16 are the h parts of 16 q rows,
    // the last 16 their l parts; threads r and r + 16 load both parts of row r,
    // for 32 keys side by side each, so the row's other half is one shuffle away.
    // The references go from tile to tile in shared memory (warp q4 of one
    // warpgroup to warp q4 of the other), each warpgroup's sums on the reference
    // they last saw.  A warp that gives up goes on through the loop without
    // waiting or writing, so that the barriers stay matched.
    const int q4 = warp & 3, wg = (warp - 4) >> 2;
    const int r = q4 * 16 + (lane & 15), kb = (lane >> 4) * 32;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int bar_wg = 1 + wg;
    constexpr int kBarAll = 3;
    const bool live = q4 * 16 < R;  // the warp has rows
    bool ok = true;
    uint32_t j = 0, piece = 0;
    // a piece's bounds for this thread's row, and what its first tile needs; asked
    // for before the output of the piece ahead
    const int32_t *row = nullptr;
    bool mine = false;
    int lo = 1, hi = 0, x = 0, e_cur = -1, b_nxt = -1;
    // group g of 16 keys of tile y (lane g and its copies): its block's stored
    // exponent, or -1 where no row may look; the block of this warpgroup's next
    // tile's group is fetched a tile ahead of its exponent
    auto block_at = [&](int y) {
      const int p = ((w.m.t_lo + y) << kPgTileLog) + (lane & 3) * 16;
      if (y >= w.t1 || p + 15 < w.m.lo_min || p > w.m.hi_max) return -1;
      const int blk = row[p >> a.shift];
      return blk >= 0 && blk < a.n_blocks ? blk : -1;
    };
    auto exp_of_block = [&](int blk) {
      return blk >= 0 ? max(63, min((int)__ldg(a.exp + blk), 247)) : -1;
    };
    auto begin = [&] {
      row = a.table + (int64_t)w.m.req * a.stride;
      mine = r < w.m.count * a.hc;
      lo = 1;
      hi = 0;
      if (mine) {
        const int i = w.m.first + r / a.hc;
        lo = a.kv_lo ? max(a.kv_lo[i], 0) : 0;
        hi = a.kv_hi ? min(a.kv_hi[i], a.pos[i]) : a.pos[i];
      }
      x = w.t0 + ((j & 1) == (uint32_t)wg ? 0 : 1);  // this warpgroup's first tile
      const int b0 = block_at(x);
      b_nxt = block_at(x + 2);
      e_cur = exp_of_block(b0);
    };
    bool more = w.next(a);
    if (more) begin();
    while (more) {
      const bool some = w.t1 > w.t0;  // else a group that sees no key
      if (ok && some)
        ok = warp_wait(&c.q_full[piece & 1], (piece >> 1) & 1, lane, abort, a.status);
      const float qf = ok && some && mine ? c.qf[piece & 1][r] : 0.f;
      float m_own = -INFINITY, l = 0.f;  // the sum l is on reference m_own
      for (uint32_t jj = j + (x - w.t0); x < w.t1; x += 2, jj += 2) {
        const int e_nxt = exp_of_block(b_nxt);
        b_nxt = block_at(x + 4);
        const int p0 = (w.m.t_lo + x) << kPgTileLog;
        const bool open = p0 >= w.m.lo_max && p0 + kPgTile - 1 <= w.m.hi_min &&
                          __all_sync(0xffffffffu, e_cur >= 0);
        // 2^e and e of the key groups
        const float kf = e_cur >= 0 ? pg_pow2(e_cur) : 1.f;
        const float ku = (float)(e_cur - 127);
        const uint32_t there = __ballot_sync(0xffffffffu, e_cur >= 0);
        if (ok) ok = warp_wait(&c.s_full[wg], (jj >> 1) & 1, lane, abort, a.status);
        tc_fence_after();
        float s[32];
        if (live && ok) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float v[16];
            const uint32_t col = tS + wg * kPgTile + lane_off + g * 16;
            tmem_ld_16x32bx2_x16<32>(col, s + 16 * g);
            tmem_ld_16x32bx2_x16<32>(col + (16u << 16), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) s[16 * g + i] = fmaf(v[i], 0.0625f, s[16 * g + i]);
          }
        }
        tc_fence_before();
        if (ok) warp_arrive(&c.s_free[wg], lane);
        // the row's largest u and t in the tile; 2^-e of the thread's two key groups
        float um = -INFINITY, tm = -INFINITY, kd[2];
        if (live && ok) {
          if (!open) {
            // NaN codes in a key that not every row may see: weight zero times
            // NaN would reach the others, so the key's values become zero (a
            // row that does see it has a NaN weight).  A NaN code makes the
            // scores of every row NaN, so any row's threads know the keys; the
            // warps share them out.
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) nan |= (uint32_t)(s[i] != s[i]) << i;
            if (__any_sync(0xffffffffu, nan != 0)) {
              // the copies are seen by this thread too (they landed long ago)
              (void)mbar_wait(&c.full[jj % NS], (jj / NS) & 1, abort, a.status);
              __syncwarp();
              for (int k = q4; k < kPgTile; k += R / 16) {
                const uint32_t nk = __shfl_sync(0xffffffffu, nan, (k >> 5) * 16);
                if (((nk >> (k & 31)) & 1) == 0) continue;
                uint4 *kr = reinterpret_cast<uint4 *>(sRing + jj % NS * kPgTileBytes +
                                                      (lane >> 3) * kPgSlot + k * 128 +
                                                      (lane & 7) * 16);
                const uint4 v = *kr;
                auto has = [](uint32_t u) {
                  const uint32_t z = ~u & 0x7F7F7F7Fu;  // a zero byte: a NaN code
                  return ((z - 0x01010101u) & ~z & 0x80808080u) != 0;
                };
                if (__any_sync(0xffffffffu, has(v.x) || has(v.y) || has(v.z) || has(v.w)))
                  *kr = make_uint4(0, 0, 0, 0);
              }
            }
          }
          // u = t + e
          float k0[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float k2 = __shfl_sync(0xffffffffu, kf, (kb >> 4) + g);
            k0[g] = __shfl_sync(0xffffffffu, ku, (kb >> 4) + g);
            const float f = qf * k2;
            // 2^-e: the exponent field mirrored about that of 1
            kd[g] = __uint_as_float((254u << 23) - __float_as_uint(k2));
#pragma unroll
            for (int i = 0; i < 16; ++i) s[16 * g + i] = fmaf(s[16 * g + i], f, k0[g]);
          }
          if (!open) {
            // a group without a block that the row attends to: its block is a bad one
            // (between the ranges of two rows of a piece a block may be anything)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int p = p0 + kb + 16 * g;
              if (((there >> ((kb >> 4) + g)) & 1) == 0 && max(lo, p) <= min(hi, p + 15))
                record_status(a.status, CPMLA_ERR_INDEX);
            }
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              const int p = p0 + kb + n;
              if (((there >> ((kb >> 4) + (n >> 4))) & 1) == 0 || p < lo || p > hi)
                s[n] = -INFINITY;
            }
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float ug = s[16 * g];
#pragma unroll
            for (int i = 1; i < 16; ++i) ug = fmaxf(ug, s[16 * g + i]);
            um = fmaxf(um, ug);
            tm = fmaxf(tm, ug - k0[g]);
          }
          um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 16));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
        }
        // the reference follows the tile's maximum when it leaves the window
        float m_old = -INFINITY, m_low = -INFINITY;
        if (x > w.t0) {
          if (ok) ok = warp_wait(&c.ref[q4], (jj - 1) & 1, lane, abort, a.status);
          if (live) {
            m_old = c.m_ref[r];
            m_low = c.m_low[r];
          }
          __syncwarp();
        }
        float m_new = m_old;
        if (mine && um > -INFINITY) {
          m_low = fmaxf(m_low, fmaxf(um - kPgFallU, tm - kPgFallT));
          const float d = um - m_old;  // +inf at a row's first key
          if (d > 15.75f) {
            m_new = um - (m_old == -INFINITY ? 6.f : 14.f);
            // from 2^25 on the difference is rounded, to 16 too, which p does not hold
            if (um - m_new > 15.75f) m_new = um;
          } else if (d < -4.f) {
            m_new = fminf(m_old, fmaxf(um, m_low) + 2.f);
          }
        }
        if (live && lane < 16) {
          c.m_ref[r] = m_new;
          c.m_low[r] = m_low;
        }
        if (ok) warp_arrive(&c.ref[q4], lane);
        if (m_new != m_own) {
          l = pg_scale(l, m_own - m_new);
          m_own = m_new;
        }
        if (x > w.t0 && named_bar_or(bar_wg, 128, m_new != m_old)) {
          // only row quarters (a warp's 16 columns of O^T) in which a row moved
          const uint32_t mv = __ballot_sync(0xffffffffu, m_new != m_old);
          if (live && lane < 16)
            c.alpha[wg][r] = m_old == -INFINITY ? 0.f : fast_exp2(m_old - m_new);
          if (lane == 0) c.mv[wg][q4] = mv;
          named_bar_sync(bar_wg, 128);
          // the PV GEMM of the tile before is done with O^T; behind that of the one ahead of
          // it, as a wait tells a phase from the next alone (jj - 3 may still run)
          if (ok && jj >= 2)
            ok = warp_wait(&c.p_free[wg], ((jj >> 1) - 1) & 1, lane, abort, a.status);
          if (ok) ok = warp_wait(&c.p_free[wg ^ 1], ((jj - 1) >> 1) & 1, lane, abort, a.status);
          tc_fence_after();
          if (ok) {
#pragma unroll 1
            for (int qr = 0; qr < R / 16; ++qr) {
              if (c.mv[wg][qr] == 0) continue;
#pragma unroll 1
              for (int cc = 0; cc < 4 * Cfg::kWide; cc += 2) {  // two at a time
                float o[2][16];
                const uint32_t col = tO + lane_off + cc * R + qr * 16;
                tmem_ld16(col, o[0]);
                tmem_ld16(col + R, o[1]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float al = c.alpha[wg][qr * 16 + i];
                  o[0][i] = o[0][i] == 0.f ? 0.f : o[0][i] * al;
                  o[1][i] = o[1][i] == 0.f ? 0.f : o[1][i] * al;
                }
                tmem_st16(col, o[0]);
                tmem_st16(col + R, o[1]);
              }
            }
            tmem_st_wait();
          }
          named_bar_sync(bar_wg, 128);  // alpha is read
        }
        // p as fp16 bits, split by cutting: an E5M2 is the upper byte of an fp16, so
        // each part is the upper byte of what is left (nothing is negative); the
        // last part is rounded
        uint32_t part[kPgParts][8];
        if (live && ok) {
          const float mm = m_new == -INFINITY ? 0.f : m_new;
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            float pv[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) pv[y] = fast_exp2(s[4 * g + y] - mm);
            sum[g >> 2] += (pv[0] + pv[1]) + (pv[2] + pv[3]);
            uint32_t a0 = pack_f16x2(pv[0], pv[1]), a1 = pack_f16x2(pv[2], pv[3]);
#pragma unroll
            for (int y = 0; y < kPgParts; ++y) {
              if (y == kPgParts - 1) {
                a0 += 0x00800080u;
                a1 += 0x00800080u;
              }
              part[y][g] = __byte_perm(a0, a1, 0x7531);
              if (y < kPgParts - 1) {
                a0 = f16x2_minus_upper(a0);
                a1 = f16x2_minus_upper(a1);
              }
            }
          }
          l = fmaf(sum[0], kd[0], fmaf(sum[1], kd[1], l));
        }
        // the PV GEMM of this buffer's last tile is done with it
        if (ok && jj >= 2)
          ok = warp_wait(&c.p_free[wg], ((jj >> 1) - 1) & 1, lane, abort, a.status);
        if (live && ok) {
          uint8_t *pr = sP + wg * Cfg::kP + r * kPgTile;
#pragma unroll
          for (int y = 0; y < kPgParts; ++y)
#pragma unroll
            for (int g = 0; g < 2; ++g)
              *reinterpret_cast<uint4 *>(pr + y * Cfg::kPart +
                                         ((((kb >> 4) + g) ^ ((r >> 1) & 3)) << 4)) =
                  make_uint4(part[y][4 * g], part[y][4 * g + 1], part[y][4 * g + 2],
                             part[y][4 * g + 3]);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        if (ok) warp_arrive(&c.p_full[wg], lane);
        e_cur = e_nxt;
      }
      j += w.t1 - w.t0;
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      // ---------------------------------------------- this piece's O and LSE
      const int r_valid = w.m.count * a.hc, h0 = w.hg * a.hc, first = w.m.first, hc = a.hc;
      const int part = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      const bool whole = w.whole();
      more = w.next(a);
      if (more) begin();
      // A warp has a quarter of the channels (its TMEM lanes) and half of the rows.
      named_bar_sync(kBarAll, 256);  // both have decided their last references
      if (live && lane < 16) {
        if (!some && wg == 0) c.m_ref[r] = -INFINITY;
        const float m = some ? c.m_ref[r] : -INFINITY;
        c.stat_l[wg][r] = pg_scale(l, m_own - m);
      }
      named_bar_sync(kBarAll, 256);
      if (ok && some) ok = warp_wait(&c.o_full, piece & 1, lane, abort, a.status);
      tc_fence_after();
      if (ok) {
        constexpr int RH = R / 2, RS = RH < 16 ? RH : 16;
        const int sw = warp - 4;
        if (lane < RH) {
          const int rr = wg * RH + lane;
          const float m = c.m_ref[rr], sl = c.stat_l[0][rr] + c.stat_l[1][rr];
          const bool empty = m == -INFINITY && sl == 0.f;  // l may be NaN
          const float l2 = empty ? -INFINITY : m + log2f(sl);
          float f = empty ? 0.f : 1.f / sl;
          int64_t orow = -1;
          if (rr < r_valid) {
            if (whole) {
              const int hh = h0 + rr % hc, i = first + rr / hc;
              const float L = l2 * 0.69314718055994530942f;
              f *= sink_factor(a.sink, hh, L);
              orow = (int64_t)(a.tokens ? a.tokens[i] : i) * a.H + hh;
              if (q4 == 0) a.lse[orow] = L;
            } else if (q4 == 0) {
              a.lse_part[(int64_t)part * R + rr] = make_float2(l2, 0.f);
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
            for (int y = 0; y < RS; ++y) o[y] *= f[y];
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
  } else if (warp >= 12) {
    // ------------------------------------------------------ q into TMEM
    const int q4 = warp & 3;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    bool ok = true;
    // q of piece k.  TMEM lanes 0-15 of this warp's 32 are the h parts of rows 16
    // q4 .., lanes 16-31 the l parts: thread 4 y + c reads 8 channels of rows y and y
    // + 8, 32 channels a step with its quad, and two 16-lane stores put the parts
    // where they belong.  The last two steps, the rope, go to shared memory.
    // (The loops are kept short: code that runs once a piece comes from L2, at
    // about 8 cycles an instruction.)
    auto load_q = [&](const PgWalk &v, uint32_t k) {
      const int r_valid = v.m.count * a.hc, y8 = lane >> 2, c4 = lane & 3;
      const uint4 *src[2];
      uint32_t mx[2] = {0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // (rows of no token read the group's first one and are not used)
        const int rr = q4 * 16 + 8 * x + y8 < r_valid ? q4 * 16 + 8 * x + y8 : 0;
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
      if (q4 * 16 < R) {
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
      // what the registers hold is split ahead of the wait
      uint32_t pre[Cfg::kQAhead > 0 ? Cfg::kQAhead : 1][8];
      if (q4 * 16 < R) {
#pragma unroll
        for (int n = 0; n < Cfg::kQAhead; n += 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) fetch(n + i, w[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) split(w[i], pre[n + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch(Cfg::kQAhead + i, w[i]);
      }
      // the softmax is done with the piece two before (its scales' place is used
      // again, and it has seen that piece's q_full), the score GEMMs with q
      if (k > 1) ok = warp_wait(&c.o_free[k & 1], ((k >> 1) - 1) & 1, lane, abort, a.status);
      if (k > 0 && ok) ok = warp_wait(&c.q_free, (k - 1) & 1, lane, abort, a.status);
      if (!ok) return;
      tc_fence_after();
      if (q4 * 16 < R) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (c4 == 0) c.qf[k & 1][q4 * 16 + 8 * x + y8] = up[x];
#pragma unroll
        for (int n = 0; n < Cfg::kQAhead; ++n) put(n, pre[n]);
#pragma unroll 1
        for (int n = Cfg::kQAhead; n < 16; n += 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[8];
            split(w[i], p);
            put(n + i, p);
            fetch(min(n + i + 4, 17), w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint2 p0 = split_q4(w[i][x].x, w[i][x].y, down[x]);
            const uint2 p1 = split_q4(w[i][x].z, w[i][x].w, down[x]);
            const int ln = q4 * 32 + 8 * x + y8, ck = i * 2 + (c4 >> 1);
            uint8_t *d = sQr + ln * 64 + ((ck ^ ((ln >> 1) & 3)) << 4) + (c4 & 1) * 8;
            *reinterpret_cast<uint2 *>(d) = make_uint2(p0.x, p1.x);
            *reinterpret_cast<uint2 *>(d + 1024) = make_uint2(p0.y, p1.y);  // lane + 16
          }
        tmem_st_wait();
        fence_proxy_async_smem();
      }
      tc_fence_before();
      warp_arrive(&c.q_full[k & 1], lane);
    };
    for (uint32_t k = 0; ok && w.next(a);)
      if (w.t1 > w.t0) load_q(w, k++);
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
  const int rc = paged_attn_args(fn, false, q, q_token_stride, H, cache, cache_exp, n_blocks, block_size,
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
  static PgKnown known;
  auto run = [&](auto kernel, auto rows, int smem) {
    a.n_cta = pg_device(fn, known, R, kernel, smem);
    if (a.n_cta < 0) return (int)CPMLA_ERR_CUDA;
    return launch_paged<decltype(rows)::value>(fn, a, kernel, kPgThreads, smem, st, tm[0], tm[1]);
  };
  return R == 64 ? run(paged_attn_kernel<64>, std::integral_constant<int, 64>{}, pg_smem<64>())
                 : run(paged_attn_kernel<16>, std::integral_constant<int, 16>{}, pg_smem<16>());
}
