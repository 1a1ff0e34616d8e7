// cross_bwd_tc.cuh -- gradients of cross attention on Blackwell tensor cores (tcgen05 + TMEM + TMA),
// bf16, head size 64 or 128.
//
// With p = exp(s - lse) and ds = p (dout . v - D) as in cross_simt.cuh, two kinds of CTA in one launch,
// each holding 128 rows of one side and streaming 128-row tiles of the other:
//
//   dk, dv   128 keys fixed (F0 = K, F1 = V), row tiles streamed (X = Q, Y = dout):
//            S^T = K Q^T, dP^T = V dout^T;  dV += P^T dout, dK += dS^T Q
//   dq       128 rows fixed (F0 = Q, F1 = dout), key tiles streamed (X = K, Y = V):
//            S = Q K^T, dP = dout V^T;  dQ += dS K
//
// so both compute S' = F0 X^T and dP' = F1 Y^T, 128 x 128 in fp32 in TMEM.  Two warpgroups share a tile,
// 64 columns each, one thread a row: p from S' while dP' is computed, then ds; both in bf16 over the
// columns the thread has read, from where the last products take them as their A operand; the streamed
// tile is their B operand, as it lies.  The score products are done twice (7 products in place of 5):
// the price of sums that stay in one CTA, with no atomics and no order of addition left to chance.  The
// kind with the longer CTAs comes first in the grid, the other fills the SMs behind it.
//
// What bounds it is the tensor pipe, 4 d cycles a 128 x 128 x d product, if nothing makes it wait, and power:
// 4096 x 16384 rows of 16 heads, d = 128, take 1.56 ms in short runs (1.23 PFLOP/s of the 7 products, 75 % of
// the measured GEMM peak) and 1.6 to 1.8 ms in long ones at 990 W.  What brought it there:
//   - Streamed tiles of 128 rows: a product's two operands from shared memory are 8 KB for 64 cycles,
//     what shared memory delivers.  With 64-row tiles (6 KB for 32 cycles) each of these products took
//     60 cycles, and the whole 2.13 ms against 1.71 ms.
//   - The fixed operand from TMEM, where there is room (dq; dk, dv at d = 64): the softmax threads copy
//     their rows there at the start, and a score product then reads 4 KB from shared memory (with the next
//     point 1.71 to 1.56 ms).
//   - The order of issue.  dk, dv: dV(j), S'(j + 1), dK(j), dP'(j + 1): ds is made under dV and S', the
//     next p under dK and dP'.  dq: S(j + 1), dQ(j), dP(j + 1): ds under S, the next p under dQ and dP.
//     (With S', dP', dV, dK in that order the products waited 760 of 3940 cycles a tile for p.)
//   - TMEM at d = 128 is full: S', dP', dV, dK of 128 columns each, or S, dP, dQ and Q, dout of 64 each.  At
//     d = 64 there is room for P of its own in dk, dv: S'(j + 1) then runs under p, whose exponentials (1024
//     cycles a tile) weigh as much as the products there, instead of after dV(j) (16 heads of 4096 x 16384
//     rows: 1350 -> 1318 us; 4 x 16 heads of 509 x 1024: 57.4 -> 56.4).
//   - The last tile as code of its own: only there may streamed rows be missing, and the others' code has no
//     selections for it (the same two cases: 1343 -> 1287 us and 52.4 -> 50.1).
//
// Rows behind a sequence's end: K of a partial key tile is loaded with zeros there (its dS is 0, and
// 0 times what the padding holds has to be 0), and scores are set aside by selection, not arithmetic.
// Streamed rows past the last one come as zeros with lse = +inf, so their p is 0; in the last tile their
// products are set to 0 besides, which are 0 times a key and a value that may hold an infinity.
#pragma once
#include <type_traits>

#include "rows_tc.cuh"

namespace pia {
namespace ctb {
using namespace tc;

constexpr int kBT = 128;               // streamed rows a tile
constexpr int kSX = 3, kSY = 2;        // ring depths: X is held from S' to the last product
constexpr int kBwdTcThreads = 64 + 256;

template <int D>
struct GSmem {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kF0 = 0;
  static constexpr int kF1 = kF0 + kTile;
  static constexpr int kX = kF1 + kTile;
  static constexpr int kY = kX + kSX * kTile;
  static constexpr int kBar = kY + kSY * kTile;
  // fixed, x_full[3], x_empty[3], y_full[2], y_empty[2], s_full, dp_full, p_full, ds_full, p_done, ds_done,
  // drain, fixed in TMEM, s_read
  static constexpr int kNumBars = 1 + 2 * kSX + 2 * kSY + 9;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kStat = (kMisc + 8 + 15) / 16 * 16;    // dk, dv: -lse2 and -D of 64 rows a warpgroup,
  static constexpr int kTotal = kStat + 2 * 2 * 2 * 64 * 4;   // two buffers
  static constexpr int kAlloc = kTotal + 512;  // (the base is checked: a kernel without static memory starts on 1 KB)
  static_assert(kX % 1024 == 0 && kY % 1024 == 0 && kBar % 8 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct GParams {
  CrossGradArgs g;
  int key_tiles, row_tiles;  // 128-key and 128-row tiles of a head
  long long n_dkv;           // CTAs of the dk, dv kind
  long long dkv_at, dq_at;   // first CTA of each kind
};

// KEYS: this CTA's fixed side is keys (dk, dv), else rows (dq).
template <int D, bool KEYS>
__device__ __forceinline__ void cross_bwd_cta(const CUtensorMap* mf0, const CUtensorMap* mf1, const CUtensorMap* mx,
                                              const CUtensorMap* my, const GParams& prm, uint32_t base, uint8_t* sbase,
                                              long long bh, int tile) {
  using L = GSmem<D>;
  const CrossGradArgs& g = prm.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)(bh / g.heads);
  const int f0 = tile * BM;                       // first fixed row
  int n = g.kv_len ? g.kv_len[b] : g.n_kv;        // keys of the sequence
  const bool bad = n < 0 || n > g.n_kv;
  if (bad) {
    if (threadIdx.x == 0) raise_error(kErrCacheLen);
    n = 0;
  }
  const int fixed_rows = KEYS ? g.n_kv : g.R;     // rows of the fixed side that are written
  const int str_rows = KEYS ? g.R : n;            // rows of the streamed side
  const int nt = KEYS && f0 >= n ? 0 : (str_rows + kBT - 1) / kBT;

  const uint32_t sF0 = base + L::kF0, sF1 = base + L::kF1, sX = base + L::kX, sY = base + L::kY;
  const uint32_t bar_fix = base + L::kBar;
  auto bar_xfull = [&](int s) { return bar_fix + 8u * (1 + s); };
  auto bar_xempty = [&](int s) { return bar_fix + 8u * (1 + kSX + s); };
  auto bar_yfull = [&](int s) { return bar_fix + 8u * (1 + 2 * kSX + s); };
  auto bar_yempty = [&](int s) { return bar_fix + 8u * (1 + 2 * kSX + kSY + s); };
  const uint32_t bar_s = bar_fix + 8u * (1 + 2 * kSX + 2 * kSY), bar_dp = bar_s + 8;  // S', dP' complete
  const uint32_t bar_p = bar_s + 16, bar_ds = bar_s + 24, bar_r = bar_s + 64;  // P, dS written; S' read
  const uint32_t bar_pdone = bar_s + 32, bar_dsdone = bar_s + 40;  // the products that read P, dS complete
  const uint32_t bar_drain = bar_s + 48, bar_ft = bar_s + 56;      // ...; the fixed rows are in TMEM
  constexpr bool kFixTmem = !KEYS || D == 64, kOwnP = KEYS && D == 64;  // P beside S', not over it
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + L::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + L::kMisc + 4);

  if (threadIdx.x == 0) {
    mbar_init(bar_fix, 1);
    for (int s = 0; s < kSX; ++s) {
      mbar_init(bar_xfull(s), 1);
      mbar_init(bar_xempty(s), 1);
    }
    for (int s = 0; s < kSY; ++s) {
      mbar_init(bar_yfull(s), 1);
      mbar_init(bar_yempty(s), 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_dp, 1);
    mbar_init(bar_ft, 8);
    mbar_init(bar_r, 8);
    mbar_init(bar_p, 8);
    mbar_init(bar_ds, 8);
    mbar_init(bar_pdone, 1);
    mbar_init(bar_dsdone, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (nt > 0) {
      mbar_expect_tx(bar_fix, 2 * L::kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        tma_load_3d(sF0 + c * BM * 128, mf0, bar_fix, c * 64, f0, (int)bh);
        tma_load_3d(sF1 + c * BM * 128, mf1, bar_fix, c * 64, f0, (int)bh);
      }
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // S' at 0, dP' at 128, dV or dQ at 256, dK at 256 + D; the fixed operands (D / 2 columns each) behind
  const uint32_t tDP = tmem + 128, tA = tmem + 256, tB = tA + D, tF = KEYS ? tB + D : tB;
  const uint32_t tPo = kOwnP ? tF + D : tmem;
  static_assert(256 + (KEYS ? 2 * D : D) + (kFixTmem ? D : 0) + (kOwnP ? 64 : 0) <= 512, "TMEM columns");

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    int nx = 0, ny = 0;
    for (int j = 0; j < nt; ++j) {
      const int sx = j % kSX, sy = j % kSY;
      if (!__all_sync(0xffffffffu, j < kSX || mbar_wait(bar_xempty(sx), (j / kSX - 1) & 1, abort_flag))) break;
      if (KEYS || (j + 1) * kBT <= n) {
        if (lane == 0) {
          mbar_expect_tx(bar_xfull(sx), L::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sX + sx * L::kTile + c * kBT * 128, mx, bar_xfull(sx), c * 64, j * kBT, (int)bh);
        }
      } else {  // the last keys, row by row, with zeros behind the sequence's end
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const int sub = lane % LPR, slot = lane / LPR;
        const long long row0 = bh * g.n_kv + (long long)j * kBT;
#pragma unroll 8
        for (int i = 0; i < kBT / RPI; ++i) {
          const int key = i * RPI + slot;
          const bool in = j * kBT + key < n;
          rtc::cp_async16(sX + sx * L::kTile + (sub >> 3) * (kBT * 128) + key * 128 + (((sub & 7) ^ (key & 7)) << 4),
                          (const __nv_bfloat16*)g.k + (in ? (row0 + key) * D + sub * 8 : 0), in ? 16 : 0);
        }
        rtc::cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_xfull(sx));
      }
      ++nx;
      if (!__all_sync(0xffffffffu, j < kSY || mbar_wait(bar_yempty(sy), (j / kSY - 1) & 1, abort_flag))) break;
      if (lane == 0) {
        mbar_expect_tx(bar_yfull(sy), L::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sY + sy * L::kTile + c * kBT * 128, my, bar_yfull(sy), c * 64, j * kBT, (int)bh);
      }
      ++ny;
    }
    if (*abort_flag) {  // let the loads in flight land before the CTA can exit
      volatile int never = 0;
      if (nt > 0) mbar_wait(bar_fix, 0, &never);
      for (int u = nx > kSX ? nx - kSX : 0; u < nx; ++u) mbar_wait(bar_xfull(u % kSX), (u / kSX) & 1, &never);
      for (int u = ny > kSY ? ny - kSY : 0; u < ny; ++u) mbar_wait(bar_yfull(u % kSY), (u / kSY) & 1, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && nt > 0) {
      constexpr uint32_t id_s = idesc_bf16(BM, kBT, 0);  // B (X, Y) K-major
      constexpr uint32_t id_a = idesc_bf16(BM, D, 1);    // B (X, Y) N-major
      // d = F X^T: F (0 or 1) from TMEM or shared memory
      auto scores = [&](uint32_t d, int f, uint32_t streamed) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          const uint64_t bd = sw128_desc(streamed + in, 16, 1024);
          if (kFixTmem) tc_mma_ts(d, tF + f * (D / 2) + 8 * kk, bd, id_s, kk > 0 ? 1u : 0u);
          else tc_mma(d, sw128_desc((f ? sF1 : sF0) + in, 16, 1024), bd, id_s, kk > 0 ? 1u : 0u);
        }
      };
      // acc += (bf16 of the two warpgroups, 32 columns at `src` and 32 at src + gap) x streamed tile
      auto last = [&](uint32_t acc, uint32_t src, int gap, uint32_t streamed, int j) {
#pragma unroll
        for (int kk = 0; kk < kBT / 16; ++kk)
          tc_mma_ts(acc, src + 8 * (kk & 3) + gap * (kk >> 2), sw128_desc(streamed + kk * 16 * 128, kBT * 128, 1024), id_a,
                    (j > 0 || kk > 0) ? 1u : 0u);
      };
      auto x_at = [&](int j) { return sX + (j % kSX) * L::kTile; };
      auto y_at = [&](int j) { return sY + (j % kSY) * L::kTile; };
      auto x_in = [&](int j) { return mbar_wait(bar_xfull(j % kSX), (j / kSX) & 1, abort_flag); };
      auto y_in = [&](int j) { return mbar_wait(bar_yfull(j % kSY), (j / kSY) & 1, abort_flag); };
      bool okw = mbar_wait(kFixTmem ? bar_ft : bar_fix, 0, abort_flag) && x_in(0) && y_in(0);
      if (okw) {
        tc_fence_after();
        scores(tmem, 0, x_at(0));
        tc_commit(bar_s);
        scores(tDP, 1, y_at(0));
        tc_commit(bar_dp);
        if (!KEYS) tc_commit(bar_yempty(0));
      }
      auto next_s = [&](int j) -> bool {
        if (!x_in(j)) return false;
        tc_fence_after();
        scores(tmem, 0, x_at(j));
        tc_commit(bar_s);
        return true;
      };
      for (int j = 0; okw && j < nt; ++j) {
        const bool more = j + 1 < nt;
        // S'(j + 1) once S'(j) has been read, or (P over it) once dV(j) has read P
        if (!KEYS || kOwnP) {
          if (more && !(mbar_wait(bar_r, j & 1, abort_flag) && next_s(j + 1))) break;
        }
        if (KEYS) {
          if (!mbar_wait(bar_p, j & 1, abort_flag)) break;
          tc_fence_after();
          last(tA, tPo, kOwnP ? 32 : 64, y_at(j), j);  // dV += P^T dout
          tc_commit(bar_pdone);
          tc_commit(bar_yempty(j % kSY));
          if (!kOwnP && more && !(mbar_wait(bar_pdone, j & 1, abort_flag) && next_s(j + 1))) break;
        }
        if (!mbar_wait(bar_ds, j & 1, abort_flag)) break;
        tc_fence_after();
        last(KEYS ? tB : tA, tDP, 64, x_at(j), j);  // dK += dS^T Q, dQ += dS K
        tc_commit(bar_dsdone);
        tc_commit(bar_xempty(j % kSX));
        if (more) {  // dP'(j + 1), over dS once that product has read it
          if (!y_in(j + 1) || !mbar_wait(bar_dsdone, j & 1, abort_flag)) break;
          tc_fence_after();
          scores(tDP, 1, y_at(j + 1));
          tc_commit(bar_dp);
          if (!KEYS) tc_commit(bar_yempty((j + 1) % kSY));
        }
      }
      tc_commit(bar_drain);
      volatile int never = 0;
      mbar_wait(bar_drain, 0, &never);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    const int wg = (warp - 2) >> 2;  // columns 64 wg .. 64 wg + 63 of every tile
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const bool live = f0 + r < (KEYS ? n : g.R);  // a row (key) with values
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int tid = (threadIdx.x - 64) & 127;
    const long long rowb = bh * g.R;
    const unsigned long long sc2 = f2pack(g.scale_log2, g.scale_log2);
    // dq: this row's -lse2 and -D; dk, dv: those of the streamed rows, through shared memory
    float nl = 0.f, nd = 0.f;
    if (!KEYS && live) {
      nl = -lse_log2(g.lse[rowb + f0 + r]);
      nd = -g.D[rowb + f0 + r];
    }
    float* const stat = reinterpret_cast<float*>(sbase + L::kStat) + wg * 4 * 64;
    // thread tid < 64: -lse2 of streamed row tid of the warpgroup's in tile j, else -D of row tid - 64
    auto row_stat = [&](int j) -> float {
      const int i = j * kBT + 64 * wg + (tid & 63);
      if (tid < 64) return i < g.R ? -lse_log2(g.lse[rowb + i]) : -INFINITY;
      return i < g.R ? -g.D[rowb + i] : 0.f;
    };
    bool ok = true;
    if (kFixTmem && nt > 0) {  // warpgroup 0 copies its rows of F0, warpgroup 1 of F1
      ok = __all_sync(0xffffffffu, mbar_wait(bar_fix, 0, abort_flag));
      if (ok) {
        uint32_t w[D / 2];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(sbase + (wg ? L::kF1 : L::kF0) + (c >> 3) * (128 * 128) + r * 128 +
                                                          (((c & 7) ^ (r & 7)) << 4));
          w[4 * c] = u.x;
          w[4 * c + 1] = u.y;
          w[4 * c + 2] = u.z;
          w[4 * c + 3] = u.w;
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tmem_st32u(tF + wg * (D / 2) + 32 * c + lane_off, w + 32 * c);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ft);
      }
    }
    float pre = KEYS && nt > 0 ? row_stat(0) : 0.f;
    // tile j; LAST: the last one, of which only some streamed rows may have values
    auto work = [&](int j, auto LAST) {
      constexpr bool kLast = decltype(LAST)::value;
      const float* st = stat + (j & 1) * 2 * 64;
      if (KEYS) {
        // into this tile's buffer (the other one may still be read by a warp on the last tile); the next
        // tile's are loaded now and land while this one is worked on
        stat[(j & 1) * 2 * 64 + tid] = pre;
        if (j + 1 < nt) pre = row_stat(j + 1);
        __syncwarp();
        asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_s, j & 1, abort_flag));
      if (!ok) return;
      tc_fence_after();
      const uint32_t tS = tmem + 64 * wg + lane_off, tP = tDP + 64 * wg + lane_off;
      const int lim = kLast ? str_rows - j * kBT - 64 * wg : 64;  // streamed rows of the half tile with values
      float p[64];
      tmem_ld64(tS, p);
      if (!KEYS || kOwnP) {  // S' has been read: the next one may come
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_r);
      }
      if (KEYS && kLast) {  // the others' lse is +inf: p = 0
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= lim) p[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        float4 l4 = make_float4(nl, nl, nl, nl);
        if (KEYS) l4 = *reinterpret_cast<const float4*>(st + e);
        f2unpack(f2fma(f2pack(p[e], p[e + 1]), sc2, f2pack(l4.x, l4.y)), p[e], p[e + 1]);
        f2unpack(f2fma(f2pack(p[e + 2], p[e + 3]), sc2, f2pack(l4.z, l4.w)), p[e + 2], p[e + 3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[e + i] = KEYS && !live ? 0.f : ex2(p[e + i]);
      }
      if (KEYS) {
        uint32_t pk[32];  // (p, and ds below, in bf16 for the products: 2^-8 of each at most; ds is made of the unrounded p)
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          __nv_bfloat162 b2 = __floats2bfloat162_rn(p[e], p[e + 1]);
          pk[e >> 1] = *reinterpret_cast<uint32_t*>(&b2);
        }
        if (kOwnP && j > 0) {  // dV of the last tile has read P
          ok = __all_sync(0xffffffffu, mbar_wait(bar_pdone, (j - 1) & 1, abort_flag));
          if (!ok) return;
          tc_fence_after();
        }
        tmem_st32u(kOwnP ? tPo + 32 * wg + lane_off : tS, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar_dp, j & 1, abort_flag));
      if (!ok) return;
      tc_fence_after();
      {
        float y[64];
        tmem_ld64(tP, y);
        if (KEYS && kLast) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= lim) y[e] = 0.f;
        }
        uint32_t dk[32];
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          float4 d4 = make_float4(nd, nd, nd, nd);
          if (KEYS) d4 = *reinterpret_cast<const float4*>(st + 64 + e);
          float s0, s1, s2, s3;
          f2unpack(f2mul(f2pack(p[e], p[e + 1]), f2add(f2pack(y[e], y[e + 1]), f2pack(d4.x, d4.y))), s0, s1);
          f2unpack(f2mul(f2pack(p[e + 2], p[e + 3]), f2add(f2pack(y[e + 2], y[e + 3]), f2pack(d4.z, d4.w))), s2, s3);
          if (KEYS ? !live : kLast && e >= lim) s0 = 0.f;
          if (KEYS ? !live : kLast && e + 1 >= lim) s1 = 0.f;
          if (KEYS ? !live : kLast && e + 2 >= lim) s2 = 0.f;
          if (KEYS ? !live : kLast && e + 3 >= lim) s3 = 0.f;
          __nv_bfloat162 b0 = __floats2bfloat162_rn(s0, s1), b1 = __floats2bfloat162_rn(s2, s3);
          dk[e >> 1] = *reinterpret_cast<uint32_t*>(&b0);
          dk[(e >> 1) + 1] = *reinterpret_cast<uint32_t*>(&b1);
        }
        tmem_st32u(tP, dk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ds);
    };
#pragma unroll 1
    for (int j = 0; j + 1 < nt; ++j) work(j, std::false_type());
    if (nt > 0) work(nt - 1, std::true_type());
    // ---- epilogue: a thread writes (a share of) its row; without tiles, and behind a sequence's keys (whose
    // sums are 0 times q and dout, which may hold an infinity), zeros; for a bad length NaN
    const bool have = __all_sync(0xffffffffu, ok && nt > 0 && mbar_wait(bar_drain, 0, abort_flag));
    if (have) tc_fence_after();
    const bool write = f0 + r < fixed_rows;
    const long long at = (bh * fixed_rows + f0 + r) * D;
    const float tau = g.scale_log2 / kLog2e, none = bad ? __int_as_float(0x7fffffff) : 0.f;
    auto put = [&](uint32_t acc, void* dst, float scale, int c_begin, int c_end) {
#pragma unroll 1
      for (int c = c_begin; c < c_end; c += 32) {
        float o[32];
        __syncwarp();  // (TMEM is read by whole warps, also where some of their rows are not written)
        if (have) tmem_ld32(acc + lane_off + c, o);
        if (!have || !live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = none;
        }
        if (!write) continue;
        uint4* const p = reinterpret_cast<uint4*>((__nv_bfloat16*)dst + at + c);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 v2 = __floats2bfloat162_rn(o[8 * u + 2 * e] * scale, o[8 * u + 2 * e + 1] * scale);
            w[e] = *reinterpret_cast<uint32_t*>(&v2);
          }
          p[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    if (have || nt == 0) {
      if (KEYS) {
        if (wg == 0) put(tB, g.dk, tau, 0, D);
        else put(tA, g.dv, 1.f, 0, D);
      } else {
        put(tA, g.dq, tau, wg * (D / 2), (wg + 1) * (D / 2));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
  }
}

template <int D>
__global__ void __launch_bounds__(kBwdTcThreads, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, GParams prm) {
  using L = GSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + L::kTotal > (uint32_t)L::kAlloc) {  // the plan does not fit: refuse, touch nothing
    if (threadIdx.x == 0) raise_error(kErrInternal);
    return;
  }
  uint8_t* const sbase = smem_raw + (base - raw);
  long long c = (long long)blockIdx.x - prm.dkv_at;
  if (c >= 0 && c < prm.n_dkv) {
    cross_bwd_cta<D, true>(&mk, &mv, &mq, &mg, prm, base, sbase, c / prm.key_tiles, (int)(c % prm.key_tiles));
  } else {
    c = (long long)blockIdx.x - prm.dq_at;
    cross_bwd_cta<D, false>(&mq, &mg, &mk, &mv, prm, base, sbase, c / prm.row_tiles, (int)(c % prm.row_tiles));
  }
}

template <int D>
cudaError_t launch_cross_bwd(const CrossGradArgs& g, long long bh, cudaStream_t s, const char** why) {
  using L = GSmem<D>;
  row_dot_kernel<__nv_bfloat16><<<(unsigned)((g.rows + 7) / 8), 256, 0, s>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap m[4];
  const void* ptr[4] = {g.q, g.dout, g.k, g.v};
  for (int i = 0; i < 4; ++i)
    if (!make_map(&m[i], ptr[i], (int)bh, i < 2 ? g.R : g.n_kv, D, BM)) {
      *why = "cuTensorMapEncodeTiled failed";
      return cudaErrorInvalidValue;
    }
  static std::atomic<bool> done[kSmemDevices];
  e = allow_smem(cross_bwd_kernel<D>, L::kAlloc, done);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute";
    return e;
  }
  GParams p;
  p.g = g;
  p.key_tiles = (g.n_kv + BM - 1) / BM;
  p.row_tiles = (g.R + BM - 1) / BM;
  p.n_dkv = bh * p.key_tiles;
  const long long n_dq = bh * p.row_tiles, grid = p.n_dkv + n_dq;
  // the kind whose CTAs take longer first: a dq CTA streams n_kv keys with three products a tile, a
  // dk, dv CTA R rows with four
  const bool dq_first = 3LL * g.n_kv > 4LL * g.R;
  p.dkv_at = dq_first ? n_dq : 0;
  p.dq_at = dq_first ? 0 : p.n_dkv;
  cross_bwd_kernel<D><<<(unsigned)grid, kBwdTcThreads, L::kAlloc, s>>>(m[0], m[1], m[2], m[3], p);
  *why = "cross-attention backward kernel launch";
  return cudaGetLastError();
}

}  // namespace ctb
}  // namespace pia
