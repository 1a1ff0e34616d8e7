// cross_bwd_tc.cuh -- gradients of cross attention on Blackwell tensor cores (tcgen05 + TMEM + TMA),
// bf16, head size 64 or 128.
//
// With p = exp(s - lse) and ds = p (dout . v - D) as in cross_simt.cuh, two kinds of CTA in one launch,
// each holding 128 rows of one side and streaming 64-row tiles of the other:
//
//   dk, dv   128 keys fixed (F0 = K, F1 = V), row tiles streamed (X = Q, Y = dout):
//            S^T = K Q^T, dP^T = V dout^T;  dV += P^T dout, dK += dS^T Q
//   dq       128 rows fixed (F0 = Q, F1 = dout), key tiles streamed (X = K, Y = V):
//            S = Q K^T, dP = dout V^T;  dQ += dS K
//
// so both compute S' = F0 X^T and dP' = F1 Y^T, 128 x 64 in fp32 in TMEM.  One thread a row of them
// forms p and ds and writes them in bf16 over the columns it has read, from where the last products
// take them as their A operand; the streamed tile is their B operand, as it lies.  The score products
// are done twice (7 products in place of 5): the price of sums that stay in one CTA, with no atomics
// and no order of addition left to chance.  The kind with the longer CTAs comes first in the grid, the
// other fills the SMs behind it.
//
// D = 128: one CTA an SM, two pairs of S', dP' and two softmax warpgroups that take the tiles in turn, so
// that the products of one tile run while the other's exponentials do (TMEM: 2 x 128 + 2 x 128
// columns).  D = 64: two CTAs an SM with one pair and one warpgroup each.
//
// Rows behind a sequence's end: K of a partial key tile is loaded with zeros there (its dS is 0, and
// 0 times what the padding holds has to be 0), and scores are set aside by selection, not arithmetic.
// Streamed rows past the last one come as zeros with lse = +inf, so their p is 0.
#pragma once
#include "rows_tc.cuh"

namespace pia {
namespace ctb {
using namespace tc;

constexpr int kStages = 4;  // of the streamed ring: a tile is held until its last product is done

template <int D>
struct GSmem {
  static constexpr int kCtas = D == 64 ? 2 : 1;
  static constexpr int kNbuf = D == 64 ? 1 : 2;
  static constexpr int kThreads = 64 + 128 * kNbuf;
  static constexpr int kFix = BM * D * 2;             // a fixed tile
  static constexpr int kStr = BN * D * 2;             // a streamed tile
  static constexpr int kF0 = 0;
  static constexpr int kF1 = kF0 + kFix;
  static constexpr int kX = kF1 + kFix;
  static constexpr int kY = kX + kStages * kStr;
  static constexpr int kBar = kY + kStages * kStr;
  // fixed, full[stages], empty[stages], s_full[nbuf], p_full[nbuf], done[nbuf], drain
  static constexpr int kNumBars = 1 + 2 * kStages + 3 * kNbuf + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kStat = (kMisc + 8 + 15) / 16 * 16;        // dk, dv: -lse2 and -D of a tile's rows,
  static constexpr int kTotal = kStat + kNbuf * 2 * 2 * BN * 4;   // two buffers a warpgroup
  static constexpr int kAlloc = kTotal + 1024 - 128;
  static constexpr int kTmem = kNbuf == 1 ? 256 : 512;
  static_assert(2 * BN * kNbuf + 2 * D <= kTmem && kTmem * kCtas <= 512, "TMEM columns");
  static_assert(kX % 1024 == 0 && kY % 1024 == 0 && kBar % 8 == 0, "alignment");
  static_assert(kAlloc <= 228 * 1024 / kCtas - 1024, "shared memory of the CTAs on one SM");
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
  constexpr int NBUF = L::kNbuf;
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
  const int nt = KEYS && f0 >= n ? 0 : (str_rows + BN - 1) / BN;

  const uint32_t sF0 = base + L::kF0, sF1 = base + L::kF1, sX = base + L::kX, sY = base + L::kY;
  const uint32_t bar_fix = base + L::kBar;
  auto bar_full = [&](int s) { return bar_fix + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return bar_fix + 8u * (1 + kStages + s); };
  auto bar_sfull = [&](int i) { return bar_fix + 8u * (1 + 2 * kStages + i); };
  auto bar_pfull = [&](int i) { return bar_fix + 8u * (1 + 2 * kStages + NBUF + i); };
  auto bar_done = [&](int i) { return bar_fix + 8u * (1 + 2 * kStages + 2 * NBUF + i); };
  const uint32_t bar_drain = bar_fix + 8u * (1 + 2 * kStages + 3 * NBUF);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + L::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + L::kMisc + 4);

  if (threadIdx.x == 0) {
    mbar_init(bar_fix, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(bar_sfull(i), 1);
      mbar_init(bar_pfull(i), 4);
      mbar_init(bar_done(i), 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (nt > 0) {
      mbar_expect_tx(bar_fix, 2 * L::kFix);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        tma_load_3d(sF0 + c * BM * 128, mf0, bar_fix, c * 64, f0, (int)bh);
        tma_load_3d(sF1 + c * BM * 128, mf1, bar_fix, c * 64, f0, (int)bh);
      }
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "n"(L::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // pair i: S' at 128 i, dP' at 128 i + 64; then dQ, or dV and dK
  const uint32_t tA = tmem + 2 * BN * NBUF, tB = tA + D;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    int issued = 0;
    for (int j = 0; j < nt; ++j) {
      const int s = j % kStages;
      if (!__all_sync(0xffffffffu, j < kStages || mbar_wait(bar_empty(s), (j / kStages - 1) & 1, abort_flag))) break;
      if (KEYS || (j + 1) * BN <= n) {
        if (lane == 0) {
          mbar_expect_tx(bar_full(s), 2 * L::kStr);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            tma_load_3d(sX + s * L::kStr + c * BN * 128, mx, bar_full(s), c * 64, j * BN, (int)bh);
            tma_load_3d(sY + s * L::kStr + c * BN * 128, my, bar_full(s), c * 64, j * BN, (int)bh);
          }
        }
      } else {  // the last keys, row by row, with zeros behind the sequence's end
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const int sub = lane % LPR, slot = lane / LPR;
        const long long row0 = bh * g.n_kv + (long long)j * BN;
#pragma unroll 4
        for (int i = 0; i < BN / RPI; ++i) {
          const int key = i * RPI + slot;
          const bool in = j * BN + key < n;
          const long long at = in ? (row0 + key) * D + sub * 8 : 0;
          const uint32_t off = s * L::kStr + (sub >> 3) * (BN * 128) + key * 128 + (((sub & 7) ^ (key & 7)) << 4);
          rtc::cp_async16(sX + off, (const __nv_bfloat16*)g.k + at, in ? 16 : 0);
          rtc::cp_async16(sY + off, (const __nv_bfloat16*)g.v + at, in ? 16 : 0);
        }
        rtc::cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_full(s));
      }
      ++issued;
    }
    if (*abort_flag) {  // let the loads in flight land before the CTA can exit
      volatile int never = 0;
      if (nt > 0) mbar_wait(bar_fix, 0, &never);
      for (int u = issued > kStages ? issued - kStages : 0; u < issued; ++u)
        mbar_wait(bar_full(u % kStages), (u / kStages) & 1, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && nt > 0) {
      constexpr uint32_t id_s = idesc_bf16(BM, BN, 0);  // B (X, Y) K-major
      constexpr uint32_t id_a = idesc_bf16(BM, D, 1);   // B (X, Y) N-major
      bool okw = mbar_wait(bar_fix, 0, abort_flag);
      auto issue_s = [&](int j) -> bool {
        const int s = j % kStages, i = j % NBUF;
        if (!mbar_wait(bar_full(s), (j / kStages) & 1, abort_flag)) return false;
        // the last products of tile j - NBUF read what this S', dP' overwrites
        if (j >= NBUF && !mbar_wait(bar_done(i), (j / NBUF - 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t tS = tmem + i * 2 * BN, tP = tS + BN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk & 3) * 32;
          tc_mma(tS, sw128_desc(sF0 + (kk >> 2) * (BM * 128) + in, 16, 1024),
                 sw128_desc(sX + s * L::kStr + (kk >> 2) * (BN * 128) + in, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk & 3) * 32;
          tc_mma(tP, sw128_desc(sF1 + (kk >> 2) * (BM * 128) + in, 16, 1024),
                 sw128_desc(sY + s * L::kStr + (kk >> 2) * (BN * 128) + in, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar_sfull(i));
        return true;
      };
      auto issue_acc = [&](int j) -> bool {
        const int s = j % kStages, i = j % NBUF;
        if (!mbar_wait(bar_pfull(i), (j / NBUF) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t tS = tmem + i * 2 * BN, tP = tS + BN;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          const uint32_t acc = (j == 0 && kk == 0) ? 0u : 1u;
          if (KEYS) {
            tc_mma_ts(tA, tS + 8 * kk, sw128_desc(sY + s * L::kStr + kk * 16 * 128, BN * 128, 1024), id_a, acc);
            tc_mma_ts(tB, tP + 8 * kk, sw128_desc(sX + s * L::kStr + kk * 16 * 128, BN * 128, 1024), id_a, acc);
          } else {
            tc_mma_ts(tA, tS + 8 * kk, sw128_desc(sX + s * L::kStr + kk * 16 * 128, BN * 128, 1024), id_a, acc);
          }
        }
        tc_commit(bar_done(i));
        tc_commit(bar_empty(s));
        return true;
      };
      // one pair: the last products of tile j - 1, then S' of tile j; two pairs: S' of tile j first
      for (int j = 0; okw; ++j) {
        const bool have = j < nt;
        if (NBUF == 1 && j > 0 && !issue_acc(j - 1)) break;
        if (have && !issue_s(j)) break;
        if (NBUF == 2 && j > 0 && !issue_acc(j - 1)) break;
        if (!have) break;
      }
      tc_commit(bar_drain);
      volatile int never = 0;
      mbar_wait(bar_drain, 0, &never);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    const int wg = (warp - 2) >> 2;  // takes the tiles j with j % NBUF == wg
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const bool live = f0 + r < (KEYS ? n : g.R);  // a row (key) with values
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + wg * 2 * BN + lane_off, tP = tS + BN;
    const int tid = (threadIdx.x - 64) & 127;
    const long long rowb = bh * g.R;
    const unsigned long long sc2 = f2pack(g.scale_log2, g.scale_log2);
    // dq: this row's -lse2 and -D; dk, dv: those of the streamed rows, through shared memory
    float nl = 0.f, nd = 0.f;
    if (!KEYS && live) {
      nl = -g.lse[rowb + f0 + r] * kLog2e;
      nd = -g.D[rowb + f0 + r];
    }
    float* const stat = reinterpret_cast<float*>(sbase + L::kStat) + wg * 4 * BN;
    // thread tid < 64: -lse2 of streamed row tid of tile j, else -D of row tid - 64
    auto row_stat = [&](int j) -> float {
      const int i = j * BN + (tid & 63);
      if (tid < 64) return i < g.R ? -g.lse[rowb + i] * kLog2e : -INFINITY;
      return i < g.R ? -g.D[rowb + i] : 0.f;
    };
    bool ok = true;
    float pre = KEYS && wg < nt ? row_stat(wg) : 0.f;
#pragma unroll 1
    for (int j = wg; j < nt; j += NBUF) {
      const float* st = stat + ((j / NBUF) & 1) * 2 * BN;
      if (KEYS) {
        // into this tile's buffer (the other one may still be read by a warp on the group's last
        // tile); the next tile's are loaded now and land while this one is worked on
        stat[((j / NBUF) & 1) * 2 * BN + tid] = pre;
        if (j + NBUF < nt) pre = row_stat(j + NBUF);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_sfull(wg), (j / NBUF) & 1, abort_flag));
      if (!ok) continue;
      tc_fence_after();
      const int lim = KEYS ? BN : n - j * BN;  // streamed rows of the tile with values
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) {
        float x[32], y[32];
        tmem_ld32(tS + 32 * c, x);
        tmem_ld32(tP + 32 * c, y);
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          unsigned long long l2, d2;
          if (KEYS) {
            const float2 a = *reinterpret_cast<const float2*>(st + 32 * c + e);
            const float2 bb = *reinterpret_cast<const float2*>(st + BN + 32 * c + e);
            l2 = f2pack(a.x, a.y);
            d2 = f2pack(bb.x, bb.y);
          } else {
            l2 = f2pack(nl, nl);
            d2 = f2pack(nd, nd);
          }
          float t0, t1, p0, p1, s0, s1;
          f2unpack(f2fma(f2pack(x[e], x[e + 1]), sc2, l2), t0, t1);
          p0 = ex2(t0);
          p1 = ex2(t1);
          f2unpack(f2mul(f2pack(p0, p1), f2add(f2pack(y[e], y[e + 1]), d2)), s0, s1);
          if (KEYS) {
            if (!live) p0 = p1 = s0 = s1 = 0.f;
          } else if (lim < BN) {
            if (32 * c + e >= lim) s0 = 0.f;
            if (32 * c + e + 1 >= lim) s1 = 0.f;
          }
          __nv_bfloat162 db = __floats2bfloat162_rn(s0, s1);
          dk[e >> 1] = *reinterpret_cast<uint32_t*>(&db);
          if (KEYS) {
            __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
            pk[e >> 1] = *reinterpret_cast<uint32_t*>(&pb);
          }
        }
        if (KEYS) {
          tmem_st16(tS + 16 * c, pk);
          tmem_st16(tP + 16 * c, dk);
        } else {
          tmem_st16(tS + 16 * c, dk);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pfull(wg));
    }
    // ---- epilogue: a thread writes (a share of) its row; without tiles zeros, for a bad length NaN
    const bool have = __all_sync(0xffffffffu, ok && nt > 0 && mbar_wait(bar_drain, 0, abort_flag));
    if (have) tc_fence_after();
    const bool write = f0 + r < fixed_rows;
    const long long at = (bh * fixed_rows + f0 + r) * D;
    const float tau = g.scale_log2 / kLog2e, none = bad ? __int_as_float(0x7fffffff) : 0.f;
    auto put = [&](uint32_t acc, void* dst, float scale, int c_begin, int c_end) {
#pragma unroll 1
      for (int c = c_begin; c < c_end; c += 32) {
        float o[32];
        if (have) {
          tmem_ld32(acc + lane_off + c, o);
        } else {
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
        if (NBUF == 1 || wg == 0) put(tB, g.dk, tau, 0, D);
        if (NBUF == 1 || wg == 1) put(tA, g.dv, 1.f, 0, D);
      } else {
        put(tA, g.dq, tau, wg * (D / NBUF), (wg + 1) * (D / NBUF));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kTmem) : "memory");
  }
}

// mq, mg, mk, mv: boxes of 128 rows; sq, sg, sk, sv: boxes of 64 rows, of q, dout, k, v
template <int D>
__global__ void __launch_bounds__(GSmem<D>::kThreads, GSmem<D>::kCtas)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                     const __grid_constant__ CUtensorMap sq, const __grid_constant__ CUtensorMap sg,
                     const __grid_constant__ CUtensorMap sk, const __grid_constant__ CUtensorMap sv, GParams prm) {
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
    cross_bwd_cta<D, true>(&mk, &mv, &sq, &sg, prm, base, sbase, c / prm.key_tiles, (int)(c % prm.key_tiles));
  } else {
    c = (long long)blockIdx.x - prm.dq_at;
    cross_bwd_cta<D, false>(&mq, &mg, &sk, &sv, prm, base, sbase, c / prm.row_tiles, (int)(c % prm.row_tiles));
  }
}

template <int D>
cudaError_t launch_cross_bwd(const CrossGradArgs& g, long long bh, cudaStream_t s, const char** why) {
  using L = GSmem<D>;
  row_dot_kernel<__nv_bfloat16><<<(unsigned)((g.rows + 7) / 8), 256, 0, s>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap m[8];
  const void* ptr[4] = {g.q, g.dout, g.k, g.v};
  for (int i = 0; i < 8; ++i)
    if (!make_map(&m[i], ptr[i & 3], (int)bh, (i & 3) < 2 ? g.R : g.n_kv, D, i < 4 ? BM : BN)) {
      *why = "cuTensorMapEncodeTiled failed";
      return cudaErrorInvalidValue;
    }
  static bool done[64] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess && !done[dev]) {
    e = cudaFuncSetAttribute(cross_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    done[dev] = e == cudaSuccess;
  }
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
  cross_bwd_kernel<D><<<(unsigned)grid, L::kThreads, L::kAlloc, s>>>(m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], p);
  *why = "cross-attention backward kernel launch";
  return cudaGetLastError();
}

}  // namespace ctb
}  // namespace pia
