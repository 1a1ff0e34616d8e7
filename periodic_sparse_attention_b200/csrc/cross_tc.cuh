// cross_tc.cuh -- cross attention of many rows on Blackwell tensor cores (tcgen05 + TMEM + TMA), bf16,
// head size 64 or 128.
//
// A CTA takes 256 rows of one key head as two 128-row tiles and walks its keys in 128-key tiles, one CTA
// an SM.  Per row tile and key tile the products take 4 x 128^2 x d flops = 8 d cycles of the tensor pipe
// and the 128^2 exponentials 1024 cycles of the special-function units, so at d = 128 the two cost the
// same and the point is to run them at once: while one row tile's softmax runs, the other's products do.
// Each row tile has its own softmax warpgroup (one row a thread).  One warp issues the products, a row
// tile's P V and its next Q K^T together before the other's: with an issuing warp for each, the two
// chains ran in step, both in their softmax and then both in their products (8192 x 16384 rows of 16
// heads, d = 128: 1.16 ms against 1.02 ms).
//
//   S = Q K^T (128 x 128, fp32 in TMEM), p = 2^(s - m) in bf16, O += P V (128 x d, fp32 in TMEM)
//
// with the lazy reference m of the prefill kernel: raised, and O rescaled, only where a tile's maximum
// passes it by more than 2^8.
//
// TMEM (512 columns): S of the two tiles (2 x 128), O (2 x d); d = 64 leaves 128 columns, which hold the
// two P (64 columns each), so that the next Q K^T is issued before this tile's P V and the softmax never
// waits for products.  At d = 128 P lies over the S columns it came from, and the next Q K^T waits for
// the P V that reads it.
// Shared units: where 256-row units would leave half of the SMs or more idle -- a call with few units, or the
// last wave of one with many -- a unit becomes a cluster of up to 8 CTAs that take a share of the keys
// each, as many as all units' clusters fit the GPU at once (a GPC's SMs set that: 74 clusters of 2, 33 of 4,
// 22 of 6, 15 of 8).  At the end every CTA leaves its sums in shared memory and finishes a slice of the
// columns of both row tiles from all of them (16 heads of 8192 x 16384 rows, d = 128, 3.46 waves: 1.02 to
// 0.91 ms, 1.21 PFLOP/s, in short runs, 1.04 ms, 1.06 PFLOP/s, in long ones at the power limit; at d = 64,
// where the exponentials alone take 0.46 ms, 0.77 ms; 16 heads of 256 x 16384 rows: 59 us against 74 in the
// few-rows kernel's 64-row CTAs).  A grid with full waves runs as clusters of two throughout, larger ones
// would not fill the SMs.
// Shared memory: Q 2 x 128 rows, rings of 128-key tiles (two of K and two of V at d = 128, four and
// four at d = 64), each loaded by TMA; V of a sequence's last keys row by row with zeros behind the end,
// since 0 times what the padding holds has to be 0.
#pragma once
#include <mutex>

#include "rows_tc.cuh"

namespace pia {
namespace ctf {
using namespace tc;

constexpr int BK = 128;
constexpr int kThreadsBig = 384;  // warp 0 loads, 1 issues, 3 holds the TMEM, 4-7 and 8-11 softmax

template <int D>
struct FSmem {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kQ = 0;                       // two tiles
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kBar = kV + kStages * kTile;
  // q, k_full, k_empty, v_full, v_empty [stages], s_full, p_full, pv_done [2], drain
  static constexpr int kNumBars = 1 + 4 * kStages + 7;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kMl = (kMisc + 8 + 15) / 16 * 16;  // shared units: m and l of the rows
  static constexpr int kTotal = kMl + 2048;
  static_assert(kStages * kTile >= 128 * D * 4, "a side's sums fit K's, the other's V's memory");
  static constexpr int kAlloc = rtc::tmem_smem(512);  // (all an SM has: the kernel holds all of its TMEM)
  static_assert(kTotal + 1024 - 128 <= kAlloc, "the plan fits");
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kBar % 8 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreadsBig, 1)
    cross_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo, RowsArgs a,
                    long long whole, int shares) {
  using L = FSmem<D>;
  constexpr int NS = L::kStages;
  constexpr bool kOver = D == 128;  // P over S
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sbase = smem_raw + (base - raw);
  if (base - raw + L::kTotal > (uint32_t)L::kAlloc) {  // the plan does not fit: refuse, touch nothing
    if (threadIdx.x == 0) raise_error(kErrInternal);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (a.R + 255) / 256;
  // units (256 rows of a head) below `whole` have a CTA, the others a cluster of `shares` CTAs
  const bool paired = blockIdx.x >= whole;
  const int rank = paired ? (int)((blockIdx.x - whole) % shares) : 0;
  const long long unit = paired ? whole + (blockIdx.x - whole) / shares : blockIdx.x;
  if (unit >= (long long)a.rows / a.R * tiles) return;  // (the grid is a whole number of clusters)
  const long long bh = unit / tiles;
  const int r0 = (int)(unit % tiles) * 256;
  int n = a.kv_len ? a.kv_len[bh / a.heads] : a.n_kv;
  const bool bad = n < 0 || n > a.n_kv;
  if (bad) {
    if (threadIdx.x == 0) raise_error(kErrCacheLen);
    n = 0;
  }
  const int all_nt = (n + BK - 1) / BK;
  // first tile of this CTA, and how many
  const int t0 = paired ? (int)((long long)all_nt * rank / shares) : 0;
  const int nt = paired ? (int)((long long)all_nt * (rank + 1) / shares) - t0 : all_nt;
  const int sides = r0 + 128 < a.R ? 2 : 1;  // row tiles that exist

  const uint32_t sQ = base + L::kQ, sK = base + L::kK, sV = base + L::kV, bar_q = base + L::kBar;
  auto bar_kfull = [&](int s) { return bar_q + 8u * (1 + s); };
  auto bar_kempty = [&](int s) { return bar_q + 8u * (1 + NS + s); };
  auto bar_vfull = [&](int s) { return bar_q + 8u * (1 + 2 * NS + s); };
  auto bar_vempty = [&](int s) { return bar_q + 8u * (1 + 3 * NS + s); };
  auto bar_sfull = [&](int i) { return bar_q + 8u * (1 + 4 * NS + i); };
  auto bar_pfull = [&](int i) { return bar_q + 8u * (3 + 4 * NS + i); };
  auto bar_pv = [&](int i) { return bar_q + 8u * (5 + 4 * NS + i); };
  const uint32_t bar_drain = bar_q + 8u * (7 + 4 * NS);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + L::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + L::kMisc + 4);

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmq) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmv) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmo) : "memory");
    mbar_init(bar_q, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_kfull(s), 1);
      mbar_init(bar_kempty(s), 1);
      mbar_init(bar_vfull(s), 1);
      mbar_init(bar_vempty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_sfull(i), 1);
      mbar_init(bar_pfull(i), 4);
      mbar_init(bar_pv(i), 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (nt > 0) {
      mbar_expect_tx(bar_q, sides * L::kTile);
      for (int i = 0; i < sides; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sQ + i * L::kTile + c * 128 * 128, &tmq, bar_q, c * 64, r0 + 128 * i, (int)bh);
    }
  }
  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // S of side i at 128 i, O at 256 + D i, P over S or (d = 64) at 384 + 64 i
  auto tS = [&](int i) { return tmem + 128 * i; };
  auto tO = [&](int i) { return tmem + 256 + D * i; };
  auto tP = [&](int i) { return kOver ? tmem + 128 * i : tmem + 384 + 64 * i; };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    int nk = 0, nv = 0;
    for (int j = 0; j < nt; ++j) {
      const int s = j % NS;
      if (!__all_sync(0xffffffffu, j < NS || mbar_wait(bar_kempty(s), (j / NS - 1) & 1, abort_flag))) break;
      if (lane == 0) {
        mbar_expect_tx(bar_kfull(s), L::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sK + s * L::kTile + c * BK * 128, &tmk, bar_kfull(s), c * 64, (t0 + j) * BK, (int)bh);
      }
      ++nk;
      if (!__all_sync(0xffffffffu, j < NS || mbar_wait(bar_vempty(s), (j / NS - 1) & 1, abort_flag))) break;
      if ((t0 + j + 1) * BK <= n) {
        if (lane == 0) {
          mbar_expect_tx(bar_vfull(s), L::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sV + s * L::kTile + c * BK * 128, &tmv, bar_vfull(s), c * 64, (t0 + j) * BK, (int)bh);
        }
      } else {
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const int sub = lane % LPR, slot = lane / LPR;
        const long long row0 = bh * a.n_kv + (long long)(t0 + j) * BK;
#pragma unroll 8
        for (int i = 0; i < BK / RPI; ++i) {
          const int key = i * RPI + slot;
          const bool in = (t0 + j) * BK + key < n;
          rtc::cp_async16(sV + s * L::kTile + (sub >> 3) * (BK * 128) + key * 128 + (((sub & 7) ^ (key & 7)) << 4),
                          (const __nv_bfloat16*)a.v + (in ? (row0 + key) * D + sub * 8 : 0), in ? 16 : 0);
        }
        rtc::cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_vfull(s));
      }
      ++nv;
    }
    if (*abort_flag) {  // let the loads in flight land before the CTA can exit
      volatile int never = 0;
      if (nt > 0) mbar_wait(bar_q, 0, &never);
      for (int u = nk > NS ? nk - NS : 0; u < nk; ++u) mbar_wait(bar_kfull(u % NS), (u / NS) & 1, &never);
      for (int u = nv > NS ? nv - NS : 0; u < nv; ++u) mbar_wait(bar_vfull(u % NS), (u / NS) & 1, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && nt > 0) {
      constexpr uint32_t id_s = idesc_bf16(128, BK, 0), id_o = idesc_bf16(128, D, 1);
      auto qk = [&](int i, int j) -> bool {
        const int s = j % NS;
        if (!mbar_wait(bar_kfull(s), (j / NS) & 1, abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          tc_mma(tS(i), sw128_desc(sQ + i * L::kTile + in, 16, 1024), sw128_desc(sK + s * L::kTile + in, 16, 1024), id_s,
                 kk > 0 ? 1u : 0u);
        }
        tc_commit(bar_sfull(i));
        if (i == sides - 1) tc_commit(bar_kempty(s));  // (covers the other side's, issued before)
        return true;
      };
      auto step = [&](int i, int j) -> bool {
        const int s = j % NS;
        if (!mbar_wait(bar_pfull(i), j & 1, abort_flag)) return false;  // every row has read S and written P
        if (!kOver && j + 1 < nt && !qk(i, j + 1)) return false;
        if (!mbar_wait(bar_vfull(s), (j / NS) & 1, abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_ts(tO(i), tP(i) + 8 * kk, sw128_desc(sV + s * L::kTile + kk * 16 * 128, BK * 128, 1024), id_o,
                    (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bar_pv(i));
        if (i == sides - 1) tc_commit(bar_vempty(s));
        return !(kOver && j + 1 < nt) || (mbar_wait(bar_pv(i), j & 1, abort_flag) && qk(i, j + 1));
      };
      bool okw = mbar_wait(bar_q, 0, abort_flag);
      for (int i = 0; okw && i < sides; ++i) okw = qk(i, 0);
      // a side's P V and its next Q K^T together, before the other side's: the sides' softmaxes then
      // run one after the other, each while the other side's products do
      for (int j = 0; okw && j < nt; ++j)
        for (int i = 0; okw && i < sides; ++i) okw = step(i, j);
      tc_commit(bar_drain);
      volatile int never = 0;
      mbar_wait(bar_drain, 0, &never);
    }
    __syncwarp();
  } else if (warp >= 4 && (warp >> 2) - 1 < sides) {
    // ---------------------------------------------------------------- softmax of side i, one row a thread
    const int i = (warp >> 2) - 1, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t S = tS(i) + lane_off, O = tO(i) + lane_off, P = tP(i) + lane_off;
    const float NEG_INF = -INFINITY;
    float m_ref = NEG_INF, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; ok && j < nt; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_sfull(i), j & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float x[128];
      tmem_ld64(S, x);
      tmem_ld64(S + 64, x + 64);
      const int lim = n - (t0 + j) * BK;
      if (lim < BK) {
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e >= lim) x[e] = NEG_INF;
      }
      float mx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float m = max3f(x[e], x[8 + e], x[16 + e]);
#pragma unroll
        for (int u = 24; u + 8 < 128; u += 16) m = max3f(m, x[u + e], x[u + 8 + e]);
        mx[e] = fmaxf(m, x[120 + e]);
      }
      const float mt =
          max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * a.scale_log2;
      // (by selection: TMEM is written by whole warps below)
      const bool up = mt > m_ref + kRescaleThreshold || (m_ref == NEG_INF && mt > NEG_INF);
      const bool rescale = up && m_ref != NEG_INF;
      const float f = rescale ? ex2(m_ref - mt) : 1.f;
      l *= f;
      m_ref = up ? mt : m_ref;
      const float neg = m_ref == NEG_INF ? 0.f : -m_ref;
      const unsigned long long sc2 = f2pack(a.scale_log2, a.scale_log2), nn = f2pack(neg, neg);
      if (!kOver && j > 0) {  // P of the last tile has been read
        ok = __all_sync(0xffffffffu, mbar_wait(bar_pv(i), (j - 1) & 1, abort_flag));
        if (!ok) break;
      }
      unsigned long long sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float t0, t1;
          f2unpack(f2fma(f2pack(x[32 * c + e], x[32 * c + e + 1]), sc2, nn), t0, t1);
          const float p0 = ex2(t0), p1 = ex2(t1);
          // (bf16 for the product: 2^-8 of a weight at most; the sum takes the weights as they are)
          __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
          pk[e >> 1] = *reinterpret_cast<uint32_t*>(&b2);
          sum[(e >> 1) & 3] = f2add(sum[(e >> 1) & 3], f2pack(p0, p1));
        }
        tmem_st16(P + 16 * c, pk);
      }
      // the last product has completed: at d = 128 this tile's Q K^T was issued after it
      if (__any_sync(0xffffffffu, rescale)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(O + 32 * c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(O + 32 * c, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pfull(i));
      float s0, s1;
      f2unpack(f2add(f2add(sum[0], sum[1]), f2add(sum[2], sum[3])), s0, s1);
      l += s0 + s1;
    }
    // ---- epilogue: the rows go through the Q tile's memory (its last product is done) to one TMA
    // store, which the tensor map clips at the head's last row
    const bool have = __all_sync(0xffffffffu, ok && nt > 0 && mbar_wait(bar_pv(i), (nt - 1) & 1, abort_flag));
    if (have) tc_fence_after();
    const float none = bad ? __int_as_float(0x7fffffff) : 0.f;
    if (paired) {
      // this CTA's sums of the side to K's (side 1: V's) memory, a column of 128 rows after the other, m
      // and l beside it.  (K and V have been read for the last time: the commit that bar_pv counts covers
      // every product issued before it, and side 1's last is the last of all.)
      float* const sums = reinterpret_cast<float*>(sbase + (i ? L::kV : L::kK));
      float* const ml = reinterpret_cast<float*>(sbase + L::kMl) + 256 * i;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (have) {
          tmem_ld32(O + c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) sums[(c + e) * 128 + r] = o[e];
      }
      ml[r] = m_ref;
      ml[128 + r] = l;
      cluster_sync();  // (for all threads of the cluster; the other warps wait below)
      const uint32_t pm = base + L::kMl + 1024 * i + 4 * r, po = (i ? sV : sK) + 4 * r;
      float w[kMaxCluster], M = NEG_INF, sum = 0.f;
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p) {
        w[p] = p < shares ? peer_f32(peer_addr(pm, p)) : NEG_INF;
        M = fmaxf(M, w[p]);
      }
      const float ref = M == NEG_INF ? 0.f : M;
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p) {
        w[p] = ex2(w[p] - ref);
        if (p < shares) sum = fmaf(peer_f32(peer_addr(pm + 512, p)), w[p], sum);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const bool row_ok = r0 + 128 * i + r < a.R;
      const long long row = bh * a.R + r0 + 128 * i + r;
#pragma unroll 1
      for (int c = 8 * rank; c < D; c += 8 * shares) {
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p)
          if (p < shares) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(peer_f32(peer_addr(po + (c + e) * 512, p)), w[p], o[e]);
          }
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          __nv_bfloat162 b2 = __floats2bfloat162_rn(bad ? none : o[2 * e] * inv, bad ? none : o[2 * e + 1] * inv);
          q[e] = *reinterpret_cast<uint32_t*>(&b2);
        }
        if (row_ok) *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + row * D + c) = make_uint4(q[0], q[1], q[2], q[3]);
      }
      if (a.lse && rank == 0 && row_ok) a.lse[row] = bad ? none : sum == 0.f ? NEG_INF : (M + log2f(sum)) * kLn2;
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (have) {
          tmem_ld32(O + 32 * c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 b2 = __floats2bfloat162_rn(bad ? none : o[8 * u + 2 * e] * inv, bad ? none : o[8 * u + 2 * e + 1] * inv);
            q[e] = *reinterpret_cast<uint32_t*>(&b2);
          }
          const int cc = 4 * c + u;  // 16-byte chunk of the row
          *reinterpret_cast<uint4*>(sbase + L::kQ + i * L::kTile + (cc >> 3) * (128 * 128) + r * 128 +
                                    (((cc & 7) ^ (r & 7)) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory");
      if (ok && q4 == 0 && lane == 0) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tma_store_3d(&tmo, sQ + i * L::kTile + c * 128 * 128, c * 64, r0 + 128 * i, (int)bh);
        tma_store_commit_and_wait_read();
      }
      if (a.lse && ok && r0 + 128 * i + r < a.R)
        a.lse[bh * a.R + r0 + 128 * i + r] = bad ? none : l == 0.f ? NEG_INF : (m_ref + log2f(l)) * kLn2;
    }
    tc_fence_before();
  }
  if (paired) {
    if (warp < 4 || (warp >> 2) - 1 >= sides) cluster_sync();
    cluster_sync();  // no CTA leaves while another reads it
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 3)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// Once per device: the shared memory above 48 KB, and how many clusters of each size are resident at once.
struct Fit {
  bool done = false;
  int sms = 0, clusters[kMaxCluster + 1] = {};
};
template <int D>
cudaError_t fit(const Fit** out) {
  static Fit fits[64];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  Fit& f = fits[dev];
  if (!f.done) {
    e = cudaFuncSetAttribute(cross_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, FSmem<D>::kAlloc);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&f.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int c = 2; e == cudaSuccess && c <= kMaxCluster; ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(c * f.sms));
      cfg.blockDim = dim3(kThreadsBig);
      cfg.dynamicSmemBytes = FSmem<D>::kAlloc;
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = (unsigned)c;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&f.clusters[c], cross_tc_kernel<D>, &cfg);
    }
    if (e != cudaSuccess) return e;
    f.done = true;
  }
  *out = &f;
  return cudaSuccess;
}

// How `units` 256-row units run: units below `whole` as one CTA each, the others as clusters of `shares`.
struct Shape {
  long long whole, grid;
  int shares;
};
inline Shape cross_shape(long long units, int n_kv, const Fit& f) {
  const int most = (n_kv + 2 * BK - 1) / (2 * BK);  // shares of two key tiles at least
  Shape p;
  if (units >= f.sms) {
    const long long rest = units % f.sms;
    const bool split = rest > 0 && rest <= f.clusters[2] && most >= 2;
    p.shares = 2;
    p.whole = split ? units - rest - (units - rest) % 2 : units;
    p.grid = split ? p.whole + 2 * (units - p.whole) : units + units % 2;
    if (!split) p.whole = p.grid;
    return p;
  }
  p.shares = 1;
  for (int c = 2; c <= kMaxCluster && c <= most; ++c)
    if (units <= f.clusters[c]) p.shares = c;
  p.whole = p.shares > 1 ? 0 : units;
  p.grid = units * p.shares;
  return p;
}

template <int D>
cudaError_t launch_cross(const RowsArgs& a, long long bh, cudaStream_t s, const char** why) {
  using L = FSmem<D>;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map(&mq, a.q, (int)bh, a.R, D, 128) || !make_map(&mk, a.k, (int)bh, a.n_kv, D, BK) ||
      !make_map(&mv, a.v, (int)bh, a.n_kv, D, BK) || !make_map(&mo, a.out, (int)bh, a.R, D, 128)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  const Fit* f = nullptr;
  cudaError_t e = fit<D>(&f);
  if (e != cudaSuccess) {
    *why = "cross-attention kernel attributes";
    return e;
  }
  const Shape shape = cross_shape(bh * ((a.R + 255) / 256), a.n_kv, *f);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)shape.grid);
  cfg.blockDim = dim3(kThreadsBig);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)shape.shares;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = shape.shares > 1 ? 1 : 0;
  *why = "cross-attention kernel launch";
  return cudaLaunchKernelEx(&cfg, cross_tc_kernel<D>, mq, mk, mv, mo, a, shape.whole, shape.shares);
}

}  // namespace ctf
}  // namespace pia
