// rows_tc.cuh -- attention of few query rows to many keys on Blackwell tensor cores (tcgen05 + TMEM),
// bf16, head size 64 or 128: a generation step's cross attention (the rows of the query heads that
// share a key head together) and the nodes of a tree of drafted tokens.
//
// With few rows the work is one pass over K and V at the memory's rate, and what matters is that
// nothing else takes longer.  A 128-row tile with the queries as its rows would leave most lanes of
// the softmax idle, so both products are taken transposed, keys first:
//
//   S^T = K Q^T      128 keys x RP rows (RP = 16, 32 or 64: the rows, padded)
//   O^T += V^T P^T   d x RP, over the tile's 128 keys
//
// One thread holds one key of the tile and its RP scores, so the exponentials of RP rows are spread
// over all 128 threads whatever RP is.  The running maximum of a row needs the other threads, but
// rarely: p is taken against a reference that is raised only where a score passes it by more than
// 2^8, which one barrier with a vote tells for the whole tile (a row without a reference yet has a bias that
// lifts every finite score past it; scores of -inf need none, their weight is 0); a warp's sums fold into
// one register a lane while the second product runs.  P goes to shared memory in bf16 (K-major, 128-byte
// swizzle) as the second product's B.
//
// A CTA takes up to 64 rows of one key head and a share of its keys (several shares where there are
// few heads).  Up to eight shares form a cluster, whose CTAs read one another's sums from shared
// memory at the end: no second launch and no workspace (a step of 8 heads over 1021 states, d = 64, in a
// replayed graph: 9.3 to 7.9 us); more shares go through a workspace and rows_join_kernel.  CG warpgroups
// of softmax (one of 16 rows' scores, two of RP / 2 rows' each from RP = 32 on: every thread of them holds
// one key and its RP / CG scores), then a warp that issues the products, one that loads K and one that
// loads V.
// A 128-key tile whose rows are consecutive comes by TMA; a tile of scattered rows (the skips, a
// ring's wrap, the drafted tokens) and a list's last tile row by row with cp.async, which fills
// entries without a row with zeros, so that nothing behind a sequence's end is ever multiplied.
// K and V have one 128-row buffer each (64 KB at d = 128): K of the next tile loads while this tile's
// softmax runs, V while the next one's does, and three CTAs an SM (two at RP = 32 and 64) cover
// what that leaves open.
//
// Measured (d = 128; in a replayed graph, and as calls among others): a step of 64 sequences x 8 key heads, 4
// rows each over up to 4096 states, 132 and 135 us, 6.0 TB/s (92 % of the measured copy); trees of up to
// 16 nodes, 64 x 32 heads, 212 and 219 us, 5.7 TB/s; of up to 64 nodes 324 and 343 us, 4.5 TB/s: there the
// softmax threads (masks, exponentials, sums of 64 rows a key) need about as long for a tile as its load
// takes.
//
// Every wait is bounded as in the prefill kernel; a wait that gives up sets the error word and the
// abort flag, every role runs out its loop without work and the CTA frees its TMEM.
#pragma once
#include "cross_simt.cuh"
#include "fwd_tc.cuh"

namespace pia {
namespace rtc {
using namespace tc;

constexpr int BK = 128;         // keys a tile
constexpr int kMaxRows = 64;    // rows a CTA
constexpr int ctas_an_sm(int rp) { return rp == 16 ? 3 : 2; }  // (80 registers a thread, 224 or 352 threads)
// The bias of a row's scores while it has no reference: the largest float, which a finite score (of |q.k| below
// 2^128, times log2(e) / 8 at most) passes the threshold with, and -inf or NaN stay what they are with
// (+inf would make NaN of -inf).  A kind of key whose prior is -inf keeps that, and one whose prior is so low
// that a score with it could overflow counts as -inf until the row has a reference.
constexpr float kNoRef = 3.402823466e38f;
__device__ __forceinline__ float bias_without_ref(float prior) {
  return prior > -0x1p127f ? kNoRef : prior <= -0x1p127f ? -INFINITY : prior;  // (NaN stays)
}

// A CTA of a cluster holds its TMEM columns while it waits for the other CTAs, and one that finds too few
// columns on its SM waits for them: two launches on two streams whose clusters met on two SMs could wait
// for each other.  So every kernel that does this asks for at least the share of an SM's shared memory (228
// KB, of which each CTA costs 1 KB beside what it asks for) that its columns are of 512: CTAs that share
// an SM then never want more columns than there are, whatever their registers would allow.
__host__ __device__ constexpr int tmem_smem(int columns) { return 228 * 1024 / 512 * columns - 1024; }

template <int D, int RP, int MODE>
struct RSmem {
  static constexpr int kCG = RP == 16 ? 1 : 2;        // softmax warpgroups
  static constexpr int kNC = RP / kCG;                // rows of each
  static constexpr int kSoft = 128 * kCG;             // softmax threads
  static constexpr int kThreads = kSoft + 96;
  static constexpr int kTile = BK * D * 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTile;
  static constexpr int kQ = kV + kTile;
  static constexpr int kP = kQ + RP * D * 2;
  static constexpr int kBar = kP + RP * BK * 2;
  // k_full, k_empty, v_full, pv_done, s_full[2], p_full, drain
  static constexpr int kNumBars = 8;
  static constexpr int kMisc = kBar + kNumBars * 8;   // tmem base, abort flag, two tree flags
  static constexpr int kRef = kMisc + 16;             // [RP] reference maxima
  static constexpr int kBl = kRef + RP * 4;           // [RP] the window's prior (cross: 0) less the reference
  static constexpr int kFac = kBl + RP * 4;           // [RP] factors; at the end 1 / sum
  static constexpr int kRed = kFac + RP * 4;          // [4][RP] the warps' maxima, sums
  static constexpr int kPl = kRed + 4 * RP * 4;       // tree: [RP] log2 priors of window and skips
  static constexpr int kPp = kPl + RP * 4;
  static constexpr int kBp = kPp + RP * 4;            // tree: [RP] the skips' prior less the reference
  static constexpr int kX = kBp + RP * 4;             // tree: [RP] depth and position modulo pi of a row
  static constexpr int kPar = kP;                     // tree: parents, then w_g[h] (only before P is
  static constexpr int kWg = kP;                      // written), depths, ancestor bits, and the rows
  static constexpr int kDep = kX + (MODE == kTree ? RP * 8 : 0);
  static constexpr int kAnc = kDep + (MODE == kTree ? kMaxTree : 0);  // (bits of a warpgroup's) at a depth
  static constexpr int kAt = kAnc + (MODE == kTree ? RP * (kMaxTree / 32) * 4 : 0);
  static constexpr int kTotal = kAt + (MODE == kTree ? kMaxTree * RP / 8 : 0);
  static constexpr int kCtas = ctas_an_sm(RP);
  static constexpr int kTmem = RP == 16 ? 64 : RP == 32 ? 128 : 256;  // two S^T, one O^T, a power of two
  static constexpr int kNeed = kTotal + 1024 - 128;
  static constexpr int kAlloc = kNeed > tmem_smem(kTmem) ? kNeed : tmem_smem(kTmem);
  static_assert(RP * BK * 2 >= kMaxTree * 4 && RP * BK * 2 >= D * 4, "the parents, w_g fit P");
  static_assert(RP * D * 4 <= kTile, "a share's sums fit K's buffer");
  static_assert(3 * RP <= kTmem && kTmem * kCtas <= 512, "TMEM columns");
  static_assert(kAlloc >= tmem_smem(kTmem), "a share of shared memory for the columns held in a cluster");
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kBar % 8 == 0 && kRef % 16 == 0 && kAt % 4 == 0, "alignment");
  static_assert(kAlloc <= 228 * 1024 / kCtas - 1024, "shared memory of the CTAs on one SM");
};

// kind::f16 descriptor with A (bit 15) and B (bit 16) K-major or MN-major
__host__ __device__ constexpr uint32_t idesc_ab(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16(M, N, b_mn) | ((uint32_t)a_mn << 15);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// barrier 1 over the softmax threads with the "or" of their votes (a warp's threads together: TMEM accesses,
// which want that, follow)
template <int N>
__device__ __forceinline__ bool vote_any(bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(N)
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void softmax_sync() {
  __syncwarp();
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
}

// Sums of N values (N = 16 or 32) over the 32 lanes by halving: of the columns two lanes hold, each
// keeps one half and gives the other away, so N - 1 shuffles (and one more for N = 16) leave every
// lane with the sum of one column, fold_column<N>(lane).
template <int N>
__device__ __forceinline__ float fold_sum(float (&v)[N], int lane) {
#pragma unroll
  for (int half = N / 2; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
    }
  }
  return N == 32 ? v[0] : v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}
template <int N>
__device__ __forceinline__ int fold_column(int lane) { return lane & (N - 1); }

// The same for maxima.
template <int N>
__device__ __forceinline__ float fold_max(float (&v)[N], int lane) {
#pragma unroll
  for (int half = N / 2; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, half));
    }
  }
  return N == 32 ? v[0] : fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, float* v) {
  if (N == 16) tmem_ld16(addr, v);
  else tmem_ld32(addr, v);
}

template <int D, int RP, int MODE>
__global__ void __launch_bounds__(RSmem<D, RP, MODE>::kThreads, RSmem<D, RP, MODE>::kCtas)
    rows_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, RowsArgs a) {
  using L = RSmem<D, RP, MODE>;
  constexpr int W = kMaxTree / 32, NC = L::kNC, kMma = 4 * L::kCG;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sbase = smem_raw + (base - raw);
  if (base - raw + L::kTotal > (uint32_t)L::kAlloc) {  // the plan does not fit: refuse, touch nothing
    if (threadIdx.x == 0) raise_error(kErrInternal);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (a.R + RP - 1) / RP;
  const long long bh = blockIdx.x / tiles;
  const int r0 = (int)(blockIdx.x % tiles) * RP;
  const int split = blockIdx.y;
  const int b = (int)(bh / a.heads), h = (int)(bh % a.heads);
  const int live = min(a.R - r0, RP);
  int rows = live, write = live;
  int* const par_s = reinterpret_cast<int*>(sbase + L::kPar);
  uint8_t* const depth_s = sbase + L::kDep;
  uint32_t* const anc_s = reinterpret_cast<uint32_t*>(sbase + L::kAnc);
  int* const flags_s = reinterpret_cast<int*>(sbase + L::kMisc + 8);

  // w_g is a float array of the caller's, of any alignment: a float a thread, on its way during the setup, then
  // through shared memory to where it is read in fours
  static_assert(D <= L::kThreads, "an element of w_g a thread");
  const float wg = MODE == kTree && threadIdx.x < D ? a.w_g[(long long)h * D + threadIdx.x] : 0.f;

  // the keys
  int n = 0;
  bool bad = false;
  TreeList tl;
  if (MODE == kCross) {
    n = a.kv_len ? a.kv_len[b] : a.n_kv;
    if (n < 0 || n > a.n_kv) {
      bad = true;
      if (threadIdx.x == 0) raise_error(kErrCacheLen);
    }
  } else {
    const int len = a.tree.cache_len[b], nodes = a.tree.tree_len ? a.tree.tree_len[b] : a.tree.T;
    bad = !tree_lengths_ok(a.tree, len, nodes);
    if (bad) {
      if (threadIdx.x == 0) raise_error(kErrCacheLen);
    } else if (!tree_setup(a.tree.parent + (long long)b * a.tree.T, nodes, r0, RP, par_s, depth_s, anc_s, flags_s)) {
      bad = true;
      write = max(0, min(nodes - r0, RP));
      if (threadIdx.x == 0) raise_error(kErrTree);
    } else {
      rows = write = max(0, min(nodes - r0, RP));
      if (rows == 0) return;  // rows past the sequence's nodes stay as they are
      tl.init(a.tree, len, nodes, flags_s[1]);
      n = tl.total();
    }
  }
  if (bad) n = 0;
  const int per = ((n + a.nsplit - 1) / a.nsplit + BK - 1) / BK * BK;
  const int e_begin = (int)min((long long)n, (long long)split * per), e_end = min(n, e_begin + per);
  const int nt = (e_end - e_begin + BK - 1) / BK;  // this CTA's tiles

  const bool shared_join = a.nsplit > 1 && a.nsplit <= kMaxCluster;

  const uint32_t sK = base + L::kK, sV = base + L::kV, sQ = base + L::kQ, sP = base + L::kP;
  const uint32_t bar_kfull = base + L::kBar, bar_kempty = bar_kfull + 8, bar_vfull = bar_kfull + 16,
                 bar_pv = bar_kfull + 24, bar_sfull = bar_kfull + 32, bar_pfull = bar_kfull + 48,
                 bar_drain = bar_kfull + 56;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + L::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + L::kMisc + 4);
  float* const ref_s = reinterpret_cast<float*>(sbase + L::kRef);
  float* const bl_s = reinterpret_cast<float*>(sbase + L::kBl);
  float* const fac_s = reinterpret_cast<float*>(sbase + L::kFac);
  float* const red_s = reinterpret_cast<float*>(sbase + L::kRed);
  float* const pl_s = reinterpret_cast<float*>(sbase + L::kPl);
  float* const pp_s = reinterpret_cast<float*>(sbase + L::kPp);
  float* const bp_s = reinterpret_cast<float*>(sbase + L::kBp);
  int2* const x_s = reinterpret_cast<int2*>(sbase + L::kX);
  uint32_t* const at_s = reinterpret_cast<uint32_t*>(sbase + L::kAt);
  float* const wg_s = reinterpret_cast<float*>(sbase + L::kWg);

  const __nv_bfloat16* const qb = (const __nv_bfloat16*)a.q + (bh * a.R + r0) * D;
  // entry e's row in the K (V) rows of this head, or null
  auto row_ptr = [&](const __nv_bfloat16* cached, const __nv_bfloat16* drafted, int e) -> const __nv_bfloat16* {
    if (e >= e_end) return nullptr;
    if (MODE == kCross) return cached + (bh * a.n_kv + e) * D;
    if (e >= tl.cached()) return drafted + (bh * a.R + (e - tl.cached())) * D;
    const int rel = tl.rel_of(e);
    return rel == kRelNone ? nullptr : cached + (bh * a.n_kv + tl.row_of(rel)) * D;
  };
  // first of 128 consecutive rows of K and V, or -1
  auto tma_row = [&](int e0) -> long long {
    if (e0 + BK > e_end) return -1;
    if (MODE == kCross) return e0;
    if (e0 + BK > tl.nwin) return -1;
    const int r = tl.row_of(e0 - tl.nwin);
    return r + BK <= a.n_kv ? r : -1;
  };

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmv) : "memory");
    mbar_init(bar_kfull, 1);
    mbar_init(bar_kempty, 1);
    mbar_init(bar_vfull, 1);
    mbar_init(bar_pv, 1);
    mbar_init(bar_sfull, 1);
    mbar_init(bar_sfull + 8, 1);
    mbar_init(bar_pfull, 4 * L::kCG);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "n"(L::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Q (zeros past the rows), 128-byte swizzle
  if (nt > 0) {
    for (int t = threadIdx.x; t < RP * (D / 8); t += L::kThreads) {
      const int r = t / (D / 8), c = t % (D / 8);
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) u = *reinterpret_cast<const uint4*>(qb + (long long)r * D + c * 8);
      *reinterpret_cast<uint4*>(sbase + L::kQ + (c >> 3) * (RP * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = u;
    }
    if (threadIdx.x < RP) {
      ref_s[threadIdx.x] = -INFINITY;
      if (MODE == kCross) bl_s[threadIdx.x] = kNoRef;  // (tree: with the priors, below)
    }
    if (MODE == kTree)
      for (int t = threadIdx.x; t < kMaxTree * RP / 32; t += L::kThreads) at_s[t] = 0u;
    if (MODE == kTree && threadIdx.x < D) wg_s[threadIdx.x] = wg;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem + 2 * RP;  // S^T buffers at tmem, tmem + RP

  if (warp > kMma) {
    // ---------------------------------------------------------------- loads: K, V
    const bool is_k = warp == kMma + 1;
    const uint32_t dst = is_k ? sK : sV, full = is_k ? bar_kfull : bar_vfull, empty = is_k ? bar_kempty : bar_pv;
    const CUtensorMap* const map = is_k ? &tmk : &tmv;
    const __nv_bfloat16* const cached = (const __nv_bfloat16*)(is_k ? a.k : a.v);
    const __nv_bfloat16* const drafted = (const __nv_bfloat16*)(is_k ? a.kt : a.vt);
    int issued = 0;
    for (int j = 0; j < nt; ++j) {
      const int e0 = e_begin + j * BK;
      if (!__all_sync(0xffffffffu, j == 0 || mbar_wait(empty, (j - 1) & 1, abort_flag))) break;
      const long long r = tma_row(e0);
      if (r >= 0) {
        if (lane == 0) {
          mbar_expect_tx(full, L::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * BK * 128, map, full, c * 64, (int)r, (int)bh);
        }
      } else {
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows an instruction
        const int sub = lane % LPR, slot = lane / LPR;
#pragma unroll 1
        for (int g = 0; g < BK / 32; ++g) {
          const unsigned long long mine = (unsigned long long)row_ptr(cached, drafted, e0 + g * 32 + lane);
#pragma unroll
          for (int i = 0; i < 32 / RPI; ++i) {
            const int key = g * 32 + i * RPI + slot;
            const unsigned long long p = __shfl_sync(0xffffffffu, mine, i * RPI + slot);
            const void* src = p ? (const void*)(p + sub * 16) : (const void*)cached;
            cp_async16(dst + (sub >> 3) * (BK * 128) + key * 128 + (((sub & 7) ^ (key & 7)) << 4), src, p ? 16 : 0);
          }
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      ++issued;
    }
    if (*abort_flag && issued > 0) {  // let the load in flight land before the CTA can exit
      volatile int never = 0;
      mbar_wait(full, (issued - 1) & 1, &never);
    }
    __syncwarp();
  } else if (warp == kMma) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && nt > 0) {
      constexpr uint32_t id_s = idesc_ab(BK, RP, 0, 0);   // K, Q both K-major
      constexpr uint32_t id_o = idesc_ab(BK, RP, 1, 0);   // V^T: V as stored, d contiguous
      // d = 64: V^T has 64 rows; the second 64 of the 128-row product repeat the first (block stride
      // 0) and are not read
      constexpr uint32_t v_blk = D == 128 ? BK * 128 : 0;
      auto qk = [&](int j) -> bool {
        if (!mbar_wait(bar_kfull, j & 1, abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk & 3) * 32;
          tc_mma(tmem + (j & 1) * RP, sw128_desc(sK + (kk >> 2) * (BK * 128) + in, 16, 1024),
                 sw128_desc(sQ + (kk >> 2) * (RP * 128) + in, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar_sfull + 8 * (j & 1));
        tc_commit(bar_kempty);
        return true;
      };
      bool okw = qk(0);
      for (int j = 0; okw && j < nt; ++j) {
        // S^T buffer (j + 1) & 1 held tile j - 1, whose P was complete before its V^T P^T was issued
        if (j + 1 < nt && !qk(j + 1)) break;
        if (!mbar_wait(bar_vfull, j & 1, abort_flag) || !mbar_wait(bar_pfull, j & 1, abort_flag)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma(tO, sw128_desc(sV + kk * 16 * 128, v_blk, 1024),
                 sw128_desc(sP + (kk >> 2) * (RP * 128) + (kk & 3) * 32, 16, 1024), id_o, (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bar_pv);
      }
      tc_commit(bar_drain);
      volatile int never = 0;
      mbar_wait(bar_drain, 0, &never);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax: one key a thread
    const int q4 = warp & 3, g0 = (warp >> 2) * NC;  // lane quarter; first of the group's rows
    const int key = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float NEG_INF = -INFINITY;
    uint32_t off[8];  // this key's place in a row of P, for rows n with n & 7 == i
#pragma unroll
    for (int i = 0; i < 8; ++i)
      off[i] = sP - base + g0 * 128 + (key >> 6) * (RP * 128) + i * 128 + ((((key >> 3) & 7) ^ i) << 4) + (key & 7) * 2;
    float l = 0.f;  // sum of the weights of row g0 + fold_column(lane) over this warp's keys
    const int l_row = g0 + fold_column<NC>(lane);
    bool ok = true;
    if (MODE == kTree && nt > 0) {  // the gate's priors and the rows' places, TPR threads a row
      constexpr int TPR = L::kSoft / RP, CH = D / 8 / TPR;
      const int r = threadIdx.x / TPR, part = threadIdx.x % TPR;
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = part * CH + i;
        float f[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(sbase + L::kQ + (c >> 3) * (RP * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)), f);
        const float4 w0 = reinterpret_cast<const float4*>(wg_s)[2 * c];
        const float4 w1 = reinterpret_cast<const float4*>(wg_s)[2 * c + 1];
        z = fmaf(f[0], w0.x, fmaf(f[1], w0.y, fmaf(f[2], w0.z, fmaf(f[3], w0.w, z))));
        z = fmaf(f[4], w1.x, fmaf(f[5], w1.y, fmaf(f[6], w1.z, fmaf(f[7], w1.w, z))));
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      z += a.b_g[h];
      if (part == 0) {  // (a padding row: the priors of a zero query at the first drafted position)
        const float pl = log_sigmoid(z) * kLog2e, pp = log_sigmoid(-z) * kLog2e;
        pl_s[r] = pl;
        pp_s[r] = pp;
        bl_s[r] = bias_without_ref(pl);
        bp_s[r] = bias_without_ref(pp);
        const int x = r < rows ? depth_s[r0 + r] : 0;
        x_s[r] = make_int2(x, tl.mod_of(x));
        const int bit = (r / NC) * kMaxTree * NC + x * NC + r % NC;  // NC bits a depth, 256 depths a warpgroup
        if (r < rows) atomicOr(at_s + (bit >> 5), 1u << (bit & 31));
      }
      softmax_sync<L::kSoft>();
    }
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      const int e0 = e_begin + j * BK, e = e0 + key;
      // `plain`: a tile in which every row reads every key as a window key.  Else the rows (bits) that
      // read this key as a window key and as a skip key.
      const bool plain = MODE == kCross ? e0 + BK <= e_end
                                        : e0 + BK <= tl.nwin && e0 + BK <= e_end && (long long)e0 - tl.nwin + tl.kwin >= flags_s[1] - 1;
      uint32_t win = 0u, skip = 0u;
      if (MODE == kTree && !plain && e < e_end) {
        const int t = e - tl.cached(), deepest = flags_s[1] - 1;
        if (e < tl.nwin || t >= 0) {
          // a window entry, a window key of every row but the deepest ones perhaps, or a drafted token
          const int rel = t >= 0 ? depth_s[t] : e - tl.nwin;
          const long long xw = (long long)tl.kwin + rel, xr = tl.reach + rel;
          if (xw >= deepest) {
            win = 0xffffffffu;
          } else {
            const int mod = tl.mod_of(rel);
#pragma unroll 4
            for (int r = 0; r < NC; ++r) {
              const int2 x = x_s[g0 + r];
              const bool w = x.x <= xw;
              win |= (uint32_t)w << r;
              skip |= (uint32_t)(!w & (x.y == mod) & (x.x <= xr)) << r;
            }
          }
          if (t >= 0) {  // of the drafted tokens only the row's ancestors
            uint32_t anc = 0u;
#pragma unroll 8
            for (int r = 0; r < NC; ++r) anc |= ((anc_s[(g0 + r) * W + (t >> 5)] >> (t & 31)) & 1u) << r;
            win &= anc;
            skip &= anc;
          }
        } else if (const int rel = tl.rel_of(e); rel != kRelNone) {
          // row o of a skip segment: the rows at depth o, and every pi deeper, as far as S*pi reaches
          const long long xr = tl.reach + rel;
          const int last = (int)(xr < deepest ? xr : deepest);
          for (int x = (e - tl.nwin) % tl.lseg; x <= last; x += tl.pi) {
            const int bit = (g0 / NC) * kMaxTree * NC + x * NC;
            skip |= at_s[bit >> 5] >> (bit & 31) & (NC == 32 ? 0xffffffffu : 0xffffu);
            if (tl.pi > kMaxTree) break;
          }
        }
      }
      const uint32_t read = MODE == kCross ? (plain || e < e_end ? 0xffffffffu : 0u) : plain ? 0xffffffffu : win | skip;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_sfull + 8 * (j & 1), (j >> 1) & 1, abort_flag));
      // s: the scores in log2 units less the rows' references, -inf for keys a row does not read
      float s[NC];
      bool raised = false;
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        bool over = false;
        if (ok) {
          tc_fence_after();
          tmem_ld_n<NC>(tmem + (j & 1) * RP + g0 + lane_off, s);
          if (plain) {
#pragma unroll
            for (int r = 0; r < NC; r += 4) {
              const float4 c = *reinterpret_cast<const float4*>(bl_s + g0 + r);
              s[r] = fmaf(s[r], a.scale_log2, c.x);
              s[r + 1] = fmaf(s[r + 1], a.scale_log2, c.y);
              s[r + 2] = fmaf(s[r + 2], a.scale_log2, c.z);
              s[r + 3] = fmaf(s[r + 3], a.scale_log2, c.w);
            }
          } else {
#pragma unroll
            for (int r = 0; r < NC; r += 4) {
              const float4 c = *reinterpret_cast<const float4*>(bl_s + g0 + r);
              const float4 k = MODE == kTree ? *reinterpret_cast<const float4*>(bp_s + g0 + r) : c;
              const float cc[4] = {c.x, c.y, c.z, c.w}, kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float t = fmaf(s[r + i], a.scale_log2, skip & (1u << (r + i)) ? kk[i] : cc[i]);
                s[r + i] = read & (1u << (r + i)) ? t : NEG_INF;
              }
            }
          }
          float top = NEG_INF;
#pragma unroll
          for (int r = 0; r + 1 < NC; r += 2) top = max3f(top, s[r], s[r + 1]);
          over = top > kRescaleThreshold;
        }
        if (pass == 1 || !vote_any<L::kSoft>(over)) break;
        // Some score passes its row's reference: raise the references that are passed, then take the
        // scores again.  (A row without a reference yet has scores with kNoRef here; the raw ones come
        // from TMEM.  A row that stays without has -inf, or NaN, for every key it reads in this tile.)
        raised = true;
        if (ok) {
#pragma unroll
          for (int c = 0; c < NC; c += 16) {
            float x[16];
            tmem_ld16(tmem + (j & 1) * RP + g0 + lane_off + c, x);
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              float4 cl = make_float4(0.f, 0.f, 0.f, 0.f), cp = cl;
              if (MODE == kTree) {
                cl = *reinterpret_cast<const float4*>(pl_s + g0 + c + r);
                cp = *reinterpret_cast<const float4*>(pp_s + g0 + c + r);
              }
              const float cc[4] = {cl.x, cl.y, cl.z, cl.w}, kk[4] = {cp.x, cp.y, cp.z, cp.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t bit = 1u << (c + r + i);
                s[c + r + i] = read & bit ? fmaf(x[r + i], a.scale_log2, skip & bit ? kk[i] : cc[i]) : NEG_INF;
              }
            }
          }
          const float top = fold_max<NC>(s, lane);
          if (lane < NC) red_s[q4 * RP + l_row] = top;
        }
        softmax_sync<L::kSoft>();
        if (const int r = threadIdx.x; r < RP) {
          const float old = ref_s[r];
          const float m = fmaxf(fmaxf(red_s[r], red_s[RP + r]), fmaxf(red_s[2 * RP + r], red_s[3 * RP + r]));
          float f = 1.f;
          if (m > old + kRescaleThreshold || (old == NEG_INF && m > NEG_INF)) {
            if (old != NEG_INF) f = ex2(old - m);
            ref_s[r] = m;
            const float bl = (MODE == kTree ? pl_s[r] : 0.f) - m, bp = (MODE == kTree ? pp_s[r] : 0.f) - m;
            bl_s[r] = bl;
            if (MODE == kTree) bp_s[r] = bp;
          }
          fac_s[r] = f;
        }
        softmax_sync<L::kSoft>();
      }
      if (raised) {
        l *= fac_s[l_row];
        if (j > 0) {  // O^T holds the earlier tiles' sums: all of them, once the last product is done
          ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_pv, (j - 1) & 1, abort_flag));
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < NC; c += 16) {
              float o[16];
              tmem_ld16(tO + g0 + lane_off + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= fac_s[g0 + c + i];
              tmem_st16(tO + g0 + lane_off + c, reinterpret_cast<const uint32_t*>(o));
            }
            tmem_wait_st();
          }
        }
      } else if (j > 0) {  // the last product has read P
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_pv, (j - 1) & 1, abort_flag));
      }
      if (ok) {
#pragma unroll
        for (int r = 0; r < NC; ++r) {
          s[r] = ex2(s[r]);
          // (bf16 for the product: 2^-8 of a weight at most; the sum l takes the weight as it is)
          *reinterpret_cast<__nv_bfloat16*>(sbase + off[r & 7] + (r >> 3) * 1024) = __float2bfloat16_rn(s[r]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar_pfull);
      if (ok) l += fold_sum<NC>(s, lane);  // while the product runs
    }
    // ---- epilogue: the sums over the 128 keys' threads, then row by row from O^T (thread = column of d)
    if (lane < NC) red_s[q4 * RP + l_row] = l;
    ok = ok && (nt == 0 || __all_sync(0xffffffffu, mbar_wait(bar_pv, (nt - 1) & 1, abort_flag)));
    softmax_sync<L::kSoft>();
    const float NaN = __int_as_float(0x7fffffff);
    if (const int key = threadIdx.x; key < RP) {
      const float sum = bad ? NaN : nt == 0 ? 0.f : (red_s[key] + red_s[RP + key]) + (red_s[2 * RP + key] + red_s[3 * RP + key]);
      const float m = nt == 0 ? NEG_INF : ref_s[key];
      fac_s[key] = bad ? NaN : sum == 0.f ? 0.f : 1.f / sum;
      if (shared_join) {
        ref_s[key] = m;
        fac_s[key] = sum;
      } else if (key < write) {
        const long long row = bh * a.R + r0 + key;
        if (a.nsplit > 1) {
          part_ml(a, split, row)[0] = bad ? 0.f : m;
          part_ml(a, split, row)[1] = sum;
        } else if (a.lse) {
          a.lse[row] = bad ? NaN : sum == 0.f ? NEG_INF : (m + log2f(sum)) * kLn2;
        }
      }
    }
    softmax_sync<L::kSoft>();
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < NC; c += 16) {
        if (g0 + c >= write && !shared_join) break;
        float o[16];
        if (nt > 0) {
          tmem_ld16(tO + g0 + lane_off + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
        if (key >= D) continue;
        if (shared_join) {  // K's buffer: every product that reads it has completed
          float* const dst = reinterpret_cast<float*>(sbase + L::kK) + (g0 + c) * D + key;
#pragma unroll
          for (int i = 0; i < 16; ++i) dst[i * D] = o[i];
          continue;
        }
        const long long at = (bh * a.R + r0 + g0 + c) * D + key;
        const int count = write - g0 - c;  // rows of the chunk that exist
        if (a.nsplit > 1) {
          float* const dst = a.part + (long long)split * a.rows * D + at;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i < count) dst[i * D] = bad ? NaN : o[i];
        } else {
          __nv_bfloat16* const dst = (__nv_bfloat16*)a.out + at;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i < count) dst[i * D] = __float2bfloat16_rn(bad ? NaN : o[i] * fac_s[g0 + c + i]);
        }
      }
    }
    tc_fence_before();
  }
  if (shared_join) {  // the shares' sums, row by row: CTA `split` of the cluster takes every nsplit-th row
    cluster_sync();
    for (int t = threadIdx.x; t < RP * (D / 4); t += L::kThreads) {
      const int r = t / (D / 4), c = t % (D / 4) * 4;
      if (r >= write || r % a.nsplit != split) continue;
      const uint32_t am = base + L::kRef + r * 4, al = base + L::kFac + r * 4, ao = sK + (r * D + c) * 4;
      float M = -INFINITY;
      for (int p = 0; p < a.nsplit; ++p) M = fmaxf(M, peer_f32(peer_addr(am, p)));
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < a.nsplit; ++p) {
        const float w = ex2(peer_f32(peer_addr(am, p)) - ref);
        const float4 v = peer_f32x4(peer_addr(ao, p));
        sum = fmaf(peer_f32(peer_addr(al, p)), w, sum);
        o.x = fmaf(v.x, w, o.x);
        o.y = fmaf(v.y, w, o.y);
        o.z = fmaf(v.z, w, o.z);
        o.w = fmaf(v.w, w, o.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long row = bh * a.R + r0 + r;
      __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + row * D + c) =
          make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
      if (a.lse && c == 0) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while another reads it
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kTmem) : "memory");
  }
}

// Rows a CTA takes: the least of 16, 32, 64 that holds them.
inline int rows_pad(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

template <int D, int RP, int MODE>
cudaError_t launch_rows_as(const RowsArgs& a, long long bh, cudaStream_t s, const char** why) {
  using L = RSmem<D, RP, MODE>;
  CUtensorMap mk, mv;
  if (!make_map(&mk, a.k, (int)bh, a.n_kv, D, BK) || !make_map(&mv, a.v, (int)bh, a.n_kv, D, BK)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  static std::atomic<bool> done[kSmemDevices];
  const cudaError_t e = allow_smem(rows_tc_kernel<D, RP, MODE>, L::kAlloc, done);
  if (e != cudaSuccess) {
    *why = "cudaFuncSetAttribute";
    return e;
  }
  const long long tiles = (a.R + RP - 1) / RP;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bh * tiles), (unsigned)a.nsplit);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 1;
  at.val.clusterDim.y = (unsigned)a.nsplit;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.nsplit > 1 && a.nsplit <= kMaxCluster ? 1 : 0;
  *why = "few-rows tensor-core kernel launch";
  return cudaLaunchKernelEx(&cfg, rows_tc_kernel<D, RP, MODE>, mk, mv, a);
}

template <int D, int MODE>
cudaError_t launch_rows(const RowsArgs& a, long long bh, cudaStream_t s, const char** why) {
  const int rp = rows_pad(a.R);
  if (rp == 16) return launch_rows_as<D, 16, MODE>(a, bh, s, why);
  if (rp == 32) return launch_rows_as<D, 32, MODE>(a, bh, s, why);
  return launch_rows_as<D, 64, MODE>(a, bh, s, why);
}

}  // namespace rtc
}  // namespace pia
