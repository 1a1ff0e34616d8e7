// cross_simt.cuh -- attention of a tile of query rows to a list of keys on CUDA cores, fp32
// throughout, for every dtype and head size up to 256: cross attention and its gradients, and the
// tree of drafted tokens.  It is the fp32 path of these operators and the path of bf16 head sizes
// the tensor-core kernels do not cover.
//
// Heads that share a key head are neighbours in q [B, H, n_q, d], so their rows together are one
// contiguous block of R = (H / H_kv) n_q rows: a key head's rows are taken as one sequence of R rows
// and the sharing needs no further attention, neither in the forward (K and V are read once for all
// of them) nor in the gradients of k and v (a sum over the R rows).
//
// A block of 16 TY threads takes 4 TY rows as a TY x 16 grid: thread (ty, tx) scores rows ty + TY a against
// keys tx + 16 b (a, b < 4) of a 64-key tile from shared memory (a row padded by 16 bytes, so that 8
// neighbouring rows start in different banks), 4 d FMAs a pair for 2 d 16-byte loads; the sixteen
// threads of a row keep its running max and sum by shuffles; then p goes through shared memory and the
// thread accumulates columns 4 (tx + 16 u) .. + 3 of its rows.  Shared memory is what bounds it, so a
// thread always holds 4 x 4 pairs: few rows take 16-row blocks of 64 threads (with 256 threads of one
// row each a 64-key tile at d = 32 took 6200 cycles of loads and products), many rows 64-row blocks of
// 256, which read each key for four times the rows.  The choice is by the number of tiles; where it
// leaves SMs idle, up to eight blocks of a cluster share a tile's keys (the gradients: what they stream)
// and add their sums in the order of their ranks, through shared memory.  Global loads are issued
// up to eight a thread and matrix before the first is used.  Measured (in a replayed graph, a
// launch of 2.5 us in each): 2 x 4 heads of 193 x 301 rows, d = 32, 10.5 us; the gradients of 2 heads of 257 x 384
// rows 14.9 us; 16 heads of 300 x 1000 rows, d = 128, 152 us (16 of the nominal 74 TFLOP/s: a thread's 4 x 4 pairs
// cost eight 16-byte reads of shared memory for 64 FMAs, and loads are not under the products), the gradients
// 463 us.
#pragma once
#include <atomic>

#include "common.cuh"
#include "tree_rule.cuh"

namespace pia {

// Host: dynamic shared memory above 48 KB is opted into once per kernel and device.  Threads that call at
// once may both find the flag unset; both then ask for the same.
constexpr int kSmemDevices = 64;
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<bool> (&done)[kSmemDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kSmemDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

constexpr int kMaxCluster = 8;  // shares of a sum joined in a cluster

// the cluster's barrier (whose aligned form wants a warp's threads together: the loops before it may have left
// them at different iterations), and a read of CTA `rank`'s shared memory at this CTA's address `a`
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
constexpr int kRowKeys = 64;  // keys a tile
enum : int { kCross = 0, kTree = 1 };

// Scores of one pass over keys [split share] of every row; nsplit > 1: partial states.
struct RowsArgs {
  const void* q;    // [BH, R, d]
  const void* k;    // [BH, n_kv, d] (tree: the cache, [BH, cap, d])
  const void* v;
  void* out;        // [BH, R, d]
  float* lse;       // [BH, R] or null
  const int* kv_len;  // cross: [B] or null
  const void* kt;   // tree: the drafted tokens' keys and values [BH, T, d]
  const void* vt;
  const float* w_g;
  const float* b_g;
  TreeArgs tree;
  float* part;      // [nsplit][BH * R][d] sums, then [nsplit][BH * R][2] (max in log2 units, sum)
  long long rows;   // BH * R
  int heads;        // heads (key heads) a batch entry
  int R, n_kv, d, nsplit;
  float scale_log2;
};

__device__ __forceinline__ float* part_ml(const RowsArgs& a, int split, long long row) {
  return a.part + (long long)a.nsplit * a.rows * a.d + ((long long)split * a.rows + row) * 2;
}

// 16 bytes of a row, widened to fp32
template <typename T>
__device__ __forceinline__ void put16(float* dst, const uint4& u) {
  if (sizeof(T) == 2) {
    float f[8];
    bf16x8_to_f32(u, f);
    *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(dst) = u;
  }
}

// `rows` rows each of two matrices (one: B null) into shared memory, row r from a(r), b(r) (null: zeros)
template <typename T, int TY, typename F, typename G>
__device__ __forceinline__ void load_rows2(float* A, float* Bm, int ld, int d, int rows, F a, G b) {
  constexpr int V = 16 / (int)sizeof(T), BATCH = TY == 4 ? 8 : 4, NT = 16 * TY;
  const int chunks = d / V, total = rows * chunks;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int t0 = threadIdx.x; t0 < total; t0 += BATCH * NT) {
    uint4 x[BATCH], y[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int t = t0 + i * NT, r = t / chunks, c = (t - r * chunks) * V;
      x[i] = y[i] = zero;
      if (t < total) {
        const T* const p = a(r);
        if (p) x[i] = *reinterpret_cast<const uint4*>(p + c);
        if (Bm) {
          const T* const q = b(r);
          if (q) y[i] = *reinterpret_cast<const uint4*>(q + c);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int t = t0 + i * NT, r = t / chunks, c = (t - r * chunks) * V;
      if (t >= total) break;
      put16<T>(A + r * ld + c, x[i]);
      if (Bm) put16<T>(Bm + r * ld + c, y[i]);
    }
  }
}
template <typename T, int TY, typename F>
__device__ __forceinline__ void load_rows(float* A, int ld, int d, int rows, F a) {
  load_rows2<T, TY>(A, nullptr, ld, d, rows, a, [](int) -> const T* { return nullptr; });
}

// dot products of rows ty + TY a of A with rows tx + 16 b of B
template <int TY>
__device__ __forceinline__ void tile_dots(const float* A, const float* Bm, int ld, int d, int ty, int tx,
                                          float (&s)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) s[a][b] = 0.f;
#pragma unroll 2
  for (int c = 0; c < d; c += 4) {
    float4 qa[4], kb[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const float4*>(A + (ty + TY * a) * ld + c);
#pragma unroll
    for (int b = 0; b < 4; ++b) kb[b] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * b) * ld + c);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[a][b] = fmaf(qa[a].x, kb[b].x, s[a][b]);
        s[a][b] = fmaf(qa[a].y, kb[b].y, s[a][b]);
        s[a][b] = fmaf(qa[a].z, kb[b].z, s[a][b]);
        s[a][b] = fmaf(qa[a].w, kb[b].w, s[a][b]);
      }
  }
}

constexpr int kPld = kRowKeys + 4;  // a row of P in shared memory

// acc[a][u] += sum_j P[ty + TY a][j] M[j][4 (tx + 16 u) ..]
template <int TY, int U>
__device__ __forceinline__ void tile_accumulate(const float* P, const float* M, int ld, int d, int ty, int tx,
                                                float4 (&acc)[4][U]) {
#pragma unroll 2
  for (int j = 0; j < kRowKeys; j += 4) {
    float4 p[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) p[a] = *reinterpret_cast<const float4*>(P + (ty + TY * a) * kPld + j);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (tx + 16 * u);
      if (c < d) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 m = *reinterpret_cast<const float4*>(M + (j + k) * ld + c);
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float w = k == 0 ? p[a].x : k == 1 ? p[a].y : k == 2 ? p[a].z : p[a].w;
            acc[a][u].x = fmaf(w, m.x, acc[a][u].x);
            acc[a][u].y = fmaf(w, m.y, acc[a][u].y);
            acc[a][u].z = fmaf(w, m.z, acc[a][u].z);
            acc[a][u].w = fmaf(w, m.w, acc[a][u].w);
          }
        }
      }
    }
  }
}

// four columns of a row
__device__ __forceinline__ void put4(float* dst, const float4& v) { *reinterpret_cast<float4*>(dst) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16* dst, const float4& v) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}
__device__ __forceinline__ void get4(float (&v)[4], const float* src) {
  const float4 u = *reinterpret_cast<const float4*>(src);
  v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
}
__device__ __forceinline__ void get4(float (&v)[4], const __nv_bfloat16* src) {
  const uint2 u = *reinterpret_cast<const uint2*>(src);
  v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ float4 scaled(const float4& v, float k, float add) {
  return make_float4(fmaf(v.x, k, add), fmaf(v.y, k, add), fmaf(v.z, k, add), fmaf(v.w, k, add));
}

__device__ __forceinline__ float half_max(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// floats of dynamic shared memory: Q, a K and a V tile, P
__host__ __device__ constexpr size_t rows_simt_smem(int d, int ty) {
  return sizeof(float) * ((size_t)(4 * ty + 2 * kRowKeys) * (d + 4) + (size_t)4 * ty * kPld);
}

template <typename T, int TY, int U, int MODE>
__global__ void __launch_bounds__(16 * TY) rows_simt_kernel(RowsArgs a) {
  constexpr int BQ = 4 * TY, NT = 16 * TY;
  extern __shared__ __align__(16) float sm[];
  const int d = a.d, ld = d + 4;
  float* const Qs = sm;
  float* const Ks = Qs + BQ * ld;
  float* const Vs = Ks + kRowKeys * ld;
  float* const Ps = Vs + kRowKeys * ld;
  __shared__ int par_s[MODE == kTree ? kMaxTree : 1], flags_s[2];
  __shared__ uint8_t depth_s[MODE == kTree ? kMaxTree : 1];
  __shared__ uint32_t anc_s[MODE == kTree ? BQ * (kMaxTree / 32) : 1];
  __shared__ int rel_s[kRowKeys], mod_s[kRowKeys];
  __shared__ float bl_s[BQ], bp_s[BQ];  // the rows' priors; at the end their maxima and sums

  const int tiles = (a.R + BQ - 1) / BQ;
  const long long bh = blockIdx.x / tiles;
  const int r0 = (int)(blockIdx.x % tiles) * BQ;
  const int split = blockIdx.y;
  const int b = (int)(bh / a.heads), h = (int)(bh % a.heads);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int live = min(a.R - r0, BQ);  // rows of the tile that exist
  int rows = live;                     // rows of the tile that are computed
  int write = live;                    // rows of the tile that are written

  // the keys: how many, and for the tree where each one is
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
    } else if (!tree_setup(a.tree.parent + (long long)b * a.tree.T, nodes, r0, BQ, par_s, depth_s, anc_s, flags_s)) {
      bad = true;
      write = max(0, min(nodes - r0, BQ));
      if (threadIdx.x == 0) raise_error(kErrTree);
    } else {
      rows = write = max(0, min(nodes - r0, BQ));
      if (rows == 0) return;  // rows past the sequence's nodes stay as they are
      tl.init(a.tree, len, nodes, flags_s[1]);
      n = tl.total();
    }
  }
  if (bad) n = 0;
  const int per = ((n + a.nsplit - 1) / a.nsplit + kRowKeys - 1) / kRowKeys * kRowKeys;
  const int e_begin = min((long long)n, (long long)split * per), e_end = min(n, e_begin + per);

  const T* const qb = (const T*)a.q + (bh * a.R + r0) * d;
  const T* const kb = (const T*)a.k + bh * (long long)a.n_kv * d;
  const T* const vb = (const T*)a.v + bh * (long long)a.n_kv * d;
  const T* const ktb = MODE == kTree ? (const T*)a.kt + bh * (long long)a.R * d : nullptr;
  const T* const vtb = MODE == kTree ? (const T*)a.vt + bh * (long long)a.R * d : nullptr;
  load_rows<T, TY>(Qs, ld, d, BQ, [&](int r) -> const T* { return r < rows ? qb + (long long)r * d : nullptr; });
  __syncthreads();
  if (MODE == kTree && !bad) {  // the gate: one warp a row
    for (int r = threadIdx.x >> 5; r < rows; r += NT / 32) {
      float z = 0.f;
      for (int c = threadIdx.x & 31; c < d; c += 32) z = fmaf(Qs[r * ld + c], a.w_g[(long long)h * d + c], z);
      z = warp_sum(z) + a.b_g[h];
      if ((threadIdx.x & 31) == 0) {
        bl_s[r] = log_sigmoid(z) * kLog2e;
        bp_s[r] = log_sigmoid(-z) * kLog2e;
      }
    }
    __syncthreads();
  }

  float m[4], l[4];
  float4 acc[4][U];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto key_row = [&](const T* cached, const T* tree, int e) -> const T* {
    if (e >= e_end) return nullptr;
    if (MODE == kCross) return cached + (long long)e * d;
    if (e >= tl.cached()) return tree + (long long)(e - tl.cached()) * d;
    const int rel = tl.rel_of(e);
    return rel == kRelNone ? nullptr : cached + (long long)tl.row_of(rel) * d;
  };
  for (int e0 = e_begin; e0 < e_end; e0 += kRowKeys) {
    __syncthreads();  // the last tile's V and P have been read
    load_rows2<T, TY>(Ks, Vs, ld, d, kRowKeys, [&](int j) { return key_row(kb, ktb, e0 + j); },
                  [&](int j) { return key_row(vb, vtb, e0 + j); });
    if (MODE == kTree && threadIdx.x < kRowKeys) {
      const int e = e0 + threadIdx.x;
      const int rel = e >= e_end ? kRelNone : e < tl.cached() ? tl.rel_of(e) : depth_s[e - tl.cached()];
      rel_s[threadIdx.x] = rel;
      mod_s[threadIdx.x] = tl.mod_of(rel);
    }
    __syncthreads();
    float s[4][4];
    tile_dots<TY>(Qs, Ks, ld, d, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + TY * i;
      int x = 0, xmod = 0;
      if (MODE == kTree && r < rows) {
        x = depth_s[r0 + r];
        xmod = tl.mod_of(x);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = tx + 16 * u, e = e0 + j;
        if (MODE == kCross) {
          s[i][u] = e < e_end ? s[i][u] * a.scale_log2 : -INFINITY;
        } else {
          int kind = r < rows && e < e_end ? tree_kind(x, xmod, rel_s[j], mod_s[j], tl.kwin, tl.reach) : 0;
          const int t = e - tl.cached();
          if (kind && t >= 0 && !((anc_s[r * (kMaxTree / 32) + (t >> 5)] >> (t & 31)) & 1u)) kind = 0;
          s[i][u] = kind ? fmaf(s[i][u], a.scale_log2, kind == 1 ? bl_s[r] : bp_s[r]) : -INFINITY;
        }
      }
      const float mt = half_max(fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3])));
      const float mn = fmaxf(m[i], mt);
      const float ref = mn == -INFINITY ? 0.f : mn;  // no key yet: every p is 0
      const float corr = exp2f(m[i] - ref);
      float ls = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float p = exp2f(s[i][u] - ref);
        Ps[r * kPld + tx + 16 * u] = p;
        ls += p;
      }
      l[i] = fmaf(l[i], corr, half_sum(ls));
      m[i] = mn;
#pragma unroll
      for (int u = 0; u < U; ++u) acc[i][u] = scaled(acc[i][u], corr, 0.f);
    }
    __syncthreads();  // P is written
    tile_accumulate<TY, U>(Ps, Vs, ld, d, ty, tx, acc);
  }

  const float NaN = __int_as_float(0x7fffffff);
  if (a.nsplit > 1) {  // the cluster's shares: max in bl_s, sum in bp_s, the weighted values in Q's place
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + TY * i;
      if (tx == 0) {
        bl_s[r] = m[i];
        bp_s[r] = bad ? NaN : l[i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (4 * (tx + 16 * u) < d) put4(Qs + r * ld + 4 * (tx + 16 * u), acc[i][u]);
    }
    cluster_sync();
    const uint32_t am = (uint32_t)__cvta_generic_to_shared(bl_s), al = (uint32_t)__cvta_generic_to_shared(bp_s),
                   ao = (uint32_t)__cvta_generic_to_shared(Qs);
    const int per_row = d / 4, mine = (write - split + a.nsplit - 1) / a.nsplit;  // rows split, split + nsplit, ...
    for (int t = threadIdx.x; t < mine * per_row; t += NT) {
      const int q = t / per_row, c = 4 * (t - q * per_row), r = split + q * a.nsplit;
      float mp[kMaxCluster], lp[kMaxCluster];
      float4 op[kMaxCluster];
      float M = -INFINITY;
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < a.nsplit) {
          mp[p] = peer_f32(peer_addr(am + 4 * r, p));
          lp[p] = peer_f32(peer_addr(al + 4 * r, p));
          op[p] = peer_f32x4(peer_addr(ao + 4 * (r * ld + c), p));
        }
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < a.nsplit) M = fmaxf(M, mp[p]);
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < a.nsplit) {
          const float w = exp2f(mp[p] - ref);
          sum = fmaf(lp[p], w, sum);
          o = make_float4(fmaf(op[p].x, w, o.x), fmaf(op[p].y, w, o.y), fmaf(op[p].z, w, o.z), fmaf(op[p].w, w, o.w));
        }
      const long long row = bh * a.R + r0 + r;
      put4((T*)a.out + row * d + c, scaled(o, sum == 0.f ? 0.f : 1.f / sum, 0.f));
      if (a.lse && c == 0) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
    cluster_sync();  // no block leaves while another reads it
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + TY * i;
    if (r >= write) continue;
    const long long row = bh * a.R + r0 + r;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no key: out 0, lse -inf (a NaN stays one)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (4 * (tx + 16 * u) < d) put4((T*)a.out + row * d + 4 * (tx + 16 * u), scaled(acc[i][u], inv, bad ? NaN : 0.f));
    if (a.lse && tx == 0) a.lse[row] = bad ? NaN : l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
}

// Joins the splits' partial states of every row: M = max m_s, out = sum acc_s 2^(m_s - M) / sum l_s 2^(m_s - M).
// A thread takes four columns of a row.  tree: rows past a sequence's nodes stay as they are.
__global__ void __launch_bounds__(256) rows_join_kernel(RowsArgs a, int tree) {
  const int per_row = a.d / 4;
  const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long row = t / per_row;
  const int c = (int)(t % per_row) * 4;
  if (row >= a.rows) return;
  if (tree && a.tree.tree_len) {
    const int b = (int)(row / a.R / a.heads), n = a.tree.tree_len[b];
    if ((int)(row % a.R) >= n && tree_lengths_ok(a.tree, a.tree.cache_len[b], n)) return;
  }
  float M = -INFINITY;
  for (int s = 0; s < a.nsplit; ++s) M = fmaxf(M, part_ml(a, s, row)[0]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.nsplit; ++s) {
    const float* ml = part_ml(a, s, row);
    const float w = exp2f(ml[0] - ref);
    const float4 p = *reinterpret_cast<const float4*>(a.part + ((long long)s * a.rows + row) * a.d + c);
    L = fmaf(ml[1], w, L);
    o.x = fmaf(p.x, w, o.x);
    o.y = fmaf(p.y, w, o.y);
    o.z = fmaf(p.z, w, o.z);
    o.w = fmaf(p.w, w, o.w);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + row * a.d + c) =
      make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  if (a.lse && c == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ---- gradients of cross attention ----------------------------------------------------------------
//   p = exp(s - lse), D = dout . out, ds = p (dout . v - D)
//   dq = tau sum_j ds k_j,  dk = tau sum_i ds q_i,  dv = sum_i p dout_i
// in two passes over the scores, by tiles of rows (dq) and by tiles of keys (dk, dv, summed over all R
// rows of the key head), in one launch.  A tile's sums stay in one block, or in the blocks of one cluster
// that add them in a fixed order: no atomics, nothing depends on scheduling.
struct CrossGradArgs {
  const void* q;      // [BH, R, d]
  const void* k;      // [BH, n_kv, d]
  const void* v;
  const void* dout;   // [BH, R, d]
  const void* out;
  const float* lse;   // [BH, R]
  float* D;           // [BH, R] (tensor cores; the CUDA-core kernel forms D from the rows it holds)
  void* dq;           // gradients in the inputs' dtype
  void* dk;
  void* dv;
  const int* kv_len;  // [B] or null
  long long rows;
  int heads, R, n_kv, d;
  float scale_log2;
};

// What p = 2^(score - lse2) takes from a row's lse: a row without keys (lse -inf) has no weights.
__device__ __forceinline__ float lse_log2(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// D of every row, for the tensor-core kernel: one warp a row
template <typename T>
__global__ void __launch_bounds__(256) row_dot_kernel(CrossGradArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  float s = 0.f;
  for (int c = (threadIdx.x & 31) * V; c < a.d; c += 32 * V) {
    __align__(16) float x[V], y[V];
    put16<T>(x, *reinterpret_cast<const uint4*>((const T*)a.out + row * a.d + c));
    put16<T>(y, *reinterpret_cast<const uint4*>((const T*)a.dout + row * a.d + c));
#pragma unroll
    for (int e = 0; e < V; ++e) s = fmaf(x[e], y[e], s);
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) a.D[row] = s;
}

// Two fixed tiles of 4 TY rows, two streamed ones of 64, and two 4 TY x 64 tiles (p and ds)
__host__ __device__ constexpr size_t cross_grad_smem(int d, int ty) {
  return sizeof(float) * (2 * (size_t)(4 * ty + kRowKeys) * (d + 4) + (size_t)2 * 4 * ty * kPld);
}

// A bad length: the error word, and NaN in every gradient of the sequence.
__device__ __forceinline__ int grad_keys(const CrossGradArgs& a, int b, bool* bad) {
  const int n = a.kv_len ? a.kv_len[b] : a.n_kv;
  *bad = n < 0 || n > a.n_kv;
  if (*bad && threadIdx.x == 0) raise_error(kErrCacheLen);
  return *bad ? 0 : n;
}

// Adds up the cluster's shares of a [rows, d] sum (in the order of the ranks) and writes the result,
// scaled; this block's share is in `sums` (row stride ld).  Rows from `live` on take the value `none`.
template <typename T, int TY>
__device__ __forceinline__ void write_joined(const float* sums, int ld, int d, int rows, int live, int shares, int rank,
                                             float scale, float none, T* dst) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(sums);
  const int per_row = d / 4;
  for (int t = threadIdx.x + 16 * TY * rank; t < rows * per_row; t += 16 * TY * shares) {
    const int r = t / per_row, c = 4 * (t - r * per_row);
    float4 v[kMaxCluster], s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kMaxCluster; ++p)
      if (p < shares) v[p] = peer_f32x4(peer_addr(at + 4 * (r * ld + c), p));
#pragma unroll
    for (int p = 0; p < kMaxCluster; ++p)
      if (p < shares) s = make_float4(s.x + v[p].x, s.y + v[p].y, s.z + v[p].z, s.w + v[p].w);
    put4(dst + (long long)r * d + c, r < live ? scaled(s, scale, 0.f) : make_float4(none, none, none, none));
  }
}

// D = dout . out of the rows ty + TY i, i < N, whose dout is in Gs: the sixteen threads of a row take four
// columns each at a time.
template <typename T, int TY, int U, int N>
__device__ __forceinline__ void row_dots(const float* Gs, int ld, int d, int rows, int ty, int tx, const T* out, float (&D)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = ty + TY * i;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (tx + 16 * u);
      if (r < rows && c < d) {
        const float4 g = *reinterpret_cast<const float4*>(Gs + r * ld + c);
        float o[4];
        get4(o, out + (long long)r * d + c);
        s = fmaf(g.x, o[0], fmaf(g.y, o[1], fmaf(g.z, o[2], fmaf(g.w, o[3], s))));
      }
    }
    D[i] = half_sum(s);
  }
}

// 4 TY rows against this block's share of the keys
template <typename T, int TY, int U>
__device__ __forceinline__ void cross_dq_block(const CrossGradArgs& a, float* sm, long long bh, int tile, int shares, int rank) {
  constexpr int BQ = 4 * TY;
  const int d = a.d, ld = d + 4;
  float* const Qs = sm;
  float* const Gs = Qs + BQ * ld;
  float* const Ks = Gs + BQ * ld;
  float* const Vs = Ks + kRowKeys * ld;
  float* const Ps = Vs + kRowKeys * ld;
  const int r0 = tile * BQ, rows = min(a.R - r0, BQ);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  bool bad;
  const int n = grad_keys(a, (int)(bh / a.heads), &bad);
  const long long row0 = bh * a.R + r0;
  load_rows2<T, TY>(Qs, Gs, ld, d, BQ, [&](int r) -> const T* { return r < rows ? (const T*)a.q + (row0 + r) * d : nullptr; },
                [&](int r) -> const T* { return r < rows ? (const T*)a.dout + (row0 + r) * d : nullptr; });
  float lse2[4], D[4];
  float4 acc[4][U];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + TY * i;
    lse2[i] = r < rows ? lse_log2(a.lse[row0 + r]) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  row_dots<T, TY, U, 4>(Gs, ld, d, rows, ty, tx, (const T*)a.out + row0 * d, D);
  const T* const kb = (const T*)a.k + bh * (long long)a.n_kv * d;
  const T* const vb = (const T*)a.v + bh * (long long)a.n_kv * d;
  const int tiles = (n + kRowKeys - 1) / kRowKeys, per = (tiles + shares - 1) / shares;
  const int t_end = min(tiles, (rank + 1) * per);
  for (int t = rank * per; t < t_end; ++t) {
    const int e0 = t * kRowKeys;
    __syncthreads();
    load_rows2<T, TY>(Ks, Vs, ld, d, kRowKeys, [&](int j) -> const T* { return e0 + j < n ? kb + (long long)(e0 + j) * d : nullptr; },
                  [&](int j) -> const T* { return e0 + j < n ? vb + (long long)(e0 + j) * d : nullptr; });
    __syncthreads();
    float s[4][4], g[4][4];
    tile_dots<TY>(Qs, Ks, ld, d, ty, tx, s);
    tile_dots<TY>(Gs, Vs, ld, d, ty, tx, g);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float p = e0 + tx + 16 * u < n ? exp2f(fmaf(s[i][u], a.scale_log2, -lse2[i])) : 0.f;
        Ps[(ty + TY * i) * kPld + tx + 16 * u] = p * (g[i][u] - D[i]);
      }
    __syncthreads();
    tile_accumulate<TY, U>(Ps, Ks, ld, d, ty, tx, acc);
  }
  const float tau = a.scale_log2 / kLog2e, none = bad ? __int_as_float(0x7fffffff) : 0.f;
  if (shares > 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (4 * (tx + 16 * u) < d) put4(Qs + (ty + TY * i) * ld + 4 * (tx + 16 * u), acc[i][u]);
    cluster_sync();
    write_joined<T, TY>(Qs, ld, d, rows, bad ? 0 : rows, shares, rank, tau, none, (T*)a.dq + row0 * d);
    cluster_sync();  // no block leaves while another reads it
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + TY * i;
    if (r >= rows) continue;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (4 * (tx + 16 * u) < d) put4((T*)a.dq + (row0 + r) * d + 4 * (tx + 16 * u), scaled(acc[i][u], tau, none));
  }
}

// 4 TY keys against this block's share of the rows
template <typename T, int TY, int U>
__device__ __forceinline__ void cross_dkv_block(const CrossGradArgs& a, float* sm, float* lse_s, float* D_s, long long bh,
                                                int tile, int shares, int rank) {
  constexpr int BK = 4 * TY;
  const int d = a.d, ld = d + 4;
  float* const Ks = sm;
  float* const Vs = Ks + BK * ld;
  float* const Qs = Vs + BK * ld;
  float* const Gs = Qs + kRowKeys * ld;
  float* const Ps = Gs + kRowKeys * ld;   // p of (key, row)
  float* const Ss = Ps + BK * kPld;       // ds of (key, row)
  const int j0 = tile * BK, keys = min(a.n_kv - j0, BK);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  bool bad;
  const int n = grad_keys(a, (int)(bh / a.heads), &bad);
  const int liv = max(0, min(n - j0, BK));  // keys of the tile inside the sequence
  const long long key0 = bh * a.n_kv + j0, rowb = bh * a.R;
  float4 dk[4][U], dv[4][U];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < U; ++u) dk[i][u] = dv[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (liv > 0) {
    load_rows2<T, TY>(Ks, Vs, ld, d, BK, [&](int j) -> const T* { return j < liv ? (const T*)a.k + (key0 + j) * d : nullptr; },
                  [&](int j) -> const T* { return j < liv ? (const T*)a.v + (key0 + j) * d : nullptr; });
    const int tiles = (a.R + kRowKeys - 1) / kRowKeys, per = (tiles + shares - 1) / shares;
    const int t_end = min(tiles, (rank + 1) * per);
    for (int t = rank * per; t < t_end; ++t) {
      const int r0 = t * kRowKeys, rows = min(a.R - r0, kRowKeys);
      __syncthreads();
      load_rows2<T, TY>(Qs, Gs, ld, d, kRowKeys,
                    [&](int r) -> const T* { return r < rows ? (const T*)a.q + (rowb + r0 + r) * d : nullptr; },
                    [&](int r) -> const T* { return r < rows ? (const T*)a.dout + (rowb + r0 + r) * d : nullptr; });
      if (threadIdx.x < kRowKeys) lse_s[threadIdx.x] = threadIdx.x < rows ? lse_log2(a.lse[rowb + r0 + threadIdx.x]) : 0.f;
      __syncthreads();
      {
        float D[kRowKeys / TY];
        row_dots<T, TY, U, kRowKeys / TY>(Gs, ld, d, rows, ty, tx, (const T*)a.out + (rowb + r0) * d, D);
        if (tx == 0)
#pragma unroll
          for (int i = 0; i < kRowKeys / TY; ++i) D_s[ty + TY * i] = D[i];
      }
      __syncthreads();
      float s[4][4], g[4][4];
      tile_dots<TY>(Ks, Qs, ld, d, ty, tx, s);
      tile_dots<TY>(Vs, Gs, ld, d, ty, tx, g);
      if (rows < kRowKeys) {  // rows that fill up the tile: 0, also against a v that holds an infinity
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (tx + 16 * u >= rows) g[i][u] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = tx + 16 * u, at = (ty + TY * i) * kPld + r;
          const float p = r < rows && ty + TY * i < liv ? exp2f(fmaf(s[i][u], a.scale_log2, -lse_s[r])) : 0.f;
          Ps[at] = p;
          Ss[at] = p * (g[i][u] - D_s[r]);
        }
      __syncthreads();
      tile_accumulate<TY, U>(Ps, Gs, ld, d, ty, tx, dv);
      tile_accumulate<TY, U>(Ss, Qs, ld, d, ty, tx, dk);
    }
  }
  const float tau = a.scale_log2 / kLog2e, none = bad ? __int_as_float(0x7fffffff) : 0.f;
  if (shares > 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (4 * (tx + 16 * u) < d) {
          put4(Ks + (ty + TY * i) * ld + 4 * (tx + 16 * u), dk[i][u]);
          put4(Vs + (ty + TY * i) * ld + 4 * (tx + 16 * u), dv[i][u]);
        }
    cluster_sync();
    write_joined<T, TY>(Ks, ld, d, keys, liv, shares, rank, tau, none, (T*)a.dk + key0 * d);
    write_joined<T, TY>(Vs, ld, d, keys, liv, shares, rank, 1.f, none, (T*)a.dv + key0 * d);
    cluster_sync();
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = ty + TY * i;
    if (j >= keys) continue;
    // keys past the sequence's end get zeros, not what 0 times an infinity of dout or q left in their sums
    const float4 rest = make_float4(none, none, none, none);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (4 * (tx + 16 * u) < d) {
        const long long at = (key0 + j) * d + 4 * (tx + 16 * u);
        put4((T*)a.dk + at, j < liv ? scaled(dk[i][u], tau, 0.f) : rest);
        put4((T*)a.dv + at, j < liv ? dv[i][u] : rest);
      }
  }
}

// One launch: the dk, dv tiles, then the dq tiles, `shares` blocks (a cluster) each.
template <typename T, int TY, int U>
__global__ void __launch_bounds__(16 * TY) cross_grad_simt_kernel(CrossGradArgs a, long long n_dkv, int shares) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float lse_s[kRowKeys], D_s[kRowKeys];
  constexpr int BT = 4 * TY;
  const long long unit = blockIdx.x / shares;
  const int rank = (int)(blockIdx.x % shares);
  if (unit < n_dkv) {
    const int tiles = (a.n_kv + BT - 1) / BT;
    cross_dkv_block<T, TY, U>(a, sm, lse_s, D_s, unit / tiles, (int)(unit % tiles), shares, rank);
  } else {
    const int tiles = (a.R + BT - 1) / BT;
    cross_dq_block<T, TY, U>(a, sm, (unit - n_dkv) / tiles, (int)((unit - n_dkv) % tiles), shares, rank);
  }
}

// ---- an accepted path into the cache ---------------------------------------------------------------
// For e < n_path[b], cache row cache_len[b] + e (mod C for a ring) of every head takes row path[b, e]
// of k_tree and v_tree, then cache_len[b] moves on by n_path[b].  One cluster of eight blocks a
// sequence: every block has read the length before the cluster's barrier, one thread writes it
// after -- one launch, no order to get wrong between the copies and the new length.
constexpr int kCommitBlocks = 8;
template <typename T>
__global__ void __cluster_dims__(kCommitBlocks, 1, 1) __launch_bounds__(256)
    cache_commit_kernel(T* __restrict__ kc, T* __restrict__ vc, const T* __restrict__ kt, const T* __restrict__ vt,
                        const int* __restrict__ path, const int* __restrict__ n_path, int* cache_len, int H, int C,
                        int Tn, int L, int d, int ring) {
  const int b = blockIdx.x / kCommitBlocks, rank = blockIdx.x % kCommitBlocks;
  const int len = *(volatile int*)(cache_len + b), cnt = n_path[b];
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  unsigned err = 0u;
  if (len < 0 || cnt < 0 || cnt > L || cnt > C || (!ring && (long long)len + cnt > C) || (long long)len + cnt > 0x7fffffffLL)
    err = kErrCacheLen;
  else
    for (int e = threadIdx.x; e < cnt; e += blockDim.x) {
      const int p = path[(long long)b * L + e];
      if (p < 0 || p >= Tn) bad_s = 1;
    }
  __syncthreads();
  if (!err && bad_s) err = kErrTree;
  if (!err) {
    constexpr int V = 16 / (int)sizeof(T);
    const int chunks = d / V;
    const long long total = (long long)H * cnt * chunks;
    for (long long t = (long long)rank * blockDim.x + threadIdx.x; t < total; t += kCommitBlocks * blockDim.x) {
      const int c = (int)(t % chunks) * V;
      const long long u = t / chunks;
      const int e = (int)(u % cnt), h = (int)(u / cnt);
      const long long bh = (long long)b * H + h;
      const long long slot = ring ? ((long long)len + e) % C : (long long)len + e;
      const long long src = (bh * Tn + path[(long long)b * L + e]) * d + c, dst = (bh * C + slot) * d + c;
      const uint4 x = *reinterpret_cast<const uint4*>(kt + src), y = *reinterpret_cast<const uint4*>(vt + src);
      *reinterpret_cast<uint4*>(kc + dst) = x;
      *reinterpret_cast<uint4*>(vc + dst) = y;
    }
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    if (err) raise_error(err);
    else cache_len[b] = len + cnt;
  }
}

}  // namespace pia
