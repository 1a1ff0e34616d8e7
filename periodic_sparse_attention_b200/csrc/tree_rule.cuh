// tree_rule.cuh -- the index rule for a tree of drafted tokens over a cache, as a list of keys.
//
// Node t of a tree sits at position i = len + x, x its depth (0 for a root) and len the cache
// length before the drafted tokens.  By the prefill rule it reads the positions i - k .. i and the
// skips i - m*pi (m0 <= m <= S): those below len are cache rows, the others are its ancestors'
// rows (and its own) among the drafted tokens.  With D distinct depths the union over the nodes of
// the cache rows is a short list, in this order, each row once:
//   window    the last min(len, k) positions
//   skips     for m = m0 .. m1 the positions len - m*pi + o, o < Lseg = min(D, pi), as far as they
//             are >= 0 and before the window (a deeper node's skip that falls into the window, or
//             into the next period's segment, is that list entry)
//   tree      the drafted tokens
// Whether a node reads an entry depends on positions alone (and, for a drafted token, on being an
// ancestor): with rel = position - len, back = x - rel is the distance to the key,
//   window key: back <= k          skip key: back > k, back <= S*pi, back a multiple of pi,
// the last tested as equal residues of position and row modulo pi (one division a key, none a pair).
#pragma once
#include "common.cuh"

namespace pia {

// flag of the device error word (after common.cuh's): a parent or path entry that names no earlier / existing node
constexpr unsigned kErrTree = 8u;

constexpr int kMaxTree = 256;      // drafted tokens of one sequence
constexpr int kRelNone = -0x7fffffff - 1;  // rel of a list entry that no row exists for

struct TreeArgs {
  const int* parent;     // [B, T]
  const int* tree_len;   // [B] or null
  const int* cache_len;  // [B]
  int T, cap, kwin, pi, S, ring;
};

// A sequence's lengths as the kernels take them: a ring holds any number of tokens that leaves room for the
// positions of a tree below 2^31.
__host__ __device__ __forceinline__ bool tree_lengths_ok(const TreeArgs& a, int len, int nodes) {
  return len >= 0 && (a.ring || len <= a.cap) && len <= 0x7fffffff - 2 * kMaxTree && nodes >= 0 && nodes <= a.T;
}

// One sequence's key list (the same in every thread of a block).
struct TreeList {
  int len, nodes;        // cache length, drafted tokens
  int nwin, nskip, lseg; // entries of the window, of the skips, rows a skip segment
  int m0;
  int cap, pi, kwin, ring;
  long long reach;       // S * pi
  int len_mod;           // len mod pi

  __host__ __device__ __forceinline__ void init(const TreeArgs& a, int len_, int nodes_, int depths) {
    len = len_;
    nodes = nodes_;
    cap = a.cap;
    pi = a.pi;
    kwin = a.kwin;
    ring = a.ring;
    reach = (long long)a.S * a.pi;
    len_mod = len % pi;
    nwin = len < kwin ? len : kwin;
    lseg = depths < pi ? depths : pi;
    m0 = first_skip_m(kwin, pi);
    long long m1 = ((long long)len + lseg - 1) / pi;  // the farthest segment with a position >= 0
    if (m1 > a.S) m1 = a.S;
    nskip = m1 >= m0 ? (int)(m1 - m0 + 1) * lseg : 0;
  }
  __host__ __device__ __forceinline__ int cached() const { return nwin + nskip; }  // entries before the tree's
  __host__ __device__ __forceinline__ int total() const { return nwin + nskip + nodes; }

  // Entry e < cached(): rel (position - len, kRelNone where there is no row to read) and the cache
  // row it sits in.
  __host__ __device__ __forceinline__ int rel_of(int e) const {
    if (e < nwin) return e - nwin;
    const int t = e - nwin, m = m0 + t / lseg, o = t % lseg;
    const long long rel = (long long)o - (long long)m * pi;
    return rel + len < 0 || rel >= -(long long)nwin ? kRelNone : (int)rel;
  }
  // (lengths stay 512 below 2^31, so positions and the sums here fit 32 bits)
  __host__ __device__ __forceinline__ int row_of(int rel) const {
    const int p = len + rel;
    return ring ? p % cap : p;
  }
  // residue of position len + rel modulo pi, -1 for an entry without a row
  __host__ __device__ __forceinline__ int mod_of(int rel) const {
    if (rel == kRelNone) return -1;
    const int r = (len_mod + rel) % pi;
    return r < 0 ? r + pi : r;
  }
};

// The rule for one (node, key): 0 not read, 1 window key, 2 skip key.
__host__ __device__ __forceinline__ int tree_kind(int x, int xmod, int rel, int mod, int kwin, long long reach) {
  if (mod < 0) return 0;  // no such row
  const int back = x - rel;
  if (back < 0) return 0;
  if (back <= kwin) return 1;
  return mod == xmod && back <= reach ? 2 : 0;
}

// Depths of a sequence's nodes and, for rows r0 .. r0 + nrows - 1, the bit set of each node's
// ancestors and itself.  All threads of the block take part (T <= kMaxTree, any block size).
//   par    kMaxTree ints of shared memory (scratch)
//   depth  kMaxTree bytes (written for every node)
//   anc    nrows x (kMaxTree / 32) words
//   flags  two ints: bad (a parent out of range), the number of depths
// Returns false where a parent is not -1 or an earlier node.
__device__ __forceinline__ bool tree_setup(const int* __restrict__ parent, int nodes, int r0, int nrows, int* par,
                                           uint8_t* depth, uint32_t* anc, int* flags) {
  constexpr int W = kMaxTree / 32;
  const int first = (int)threadIdx.x < nodes ? parent[threadIdx.x] : 0;  // on its way during the zeroing
  if (threadIdx.x == 0) flags[0] = flags[1] = 0;
  for (int t = threadIdx.x; t < nrows * W; t += blockDim.x) anc[t] = 0u;
  __syncthreads();
  for (int t = threadIdx.x; t < nodes; t += blockDim.x) {
    const int p = t == (int)threadIdx.x ? first : parent[t];
    par[t] = p;
    if (p < -1 || p >= t) flags[0] = 1;
  }
  __syncthreads();
  if (flags[0]) return false;
  int deepest = 0;
  for (int t = threadIdx.x; t < nodes; t += blockDim.x) {
    const bool mine = t >= r0 && t < r0 + nrows;
    int n = 0;
    for (int u = t; u >= 0; u = par[u], ++n)  // a parent is an earlier node: at most t + 1 steps
      if (mine) anc[(t - r0) * W + (u >> 5)] |= 1u << (u & 31);
    depth[t] = (uint8_t)(n - 1);
    deepest = n > deepest ? n : deepest;
  }
  if (deepest) atomicMax(&flags[1], deepest);
  __syncthreads();
  return true;
}

}  // namespace pia
