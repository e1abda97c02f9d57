// verify.cu -- verification of drafted tokens against the target's
// probabilities (rejection sampling down a tree), from given random numbers.
//
// Repeatedly replacing p by the normalised positive part of p - q needs no
// row of state: with r_0 = p and S_0 = 1, the k-th rejection leaves
//   r_k = max(p - c_k q, 0),   c_k = S_0 + ... + S_(k-1),   S_k = sum r_k,
// because max(max(p - c q, 0) - S q, 0) = max(p - (c + S) q, 0) for S, q >= 0.  So
// a rejection costs one sum over the rows p and q, and the next token one
// more; an acceptance reads two numbers.  Sums and comparisons are in 64 bits:
// a token's probability mass can be as small as the rounding of a 32-bit sum
// over the vocabulary, and the token that comes out must not depend on it.
//
// One cluster of 8 CTAs per sequence shares the vocabulary: each warp
// of the cluster owns one contiguous run of it, sums it, and the sums meet in
// rank 0's .. 7's shared memory in a fixed order.  The same per-warp sums find
// the warp whose run holds the next token, and only that run is read again.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kv.h"

namespace strata {

namespace cg = cooperative_groups;

namespace vd {
constexpr int CLUSTER = 8;
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int NODES = STRATA_TREE_MAX_NODES;
}  // namespace vd

// The remaining target row r of one node: p - c q (or p without the rejected
// tokens), read in 16-byte blocks that start at the row's own alignment.
struct RestRow {
  const float* p;       // first element of the row
  const float* q;       // nullptr: rejected tokens instead
  double c;
  int V;
  int shift;            // elements between the 16-byte boundary below p and p
  const int* gone;      // rejected tokens of the node (q == nullptr)
  int n_gone;

  __device__ __forceinline__ double rest(float pv, float qv) const {
    const double r = fma(-c, (double)qv, (double)pv);
    return r > 0.0 ? r : 0.0;
  }
  __device__ __forceinline__ double one(float pv, float qv, int x) const {
    if (q) return rest(pv, qv);
    for (int i = 0; i < n_gone; ++i)
      if (gone[i] == x) return 0.0;
    return (double)pv;
  }
  // The four values of block `blk` (elements 4 * blk - shift ..), 0 outside
  // the row.
  __device__ __forceinline__ void load(int blk, float (&pv)[4], float (&qv)[4]) const {
    const int x0 = 4 * blk - shift;
    if (x0 >= 0 && x0 + 4 <= V) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + x0));
      pv[0] = a.x; pv[1] = a.y; pv[2] = a.z; pv[3] = a.w;
      if (q) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(q + x0));
        qv[0] = b.x; qv[1] = b.y; qv[2] = b.z; qv[3] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = x0 + j >= 0 && x0 + j < V;
        pv[j] = in ? __ldg(p + x0 + j) : 0.f;
        qv[j] = in && q ? __ldg(q + x0 + j) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void values(int blk, const float (&pv)[4], const float (&qv)[4],
                                         double (&r)[4]) const {
    const int x0 = 4 * blk - shift;
#pragma unroll
    for (int j = 0; j < 4; ++j)      // (elements outside the row were loaded as 0)
      r[j] = q ? rest(pv[j], qv[j]) : (double)pv[j];
    if (!q)
      for (int i = 0; i < n_gone; ++i) {
        const int d = gone[i] - x0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d == j) r[j] = 0.0;
      }
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum of blocks [b0, b1) by one warp, the same in every lane.
template <bool Q>
__device__ __forceinline__ double run_sum(const RestRow& row, int b0, int b1, int lane) {
  constexpr int U = 2;
  double s0 = 0.0, s1 = 0.0;
  auto add = [](double& s, double r) {
    if (r > 0.0) s += r;
  };
  for (int blk = b0 + lane; blk < b1; blk += 32 * U) {
    float pv[U][4], qv[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pv[u][j] = qv[u][j] = 0.f;
      if (blk + 32 * u < b1) row.load(blk + 32 * u, pv[u], qv[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (Q) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          add(s0, fma(-row.c, (double)qv[u][j], (double)pv[u][j]));
          add(s1, fma(-row.c, (double)qv[u][j + 1], (double)pv[u][j + 1]));
        }
      } else {
        double r[4];
        row.values(blk + 32 * u, pv[u], qv[u], r);
        s0 += r[0] + r[1];
        s1 += r[2] + r[3];
      }
    }
  }
  return warp_sum(s0 + s1);
}

__global__ void __cluster_dims__(vd::CLUSTER, 1, 1) __launch_bounds__(vd::THREADS, 2)
    verify_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ parent,
                  const int32_t* __restrict__ count, const float* __restrict__ p,
                  const float* __restrict__ q, const float* __restrict__ u_accept,
                  const float* __restrict__ u_sample, int N, int V, int32_t* __restrict__ path,
                  int32_t* __restrict__ path_len, int32_t* __restrict__ out_tokens,
                  unsigned* err) {
  using namespace vd;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / CLUSTER;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // sums of every warp's run, two copies used in turn: a CTA may still read
  // one while another CTA already writes the next
  __shared__ double sums[2][CLUSTER * WARPS];
  __shared__ int gone[NODES], nodes[NODES];
  __shared__ int tok_s[NODES], par_s[NODES];
  __shared__ float u_s[NODES], p_s[NODES], q_s[NODES];
  int n = count ? count[b] : N;
  if (n < 0 || n > N) {
    if (rank == 0 && threadIdx.x == 0) atomicOr(err, kErrIndex);
    n = 0;
  }
  if (n == 0) {            // the whole cluster leaves: nothing to synchronise
    if (rank == 0) {
      for (int i = threadIdx.x; i < N; i += THREADS) {
        path[(int64_t)b * N + i] = -1;
        out_tokens[(int64_t)b * N + i] = -1;
      }
      if (threadIdx.x == 0) path_len[b] = 0;
    }
    return;
  }
  if ((int)threadIdx.x < n) {
    const int i = threadIdx.x;
    const int64_t at = (int64_t)b * N + i;
    int pa = parent ? parent[at] : i - 1;
    if (pa < -1 || pa >= i) {
      if (rank == 0) atomicOr(err, kErrIndex);
      pa = -1;
    }
    const int x = tokens[at];
    if (i > 0 && (unsigned)x >= (unsigned)V && rank == 0) atomicOr(err, kErrIndex);
    tok_s[i] = x;
    par_s[i] = pa;
    u_s[i] = u_accept[at];
    // the token's own probabilities after its parent, should it be asked for
    float pv = 0.f, qv = 1.f;
    if (i > 0 && pa >= 0 && (unsigned)x < (unsigned)V) {
      const int64_t px = ((int64_t)b * N + pa) * V + x;
      pv = __ldg(p + px);
      if (q) qv = __ldg(q + px);
    }
    p_s[i] = pv;
    q_s[i] = qv;
  }
  cluster.sync();            // every CTA runs: its shared memory may be written from now on

  int turn = 0;
  // The sum of r over the row, equal in every thread of the cluster; leaves the
  // warps' sums in sums[turn].
  auto total = [&](const RestRow& row) -> double {
    turn ^= 1;
    const int blocks = (row.shift + V + 3) / 4;
    const int per = (blocks + CLUSTER * WARPS - 1) / (CLUSTER * WARPS);
    const int w = rank * WARPS + warp;
    const int b0 = min(w * per, blocks), b1 = min(b0 + per, blocks);
    const double s = row.q ? run_sum<true>(row, b0, b1, lane) : run_sum<false>(row, b0, b1, lane);
    if (lane < CLUSTER) cluster.map_shared_rank(&sums[turn][0], lane)[w] = s;
    cluster.sync();
    double t = 0.0;
    for (int i = lane; i < CLUSTER * WARPS; i += 32) t += sums[turn][i];
    return warp_sum(t);
  };

  int cur = 0, n_path = 1, n_gone = 0;
  double c = 0.0, S = 1.0;
  bool known = true;         // S is the sum of r
  auto row_at = [&]() {
    RestRow r;
    const int64_t off = ((int64_t)b * N + cur) * V;
    r.p = p + off;
    // nothing rejected yet: r is p, whatever q is
    r.q = q && c != 0.0 ? q + off : nullptr;
    r.c = c;
    r.V = V;
    r.shift = (int)(off & 3);
    r.gone = gone;
    r.n_gone = q ? 0 : n_gone;
    return r;
  };
  if (threadIdx.x == 0) nodes[0] = 0;
  for (int i = 1; i < n; ++i) {
    if (par_s[i] != cur) continue;
    const int x = tok_s[i];
    if ((unsigned)x >= (unsigned)V) continue;
    if (!known) S = total(row_at());
    known = true;
    if ((double)u_s[i] * (double)q_s[i] * S < row_at().one(p_s[i], q_s[i], x)) {
      cur = i;
      c = 0.0;
      S = 1.0;
      __syncthreads();       // everyone is done with gone[]
      n_gone = 0;
      if (threadIdx.x == 0) nodes[n_path] = i;
      ++n_path;
    } else {
      c += S;
      known = false;
      if (threadIdx.x == 0) gone[n_gone] = x;
      ++n_gone;
      __syncthreads();
    }
  }
  // the next token
  const RestRow row = row_at();
  __syncthreads();
  const double sum = total(row);
  const double want = (double)u_sample[b] * sum;
  // the run that holds it: the first whose running sum exceeds `want`, else
  // the last with a positive sum.  Every warp scans the sums, four to a lane.
  constexpr int RPL = CLUSTER * WARPS / 32;
  double mine[RPL], upto = 0.0;
#pragma unroll
  for (int j = 0; j < RPL; ++j) {
    mine[j] = sums[turn][lane * RPL + j];
    upto += mine[j];
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  double at = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) at = 0.0;
  int hit = -1, last = -1;
  double hit_at = 0.0, last_at = 0.0;
#pragma unroll
  for (int j = 0; j < RPL; ++j) {
    if (mine[j] > 0.0) {
      last = lane * RPL + j;
      last_at = at;
      if (hit < 0 && at + mine[j] > want) {
        hit = last;
        hit_at = at;
      }
    }
    at += mine[j];
  }
  const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
  const unsigned some = __ballot_sync(0xffffffffu, last >= 0);
  const int from = hits ? __ffs(hits) - 1 : some ? 31 - __clz(some) : 0;
  int run = __shfl_sync(0xffffffffu, hits ? hit : last, from);
  const double below_run = __shfl_sync(0xffffffffu, hits ? hit_at : last_at, from);
  if (run < 0) {
    run = 0;
    if (rank == 0 && threadIdx.x == 0) atomicOr(err, kErrIndex);
  }
  if (rank == run / WARPS && warp == run % WARPS) {
    const int blocks = (row.shift + V + 3) / 4;
    const int per = (blocks + CLUSTER * WARPS - 1) / (CLUSTER * WARPS);
    const int b0 = min(run * per, blocks), b1 = min(b0 + per, blocks);
    // each lane takes a contiguous share, U blocks of it at a time
    constexpr int U = 4;
    int found = -1, fallback = -1;
    double base = below_run;
    for (int k0 = b0; k0 < b1 && found < 0; k0 += 32 * U) {
      const int share = min(U, (b1 - k0 + 31) / 32);
      const int l0 = k0 + lane * share;
      float pv[U][4], qv[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < share && l0 + u < b1) row.load(l0 + u, pv[u], qv[u]);
      double mine_sum = 0.0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < share && l0 + u < b1) {
          double r[4];
          row.values(l0 + u, pv[u], qv[u], r);
          mine_sum += (r[0] + r[1]) + (r[2] + r[3]);
        }
      double to = mine_sum;                      // sum of lanes 0 .. lane
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, to, off);
        if (lane >= off) to += o;
      }
      const double before = __shfl_up_sync(0xffffffffu, to, 1);
      double run_at = base + (lane ? before : 0.0);
      int x_hit = -1, x_pos = -1;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < share && l0 + u < b1) {
          double r[4];
          row.values(l0 + u, pv[u], qv[u], r);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            run_at += r[j];
            if (r[j] > 0.0) {
              x_pos = 4 * (l0 + u) - row.shift + j;
              if (x_hit < 0 && run_at > want) x_hit = x_pos;
            }
          }
        }
      const unsigned x_hits = __ballot_sync(0xffffffffu, x_hit >= 0);
      const unsigned x_some = __ballot_sync(0xffffffffu, x_pos >= 0);
      if (x_some) fallback = __shfl_sync(0xffffffffu, x_pos, 31 - __clz(x_some));
      if (x_hits) found = __shfl_sync(0xffffffffu, x_hit, __ffs(x_hits) - 1);
      base += __shfl_sync(0xffffffffu, to, 31);
    }
    if (found < 0) found = fallback < 0 ? 0 : fallback;
    for (int i = lane; i < N; i += 32) {
      const int64_t at = (int64_t)b * N + i;
      path[at] = i < n_path ? nodes[i] : -1;
      out_tokens[at] = i < n_path - 1 ? tok_s[nodes[i + 1]] : i == n_path - 1 ? found : -1;
    }
    if (lane == 0) path_len[b] = n_path;
  }
  // no CTA leaves while another may still write its shared memory: every
  // remote write came before the last cluster barrier
}

cudaError_t launch_verify(const int32_t* tokens, const int32_t* parent, const int32_t* count,
                          const float* p, const float* q, const float* u_accept,
                          const float* u_sample, int B, int N, int V, int32_t* path,
                          int32_t* path_len, int32_t* out_tokens, unsigned* err,
                          cudaStream_t stream) {
  verify_kernel<<<B * vd::CLUSTER, vd::THREADS, 0, stream>>>(tokens, parent, count, p, q, u_accept,
                                                             u_sample, N, V, path, path_len,
                                                             out_tokens, err);
  return cudaGetLastError();
}

}  // namespace strata
