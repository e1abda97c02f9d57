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
// rank 0's .. 7's shared memory in a fixed order.  On the pass for the next
// token the sums of every four values stay in shared memory, so finding it
// takes one more load.
//
// Bound by the chain of passes of the sequence with the most rejections: a
// pass over 100,003 tokens of p and q takes about 4.2 us (2.7 us the sums, of which
// 0.8 us are the conversions to 64 bits, 0.9 us the cluster's barrier); a greedy
// chain of 3 drafts at 32,000 tokens takes 6.2 us in all, 32 trees of 16 nodes at
// 100,003 tokens 24 to 31 us, by how many passes the longest of them needs.
// Holding a node's rows in shared memory between its passes was no faster (29.7
// against 31.4 us then, and slower without rejections), nor were 256 or 1024 threads.
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
      const uint4 a = ld_v4(p + x0);
      pv[0] = __uint_as_float(a.x);
      pv[1] = __uint_as_float(a.y);
      pv[2] = __uint_as_float(a.z);
      pv[3] = __uint_as_float(a.w);
      if (q) {
        const uint4 b = ld_v4(q + x0);
        qv[0] = __uint_as_float(b.x);
        qv[1] = __uint_as_float(b.y);
        qv[2] = __uint_as_float(b.z);
        qv[3] = __uint_as_float(b.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = x0 + j >= 0 && x0 + j < V;
        pv[j] = in ? ld_f32(p + x0 + j) : 0.f;
        qv[j] = in && q ? ld_f32(q + x0 + j) : 0.f;
      }
    }
  }
  template <bool Q>
  __device__ __forceinline__ void values(int blk, const float (&pv)[4], const float (&qv)[4],
                                         double (&r)[4]) const {
    const int x0 = 4 * blk - shift;
#pragma unroll
    for (int j = 0; j < 4; ++j)      // (elements outside the row were loaded as 0)
      r[j] = Q ? rest(pv[j], qv[j]) : (double)pv[j];
    if (!Q)
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

// Sum of blocks [b0, b1) by one warp, the same in every lane.  `keep`, when
// given, gets the blocks' own sums.
template <bool Q>
__device__ __forceinline__ double run_sum(const RestRow& row, int b0, int b1, int lane,
                                          double* keep) {
  constexpr int U = 2;     // 3, 4 and 8 were no faster: the rows come from L2 or once
  double sum = 0.0;
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
      double r[4];
      row.values<Q>(blk + 32 * u, pv[u], qv[u], r);
      const double s = (r[0] + r[1]) + (r[2] + r[3]);
      sum += s;
      if (keep && blk + 32 * u < b1) keep[blk + 32 * u - b0] = s;
    }
  }
  return warp_sum(sum);
}

__global__ void __cluster_dims__(vd::CLUSTER, 1, 1) __launch_bounds__(vd::THREADS, 2)
    verify_kernel(const int32_t* tokens, const int32_t* parent, const int32_t* count,
                  const float* p, const float* q, const float* u_accept,
                  const float* u_sample, int N, int V, int32_t* path, int32_t* path_len,
                  int32_t* out_tokens, unsigned* err) {
  using namespace vd;
  extern __shared__ double block_sums[];     // of this CTA's blocks, for the next token
  stream_order_begin();
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
      pv = ld_f32(p + px);
      if (q) qv = ld_f32(q + px);
    }
    p_s[i] = pv;
    q_s[i] = qv;
  }
  cluster.sync();            // every CTA runs: its shared memory may be written from now on

  int turn = 0;
  // The sum of r over the row, equal in every thread of the cluster; leaves the
  // warps' sums in sums[turn].
  auto total = [&](const RestRow& row, bool keep) -> double {
    turn ^= 1;
    const int blocks = (row.shift + V + 3) / 4;
    const int per = (blocks + CLUSTER * WARPS - 1) / (CLUSTER * WARPS);
    const int w = rank * WARPS + warp;
    const int b0 = min(w * per, blocks), b1 = min(b0 + per, blocks);
    double* at = keep ? block_sums + warp * per : nullptr;
    const double s = row.q ? run_sum<true>(row, b0, b1, lane, at) : run_sum<false>(row, b0, b1, lane, at);
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
    if (!known) S = total(row_at(), false);
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
  const double sum = total(row, true);
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
    // the block: each lane takes a contiguous share of the run's sums
    const double* sum_of = block_sums + warp * per;
    const int share = (b1 - b0 + 31) / 32;
    const int l0 = min(lane * share, b1 - b0), l1 = min(l0 + share, b1 - b0);
    double mine_sum = 0.0;
    for (int i = l0; i < l1; ++i) mine_sum += sum_of[i];
    double to = mine_sum;                        // sum of lanes 0 .. lane
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, to, off);
      if (lane >= off) to += o;
    }
    double run_at = __shfl_up_sync(0xffffffffu, to, 1);
    run_at = below_run + (lane ? run_at : 0.0);
    int blk_hit = -1, blk_pos = -1;
    double hit_from = 0.0, pos_from = 0.0;
    for (int i = l0; i < l1; ++i) {
      const double s = sum_of[i];
      if (s > 0.0) {
        blk_pos = i;
        pos_from = run_at;
        if (blk_hit < 0 && run_at + s > want) {
          blk_hit = i;
          hit_from = run_at;
        }
      }
      run_at += s;
    }
    const unsigned b_hits = __ballot_sync(0xffffffffu, blk_hit >= 0);
    const unsigned b_some = __ballot_sync(0xffffffffu, blk_pos >= 0);
    const int src = b_hits ? __ffs(b_hits) - 1 : b_some ? 31 - __clz(b_some) : 0;
    const int in = __shfl_sync(0xffffffffu, b_hits ? blk_hit : blk_pos, src);
    run_at = __shfl_sync(0xffffffffu, b_hits ? hit_from : pos_from, src);
    // the token in it
    int found = -1, fallback = -1;
    if (in >= 0) {
      const int blk = b0 + in;
      float pv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
      row.load(blk, pv, qv);
      double r[4];
      if (row.q)
        row.values<true>(blk, pv, qv, r);
      else
        row.values<false>(blk, pv, qv, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        run_at += r[j];
        if (r[j] > 0.0) {
          fallback = 4 * blk - row.shift + j;
          if (found < 0 && run_at > want) found = fallback;
        }
      }
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
  auto sums_bytes = [](int v) {
    const int per = ((v + 3) / 4 + 1 + vd::CLUSTER * vd::WARPS - 1) / (vd::CLUSTER * vd::WARPS);
    return per * vd::WARPS * (int)sizeof(double);
  };
  const int bytes = sums_bytes(V);
  // Asked for from well below 48 KB on, which the kernel's other shared memory
  // counts towards, and always the most, whatever V is: another thread's call
  // may set it between this and the launch.
  if (bytes > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sums_bytes(STRATA_VERIFY_MAX_VOCAB));
    if (e != cudaSuccess) return e;
  }
  return launch_in_order(verify_kernel, B * vd::CLUSTER, vd::THREADS, bytes, stream, 0, tokens,
                         parent, count, p, q, u_accept, u_sample, N, V, path, path_len, out_tokens,
                         err);
}

}  // namespace strata
