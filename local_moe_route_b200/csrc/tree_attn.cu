// tree_attn.cu -- attention of the nodes of a draft tree over the 8-bit paged
// KV cache.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.h"

namespace strata {

namespace ta {
constexpr int THREADS = 128;
constexpr int NODES = STRATA_TREE_MAX_NODES;
}  // namespace ta

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

// One CTA per (node, query head, sequence): 128 positions at a time, one
// thread per position for the scores and one per feature for the sum.
template <int D>
__global__ void __launch_bounds__(ta::THREADS)
    tree_attn_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, const int32_t* __restrict__ parent,
                     const uint16_t* __restrict__ q, int64_t q_stride, int Hq, float scale,
                     uint16_t* __restrict__ out, unsigned* err) {
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, th = threadIdx.x;
  const int hk = h / (Hq / c.Hkv);
  bool bad;
  const SeqRange sq = seq_range(s, b, &bad);
  if (bad && th == 0) atomicOr(err, kErrIndex);
  if (i >= sq.count) return;
  __shared__ float qs[D], ws[ta::THREADS], red[ta::THREADS / 32];
  __shared__ int64_t rows[ta::THREADS];
  __shared__ unsigned long long sees;
  const int64_t tok = (int64_t)b * s.N + i;
  if (th < D) qs[th] = __uint_as_float((uint32_t)q[tok * q_stride + h * D + th] << 16);
  if (th == 0) {
    unsigned long long m = 0;
    for (int j = i; j >= 0;) {
      m |= 1ull << j;
      int pa = parent ? parent[(int64_t)b * s.N + j] : j - 1;
      if (pa < -1 || pa >= j) {
        atomicOr(err, kErrIndex);
        pa = -1;
      }
      j = pa;
    }
    sees = m;
  }
  __syncthreads();
  const int64_t end = (int64_t)sq.pos + sq.count;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int64_t t0 = 0; t0 < end; t0 += ta::THREADS) {
    const int64_t t = t0 + th;
    int64_t row = -1;
    float x = -INFINITY;
    if (t < end && (t < sq.pos || ((sees >> (t - sq.pos)) & 1))) {
      row = row_of(c, s, b, t);
      if (row < 0) {
        atomicOr(err, kErrIndex);
      } else {
        row += (int64_t)hk * c.page;
        const int e = c.k_exp[row];
        if (e == 0) {
          row = -1;
        } else {
          x = 0.f;
          for (int d = 0; d < D; ++d) x = fmaf(qs[d], e4m3_value(c.k[row * D + d]), x);
          x *= scale * __uint_as_float((uint32_t)e << 23);
        }
      }
    }
    rows[th] = row;
    float top = x;
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (th % 32 == 0) red[th / 32] = top;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    ws[th] = row < 0 ? 0.f : expf(x - mn);
    const float keep = m == -INFINITY ? 0.f : expf(m - mn);
    __syncthreads();
    l *= keep;
    o *= keep;
    for (int j = 0; j < ta::THREADS; ++j) {
      if (rows[j] < 0) continue;
      l += ws[j];
      if (th < D)
        o = fmaf(ws[j] * __uint_as_float((uint32_t)c.v_exp[rows[j]] << 23),
                 e4m3_value(c.v[rows[j] * D + th]), o);
    }
    m = mn;
    __syncthreads();
  }
  if (th < D)
    out[(tok * Hq + h) * D + th] =
        __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.f ? 0.f : o / l));
}

size_t tree_attn_scratch(const strata_kv_cache_t&, const strata_kv_seqs_t&, int) { return 256; }

cudaError_t launch_tree_attn(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* parent, const uint16_t* q, int64_t q_stride, int Hq,
                             float scale, uint16_t* out, void*, unsigned* err,
                             cudaStream_t stream) {
  const dim3 grid(s.N, Hq, s.B);
  if (c.D == 128)
    tree_attn_kernel<128><<<grid, ta::THREADS, 0, stream>>>(c, s, parent, q, q_stride, Hq, scale,
                                                            out, err);
  else
    tree_attn_kernel<64><<<grid, ta::THREADS, 0, stream>>>(c, s, parent, q, q_stride, Hq, scale,
                                                           out, err);
  return cudaGetLastError();
}

}  // namespace strata
