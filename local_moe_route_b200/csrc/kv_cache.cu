// kv_cache.cu -- the 8-bit paged KV cache: quantising rows as they are
// written, reading them back, and moving the accepted path's rows.
//
// A row x (one position of one head, K or V, D values) is held as e4m3 codes
// and one exponent e, the smallest in [-126, 119] with max|x| <= 448 * 2^e.
// Dividing by a power of two is exact, so the one rounding is that of the
// code (half a step, 2^-4 of the value, as for any scale: e4m3 is a floating
// format, a finer scale would not make its steps smaller), and the exponent
// comes from the bf16 bits with integer operations alone.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.h"

namespace strata {

namespace kvc {
constexpr int THREADS = 256;
constexpr int UNROLL = 2;    // rows in flight per thread group
}  // namespace kvc

__device__ __forceinline__ float pow2_biased(int biased) {   // 2^(biased - 127), biased in 1..254
  return __uint_as_float((uint32_t)biased << 23);
}

// Eight bf16 values per lane, D / 8 lanes per row: codes (8 bytes) and the
// row's biased exponent.
template <int D>
__device__ __forceinline__ uint2 quantise8(const uint4& x, int* biased) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // largest finite magnitude, as bf16 bits
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    if (lo < 0x7F80u) top = max(top, lo);
    if (hi < 0x7F80u) top = max(top, hi);
  }
#pragma unroll
  for (int off = D / 16; off > 0; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  // 448 = 1.75 * 2^8: mantissas above 1.75 take the next exponent
  int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  e = min(max(e, -126), 119);
  *biased = e + 127;
  const float s = pow2_biased(127 - e);
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    c[h] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float a = bf16_lo(w[2 * h + j]), b = bf16_hi(w[2 * h + j]);
      // 0 * x is NaN for an infinity (which has no code) and 0 otherwise
      const float2 y = make_float2(fmaf(a, s, 0.f * a), fmaf(b, s, 0.f * b));
      c[h] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * j);
    }
  }
  return make_uint2(c[0], c[1]);
}

// One group of D / 8 lanes per row; rows in the order (token, head, K or V).
template <int D>
__global__ void __launch_bounds__(kvc::THREADS)
    kv_append_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, const uint16_t* __restrict__ k,
                     const uint16_t* __restrict__ v, int64_t stride, unsigned* err) {
  constexpr int LPR = D / 8;                       // lanes per row
  constexpr int GROUPS = kvc::THREADS / LPR;       // rows per CTA and step
  const int lane = threadIdx.x % LPR;
  const int rows = s.B * s.N * c.Hkv * 2;
  // the whole CTA runs every step: the row maximum uses full-warp shuffles
  for (int base = blockIdx.x * GROUPS * kvc::UNROLL; base < rows;
       base += gridDim.x * GROUPS * kvc::UNROLL) {
    uint4 x[kvc::UNROLL];
    int64_t row[kvc::UNROLL];
    bool is_v[kvc::UNROLL];
#pragma unroll
    for (int u = 0; u < kvc::UNROLL; ++u) {
      const int r = base + u * GROUPS + (int)threadIdx.x / LPR;
      row[u] = -1;
      x[u] = make_uint4(0, 0, 0, 0);
      if (r >= rows) continue;
      const int kv = r & 1, th = r >> 1, h = th % c.Hkv, tok = th / c.Hkv;
      const int b = tok / s.N, i = tok % s.N;
      bool bad;
      const SeqRange q = seq_range(s, b, &bad);
      if (bad) atomicOr(err, kErrIndex);
      if (i >= q.count) continue;
      row[u] = row_of(c, s, b, (int64_t)q.pos + i);
      if (row[u] < 0) {
        atomicOr(err, kErrIndex);
        continue;
      }
      row[u] += (int64_t)h * c.page;
      is_v[u] = kv != 0;
      x[u] = ld_nc_v4((kv ? v : k) + tok * stride + h * D + lane * 8);
    }
#pragma unroll
    for (int u = 0; u < kvc::UNROLL; ++u) {
      int biased;
      const uint2 code = quantise8<D>(x[u], &biased);
      if (row[u] < 0) continue;
      *reinterpret_cast<uint2*>((is_v[u] ? c.v : c.k) + row[u] * D + lane * 8) = code;
      if (lane == 0) (is_v[u] ? c.v_exp : c.k_exp)[row[u]] = (uint8_t)biased;
    }
  }
}

__device__ __forceinline__ uint32_t dequantise2(uint32_t codes, float f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  const float2 y = __half22float2(__half2(h));
  return pack_bf16x2(y.x * f, y.y * f);
}

template <int D>
__global__ void __launch_bounds__(kvc::THREADS)
    kv_read_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, uint16_t* __restrict__ k_out,
                   uint16_t* __restrict__ v_out, unsigned* err) {
  constexpr int LPR = D / 8;
  constexpr int GROUPS = kvc::THREADS / LPR;
  const int lane = threadIdx.x % LPR;
  const int rows = s.B * s.N * c.Hkv * 2;
  for (int base = blockIdx.x * GROUPS * kvc::UNROLL; base < rows;
       base += gridDim.x * GROUPS * kvc::UNROLL) {
    uint2 code[kvc::UNROLL];
    float f[kvc::UNROLL];
    uint16_t* dst[kvc::UNROLL];
#pragma unroll
    for (int u = 0; u < kvc::UNROLL; ++u) {
      const int r = base + u * GROUPS + (int)threadIdx.x / LPR;
      dst[u] = nullptr;
      code[u] = make_uint2(0, 0);
      f[u] = 0.f;
      if (r >= rows) continue;
      const int kv = r & 1, th = r >> 1, h = th % c.Hkv, tok = th / c.Hkv;
      const int b = tok / s.N, i = tok % s.N;
      uint16_t* out = kv ? v_out : k_out;
      if (!out) continue;
      bool bad;
      const SeqRange q = seq_range(s, b, &bad);
      if (bad) atomicOr(err, kErrIndex);
      if (i >= q.count) continue;
      dst[u] = out + ((int64_t)tok * c.Hkv + h) * D + lane * 8;
      int64_t row = row_of(c, s, b, (int64_t)q.pos + i);
      if (row < 0) {
        atomicOr(err, kErrIndex);
        continue;
      }
      row += (int64_t)h * c.page;
      const int e = (kv ? c.v_exp : c.k_exp)[row];
      if (e == 0) continue;                        // nothing held: zeros
      code[u] = ld_nc_v2((kv ? c.v : c.k) + row * D + lane * 8);
      f[u] = pow2_biased(e);
    }
#pragma unroll
    for (int u = 0; u < kvc::UNROLL; ++u) {
      if (!dst[u]) continue;
      uint4 y;
      y.x = dequantise2(code[u].x & 0xFFFFu, f[u]);
      y.y = dequantise2(code[u].x >> 16, f[u]);
      y.z = dequantise2(code[u].y & 0xFFFFu, f[u]);
      y.w = dequantise2(code[u].y >> 16, f[u]);
      *reinterpret_cast<uint4*>(dst[u]) = y;
    }
  }
}

// One CTA per sequence.  A thread owns one 16-byte column of a head's K or V
// rows (or a head's exponents) and moves it for the whole path in ascending
// order, several loads ahead of the stores.  Sources are never below their
// destinations (path[i] >= i), so a row is read before it is overwritten:
// row i is written after the rows path[0..i] are read, and a later entry
// reads at its own index or above.
template <int D>
__global__ void __launch_bounds__(kvc::THREADS)
    kv_commit_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, const int32_t* __restrict__ path,
                     const int32_t* __restrict__ path_len, int32_t* pos_out, unsigned* err) {
  constexpr int CPR = D / 16;                      // 16-byte columns per row
  constexpr int AHEAD = 8;
  __shared__ int64_t src[STRATA_TREE_MAX_NODES + AHEAD], dst[STRATA_TREE_MAX_NODES + AHEAD];
  const int b = blockIdx.x;
  const int pos = s.pos[b];
  int n = path_len[b];
  bool bad = n < 0 || n > s.N || pos < 0;
  if (bad) n = 0;
  for (int i = threadIdx.x; i < STRATA_TREE_MAX_NODES + AHEAD; i += kvc::THREADS) {
    int64_t from = -1, to = -1;
    if (i < n) {
      const int p = path[(int64_t)b * s.N + i];
      if (p < i || p >= s.N) {
        bad = true;
      } else if (p > i) {
        from = row_of(c, s, b, (int64_t)pos + p);
        to = row_of(c, s, b, (int64_t)pos + i);
        if (from < 0 || to < 0) {
          bad = true;
          from = -1;
        }
      }
    }
    src[i] = from;
    dst[i] = to;
  }
  if (bad) atomicOr(err, kErrIndex);
  __syncthreads();
  for (int it = threadIdx.x; it < c.Hkv * 2 * (CPR + 1); it += kvc::THREADS) {
    const int col = it % (CPR + 1), kv = (it / (CPR + 1)) & 1, h = it / (CPR + 1) / 2;
    const int64_t head = (int64_t)h * c.page;
    uint8_t* codes = kv ? c.v : c.k;
    uint8_t* exps = kv ? c.v_exp : c.k_exp;
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
      if (col < CPR) {
        uint4 x[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (src[i0 + u] >= 0)
            x[u] = *reinterpret_cast<const uint4*>(codes + (src[i0 + u] + head) * D + col * 16);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (src[i0 + u] >= 0)
            *reinterpret_cast<uint4*>(codes + (dst[i0 + u] + head) * D + col * 16) = x[u];
      } else {
        uint8_t x[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (src[i0 + u] >= 0) x[u] = exps[src[i0 + u] + head];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (src[i0 + u] >= 0) exps[dst[i0 + u] + head] = x[u];
      }
    }
  }
  // every thread of the CTA read pos before the barrier above
  if (threadIdx.x == 0) pos_out[b] = pos + n;
}

static int row_grid(const strata_kv_cache_t& c, const strata_kv_seqs_t& s) {
  const int64_t rows = (int64_t)s.B * s.N * c.Hkv * 2;
  const int per = kvc::THREADS / (c.D / 8) * kvc::UNROLL;
  const int64_t ctas = (rows + per - 1) / per;
  return (int)(ctas < 148 * 32 ? ctas : 148 * 32);
}

cudaError_t launch_kv_append(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const uint16_t* k, const uint16_t* v, int64_t stride, unsigned* err,
                             cudaStream_t stream) {
  if (c.D == 128)
    kv_append_kernel<128><<<row_grid(c, s), kvc::THREADS, 0, stream>>>(c, s, k, v, stride, err);
  else
    kv_append_kernel<64><<<row_grid(c, s), kvc::THREADS, 0, stream>>>(c, s, k, v, stride, err);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, uint16_t* k_out,
                           uint16_t* v_out, unsigned* err, cudaStream_t stream) {
  if (c.D == 128)
    kv_read_kernel<128><<<row_grid(c, s), kvc::THREADS, 0, stream>>>(c, s, k_out, v_out, err);
  else
    kv_read_kernel<64><<<row_grid(c, s), kvc::THREADS, 0, stream>>>(c, s, k_out, v_out, err);
  return cudaGetLastError();
}

cudaError_t launch_kv_commit(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* path, const int32_t* path_len, int32_t* pos_out,
                             unsigned* err, cudaStream_t stream) {
  if (c.D == 128)
    kv_commit_kernel<128><<<s.B, kvc::THREADS, 0, stream>>>(c, s, path, path_len, pos_out, err);
  else
    kv_commit_kernel<64><<<s.B, kvc::THREADS, 0, stream>>>(c, s, path, path_len, pos_out, err);
  return cudaGetLastError();
}

}  // namespace strata
