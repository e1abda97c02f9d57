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
#include "internal.h"
#include "kv.h"

namespace strata {

namespace kvc {
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
}  // namespace kvc

__device__ __forceinline__ float pow2_biased(int biased) {   // 2^(biased - 127), biased in 1..254
  return __uint_as_float((uint32_t)biased << 23);
}

// Biased exponent of a row whose largest magnitude has the bf16 bits `top`:
// 448 = 1.75 * 2^8, so mantissas above 1.75 take the next exponent.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  return min(max(e, -126), 119) + 127;
}

// Sixteen bf16 values per lane, D / 16 lanes per row: codes (16 bytes) and the
// row's biased exponent.  Called by whole warps.  Two 16-bit maxima per
// instruction and two scaled values per multiplication: with one value at a time
// and the infinities looked for in each, the kernel was bound by this
// arithmetic (four 6144-token chunks 18.0 us).
template <int D>
__device__ __forceinline__ uint4 quantise16(const uint4& x0, const uint4& x1, int* biased) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, w[i] & 0x7FFF7FFFu);
  uint32_t top = max(top2 >> 16, top2 & 0xFFFFu);
  const bool odd = __any_sync(0xffffffffu, top >= 0x7F80u);   // an infinity or a NaN
  if (odd) {                             // the largest finite magnitude
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
  }
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  *biased = row_exponent(top);
  const float f = pow2_biased(254 - *biased);
  uint32_t c[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    c[h] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t v = w[2 * h + j];
      float2 y = __fmul2_rn(make_float2(bf16_lo(v), bf16_hi(v)), make_float2(f, f));
      if (odd) {                         // infinities have no code: NaN, as 0 * x says
        y.x += 0.f * bf16_lo(v);
        y.y += 0.f * bf16_hi(v);
      }
      c[h] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * j);
    }
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// How the lanes of a warp share the rows of the call.  D / 16 lanes take a row
// (16 values each), so a warp takes RPS = 512 / D rows at a time.  A token's
// 2 * Hkv rows (K of every head, then V of every head) go to one warp or several in
// steps of RPS; when they are fewer than RPS, several tokens share the warp.
template <int D>
struct RowLanes {
  static constexpr int LPR = D / 16, RPS = 32 / LPR;
  int ch, r, step;        // 16-value piece, first row, rows per step
  int tok;                // the lane's token, -1: none
  __device__ __forceinline__ RowLanes(const strata_kv_cache_t& c, const strata_kv_seqs_t& s) {
    const int lane = threadIdx.x % 32, sub = lane / LPR, rows = 2 * c.Hkv;
    const int warp = blockIdx.x * kvc::WARPS + threadIdx.x / 32;
    const int tpw = rows < RPS ? RPS / rows : 1;
    const int mine = rows < RPS ? sub / rows : 0;
    ch = lane % LPR;
    r = sub - mine * rows;
    step = rows < RPS ? rows : RPS;
    const int64_t t = (int64_t)warp * tpw + mine;
    tok = mine < tpw && t < (int64_t)s.B * s.N ? (int)t : -1;
  }
  // CTAs for all tokens (x) and how many warps share a token's rows (y), each of
  // which takes every y-th lot of `lot` steps: one lot per warp up to two CTAs per
  // SM, two up to four CTAs per SM, four beyond.  Every warp pays the chain
  // position -> page, every lot its loads.  Appending to 32 heads of D = 128 (16 lots),
  // one warp per token -> this: 32 tokens 9.5 -> 2.1 us, 256 tokens 9.7 -> 2.9, 2048
  // tokens 17.8 -> 10.7; 4 heads (2 lots), 32 tokens 2.5 -> 2.0, 24,576 tokens 14.3 and
  // 18.5 with one lot per warp.  Reading 64 positions of 3 sequences at 32 heads 4.3 ->
  // 2.6.
  static dim3 grid(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int lot) {
    const int rows = 2 * c.Hkv, tpw = rows < RPS ? RPS / rows : 1;
    const int64_t x = ((int64_t)s.B * s.N + kvc::WARPS * tpw - 1) / (kvc::WARPS * tpw);
    const int n = (rows + lot * RPS - 1) / (lot * RPS), sms = sm_count();
    const int y = x * n <= 2 * sms ? n : x * ((n + 1) / 2) <= 4 * sms ? (n + 1) / 2 : (n + 3) / 4;
    return dim3((unsigned)x, (unsigned)y);
  }
};

// The position of token `tok` of the call, -1 when its slot is not in use.
__device__ __forceinline__ int64_t token_pos(const strata_kv_seqs_t& s, int tok, int* b,
                                             unsigned* err) {
  if (tok < 0) return -1;
  *b = tok / s.N;
  const int i = tok - *b * s.N;
  bool bad;
  const SeqRange q = seq_range(s, *b, &bad);
  if (bad) atomicOr(err, kErrIndex);
  return i < q.count ? (int64_t)q.pos + i : -1;
}

// Bound by its bytes once there are tens of thousands of rows, by the chain
// position -> page -> row below; the rows' loads are in flight while the page is
// looked up (their addresses do not depend on it).  Four 6144-token chunks (57 MB)
// take 14.3 us, 4.0 TB/s; two steps in flight per warp 16.3 us (more registers,
// fewer warps), two tokens per warp 10 % more.
template <int D>
__global__ void __launch_bounds__(kvc::THREADS)
    kv_append_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, const uint16_t* k, const uint16_t* v,
                     int64_t stride, unsigned* err) {
  stream_order_begin();
  const RowLanes<D> w(c, s);
  int b = 0;
  const int64_t pos = token_pos(s, w.tok, &b, err);
  const int rows = 2 * c.Hkv;
  int row = -1;
  const int first = blockIdx.y * w.step;
  for (int r0 = first; r0 < rows; r0 += gridDim.y * w.step) {
    const int r = r0 + w.r;
    const bool is_v = r >= c.Hkv;
    const int h = is_v ? r - c.Hkv : r;
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (r < rows && pos >= 0) {
      const uint16_t* src = (is_v ? v : k) + w.tok * stride + (int64_t)h * D + w.ch * 16;
      x[0] = ld_v4(src);
      x[1] = ld_v4(src + 8);
    }
    if (r0 == first && pos >= 0) {
      row = (int)row_of(c, s, b, pos);
      if (row < 0) atomicOr(err, kErrIndex);
    }
    int biased;
    const uint4 code = quantise16<D>(x[0], x[1], &biased);
    if (r >= rows || row < 0) continue;
    const int64_t at = row + h * c.page;
    *reinterpret_cast<uint4*>((is_v ? c.v : c.k) + at * D + w.ch * 16) = code;
    if (w.ch == 0) (is_v ? c.v_exp : c.k_exp)[at] = (uint8_t)biased;
  }
}

__device__ __forceinline__ void st_v8(void* p, const uint32_t (&x)[8]) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

__device__ __forceinline__ uint32_t dequantise2(uint32_t codes, float f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  const float2 y = __fmul2_rn(__half22float2(__half2(h)), make_float2(f, f));
  return pack_bf16x2(y.x, y.y);
}

// 34,000 positions at 4 heads (105 MB, two thirds of them written) take 19.1 us,
// 5.5 TB/s.  The sixteen values of a lane leave in one store of 32 bytes (WIDE) where
// the outputs start on such a boundary (every allocation of its own does): two of
// 16 bytes, half a sector each, took 22.6 us.  Eight CTAs per SM (32 registers)
// instead of five 19.7 for 20.6; one or four steps in flight instead of two 20.7
// and 24.3, 128 or 512 threads 21.3 and 25.6.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kvc::THREADS, 8)
    kv_read_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, uint16_t* k_out, uint16_t* v_out,
                   unsigned* err) {
  constexpr int U = 2;
  stream_order_begin();
  const RowLanes<D> w(c, s);
  int b = 0;
  const int64_t pos = token_pos(s, w.tok, &b, err);
  if (pos < 0) return;
  const int row = (int)row_of(c, s, b, pos);
  if (row < 0) atomicOr(err, kErrIndex);
  const int rows = 2 * c.Hkv;
  for (int r0 = blockIdx.y * U * w.step; r0 < rows; r0 += gridDim.y * U * w.step) {
    uint4 code[U];
    int e[U];
    uint16_t* out[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * w.step + w.r;
      const bool is_v = r >= c.Hkv;
      const int h = is_v ? r - c.Hkv : r;
      out[u] = r < rows ? (is_v ? v_out : k_out) : nullptr;
      code[u] = make_uint4(0, 0, 0, 0);
      e[u] = 0;
      if (out[u] && row >= 0) {
        const int64_t at = row + h * c.page;
        e[u] = (is_v ? c.v_exp : c.k_exp)[at];
        code[u] = ld_v4((is_v ? c.v : c.k) + at * D + w.ch * 16);
      }
      if (out[u]) out[u] += ((int64_t)w.tok * c.Hkv + h) * D + w.ch * 16;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!out[u]) continue;
      if (e[u] == 0) code[u] = make_uint4(0, 0, 0, 0);         // nothing held: zeros
      const float f = pow2_biased(e[u]);
      const uint32_t x[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = dequantise2(x[i] & 0xFFFFu, f);
        y[2 * i + 1] = dequantise2(x[i] >> 16, f);
      }
      if (WIDE) {
        st_v8(out[u], y);
      } else {
        reinterpret_cast<uint4*>(out[u])[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4*>(out[u])[1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
  }
}

// One cluster per sequence, one of its CTAs per 256 / D heads.  A warp moves
// the K and V rows of those heads at one position with one 16-byte piece per
// lane; all of the path's rows are read before any is written (a barrier between),
// so the order of the moves does not matter and every read is in flight at
// once.  Moving them in path order, eight at a time, took 9.6 us for 256 paths of
// up to 64 nodes at 8 heads.
namespace kvc {
constexpr int MOVE_WARPS = 16;
}  // namespace kvc

template <int D>
__global__ void __launch_bounds__(kvc::MOVE_WARPS * 32)
    kv_commit_kernel(strata_kv_cache_t c, strata_kv_seqs_t s, const int32_t* path,
                     const int32_t* path_len, int32_t* pos_out, unsigned* err) {
  using namespace kvc;
  constexpr int NODES = STRATA_TREE_MAX_NODES;
  constexpr int CPR = D / 16, HEADS = 256 / D;     // pieces per row; heads per warp
  constexpr int U = NODES / MOVE_WARPS;            // rows per warp
  __shared__ int64_t src[NODES], dst[NODES];
  // the next kernel's CTAs wait until this one is done: let in early, they took 1.6
  // us from 256 sequences' 64-node trees (8.7 us in a graph, this way 7.1; 7.5
  // without programmatic launches)
  stream_order_wait();
  const int b = blockIdx.y, th = threadIdx.x, warp = th / 32, lane = th % 32;
  const int pos = s.pos[b];
  int n = path_len[b];
  bool bad = n < 0 || n > s.N || pos < 0;
  if (bad) n = 0;
  if (th < NODES) {
    int64_t from = -1, to = -1;
    if (th < n) {
      const int p = path[(int64_t)b * s.N + th];
      if (p < th || p >= s.N) {
        bad = true;
      } else if (p > th) {
        from = row_of(c, s, b, (int64_t)pos + p);
        to = row_of(c, s, b, (int64_t)pos + th);
        if (from < 0 || to < 0) {
          bad = true;
          from = -1;
        }
      }
    }
    src[th] = from;
    dst[th] = to;
  }
  if (bad) atomicOr(err, kErrIndex);
  __syncthreads();
  const int piece = lane % CPR;
  const bool v = lane / CPR % 2;
  for (int h0 = blockIdx.x * HEADS; h0 < c.Hkv; h0 += gridDim.x * HEADS) {
    const int h = h0 + lane / CPR / 2;
    uint8_t* codes = (v ? c.v : c.k) + (int64_t)h * c.page * D + piece * 16;
    uint8_t* exps = (v ? c.v_exp : c.k_exp) + (int64_t)h * c.page;
    uint4 x[U];
    uint8_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t from = src[u * MOVE_WARPS + warp];
      if (from >= 0 && h < c.Hkv) {
        x[u] = *reinterpret_cast<const uint4*>(codes + from * D);
        e[u] = exps[from];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t from = src[u * MOVE_WARPS + warp], to = dst[u * MOVE_WARPS + warp];
      if (from >= 0 && h < c.Hkv) {
        *reinterpret_cast<uint4*>(codes + to * D) = x[u];
        if (piece == 0) exps[to] = e[u];
      }
    }
  }
  // pos_out may be pos itself: written once the whole cluster has read it
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (blockIdx.x == 0 && th == 0) pos_out[b] = pos + n;
}

cudaError_t launch_kv_append(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const uint16_t* k, const uint16_t* v, int64_t stride, unsigned* err,
                             cudaStream_t stream) {
  if (c.D == 128)
    return launch_in_order(kv_append_kernel<128>, RowLanes<128>::grid(c, s, 1), kvc::THREADS, 0,
                           stream, 0, c, s, k, v, stride, err);
  return launch_in_order(kv_append_kernel<64>, RowLanes<64>::grid(c, s, 1), kvc::THREADS, 0, stream,
                         0, c, s, k, v, stride, err);
}

cudaError_t launch_kv_read(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, uint16_t* k_out,
                           uint16_t* v_out, unsigned* err, cudaStream_t stream) {
  const bool wide =
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  if (c.D == 128)
    return launch_in_order(wide ? kv_read_kernel<128, true> : kv_read_kernel<128, false>,
                           RowLanes<128>::grid(c, s, 2), kvc::THREADS, 0, stream, 0, c, s,
                           k_out, v_out, err);
  return launch_in_order(wide ? kv_read_kernel<64, true> : kv_read_kernel<64, false>,
                         RowLanes<64>::grid(c, s, 2), kvc::THREADS, 0, stream, 0, c, s, k_out,
                         v_out, err);
}

cudaError_t launch_kv_commit(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* path, const int32_t* path_len, int32_t* pos_out,
                             unsigned* err, cudaStream_t stream) {
  const int heads = 256 / c.D, groups = (c.Hkv + heads - 1) / heads;
  // Two CTAs per SM, a cluster of 8 per sequence at most.  More of them wait
  // for a place and pay the chain position -> path -> page again: 256 paths at 8
  // heads took 7.2 us with one CTA per sequence (7.0 with programmatic launches),
  // 8.9 and 11.1 us with two and four; 32 paths 3.7 us with four.
  int ctas = 2 * sm_count() / s.B;
  ctas = ctas < 1 ? 1 : ctas > 8 ? 8 : ctas;
  if (ctas > groups) ctas = groups;
  return launch_in_order(c.D == 128 ? kv_commit_kernel<128> : kv_commit_kernel<64>, dim3(ctas, s.B),
                         kvc::MOVE_WARPS * 32, 0, stream, (unsigned)ctas, c, s, path, path_len,
                         pos_out, err);
}

}  // namespace strata
