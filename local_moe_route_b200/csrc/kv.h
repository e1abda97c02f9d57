// kv.h -- device-side views of the paged KV cache and the host-side launch
// functions of its kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/strata_kv.h"

namespace strata {

unsigned* check_word();   // device address of the check word of the current device (api.cu)

cudaError_t launch_kv_append(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const uint16_t* k, const uint16_t* v, int64_t stride, unsigned* err,
                             cudaStream_t stream);
cudaError_t launch_kv_read(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, uint16_t* k_out,
                           uint16_t* v_out, unsigned* err, cudaStream_t stream);
cudaError_t launch_kv_commit(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* path, const int32_t* path_len, int32_t* pos_out,
                             unsigned* err, cudaStream_t stream);

size_t tree_attn_scratch(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int Hq);
cudaError_t launch_tree_attn(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* parent, const uint16_t* q, int64_t q_stride, int Hq,
                             float scale, uint16_t* out, void* ws, unsigned* err,
                             cudaStream_t stream);

cudaError_t launch_verify(const int32_t* tokens, const int32_t* parent, const int32_t* count,
                          const float* p, const float* q, const float* u_accept,
                          const float* u_sample, int B, int N, int V, int32_t* path,
                          int32_t* path_len, int32_t* out_tokens, unsigned* err,
                          cudaStream_t stream);

#ifdef __CUDACC__
// These kernels are launched so that their CTAs may be set up while the kernel
// before them in the stream still runs (programmatic stream serialization): a
// step is a chain of calls of a few microseconds each, and the gap between two
// launches is about one.  Every kernel waits, in all its threads and before it
// touches global memory, until the kernel before it is complete and its writes
// are visible, so the order of the stream's work is what it always is; it lets the
// next one in as soon as all its own CTAs run.  What another kernel may have
// written is read with plain loads: the read-only path asks for data that does not
// change while the kernel is resident, and it may be resident early.  Calls of one
// token per sequence one after another from Python: append 8.1 -> 7.5 us, attention
// 12.4 -> 11.2; in a graph 2.7 -> 2.6 and 11.1 -> 11.0.
__device__ __forceinline__ void stream_order_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void stream_order_begin() {
  stream_order_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// `cluster`: CTAs per cluster along x, 0 when the kernel says it itself.
template <class... P, class... A>
inline cudaError_t launch_in_order(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                   cudaStream_t stream, unsigned cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The first position and the number of tokens of sequence b in this call; a
// negative position or a count outside 0 .. N leaves it without tokens.
struct SeqRange {
  int pos, count;
};
__device__ __forceinline__ SeqRange seq_range(const strata_kv_seqs_t& s, int b, bool* bad) {
  SeqRange r;
  r.pos = s.pos[b];
  r.count = s.count ? s.count[b] : s.N;
  *bad = r.pos < 0 || r.count < 0 || r.count > s.N;
  if (*bad) r = {0, 0};
  return r;
}

// Row (page * Hkv + head) * page_size + offset of position t of sequence b
// and head 0, or -1 when the table has no valid page for it.
__device__ __forceinline__ int64_t row_of(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                                          int b, int64_t t) {
  const int64_t col = t / c.page;
  if (col >= s.max_pages) return -1;
  const int pg = s.table[(int64_t)b * s.max_pages + col];
  if ((unsigned)pg >= (unsigned)c.pages) return -1;
  return (int64_t)pg * c.Hkv * c.page + t % c.page;
}
#endif

}  // namespace strata
