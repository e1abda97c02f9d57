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
