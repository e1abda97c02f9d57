// api_kv.cu -- the C ABI declared in include/strata_kv.h: host-side argument
// validation and the launches of each entry point.
#include <math.h>

#include "internal.h"
#include "kv.h"

using namespace strata;

namespace {

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_opt(const void* p) { return p == nullptr || ok_ptr(p); }
strata_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? STRATA_OK : STRATA_ERR_CUDA; }

strata_status_t check_cache_dims(const strata_kv_cache_t& c) {
  if (c.pages <= 0 || c.page <= 0 || c.Hkv <= 0 || c.D <= 0) return STRATA_ERR_INVALID_ARG;
  if ((c.D != 64 && c.D != 128) || (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128))
    return STRATA_ERR_UNSUPPORTED;
  if (c.Hkv > 65535 || (int64_t)c.pages * c.Hkv >= (int64_t(1) << 31) / c.page)
    return STRATA_ERR_UNSUPPORTED;
  return STRATA_OK;
}

strata_status_t check_seqs_dims(const strata_kv_cache_t& c, const strata_kv_seqs_t& s) {
  if (s.B < 0 || s.N <= 0 || s.max_pages <= 0) return STRATA_ERR_INVALID_ARG;
  if ((int64_t)s.B * s.N >= (1 << 24) || (int64_t)s.max_pages * c.page >= (int64_t(1) << 31) ||
      (int64_t)s.B * s.N * c.Hkv >= (1 << 29))
    return STRATA_ERR_UNSUPPORTED;
  return STRATA_OK;
}

bool cache_ptrs(const strata_kv_cache_t& c) {
  return ok_ptr(c.k) && ok_ptr(c.v) && ok_ptr(c.k_exp) && ok_ptr(c.v_exp);
}
bool seqs_ptrs(const strata_kv_seqs_t& s) {
  return ok_ptr(s.table) && ok_ptr(s.pos) && ok_opt(s.count);
}

// Sizes of the cache and the sequences, then their pointers.
strata_status_t check_both(const strata_kv_cache_t& c, const strata_kv_seqs_t& s) {
  strata_status_t st = check_cache_dims(c);
  if (st == STRATA_OK) st = check_seqs_dims(c, s);
  if (st == STRATA_OK && s.B > 0 && (!cache_ptrs(c) || !seqs_ptrs(s))) st = STRATA_ERR_INVALID_ARG;
  return st;
}

// A row stride in elements: 0 stands for `width`.  Returns false when it is
// too small, not a multiple of 8, or takes offsets past 2^62.
bool ok_stride(int64_t* stride, int64_t width) {
  if (*stride == 0) *stride = width;
  return *stride >= width && *stride % 8 == 0 && *stride < (int64_t(1) << 36);
}

strata_status_t check_tree_dims(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int Hq) {
  strata_status_t st = check_cache_dims(c);
  if (st == STRATA_OK) st = check_seqs_dims(c, s);
  if (st != STRATA_OK) return st;
  if (Hq <= 0 || Hq % c.Hkv) return STRATA_ERR_INVALID_ARG;
  if (s.N > STRATA_TREE_MAX_NODES || Hq / c.Hkv > 64 || (int64_t)s.B * s.N * Hq >= (1 << 30))
    return STRATA_ERR_UNSUPPORTED;
  // the attention counts its tiles (and rows in blocks of 16 at least) in 31 bits
  const int64_t blocks = ((int64_t)s.N * (Hq / c.Hkv) + 15) / 16;
  if ((double)s.B * c.Hkv * blocks * ((double)s.max_pages * c.page / 256 + 4) >= 2147483648.0)
    return STRATA_ERR_UNSUPPORTED;
  return STRATA_OK;
}

}  // namespace

extern "C" {

strata_status_t strata_kv_append(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                 const uint16_t* k, const uint16_t* v, int64_t stride,
                                 strata_stream_t stream) {
  const strata_status_t st = check_both(cache, seqs);
  if (st != STRATA_OK) return st;
  if (!ok_stride(&stride, (int64_t)cache.Hkv * cache.D)) return STRATA_ERR_INVALID_ARG;
  if (seqs.B == 0) return STRATA_OK;
  if (!ok_ptr(k) || !ok_ptr(v)) return STRATA_ERR_INVALID_ARG;
  unsigned* err = check_word();
  if (!err) return STRATA_ERR_CUDA;
  return cuda_status(launch_kv_append(cache, seqs, k, v, stride, err,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

strata_status_t strata_kv_read(strata_kv_cache_t cache, strata_kv_seqs_t seqs, uint16_t* k_out,
                               uint16_t* v_out, strata_stream_t stream) {
  const strata_status_t st = check_both(cache, seqs);
  if (st != STRATA_OK) return st;
  if (!ok_opt(k_out) || !ok_opt(v_out)) return STRATA_ERR_INVALID_ARG;
  if (seqs.B == 0 || (!k_out && !v_out)) return STRATA_OK;
  unsigned* err = check_word();
  if (!err) return STRATA_ERR_CUDA;
  return cuda_status(
      launch_kv_read(cache, seqs, k_out, v_out, err, reinterpret_cast<cudaStream_t>(stream)));
}

size_t strata_tree_attention_workspace_bytes(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                             int32_t Hq) {
  if (check_tree_dims(cache, seqs, Hq) != STRATA_OK) return 0;
  return tree_attn_scratch(cache, seqs, Hq);
}

strata_status_t strata_tree_attention(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                      const int32_t* parent, const uint16_t* q, int64_t q_stride,
                                      int32_t Hq, float scale, uint16_t* out, void* ws,
                                      size_t ws_bytes, strata_stream_t stream) {
  strata_status_t st = check_tree_dims(cache, seqs, Hq);
  if (st == STRATA_OK) st = check_both(cache, seqs);
  if (st != STRATA_OK) return st;
  if (!ok_stride(&q_stride, (int64_t)Hq * cache.D)) return STRATA_ERR_INVALID_ARG;
  if (seqs.B == 0) return STRATA_OK;
  if (!ok_opt(parent) || !ok_ptr(q) || !ok_ptr(out)) return STRATA_ERR_INVALID_ARG;
  if (!ok_ptr(ws) || ws_bytes < tree_attn_scratch(cache, seqs, Hq)) return STRATA_ERR_WORKSPACE;
  unsigned* err = check_word();
  if (!err) return STRATA_ERR_CUDA;
  if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)cache.D);
  return cuda_status(launch_tree_attn(cache, seqs, parent, q, q_stride, Hq, scale, out, ws, err,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

strata_status_t strata_verify_drafts(const int32_t* tokens, const int32_t* parent,
                                     const int32_t* count, const float* p, const float* q,
                                     const float* u_accept, const float* u_sample,
                                     strata_verify_dims_t dims, int32_t* path, int32_t* path_len,
                                     int32_t* out_tokens, strata_stream_t stream) {
  if (dims.B < 0 || dims.N <= 0 || dims.V <= 0) return STRATA_ERR_INVALID_ARG;
  if (dims.N > STRATA_TREE_MAX_NODES || (int64_t)dims.B * dims.N >= (1 << 24) ||
      dims.V > STRATA_VERIFY_MAX_VOCAB)
    return STRATA_ERR_UNSUPPORTED;
  if (dims.B == 0) return STRATA_OK;
  if (!ok_ptr(tokens) || !ok_opt(parent) || !ok_opt(count) || !ok_ptr(p) || !ok_opt(q) ||
      !ok_ptr(u_accept) || !ok_ptr(u_sample) || !ok_ptr(path) || !ok_ptr(path_len) ||
      !ok_ptr(out_tokens))
    return STRATA_ERR_INVALID_ARG;
  unsigned* err = check_word();
  if (!err) return STRATA_ERR_CUDA;
  return cuda_status(launch_verify(tokens, parent, count, p, q, u_accept, u_sample, dims.B, dims.N,
                                   dims.V, path, path_len, out_tokens, err,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

strata_status_t strata_kv_commit(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                 const int32_t* path, const int32_t* path_len, int32_t* pos_out,
                                 strata_stream_t stream) {
  const strata_status_t st = check_both(cache, seqs);
  if (st != STRATA_OK) return st;
  if (seqs.N > STRATA_TREE_MAX_NODES || seqs.B > 65535) return STRATA_ERR_UNSUPPORTED;
  if (seqs.B == 0) return STRATA_OK;
  if (!ok_ptr(path) || !ok_ptr(path_len) || !ok_ptr(pos_out)) return STRATA_ERR_INVALID_ARG;
  unsigned* err = check_word();
  if (!err) return STRATA_ERR_CUDA;
  return cuda_status(launch_kv_commit(cache, seqs, path, path_len, pos_out, err,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
