/*
 * strata_kv.h -- C ABI of one speculative-decoding step over an 8-bit paged
 * KV cache on B200 (sm_100a), beside the expert layer of strata_moe.h.
 *
 * The expert layer runs verify batches (the last accepted token and a few
 * drafted ones); these entry points run what stands around it in such a step:
 *
 *   strata_kv_append        quantise the new tokens' K and V into the cache
 *   strata_tree_attention   attention of every node of the draft tree over the
 *                           committed positions and the node's ancestors
 *   strata_verify_drafts    which drafts the target accepts, and the next token
 *   strata_kv_commit        the accepted path's rows moved to their positions
 *   strata_kv_read          a range of positions read back as bf16
 *
 * The conventions of strata_moe.h hold here too: device pointers owned by the
 * caller and 16-byte aligned, work enqueued on `stream`, no host
 * synchronisation and no allocation (every call can be captured in a CUDA
 * graph), arguments validated on the host before any launch, results
 * bit-identical from run to run, indices found out of range on the device
 * reported through strata_moe_device_status().  Nothing is kept between calls:
 * calls on different streams may overlap as long as their outputs and their
 * workspaces do not.
 */
#ifndef STRATA_KV_H
#define STRATA_KV_H

#include "strata_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most nodes of a draft tree (strata_tree_attention, strata_verify_drafts,
 * strata_kv_commit). */
#define STRATA_TREE_MAX_NODES 64

/* The cache: a pool of pages of `page` positions each, shared by all
 * sequences.
 *   pages    pages in the pool                page   16, 32, 64 or 128
 *   Hkv      KV heads                         D      head size, 64 or 128
 *   k, v     [pages][Hkv][page][D] e4m3 codes (no infinities, 0x7F and 0xFF
 *            are NaN)
 *   k_exp, v_exp [pages][Hkv][page] exponents, biased by 127
 * A row (one position of one head, K or V) stands for the values
 * code * 2^(exp - 127); strata_kv_append writes exponents of 1 .. 246.  A row whose
 * exponent byte is 0 holds nothing: attention passes over it (over V alone when K is
 * held: the position keeps its weight), strata_kv_read gives zeros for it.  A byte of
 * 255 is not to be used.
 * pages * Hkv * page < 2^31. */
typedef struct {
  int32_t pages, page, Hkv, D;
  uint8_t *k, *v, *k_exp, *v_exp;
} strata_kv_cache_t;

/* Which positions of which sequences a call deals with: tokens pos[b] ..
 * pos[b] + count[b] - 1 of sequence b.
 *   B        sequences (B = 0: nothing runs)
 *   N        token slots per sequence in the call's tensors
 *   max_pages columns of the page table
 *   table    [B][max_pages]: position t of sequence b lies in page
 *            table[b][t / page], at t % page
 *   pos      [B] position of the sequence's first token of this call (for the
 *            attention: the committed length)
 *   count    [B] tokens in this call, 0 .. N; NULL = N for every sequence.
 *            Rows of the slots behind a sequence's count are neither read nor
 *            written.
 * B * N < 2^24, B * N * Hkv < 2^29, max_pages * page < 2^31.  Reported through
 * strata_moe_device_status(): a page outside [0, pages) and a position behind
 * max_pages * page (no row is read or written there; attention passes over
 * it), a negative pos and a count outside 0 .. N (the sequence counts as having
 * no tokens).  Pages written by one call must be distinct. */
typedef struct {
  int32_t B, N, max_pages;
  const int32_t *table, *pos, *count;
} strata_kv_seqs_t;

/* Writes the tokens' K and V into the cache, quantised row by row: the
 * exponent is the smallest e in [-126, 119] with max|x| <= 448 * 2^e over the
 * row's finite values, each code the e4m3 nearest to x / 2^e (ties to even,
 * magnitudes above 448 to 448).  The scale is a power of two so that x / 2^e
 * is exact and the code the only rounding.  Infinities and NaN become NaN
 * codes and leave the row's other values alone.
 *   k, v     token i of sequence b at (b * N + i) * stride: its Hkv * D bf16
 *            values, [Hkv][D]
 *   stride   elements from one token to the next: Hkv * D or more, a multiple
 *            of 8 (parts of a fused projection's rows can be passed as they
 *            are); 0 = Hkv * D */
STRATA_API strata_status_t strata_kv_append(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                 const uint16_t* k, const uint16_t* v, int64_t stride,
                                 strata_stream_t stream);

/* Reads positions back as bf16 (codes times the power of two, rounded to
 * nearest even where bf16's exponent range cuts them).
 *   k_out, v_out [B][N][Hkv][D] bf16; either may be NULL.  Positions without a
 *   valid page give zeros. */
STRATA_API strata_status_t strata_kv_read(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                               uint16_t* k_out, uint16_t* v_out, strata_stream_t stream);

/* Attention of the nodes of a draft tree (1 <= N <= STRATA_TREE_MAX_NODES
 * nodes per sequence) over the cache.  Node i of sequence b lies at position
 * pos[b] + i, its K and V already appended; it sees the positions below pos[b],
 * its ancestors and itself:
 *   o[b][i][h] = sum_t softmax_t(scale * q[b][i][h] . K[t][h / (Hq / Hkv)])
 *                V[t][h / (Hq / Hkv)]
 *   parent   [B][N] int32: the node above node i, below i, or -1 for none; NULL
 *            = i - 1 (a chain of drafts; N = 1 is plain decoding).  Another value
 *            is reported and counts as -1.
 *   q        node i of sequence b at (b * N + i) * q_stride: [Hq][D] bf16
 *   q_stride elements, Hq * D or more, a multiple of 8; 0 = Hq * D
 *   Hq       query heads, Hq % Hkv == 0, Hq / Hkv <= 64, B * N * Hq < 2^30, and
 *            B * Hkv * ceil(N * Hq / Hkv / 16) * (max_pages * page / 256 + 4)
 *            < 2^31
 *   scale    <= 0 means 1 / sqrt(D)
 *   out      [B][N][Hq][D] bf16; rows of slots behind count[b] are left as they
 *            were; a node that sees no row gets zeros; may be q itself
 *            (q_stride = Hq * D)
 * Values at positions a node does not see, NaN among them, do not reach it.
 * The sums over the positions hold 448 times the weights and V: with |V| up to
 * 2^87 they stay finite at any length, up to 2^103 at 32,768 positions.
 * Scores, softmax and sums in fp32 (values of q below 2^-13.8 of their row's largest
 * are rounded to 2^-21.8 of it, all others taken as they are); for the product with
 * V what a position adds to a row (its weight times 2^(v_exp - 127)) is rounded to
 * 2^-9 of its value, or to 2^-17.8 of the row's largest in the same tile of 256
 * positions where that is more: a large V without weight takes nothing from the
 * others.
 *   ws       scratch of strata_tree_attention_workspace_bytes() bytes, which
 *            reads the sizes of `cache` and `seqs` only (0 = refused) */
STRATA_API size_t strata_tree_attention_workspace_bytes(strata_kv_cache_t cache,
                                             strata_kv_seqs_t seqs, int32_t Hq);
STRATA_API strata_status_t strata_tree_attention(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                      const int32_t* parent, const uint16_t* q,
                                      int64_t q_stride, int32_t Hq, float scale, uint16_t* out,
                                      void* ws, size_t ws_bytes, strata_stream_t stream);

/* Verification of drafted tokens by rejection sampling, from given random
 * numbers: the tokens that come out are distributed as if drawn from the
 * target one by one.
 *   B sequences, N nodes (1 .. STRATA_TREE_MAX_NODES), V tokens in the vocabulary;
 *   B * N < 2^24, V <= STRATA_VERIFY_MAX_VOCAB (a sequence's sums of four
 *   probabilities stay in shared memory) */
#define STRATA_VERIFY_MAX_VOCAB 800000
typedef struct {
  int32_t B, N, V;
} strata_verify_dims_t;

/* Node 0 is the sequence's last token, nodes 1 .. count[b] - 1 are drafts.
 *   tokens   [B][N] int32 (tokens[b][0] is not used)
 *   parent   [B][N] int32 or NULL (chain), as for strata_tree_attention
 *   count    [B] int32 or NULL (N); a sequence of 0 nodes gets path_len 0
 *   p        [B][N][V] fp32: the target's probabilities after node i
 *   q        [B][N][V] fp32: the draft's probabilities after node i, which the
 *            children of node i were drawn from; NULL = the drafter put all
 *            its weight on the drafted token (greedy drafts)
 *   u_accept [B][N] fp32 in [0, 1): for the test of node i
 *   u_sample [B] fp32 in [0, 1): for the next token
 * From node 0 down, the children of the current node are tried in ascending
 * order.  With r = p of the current node, c = 0, S = 1 at first, child i with
 * token x is accepted and becomes the current node when
 *   u_accept[i] * q(x) * S < r(x);
 * otherwise c grows by S, r = max(p - c q, 0) and S = sum r (q = NULL: q(x) = 1 in
 * the test, and r is p without the tokens rejected at this node).  This is the
 * repeated "accept, else sample from the normalised positive part of p - q" with
 * the normalisations carried in c.  Below the last accepted node the next token
 * is the lowest index at which the running sum of r exceeds u_sample * sum r (the
 * last index with r > 0 should none; 0 and a report when r has no positive
 * value).  All of it in 64 bits.  A token outside [0, V) is reported and
 * rejected without changing r.
 *   path     [B][N] int32 out: the accepted nodes from node 0, then -1
 *   path_len [B] int32 out: their number, 1 + accepted drafts
 *   out_tokens [B][N] int32 out: the path_len new tokens (accepted drafts, then
 *            the next token), then -1 */
STRATA_API strata_status_t strata_verify_drafts(const int32_t* tokens, const int32_t* parent,
                                     const int32_t* count, const float* p, const float* q,
                                     const float* u_accept, const float* u_sample,
                                     strata_verify_dims_t dims, int32_t* path,
                                     int32_t* path_len, int32_t* out_tokens,
                                     strata_stream_t stream);

/* Keeps the accepted path: the rows at pos[b] + path[b][i] move to pos[b] + i
 * for i < path_len[b], all of them as they were before the call.
 *   path     [B][N] int32 (N <= STRATA_TREE_MAX_NODES), as strata_verify_drafts
 *            writes it; an entry outside [i, N) is reported and its row not moved
 *            (pos_out counts it all the same: what position pos[b] + i held stays)
 *   path_len [B] int32; outside 0 .. N is reported and counts as 0
 *   pos_out  [B] int32 out: pos[b] + path_len[b]; may be pos itself
 * seqs.count is not used; B <= 65535. */
STRATA_API strata_status_t strata_kv_commit(strata_kv_cache_t cache, strata_kv_seqs_t seqs,
                                 const int32_t* path, const int32_t* path_len,
                                 int32_t* pos_out, strata_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* STRATA_KV_H */
