// tree_attn.cu -- attention of the nodes of a draft tree over the 8-bit paged
// KV cache.
//
// Per sequence b and KV head: the rows are the (node, query head) pairs that
// share the head, N * Hq / Hkv of them, and every row attends over the same
// positions, so each K and V byte is read once for all rows.  With few
// rows the bytes of the cache are the bound (258 bytes per position and head
// at D = 128), with many rows the products are.
//
// The products run on the e4m3 codes as they lie in the cache (tcgen05
// kind::f8f6f4), transposed, so that the 128 rows of the instruction are
// positions (scores) or features (output) and the query rows are its
// narrow side:
//   S^T [128 positions][2R] = K tile [128][D] . [q_hi ; q_lo]^T
//   O^T [D][2R]             = V tile^T [D][128] . [P_hi | P_lo]
// A bf16 q (8 significant bits) times a power of two is the sum of two e4m3
// values (4 bits each), so the scores are sums of exact products.  The high part
// leaves 16 of 448 at most, so the low part is held times 16: together they are
// exact for values of q above 2^-13.8 of the row's largest and off by 2^-21.8 of
// that at most below (2^-9.8 and 2^-17.8 with both parts on one scale).  The weights are
// split the same way: p (fp32) is rounded to fp16 (2^-11), to e4m3, and
// the remainder to e4m3 again, 2^-9 of the value in all.  Against one bf16
// rounding of p (2^-8) that is half the error, and the tensor pipe never
// waits for codes to be widened.  High and low parts are separate columns
// of one product (the K or V tile is read from shared memory once) and are
// added in fp32 registers.
//
// A position's K exponent multiplies its scores, one factor per thread,
// because a thread is a position there.  Its V exponent goes into the weight,
//   P = 2^(s + ev - r) * 448,   r = ceil(max (s + ev)) over what the row sees,
// and the tile's O is added to the running sum as O * 2^r.  e4m3 reaches only
// 2^-9 (2^-17.8 of the tile's largest weight), so what is scaled to that range is what
// a position adds to the output, score and V scale together, per row and tile: a
// large V that a row gives no weight to, or that another node sees, takes nothing
// from the others, and positions of a tile far below an earlier tile's maximum keep
// their precision.  ev enters with the multiplication by the K factor, so the weight
// is one exponential and the softmax's sum takes it times 2^(largest ev - ev), a factor
// per position.  Where a tile's exponents lie too far apart for that, e.g. beside a V
// row of zeros, the sum has a reference and exponentials of its own (a third barrier).
// References are integers (log2 domain), so rescaling is an exponent addition.
//
// Work: the tiles (256 positions) of all (sequence, KV head, block of R rows)
// units in one line, cut into equal runs, one per CTA, whatever the lengths are.
// A unit that lies in one run is finished there; the others leave partial sums
// that tree_attn_combine_kernel joins in run order (no atomics, so results do
// not depend on the order in which CTAs run).
//
// Roles per CTA: a warp that follows the run, announces its units and issues
// the TMA copies of pages (K, V, exponents, query rows) into rings of tiles, a
// warp that issues the MMAs, and one warpgroup per 16 row columns for the
// softmax, the weights and the running sums.  K and V places come free at
// different times (after the scores, after the output), so they are separate
// rings; the next tile's scores are issued as soon as these have left TMEM.
//
// R, the rows per block, is 16 when all rows of N nodes fit and 32 otherwise,
// with two CTAs per SM (their TMEM and registers).  Blocks of 64 rows (one CTA per
// SM) were 5 % faster on 64-node trees of 4 sequences and 10 to 20 % slower on 8-node
// and on few trees; blocks of 16 for all rows 36 % slower on 24-node trees.
//
// Measured (D = 128, 4 KV heads, 32 query heads, one call): 32 sequences of 4 nodes
// behind up to 34,000 positions 105 us in a graph at burst clocks, 5.5 TB/s of the
// cache's bytes (0.84 of the copy rate; with one node 98 us), 125 us called without a
// pause (4.7 TB/s, 0.71: the clock falls to 1.66 GHz); one sequence behind 34,000
// 21 us; one token behind 300 positions 10 us, of which 2 us are the launch, 6 us the
// first tile's chain of dependent steps (lengths -> page -> copy -> scores) and 2 us
// the join.  In a long line a tile takes a CTA 3.3 us, with two CTAs per SM near what
// its 66 KB take at the copy rate; D = 64 halves the bytes but not the arithmetic
// (97 us): 25 to 27 instructions a weight, issued in about half of the cycles, the
// softmax warps waiting for tensor memory and for each other the rest.  Steps that did not
// help: the last fifth of the line in small runs taken from a counter (141 us
// against 126: a run costs two tiles), one barrier per tile with every warp
// working out the references (112 against 108), 8 columns per warpgroup.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "kv.h"
#include "tree_parts.h"

namespace strata {

namespace ta {
constexpr int SUB = 128;                    // positions per MMA tile
constexpr int TILE = 2 * SUB;               // positions per softmax step
constexpr int NODES = STRATA_TREE_MAX_NODES;
constexpr float LOG2_WSCALE = 8.807354922f; // weights are scaled to e4m3's largest value, 448
constexpr float QLO = 16.f;                 // the low parts of q are held times this
// V exponents of a tile that lie no further apart: the scores need no reference of
// their own (the sums then hold up to 2^SPREAD times the weights).
constexpr int SPREAD = 30;
// What a unit costs besides its tiles (its query rows, the tree's masks, its
// results), in tiles: units take that much more of the line.  On short lines
// the number of tiles per CTA counts, not their even cost.  With a cost of 0, 1, 2
// and 3: 8 tiles 10.2, 12.5, 11.4, 12.5 us; 8 nodes of 12 short sequences (0.8 tiles
// per CTA) 14.7, 16.4, 17.5, 18.4; 4 nodes behind 34,000 (1.8 per CTA) 24.1, 21.4, 21.3,
// 21.3; 24 sequences to 3,000 (2 per CTA) 25.3, 22.9, 22.1, 23.3, but 9 of them (just
// above 1) 16.5 with 1 and 17.1 with 2; 24-node trees of 16 (10 per CTA) 52.5, 46.5, 45.7,
// 46.3; 32 sequences to 34,000 (30 per CTA) 116.9, 111.8, 109.9, 108.0.
__host__ __device__ constexpr uint32_t unit_cost(uint32_t tiles, uint32_t ctas) {
  return tiles >= 16 * ctas ? 3 : tiles >= 4 * ctas ? 2 : tiles > ctas ? 1 : 0;
}
constexpr int UNITS = 4;                    // units announced ahead
constexpr int C = 16;                       // row columns per softmax warpgroup
constexpr int CTAS = 2;                     // per SM

template <int D, int R>
struct Cfg {
  static constexpr int NWG = R / C;                    // softmax warpgroups
  // K and V rings, in MMA tiles
  static constexpr int KS = D == 64 ? 4 : 2;
  static constexpr int VS = D == 64 ? 4 : 2;
  static constexpr int ES = 4;                         // exponents, in softmax tiles
  static_assert(ES >= KS / 2 + 2, "see load_e");
  static constexpr int SOFT = NWG * 128;
  static constexpr int THREADS = SOFT + 64;
  static constexpr int KV_BYTES = SUB * D;             // one operand tile
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + KS * KV_BYTES;
  static constexpr int Q_OFF = V_OFF + VS * KV_BYTES;          // [2R][D] codes
  static constexpr int QR_OFF = Q_OFF + 2 * R * D;             // [R][D] bf16, as they come
  static constexpr int P_OFF = QR_OFF + 2 * R * D;             // [TILE][2R] codes
  static constexpr int E_OFF = P_OFF + TILE * 2 * R;           // [ES][K, V][TILE] exponents
  static constexpr int MISC_OFF = E_OFF + ES * 2 * TILE;
  static constexpr int O_COL = 4 * R;                  // TMEM: the scores, then O
  static constexpr int TMEM_COLS = R == 32 ? 256 : 128;
};

// One unit as a run sees it: tiles first .. stop - 1 of (sequence, KV head,
// block of rows).
struct Unit {
  int b, hk, rb, pos, count, tiles, first, stop;
  unsigned end;              // positions with a column in the page table
  int run, follow;           // the run, and how many runs after it go on with the unit
  int last;                  // no unit: the CTA is done
};

template <class F, int R>
struct Misc {
  uint64_t k_full[F::KS], k_empty[F::KS], v_full[F::VS], v_empty[F::VS], e_full[F::ES];
  uint64_t s_full, s_free, p_ready, o_full, q_full, qr_full, qr_empty;
  uint64_t u_full[UNITS], u_empty[UNITS];
  uint32_t seen_by[NODES];           // rows that see the node
  unsigned long long nan_nodes;      // nodes whose V holds a NaN
  Unit unit[UNITS];
  uint32_t tmem;
  int abort;
  unsigned long long sees[UNITS][R]; // nodes that a row sees
  int row[UNITS][R];                 // a row's node and query head: node * Hq + head
  int row_node[UNITS][R];
  uint2 scan[F::THREADS / 32];
  uint32_t start_off;
  int start_b;
  int nan_row[R];
  alignas(16) float qf[R];                    // score factor of the row
  // per warp: largest score plus V exponent of the tile; largest score
  alignas(16) float wmax[F::NWG][4][C], wscore[F::NWG][4][C];
  uint2 wexp[F::NWG][4];      // per warp: largest V exponent that a row sees; 255 - the smallest
  alignas(16) float mref[F::NWG][C], beta[F::NWG][C], alpha[F::NWG][C];
  alignas(16) float beta_o[F::NWG][2][C];
  alignas(16) float sref[F::NWG][C];          // mref of the scores, where they have their own
  alignas(16) float lsum[F::NWG][4][C];       // per warp: sums of the weights
  alignas(16) float inv[R];                   // 1 / sum
};

__host__ __device__ constexpr size_t slot_floats(int R, int D) { return (size_t)R * (D + 2); }
}  // namespace ta

struct TreeArgs {
  strata_kv_cache_t c;
  strata_kv_seqs_t s;
  const int32_t* parent;
  const uint16_t* q;
  int64_t q_stride;
  int Hq, G;              // query heads, query heads per KV head
  int blocks;             // blocks of R rows per sequence and KV head when it has N nodes
  float scale;            // times log2(e)
  uint16_t* out;
  ta::Head* heads;
  float* parts;
  unsigned* err;
};

// One sequence's extent in this call.
struct TreeSeq {
  int pos, count, tiles, blocks;
  unsigned end;           // positions with a column in the page table
  __device__ __forceinline__ uint32_t units(const TreeArgs& a) const {
    return tiles ? (uint32_t)(blocks * a.c.Hkv) : 0u;
  }
};

template <int R>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  TreeSeq t;
  bool bad;
  const SeqRange r = seq_range(a.s, b, &bad);
  t.pos = r.pos;
  t.count = r.count;
  const unsigned room = (unsigned)a.s.max_pages * (unsigned)a.c.page;
  t.end = (unsigned)r.pos + (unsigned)r.count;
  if (t.end > room) {
    bad = r.count > 0;
    t.end = room;
  }
  t.tiles = r.count > 0 ? (int)((t.end + ta::TILE - 1) / ta::TILE) : 0;
  t.blocks = (r.count * a.G + R - 1) / R;
  if (bad && report) atomicOr(a.err, kErrIndex);
  return t;
}

// The line of all units' tiles, each unit with its cost in front, and how it is
// cut into runs, one per CTA.
struct Line {
  uint32_t cost, total, runs, q, rem;
  __device__ __forceinline__ Line(uint32_t tiles, uint32_t units, uint32_t ctas) {
    cost = ta::unit_cost(tiles, ctas);
    total = tiles + cost * units;
    runs = min(tiles, ctas);
    q = runs ? total / runs : 0;
    rem = total - q * runs;
  }
  __device__ __forceinline__ uint32_t start(uint32_t r) const { return r * q + min(r, rem); }
  __device__ __forceinline__ uint32_t run_of(uint32_t w) const {
    return w < rem * (q + 1) ? w / (q + 1) : rem + (w - rem * (q + 1)) / q;
  }
};

// The units of a run in order.  A unit takes cost + tiles places of the
// line; a run that holds only its first places leaves all its tiles to
// the next run.
template <int R>
struct Cursor {
  TreeSeq t;
  int b, hk, rb;
  int cost;
  uint32_t off;           // place in the unit
  uint32_t at, left;      // place in the line; places left in the run
  __device__ __forceinline__ void start(const TreeArgs& a, const Line& line, int b0, uint32_t o,
                                        uint32_t w, uint32_t n) {
    b = b0;
    cost = (int)line.cost;
    at = w;
    left = n;
    t = tree_seq<R>(a, b, false);
    const uint32_t len = t.tiles + cost, u = o / len;
    off = o - u * len;
    hk = (int)(u / t.blocks);
    rb = (int)u - hk * t.blocks;
  }
  __device__ __forceinline__ void advance(const TreeArgs& a) {
    off = 0;
    if (++rb < t.blocks) return;
    rb = 0;
    if (++hk < a.c.Hkv) return;
    hk = 0;
    do {
      ++b;
      t = tree_seq<R>(a, b, false);
    } while (t.tiles == 0);
  }
  // The next unit with tiles in run `run`; false when there is none.
  __device__ __forceinline__ bool next(const TreeArgs& a, const Line& line, int run, ta::Unit* u) {
    while (left > 0) {
      const uint32_t len = t.tiles + cost;
      const uint32_t upto = min(len, off + left);
      const int first = max(0, (int)off - cost);
      const int stop = max(0, (int)upto - cost);
      u->b = b;
      u->hk = hk;
      u->rb = rb;
      u->pos = t.pos;
      u->count = t.count;
      u->tiles = t.tiles;
      u->first = first;
      u->stop = stop;
      u->end = t.end;
      u->run = run;
      u->follow = upto == len ? 0 : (int)line.run_of(at + (len - off) - 1) - run;
      u->last = 0;
      at += upto - off;
      left -= upto - off;
      if (left > 0)
        advance(a);
      else
        off = upto;
      if (stop > first) return true;
    }
    return false;
  }
};

// 32 lanes x 16 consecutive columns from either address, waited for.
__device__ __forceinline__ void tmem_load2(uint32_t at0, uint32_t at1, uint32_t (&x)[16],
                                           uint32_t (&y)[16]) {
  tmem_ld_32x32b_x16(at0, x);
  tmem_ld_32x32b_x16(at1, y);
  tmem_ld_wait_regs(x);
  tmem_ld_wait_regs(y);
}

// mbar_wait_warp with its slow path out of line: the waits are many and the
// code between them runs from the instruction cache.
__device__ __noinline__ bool ta_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          unsigned* err) {
  return mbar_wait_warp(bar, parity, abort, err);
}
__device__ __forceinline__ bool ta_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        unsigned* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity))) return true;
  return ta_wait_slow(bar, parity, abort, err);
}

// Pairs of fp32 values, one instruction for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(uint32_t x, uint32_t y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ f32x2 pair(float x, float y) {
  return pair(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ void unpair(f32x2 v, float& x, float& y) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  x = __uint_as_float(a);
  y = __uint_as_float(b);
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float ta_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for integers e (0 below the normal range, no value above it arises)
__device__ __forceinline__ float pow2i(int e) {
  return e < -126 ? 0.f : __uint_as_float((uint32_t)(min(e, 127) + 127) << 23);
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t sbo, uint64_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(sbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1u << 46) | (swizzle << 61);
}
// Swizzle mode for rows of `bytes` bytes, and the same permutation of 16-byte
// chunks for stores.
__host__ __device__ constexpr uint64_t sw_mode(int bytes) {
  return bytes == 128 ? 2 : bytes == 64 ? 4 : 6;
}
template <int BYTES>
__device__ __forceinline__ uint32_t sw_off(uint32_t row, uint32_t byte) {
  const uint32_t off = row * BYTES + byte;
  return BYTES == 128 ? off ^ ((row & 7) << 4)
         : BYTES == 64 ? off ^ (((row >> 1) & 3) << 4)
                       : off ^ (((row >> 2) & 1) << 4);
}

__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// e4m3 operands, fp32 sums; majors: 0 = K, 1 = M or N
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Four weights to e4m3 pairs: the values rounded to fp16, their codes (hi),
// and the codes of what those leave (lo).
__device__ __forceinline__ void split4(uint32_t h01, uint32_t h23, uint32_t* hi, uint32_t* lo) {
  const uint32_t h[2] = {h01, h23};
  *hi = *lo = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    __half2_raw x;
    x.x = (unsigned short)(h[i] & 0xFFFFu);
    x.y = (unsigned short)(h[i] >> 16);
    const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const __half2 left = __hsub2(__half2(x), __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    const __nv_fp8x2_storage_t r =
        __nv_cvt_halfraw2_to_fp8x2(__half2_raw(left), __NV_SATFINITE, __NV_E4M3);
    *hi |= (uint32_t)c << (16 * i);
    *lo |= (uint32_t)r << (16 * i);
  }
}

// The nodes that `node` sees (itself and those above it, as bits), per lane, from
// the parents of nodes lane and lane + 32 (-1: none; below the node itself): every
// round doubles the number of generations a node knows of.  Followed one by one,
// the parents of a chain of 64 nodes cost 3.2 of 18.7 us.
__device__ __forceinline__ unsigned long long row_sees(int (&up)[2], int node, int lane) {
  const uint32_t all = 0xffffffffu;
  uint32_t low = 1u << lane, low2 = 0, high2 = 1u << lane;     // of nodes lane, lane + 32
#pragma unroll 1
  while (__any_sync(all, up[0] >= 0 || up[1] >= 0)) {
    const uint32_t m0 = __shfl_sync(all, low, up[0]), m1 = __shfl_sync(all, low, up[1]);
    const uint32_t n1 = __shfl_sync(all, low2, up[1]), h1 = __shfl_sync(all, high2, up[1]);
    const int u0 = __shfl_sync(all, up[0], up[0]), u1 = __shfl_sync(all, up[0], up[1]);
    const int v1 = __shfl_sync(all, up[1], up[1]);
    if (up[0] >= 0) {
      low |= m0;
      up[0] = u0;
    }
    if (up[1] >= 32) {
      low2 |= n1;
      high2 |= h1;
      up[1] = v1;
    } else if (up[1] >= 0) {
      low2 |= m1;
      up[1] = u1;
    }
  }
  const uint32_t a = __shfl_sync(all, low, node), b = __shfl_sync(all, low2, node),
                 c = __shfl_sync(all, high2, node);
  return node < 32 ? a : node < 64 ? (unsigned long long)c << 32 | b : 0ull;
}

// Waits (with a limit) for the copies in flight into a ring of N stages, of
// which `n` uses were armed: shared memory must outlive them.
template <int N>
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t n) {
  for (uint32_t i = n > (uint32_t)N ? n - N : 0; i < n; ++i) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(smem_addr(&full[i % N]), (i / N) & 1) &&
           global_ns() - t0 < kWaitLimitNs) {
    }
  }
}

template <int D, int R>
__global__ void __launch_bounds__(ta::Cfg<D, R>::THREADS, ta::CTAS)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const TreeArgs a) {
  using namespace ta;
  using F = Cfg<D, R>;
  constexpr int NWG = F::NWG, KS = F::KS, VS = F::VS, ES = F::ES;
  using M = Misc<F, R>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem + F::K_OFF;
  uint8_t* sV = smem + F::V_OFF;
  uint8_t* sQ = smem + F::Q_OFF;
  uint8_t* sP = smem + F::P_OFF;
  uint8_t* sE = smem + F::E_OFF;
  M& m = *reinterpret_cast<M*>(smem + F::MISC_OFF);
  volatile int* abort_flag = &m.abort;
  const int th = threadIdx.x, warp = th / 32, lane = th % 32;
  constexpr int W_TMA = NWG * 4, W_MMA = NWG * 4 + 1;
  const bool reporter = blockIdx.x == 0;

  if (th == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&m.k_full[i], 1);
      mbar_init(&m.k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&m.v_full[i], 1);
      mbar_init(&m.v_empty[i], 1);
    }
    for (int i = 0; i < ES; ++i) mbar_init(&m.e_full[i], 1);
    mbar_init(&m.s_full, 1);
    mbar_init(&m.s_free, F::SOFT);
    mbar_init(&m.qr_full, 1);
    mbar_init(&m.qr_empty, 1);
    mbar_init(&m.p_ready, F::SOFT);
    mbar_init(&m.o_full, 1);
    mbar_init(&m.q_full, F::SOFT);
    for (int i = 0; i < UNITS; ++i) {
      mbar_init(&m.u_full[i], 1);
      mbar_init(&m.u_empty[i], 2);       // the MMA warp and the softmax
    }
    m.abort = 0;
    fence_mbar_init();
  }
  if (warp == W_TMA && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == W_MMA) tmem_alloc(&m.tmem, F::TMEM_COLS);
  stream_order_begin();

  // ---- the line: sequences in contiguous shares per thread, their lengths
  // scanned over the CTA
  const int per = (a.s.B + F::THREADS - 1) / F::THREADS;
  const int sb0 = min(th * per, a.s.B), sb1 = min(sb0 + per, a.s.B);
  uint2 mine = {0, 0};                 // tiles, units
  for (int b = sb0; b < sb1; ++b) {
    const TreeSeq t = tree_seq<R>(a, b, reporter);
    const uint32_t n = t.units(a);
    mine.x += n * t.tiles;
    mine.y += n;
  }
  uint2 incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, off);
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl.y, off);
    if (lane >= off) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) m.scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint2 below = {incl.x - mine.x, incl.y - mine.y}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < F::THREADS / 32; ++w) {
    const uint2 n = m.scan[w];
    if (w < warp) {
      below.x += n.x;
      below.y += n.y;
    }
    all.x += n.x;
    all.y += n.y;
  }
  const Line line(all.x, all.y, gridDim.x);
  const int cta = blockIdx.x;
  const bool active = cta < (int)line.runs;
  const uint32_t w0 = active ? line.start(cta) : 0;
  const uint32_t before = below.x + line.cost * below.y;
  if (active && w0 >= before && w0 < before + mine.x + line.cost * mine.y) {
    uint32_t at = before;
    for (int b = sb0; b < sb1; ++b) {
      const TreeSeq t = tree_seq<R>(a, b, false);
      const uint32_t n = t.units(a) * (t.tiles + line.cost);
      if (w0 < at + n) {
        m.start_b = b;
        m.start_off = w0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const uint32_t tmem = m.tmem;
  if (!active) {
    // more runs than work
  } else if (warp == W_TMA) {
    // ------------------------------------------------ units and page copies
    // In the order in which the places come free: exponents and K of a tile,
    // then V of the tile before it.
    Cursor<R> cu;
    cu.start(a, line, m.start_b, m.start_off, w0, line.start(cta + 1) - w0);
    uint32_t jk = 0, jv = 0, g = 0, un = 0, nq = 0;
    int64_t row[2] = {-1, -1};         // of the tile, per MMA tile: this lane's page
    bool dead = false;
    const int page = a.c.page, page_bits = 31 - __clz(page);
    auto load_k = [&]() -> bool {
#pragma unroll
      for (int h = 0; h < 2; ++h, ++jk) {
        const int ks = jk % KS;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, row[h] >= 0));
        if (jk >= (uint32_t)KS &&
            !ta_wait(&m.k_empty[ks], (jk / KS - 1) & 1, abort_flag, a.err))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&m.k_full[ks], n * page * D);
        __syncwarp();
        if (row[h] >= 0)
          tma_load_2d(sK + ks * F::KV_BYTES + lane * page * D, &map_k, 0, (int)row[h],
                      &m.k_full[ks]);
      }
      return true;
    };
    auto load_v = [&]() -> bool {
#pragma unroll
      for (int h = 0; h < 2; ++h, ++jv) {
        const int vs = jv % VS;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, row[h] >= 0));
        if (jv >= (uint32_t)VS &&
            !ta_wait(&m.v_empty[vs], (jv / VS - 1) & 1, abort_flag, a.err))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&m.v_full[vs], n * page * D);
        __syncwarp();
        if (row[h] >= 0)
          tma_load_2d(sV + vs * F::KV_BYTES + lane * page * D, &map_v, 0, (int)row[h],
                      &m.v_full[vs]);
      }
      return true;
    };
    // The slot's last tile is done with: this warp has waited until the K tile
    // KS / 2 tiles back was read, which comes after the weights KS / 2 + 2 tiles
    // back were finished (ES >= KS / 2 + 2).
    auto load_e = [&]() {
      const int es = g % ES;
      uint8_t* e = sE + es * 2 * TILE + lane * page;
      uint32_t n = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        n += __popc(__ballot_sync(0xffffffffu, row[h] >= 0));
        if (lane * page < SUB && row[h] < 0) {         // no page: nothing held there
          for (int i = 0; i < page; i += 16)
            *reinterpret_cast<uint4*>(e + h * SUB + i) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();                    // before a later copy to the same place
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&m.e_full[es], n * page * 2);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (row[h] >= 0) {
          bulk_load(e + h * SUB, a.c.k_exp + row[h], page, &m.e_full[es]);
          bulk_load(e + TILE + h * SUB, a.c.v_exp + row[h], page, &m.e_full[es]);
        }
      ++g;
    };
    // Tells the other warps of unit u (or that there is none left): its rows, the
    // nodes' parents when the run reaches the tree, the rows' values.
    auto announce = [&](const Unit& u, bool some) -> bool {
      const int us = un % UNITS;
      if (un >= (uint32_t)UNITS &&
          !ta_wait(&m.u_empty[us], (un / UNITS - 1) & 1, abort_flag, a.err))
        return false;
      if (some) {
        const bool drafts = (unsigned)u.stop * TILE > (unsigned)u.pos;
        static_assert(NODES == 64, "two nodes per lane");
        const int flat = u.rb * R + lane;              // R <= 32: a row per lane
        int node = flat / a.G;
        const int head = u.hk * a.G + flat - node * a.G, row_q = node * a.Hq + head;
        if (lane < R) {
          m.row_node[us][lane] = node;
          m.row[us][lane] = row_q;
        } else {
          node = u.count;
        }
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, node < u.count));
        int up[NODES / 32];
#pragma unroll
        for (int j = 0; j < NODES / 32; ++j) {
          const int i = j * 32 + lane;
          up[j] = i < u.count ? i - 1 : -1;
          if (drafts && a.parent && i < u.count) up[j] = a.parent[(int64_t)u.b * a.s.N + i];
        }
        if (un > 0 && !ta_wait(&m.qr_empty, (un - 1) & 1, abort_flag, a.err)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&m.qr_full, n * D * 2);
        __syncwarp();
        ++nq;
        if (node < u.count)
          bulk_load(smem + F::QR_OFF + lane * D * 2,
                    a.q + ((int64_t)u.b * a.s.N + node) * a.q_stride + (int64_t)head * D, D * 2,
                    &m.qr_full);
        if (drafts) {
#pragma unroll
          for (int j = 0; j < NODES / 32; ++j) {
            const int i = j * 32 + lane;
            if (up[j] < -1 || up[j] >= i) {
              atomicOr(a.err, kErrIndex);
              up[j] = -1;
            }
          }
          const unsigned long long sees = row_sees(up, node, lane);
          if (lane < R) m.sees[us][lane] = sees;
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (some) m.unit[us] = u;
        m.unit[us].last = !some;
        mbar_arrive(&m.u_full[us]);
      }
      __syncwarp();
      ++un;
      return true;
    };
    Unit u;
    while (!dead && cu.next(a, line, cta, &u)) {
      for (int tile = u.first; tile < u.stop; ++tile) {
        // this lane's page of either MMA tile; its number is on the way while a
        // new unit is announced
        unsigned first[2];
        int pg[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          first[h] = (unsigned)tile * TILE + h * SUB + (unsigned)(lane * page);
          pg[h] = -1;
          if (lane * page < SUB && first[h] < u.end)
            pg[h] = a.s.table[(int64_t)u.b * a.s.max_pages + (first[h] >> page_bits)];
        }
        if (tile == u.first && !announce(u, true)) {
          dead = true;
          break;
        }
        int64_t now[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          now[h] = -1;
          if (lane * page < SUB && first[h] < u.end) {
            if ((unsigned)pg[h] < (unsigned)a.c.pages)
              now[h] = ((int64_t)pg[h] * a.c.Hkv + u.hk) * page;
            else
              atomicOr(a.err, kErrIndex);
          }
        }
        const int64_t was[2] = {row[0], row[1]};
        row[0] = now[0];
        row[1] = now[1];
        // the exponents' slot is free once the first K place is
        if (jk >= (uint32_t)KS &&
            !ta_wait(&m.k_empty[jk % KS], (jk / KS - 1) & 1, abort_flag, a.err)) {
          dead = true;
          break;
        }
        load_e();
        if (!load_k()) {
          dead = true;
          break;
        }
        if (g > 1) {
          row[0] = was[0];
          row[1] = was[1];
          if (!load_v()) {
            dead = true;
            break;
          }
          row[0] = now[0];
          row[1] = now[1];
        }
      }
    }
    if (!dead) dead = !announce(Unit(), false);
    if (!dead && g > 0) dead = !load_v();
    if (dead) {
      drain_ring<KS>(m.k_full, jk);
      drain_ring<VS>(m.v_full, jv);
      drain_ring<ES>(m.e_full, g);
      drain_ring<1>(&m.qr_full, nq);
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------ MMA issue
    const bool leader = elect_one();
    constexpr uint32_t ID_S = idesc_e4m3(SUB, 2 * R, 0, 0);
    constexpr uint32_t ID_O = idesc_e4m3(D, 2 * R, 1, 1);
    uint32_t g = 0;                                        // tiles
    auto scores = [&](uint32_t i) -> bool {
      for (int h = 0; h < 2; ++h) {
        const uint32_t j = 2 * i + h;
        const int ks = j % KS;
        if (!ta_wait(&m.k_full[ks], (j / KS) & 1, abort_flag, a.err)) return false;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8_ss(tmem + h * 2 * R,
                      smem_desc(smem_addr(sK + ks * F::KV_BYTES) + 32 * k, 8 * D, sw_mode(D)),
                      smem_desc(smem_addr(sQ) + 32 * k, 8 * D, sw_mode(D)), ID_S, k > 0);
          mma_commit(&m.k_empty[ks]);
          if (h == 1) mma_commit(&m.s_full);
        }
        __syncwarp();
      }
      return true;
    };
    auto output = [&](uint32_t i) -> bool {
      for (int h = 0; h < 2; ++h) {
        const uint32_t j = 2 * i + h;
        const int vs = j % VS;
        if (!ta_wait(&m.v_full[vs], (j / VS) & 1, abort_flag, a.err)) return false;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < SUB / 32; ++k)
            mma_f8_ss(tmem + F::O_COL,
                      smem_desc(smem_addr(sV + vs * F::KV_BYTES) + 32 * k * D, 8 * D, sw_mode(D)),
                      smem_desc(smem_addr(sP) + (h * SUB + 32 * k) * 2 * R, 16 * R,
                                sw_mode(2 * R)),
                      ID_O, h > 0 || k > 0);
          mma_commit(&m.v_empty[vs]);
          if (h == 1) mma_commit(&m.o_full);
        }
        __syncwarp();
      }
      return true;
    };
    bool dead = false;
    for (uint32_t un = 0; !dead; ++un) {
      const int us = un % UNITS;
      if (!ta_wait(&m.u_full[us], (un / UNITS) & 1, abort_flag, a.err)) break;
      const int tiles = m.unit[us].stop - m.unit[us].first;
      const bool last = m.unit[us].last;
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.u_empty[us]);
      if (last) break;
      if (!ta_wait(&m.q_full, un & 1, abort_flag, a.err)) break;
      tc_fence_after();
      if (!scores(g)) break;
      for (int i = 0; i < tiles; ++i, ++g) {
        // the next scores as soon as these have left TMEM
        if (i + 1 < tiles) {
          if (!ta_wait(&m.s_free, g & 1, abort_flag, a.err)) {
            dead = true;
            break;
          }
          tc_fence_after();
          if (!scores(g + 1)) {
            dead = true;
            break;
          }
        }
        if (!ta_wait(&m.p_ready, g & 1, abort_flag, a.err)) {
          dead = true;
          break;
        }
        tc_fence_after();
        if (!output(g)) {
          dead = true;
          break;
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax
    const int wg = warp / 4, wq = warp % 4, lt = th % 128;   // lt: position in an MMA tile
    constexpr uint32_t ALL = F::SOFT;
    const uint32_t lanes_at = tmem + ((uint32_t)(wq * 32) << 16) + wg * C;
    const uint32_t bar_wg = 2 + wg;
    // the feature whose sums this thread keeps (D = 64: 16 lanes per warp)
    const int feat = D == 128 ? lt : wq * 16 + lane;
    const bool has_feat = D == 128 || lane < 16;
    f32x2 acc[C / 2], l[C / 2];
    uint32_t g = 0;
    bool ok = true, dead = false;

    // O of tile i (sum of its high and low columns) into acc
    auto add_o = [&](uint32_t i) {
      ok = ta_wait(&m.o_full, i & 1, abort_flag, a.err) && ok;
      tc_fence_after();
      const float* bo = m.beta_o[wg][i & 1];
      uint32_t hi[C], lo[C];
      tmem_load2(lanes_at + F::O_COL, lanes_at + F::O_COL + R, hi, lo);
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 b4 = *reinterpret_cast<const float4*>(bo + c);
        acc[c / 2] = fma2(add2(pair(hi[c], hi[c + 1]), pair(lo[c], lo[c + 1])), pair(b4.x, b4.y),
                          acc[c / 2]);
        acc[c / 2 + 1] = fma2(add2(pair(hi[c + 2], hi[c + 3]), pair(lo[c + 2], lo[c + 3])),
                              pair(b4.z, b4.w), acc[c / 2 + 1]);
      }
    };

    // The unit's results: rounded to the output when the run holds all of it,
    // its part otherwise.
    auto finish_unit = [&](const Unit& u, int us) {
      float o[C];
#pragma unroll
      for (int c = 0; c < C; c += 2) unpair(acc[c / 2], o[c], o[c + 1]);
      unsigned long long nan_nodes = (unsigned)u.stop * TILE > (unsigned)u.pos ? m.nan_nodes : 0;
      while (nan_nodes) {
        const int j = __ffsll((long long)nan_nodes) - 1;
        nan_nodes &= nan_nodes - 1;
        const int64_t row = row_of(a.c, a.s, u.b, (int64_t)u.pos + j) + (int64_t)u.hk * a.c.page;
        const bool nan = has_feat && (a.c.v[row * D + feat] & 0x7F) == 0x7F;
        const uint32_t by = m.seen_by[j] >> (wg * C);
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (nan && ((by >> c) & 1)) o[c] = __uint_as_float(0x7FC00000u);
      }
      if (!has_feat) return;
      if (u.first == 0 && u.stop == u.tiles) {
        uint16_t* out = a.out + (int64_t)u.b * a.s.N * a.Hq * D + feat;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (m.row_node[us][wg * C + c] < u.count)
            out[(int64_t)m.row[us][wg * C + c] * D] =
                __bfloat16_as_ushort(__float2bfloat16_rn(o[c] * m.inv[wg * C + c]));
      } else {
        float* part = a.parts + (size_t)(2 * u.run + (u.first == 0)) * slot_floats(R, D) +
                      wg * C * D + feat;
#pragma unroll
        for (int c = 0; c < C; ++c) part[c * D] = o[c];
      }
    };

    for (uint32_t un = 0;; ++un) {
      // ---- a unit begins: its query rows, split and scaled, and what they see
      const int us = un % UNITS;
      const Unit& u = m.unit[us];
      dead = !ta_wait(&m.u_full[us], (un / UNITS) & 1, abort_flag, a.err);
      if (named_barrier_or(1, ALL, dead)) break;
      if (u.last) break;
      const unsigned pos = (unsigned)u.pos;
      const bool drafts = (unsigned)u.stop * TILE > pos;     // the run reaches the tree
      if (drafts) {
        constexpr int NPW = NODES / (ALL / 32);          // nodes per warp
        const unsigned long long sees = lane < R ? m.sees[us][lane] >> (warp * NPW) : 0;
        uint32_t by = 0;
#pragma unroll
        for (int i = 0; i < NPW; ++i) {
          const uint32_t b = __ballot_sync(0xffffffffu, (sees >> i) & 1);
          if (lane == i) by = b;
        }
        if (lane < NPW) m.seen_by[warp * NPW + lane] = by;
      }
      if (th == 0) m.nan_nodes = 0;
      ok = ta_wait(&m.qr_full, un & 1, abort_flag, a.err) && ok;
      constexpr int LPR = D / 8;             // lanes per row, 8 values each
#pragma unroll 1
      for (int r0 = 0; r0 < R; r0 += ALL / LPR) {
        const int r = r0 + th / LPR, ch = th % LPR;
        if (r0 + ALL / LPR > R && r >= R) continue;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (m.row_node[us][r] < u.count)
          x = *reinterpret_cast<const uint4*>(smem + F::QR_OFF + (r * D + ch * 8) * 2);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, off, LPR));
        const bool nan = top >= 0x7F80u;     // an infinity's scores are NaN as well
        int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
        e = nan ? 0 : min(max(e, -126), 119);
        const float s = pow2i(-e);
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (nan) break;
          const float2 y = make_float2(bf16_lo(w[i]) * s, bf16_hi(w[i]) * s);
          const __nv_fp8x2_storage_t c8 = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
          const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c8, __NV_E4M3)));
          const __nv_fp8x2_storage_t r8 = __nv_cvt_float2_to_fp8x2(
              make_float2(QLO * (y.x - back.x), QLO * (y.y - back.y)), __NV_SATFINITE, __NV_E4M3);
          hi[i / 2] |= (uint32_t)c8 << (16 * (i & 1));
          lo[i / 2] |= (uint32_t)r8 << (16 * (i & 1));
        }
        *reinterpret_cast<uint2*>(sQ + sw_off<D>(r, ch * 8)) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(sQ + sw_off<D>(R + r, ch * 8)) = make_uint2(lo[0], lo[1]);
        if (ch == 0) {
          m.qf[r] = a.scale * pow2i(e);
          m.nan_row[r] = nan;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&m.q_full);
      dead = named_barrier_or(1, ALL, !ok);
      if (th == 0) mbar_arrive(&m.qr_empty);

      float m_run = -INFINITY;               // of column lt, in threads lt < C
#pragma unroll
      for (int c = 0; c < C / 2; ++c) acc[c] = l[c] = pair(0.f, 0.f);
      const int first_tile = u.first, stop = dead ? u.first : u.stop;
      const unsigned end = u.end;
      for (int tile = first_tile; tile < stop; ++tile, ++g) {
        ok = ta_wait(&m.e_full[g % ES], (g / ES) & 1, abort_flag, a.err) && ok;
        const uint8_t* e = sE + (g % ES) * 2 * TILE + lt;
        const uint32_t ke[2] = {e[0], e[SUB]}, ve[2] = {e[TILE], e[TILE + SUB]};
        const bool tree = (unsigned)(tile + 1) * TILE > pos;  // nodes, or the end
        // positions to mask or to keep from the product
        const bool odd =
            __any_sync(0xffffffffu, tree || !ke[0] || !ke[1] || !ve[0] || !ve[1]);
        uint32_t vis[2] = {~0u, ~0u};        // rows of this warpgroup that see the position
        if (odd) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned t = (unsigned)tile * TILE + h * SUB + lt;
            if (t >= end || ke[h] == 0)
              vis[h] = 0;
            else if (t >= pos)
              vis[h] = m.seen_by[t - pos] >> (wg * C);
          }
        }
        ok = ta_wait(&m.s_full, g & 1, abort_flag, a.err) && ok;
        tc_fence_after();
        float s[2][C];                       // score plus V exponent
        const f32x2 q_lo = pair(1.f / QLO, 1.f / QLO);
        const float ev[2] = {(float)((int)ve[0] - 127), (float)((int)ve[1] - 127)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x2 kf = pair(ke[h] << 23, ke[h] << 23), e2 = pair(ev[h], ev[h]);
          uint32_t hi[C], lo[C];
          tmem_load2(lanes_at + h * 2 * R, lanes_at + h * 2 * R + R, hi, lo);
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(&m.qf[wg * C + c]);
            unpair(fma2(fma2(pair(lo[c], lo[c + 1]), q_lo, pair(hi[c], hi[c + 1])),
                        mul2(pair(f4.x, f4.y), kf), e2),
                   s[h][c], s[h][c + 1]);
            unpair(fma2(fma2(pair(lo[c + 2], lo[c + 3]), q_lo, pair(hi[c + 2], hi[c + 3])),
                        mul2(pair(f4.z, f4.w), kf), e2),
                   s[h][c + 2], s[h][c + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(&m.s_free);
        if (odd) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (!((vis[h] >> c) & 1)) s[h][c] = -INFINITY;
          }
        }
        {
          float w[C];
#pragma unroll
          for (int c = 0; c < C; ++c) w[c] = warp_max(fmaxf(s[0][c], s[1][c]));
          if (lane == 0) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
              *reinterpret_cast<float4*>(&m.wmax[wg][wq][c]) =
                  make_float4(w[c], w[c + 1], w[c + 2], w[c + 3]);
          }
          uint2 e;
          e.x = __reduce_max_sync(0xffffffffu, max(vis[0] ? ve[0] : 0u, vis[1] ? ve[1] : 0u));
          e.y = __reduce_max_sync(0xffffffffu,
                                  max(vis[0] ? 255u - ve[0] : 0u, vis[1] ? 255u - ve[1] : 0u));
          if (lane == 0) m.wexp[wg][wq] = e;
        }
        named_barrier_sync(bar_wg, 128);
        int etop = 0, elow = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          etop = max(etop, (int)m.wexp[wg][i].x);
          elow = max(elow, (int)m.wexp[wg][i].y);
        }
        elow = 255 - elow;
        // V exponents too far apart: the scores need a maximum of their own
        const bool per_row = etop - elow > SPREAD;
        // (The exponents are read again where the scores are wanted without them: kept in
        // registers they cost 32 long sequences 106.4 us for 105.1.)
        auto exponent = [&](int h) { return (float)((int)e[TILE + h * SUB] - 127); };
        if (per_row) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float w = warp_max(fmaxf(s[0][c] - exponent(0), s[1][c] - exponent(1)));
            if (lane == 0) m.wscore[wg][wq][c] = w;
          }
          named_barrier_sync(bar_wg, 128);
        }
        bool moved = false;
        if (lt < C) {
          const float top = fmaxf(fmaxf(m.wmax[wg][0][lt], m.wmax[wg][1][lt]),
                                  fmaxf(m.wmax[wg][2][lt], m.wmax[wg][3][lt]));
          // the reference of the row's scores, and that of its weights above it
          float ref = ceilf(top) - (float)(etop - 127);
          int lift = etop - 127;
          if (per_row) {
            ref = ceilf(fmaxf(fmaxf(m.wscore[wg][0][lt], m.wscore[wg][1][lt]),
                              fmaxf(m.wscore[wg][2][lt], m.wscore[wg][3][lt])));
            lift = min(max((int)(ceilf(top) - ref), -127), 127);
          }
          // a tile without a visible position changes nothing
          if (top == -INFINITY) ref = m_run == -INFINITY ? 0.f : m_run;
          m.mref[wg][lt] = LOG2_WSCALE - (top == -INFINITY ? 0.f : ceilf(top));
          m.sref[wg][lt] = LOG2_WSCALE - ref;
          const float now = top == -INFINITY ? m_run : fmaxf(m_run, ref);
          float al = 1.f;
          if (now != m_run) {
            al = m_run == -INFINITY ? 0.f : pow2i((int)fmaxf(m_run - now, -200.f));
            moved = true;
          }
          const int d = now == -INFINITY ? 0 : (int)fmaxf(ref - now, -200.f);
          m_run = now;
          m.alpha[wg][lt] = al;
          m.beta[wg][lt] = pow2i(d);
          m.beta_o[wg][g & 1][lt] = pow2i(d + lift);
        }
        // (the references, and whether any moved or a wait gave up)
        const bool rescale = named_barrier_or(bar_wg, 128, moved || !ok);
        if (rescale && (dead = named_barrier_or(bar_wg, 128, !ok))) break;
        // weights; their sums per position in l, scaled to the running maximum
        if (rescale) {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 a4 = *reinterpret_cast<const float4*>(&m.alpha[wg][c]);
            l[c / 2] = mul2(l[c / 2], pair(a4.x, a4.y));
            l[c / 2 + 1] = mul2(l[c / 2 + 1], pair(a4.z, a4.w));
          }
        }
        if (per_row) {
#pragma unroll
          for (int c = 0; c < C; c += 2) {
            const float r0 = m.sref[wg][c], r1 = m.sref[wg][c + 1];
            f32x2 p[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              p[h] = pair(ta_exp2((s[h][c] - exponent(h)) + r0),
                          ta_exp2((s[h][c + 1] - exponent(h)) + r1));
            l[c / 2] = fma2(add2(p[0], p[1]), pair(m.beta[wg][c], m.beta[wg][c + 1]), l[c / 2]);
          }
        }
        // The weights go to the codes as they are (with the scale and the rounding to fp16
        // in a pass of their own 24-node trees took 46.1 us for 44.3); the softmax's own,
        // whose sum the row is divided by, are these times 2^(lift - ev).
        uint32_t ph[2][C / 2];
        f32x2 back[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (bounded where the weight is 0 and the exponent any)
          const int up = min(max(etop - (int)ve[h], -126), SPREAD) + 127;
          back[h] = pair((uint32_t)up << 23, (uint32_t)up << 23);
        }
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 r4 = *reinterpret_cast<const float4*>(&m.mref[wg][c]);
          const float4 b4 = *reinterpret_cast<const float4*>(&m.beta[wg][c]);
          const f32x2 rr[2] = {pair(r4.x, r4.y), pair(r4.z, r4.w)};
          const f32x2 bb[2] = {pair(b4.x, b4.y), pair(b4.z, b4.w)};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x2 p[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x, y;
              unpair(add2(pair(s[h][c + 2 * j], s[h][c + 2 * j + 1]), rr[j]), x, y);
              x = ta_exp2(x);
              y = ta_exp2(y);
              p[h] = pair(x, y);
              ph[h][c / 2 + j] = pack_f16x2(x, y);
            }
            if (!per_row)
              l[c / 2 + j] = fma2(fma2(p[0], back[0], mul2(p[1], back[1])), bb[j], l[c / 2 + j]);
          }
        }
        // the tile before: its output, now that its product is done
        if (tile > first_tile) add_o(g - 1);
        if (rescale) {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 a4 = *reinterpret_cast<const float4*>(&m.alpha[wg][c]);
            acc[c / 2] = mul2(acc[c / 2], pair(a4.x, a4.y));
            acc[c / 2 + 1] = mul2(acc[c / 2 + 1], pair(a4.z, a4.w));
          }
        }
        if (odd && wg == 0) {
          // V rows that must not reach the product: nothing held (stale
          // bytes), or a node's NaN, which only the nodes that see it may get.
          // Here the last tile's product is done, so its V tile has landed and the
          // barriers' phases are unambiguous.
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t j = 2 * g + h;
            ok = ta_wait(&m.v_full[j % VS], (j / VS) & 1, abort_flag, a.err) && ok;
            const unsigned t = (unsigned)tile * TILE + h * SUB + lt;
            uint4* vr = reinterpret_cast<uint4*>(sV + (j % VS) * F::KV_BYTES + lt * D);
            // eight lanes' 16-byte pieces lie in different banks (one token behind 300
            // positions 10.2 us; 10.8 with all lanes' pieces in one)
            const int rot = D == 128 ? lane : lane / 2;
            if (t >= end || e[h * SUB] == 0 || e[TILE + h * SUB] == 0) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) vr[(i + rot) % (D / 16)] = make_uint4(0, 0, 0, 0);
            } else if (t >= pos) {
              uint32_t any = 0;        // a byte 0x7F without its sign carries into bit 7
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint4 x = vr[(i + rot) % (D / 16)];
                any |= ((x.x & 0x7F7F7F7Fu) + 0x01010101u) | ((x.y & 0x7F7F7F7Fu) + 0x01010101u) |
                       ((x.z & 0x7F7F7F7Fu) + 0x01010101u) | ((x.w & 0x7F7F7F7Fu) + 0x01010101u);
              }
              any &= 0x80808080u;
              if (any) {
                uint32_t* vw = reinterpret_cast<uint32_t*>(vr);
#pragma unroll 1
                for (int i = 0; i < D / 4; ++i)
                  vw[i] &= ~__vcmpeq4(vw[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              }
              if (any) atomicOr(&m.nan_nodes, 1ull << (t - pos));
            }
          }
        }
        // the weights' codes
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi[C / 4], lo[C / 4];
#pragma unroll
          for (int i = 0; i < C / 4; ++i) split4(ph[h][2 * i], ph[h][2 * i + 1], &hi[i], &lo[i]);
          uint8_t* to_hi = sP + sw_off<2 * R>(h * SUB + lt, wg * C);
          uint8_t* to_lo = sP + sw_off<2 * R>(h * SUB + lt, R + wg * C);
          *reinterpret_cast<uint4*>(to_hi) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to_lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // also orders this thread's reads of the exponents before a later copy there
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&m.p_ready);
      }
      // ---- what the unit leaves: sums over the positions, the last product
      if (!dead) {
        float x[C];
#pragma unroll
        for (int c = 0; c < C; c += 2) unpair(l[c / 2], x[c], x[c + 1]);
        // over the warp's lanes: each step halves the columns a lane keeps
#pragma unroll
        for (int w = C / 2, bit = 16; w > 0; w /= 2, bit /= 2) {
#pragma unroll
          for (int c = 0; c < w; ++c) {
            const float give = lane & bit ? x[c] : x[c + w], keep = lane & bit ? x[c + w] : x[c];
            x[c] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
          }
        }
#pragma unroll
        for (int bit = 16 / C; bit > 0; bit /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], bit);
        if (lane % (32 / C) == 0) m.lsum[wg][wq][lane / (32 / C)] = x[0];
        named_barrier_sync(bar_wg, 128);
        const bool whole = u.first == 0 && u.stop == u.tiles;
        if (lt < C) {
          const int r = wg * C + lt;
          float sum = (m.lsum[wg][0][lt] + m.lsum[wg][1][lt]) +
                      (m.lsum[wg][2][lt] + m.lsum[wg][3][lt]);
          // (its scores are 0: without a position it sees nothing was added)
          if (m.nan_row[r] && sum != 0.f) sum = __uint_as_float(0x7FC00000u);
          m.inv[r] = sum == 0.f ? 0.f : 1.f / sum;
          if (!whole) {
            float* part =
                a.parts + (size_t)(2 * u.run + (u.first == 0)) * slot_floats(R, D) + R * D + 2 * r;
            part[0] = m_run;
            part[1] = sum;
          }
        }
        if (u.first == 0 && th == 64) {
          Head hd;
          hd.run = u.run;
          hd.follow = u.follow;
          a.heads[((int64_t)u.b * a.c.Hkv + u.hk) * a.blocks + u.rb] = hd;
        }
        add_o(g - 1);
        dead = named_barrier_or(bar_wg, 128, !ok);
        if (!dead) finish_unit(u, us);
      }
      // all warpgroups are done with the unit and its rows, or stop together
      if (named_barrier_or(1, ALL, dead)) break;
      if (th == 0) mbar_arrive(&m.u_empty[un % UNITS]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, F::TMEM_COLS);
  }
}

// Joins the parts of the units that lie in more than one run, in run order:
// one CTA of 8 warps per unit and 8 / WPR of its rows.
template <int D, int R, int WPR>
__global__ void __launch_bounds__(256) tree_attn_combine_kernel(const TreeArgs a) {
  using namespace ta;
  constexpr int V = D / 32, U = 8;
  __shared__ float part_o[8][D], part_l[8], part_m[8];
  stream_order_begin();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int unit = blockIdx.x;
  const int rb = unit % a.blocks, hk = unit / a.blocks % a.c.Hkv, b = unit / a.blocks / a.c.Hkv;
  const Head hd = a.heads[unit];
  const TreeSeq t = tree_seq<R>(a, b, false);
  // units of fewer nodes than N may not exist: their entry was not written
  if (rb >= t.blocks || hd.follow == 0) return;
  if (!parts_within(hd)) {         // not written: a wait gave up before this unit
    if (threadIdx.x == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  const int r = blockIdx.y * (8 / WPR) + warp / WPR;
  const int flat = rb * R + r, node = flat / a.G, h = hk * a.G + flat % a.G;
  const int n = hd.follow + 1;
  float o[V], sum = 0.f, top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = 0.f;
  for (int i0 = warp % WPR; i0 < n; i0 += WPR * U) {
    float2 ml[U];
    float v[U][V], most = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * WPR;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (i >= n) continue;
      const float* p = a.parts + (size_t)part_slot(hd, i) * slot_floats(R, D);
      ml[u] = *reinterpret_cast<const float2*>(p + R * D + 2 * r);
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + r * D + lane * 4);
        v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p + r * D + lane * 2);
        v[u][0] = x.x; v[u][1] = x.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) most = fmaxf(most, ml[u].x);
    const float keep = top == -INFINITY ? 0.f : pow2i((int)fmaxf(top - most, -200.f));
    top = most;
    sum *= keep;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] *= keep;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * WPR >= n) continue;
      const float f = ml[u].x == -INFINITY ? 0.f : pow2i((int)fmaxf(ml[u].x - top, -200.f));
      sum = fmaf(ml[u].y, f, sum);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = fmaf(v[u][j], f, o[j]);
    }
  }
  if (WPR > 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) part_o[warp][lane * V + j] = o[j];
    if (lane == 0) {
      part_l[warp] = sum;
      part_m[warp] = top;
    }
    __syncthreads();
    if (warp % WPR != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = fmaxf(top, part_m[warp + w]);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float pm = part_m[warp + w];
      const float f = pm == -INFINITY ? 0.f : pow2i((int)fmaxf(pm - top, -200.f));
      sum = fmaf(part_l[warp + w], f, sum);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = fmaf(part_o[warp + w][lane * V + j], f, o[j]);
    }
  }
  if (node >= t.count) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* dst = a.out + (((int64_t)b * a.s.N + node) * a.Hq + h) * D + lane * V;
#pragma unroll
  for (int j = 0; j < V; j += 2)
    *reinterpret_cast<uint32_t*>(dst + j) =
        sum == 0.f ? 0u : pack_bf16x2(o[j] * inv, o[j + 1] * inv);
}

static int tree_block_rows(int N, int G) {
  const int rows = N * G;
  return rows <= 16 ? 16 : 32;
}

// CTAs on `sms` SMs, as many as the workspace has room for at most.
static int tree_ctas(int sms) {
  const int n = sms * ta::CTAS;
  return n < ta::MAX_CTAS ? n : ta::MAX_CTAS;
}
static int tree_blocks(int N, int G) {
  const int R = tree_block_rows(N, G);
  return (N * G + R - 1) / R;
}
static size_t tree_heads_bytes(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int Hq) {
  const size_t units = (size_t)s.B * c.Hkv * tree_blocks(s.N, Hq / c.Hkv);
  return (units * sizeof(ta::Head) + 255) & ~size_t(255);
}

size_t tree_attn_scratch(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int Hq) {
  const int R = tree_block_rows(s.N, Hq / c.Hkv);
  return tree_heads_bytes(c, s, Hq) +
         (size_t)ta::MAX_CTAS * 2 * ta::slot_floats(R, c.D) * sizeof(float);
}

template <int D, int R>
static cudaError_t launch_tree(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                               cudaStream_t stream) {
  using F = ta::Cfg<D, R>;
  constexpr int SMEM = F::MISC_OFF + (int)sizeof(ta::Misc<F, R>);
  static_assert(ta::CTAS * (SMEM + 1024) <= 233472, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, R>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const int grid = tree_ctas(sm_count());
  e = launch_in_order(tree_attn_kernel<D, R>, grid, F::THREADS, SMEM, stream, 0, mk, mv, a);
  if (e != cudaSuccess) return e;
  // Many parts per unit: a row's parts over 8 warps; few: a row per warp.  The whole
  // call with 4 KV heads of 4 nodes, over 8 warps and one: behind 34,000 positions 4 units
  // 21.4 and 33.4 us, 16 31.9 and 33.7, 24 35.6 and 36.5, 28 40.2 and 39.6, 36 49.3 and
  // 47.1, 72 77.3 and 69.2; behind 3,000 or fewer 4 to 20 units 13.9 to 20.2 and 17.6 to
  // 21.5, 36 19.0 and 16.5, 72 26.3 and 19.1.
  const int units = a.s.B * a.c.Hkv * a.blocks;
  const bool wide = grid / units >= 12;
  return launch_in_order(
      wide ? tree_attn_combine_kernel<D, R, 8> : tree_attn_combine_kernel<D, R, 1>,
      dim3(units, wide ? R : R / 8), 256, 0, stream, 0, a);
}

cudaError_t launch_tree_attn(const strata_kv_cache_t& c, const strata_kv_seqs_t& s,
                             const int32_t* parent, const uint16_t* q, int64_t q_stride, int Hq,
                             float scale, uint16_t* out, void* ws, unsigned* err,
                             cudaStream_t stream) {
  TreeArgs a;
  a.c = c;
  a.s = s;
  a.parent = parent;
  a.q = q;
  a.q_stride = q_stride;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.scale = scale * 1.4426950408889634f;
  a.out = out;
  a.heads = static_cast<ta::Head*>(ws);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + tree_heads_bytes(c, s, Hq));
  a.blocks = tree_blocks(s.N, a.G);
  a.err = err;
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)c.pages * c.Hkv * c.page;
  const CUtensorMapSwizzle sw = c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (encode_tmap_2d(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.k, c.D, rows, c.D, c.D, c.page, sw,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != CUDA_SUCCESS ||
      encode_tmap_2d(&mv, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.v, c.D, rows, c.D, c.D, c.page, sw,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int R = tree_block_rows(s.N, a.G);
  if (c.D == 128)
    return R == 16 ? launch_tree<128, 16>(a, mk, mv, stream) : launch_tree<128, 32>(a, mk, mv, stream);
  return R == 16 ? launch_tree<64, 16>(a, mk, mv, stream) : launch_tree<64, 32>(a, mk, mv, stream);
}

}  // namespace strata
