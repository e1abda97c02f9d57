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
// values (4 bits each), so the scores are sums of exact products: the low
// part is exact down to 2^-17 of the row's largest value.  The weights are
// split the same way: p (fp32) is rounded to fp16 (2^-11), to e4m3, and
// the remainder to e4m3 again, 2^-9 of the value in all.  Against one bf16
// rounding of p (2^-8) that is half the error, and the tensor pipe never
// waits for codes to be widened.  High and low parts are separate columns
// of one product (the K or V tile is read from shared memory once) and are
// added in fp32 registers.
//
// A position's K exponent multiplies its scores, one factor per thread,
// because a thread is a position there.  Its V exponent goes into the weight:
// P = p * 2^(ev - E) * 448 with E the largest V exponent of the tile, and the
// tile's O is added to the running sum as O * 2^E.  A tile's weights
// are scaled to its own maximum, not to the running one, since e4m3 reaches
// only 2^-9 (2^-17.8 of the tile's largest weight): positions of a tile far
// below an earlier tile's maximum keep their precision.  References are
// integers (log2 domain), so rescaling is an exponent addition.
//
// Work: the tiles of all (sequence, KV head, block of R rows) units in one
// line, cut into equal runs, one per CTA, whatever the lengths are.  A unit
// that lies in one run is finished there; the others leave partial sums
// that tree_attn_combine_kernel joins in run order.
//
// Roles per CTA: a warp that issues the TMA copies of pages (K, V, exponents)
// into a ring of tiles, a warp that issues the MMAs, and one warpgroup per 32
// row columns (16 when R = 16) for the softmax, the weights and the running sums.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "kv.h"

namespace strata {

namespace ta {
constexpr int TILE = 128;                   // positions per tile
constexpr int NODES = STRATA_TREE_MAX_NODES;
constexpr int MAX_CTAS = 148 * 4;           // runs the workspace has room for
constexpr float WSCALE = 448.f;             // weights are scaled to e4m3's largest value

template <int D, int R>
struct Cfg {
  static constexpr int NWG = R == 64 ? 2 : 1;          // softmax warpgroups
  static constexpr int C = R / NWG;                    // row columns per warpgroup
  static constexpr int CTAS = R == 64 ? 1 : 2;         // per SM
  static constexpr int STAGES =
      D == 128 ? (R == 64 ? 5 : R == 32 ? 2 : 3) : (R == 64 ? 8 : R == 32 ? 5 : 6);
  static constexpr int THREADS = NWG * 128 + 64;
  static constexpr int KV_BYTES = TILE * D;            // one operand tile
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + STAGES * KV_BYTES;
  static constexpr int Q_OFF = V_OFF + STAGES * KV_BYTES;      // [2R][D] codes
  static constexpr int P_OFF = Q_OFF + 2 * R * D;              // [128][2R] codes
  static constexpr int E_OFF = P_OFF + TILE * 2 * R;           // [STAGES][2][128] exponents
  static constexpr int MISC_OFF = E_OFF + STAGES * 256;
  static constexpr int S_COLS = 2 * R;                 // TMEM: two S tiles, one O tile
  static constexpr int TMEM_COLS = R == 64 ? 512 : R == 32 ? 256 : 128;
};

template <int R, int NWG, int C, int STAGES>
struct Misc {
  uint64_t full[STAGES], empty[STAGES], s_full[2], p_ready, o_full, q_full;
  uint64_t sees[R];                  // nodes that the row's node sees
  unsigned long long nan_nodes;      // nodes whose V holds a NaN
  uint32_t tmem;
  int abort;
  int parent[NODES];
  int64_t scan[16];
  int64_t total, start_off;
  int start_b;
  alignas(16) float qf[R];                       // score factor of the row
  int nan_row[R];
  alignas(16) float wmax[NWG][C][4];             // per warp: largest score of the tile
  alignas(16) uint32_t wexp[NWG][C][4];          // per warp: largest visible V exponent
  alignas(16) uint32_t wtop[NWG][4];
  alignas(16) float mref[NWG][C], beta[NWG][C], alpha[NWG][C];
  alignas(16) float beta_o[NWG][2][C];
  alignas(16) uint32_t ecol[NWG][C];
  alignas(16) float lsum[NWG][C][4];
};

// A run's first unit may have begun in an earlier run: slot 0; its last may go
// on in the next: slot 1.
struct Head {
  int follow;      // runs after this one that continue the unit of slot 1
  int b, hk, rb;
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
  float scale;            // times log2(e)
  uint16_t* out;
  ta::Head* heads;
  float* parts;
  unsigned* err;
};

// One sequence's extent in this call.
struct TreeSeq {
  int pos, count, tiles, blocks;
  int64_t end;            // positions with a column in the page table
};

template <int R>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  TreeSeq t;
  bool bad;
  const SeqRange r = seq_range(a.s, b, &bad);
  t.pos = r.pos;
  t.count = r.count;
  const int64_t room = (int64_t)a.s.max_pages * a.c.page;
  t.end = (int64_t)r.pos + r.count;
  if (t.end > room) {
    bad = r.count > 0;
    t.end = room;
  }
  t.tiles = r.count > 0 ? (int)((t.end + ta::TILE - 1) / ta::TILE) : 0;
  t.blocks = (r.count * a.G + R - 1) / R;
  if (bad && report) atomicOr(a.err, kErrIndex);
  return t;
}

// A run's position in the line of tiles.
template <int R>
struct Cursor {
  int b, hk, rb, tile;
  TreeSeq t;
  __device__ __forceinline__ void at(const TreeArgs& a, int b0, int64_t off) {
    b = b0;
    t = tree_seq<R>(a, b, false);
    tile = (int)(off % t.tiles);
    const int64_t u = off / t.tiles;
    rb = (int)(u % t.blocks);
    hk = (int)(u / t.blocks);
  }
  // To the next unit; only called while tiles are left in the run.
  __device__ __forceinline__ void next_unit(const TreeArgs& a) {
    tile = 0;
    if (++rb < t.blocks) return;
    rb = 0;
    if (++hk < a.c.Hkv) return;
    hk = 0;
    do {
      ++b;
      t = tree_seq<R>(a, b, false);
    } while (t.tiles == 0);
  }
};

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

template <int D, int R>
__global__ void __launch_bounds__(ta::Cfg<D, R>::THREADS, ta::Cfg<D, R>::CTAS)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const TreeArgs a) {
  using namespace ta;
  using F = Cfg<D, R>;
  constexpr int NWG = F::NWG, C = F::C, STAGES = F::STAGES;
  using M = Misc<R, NWG, C, STAGES>;
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

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (th == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    mbar_init(&m.s_full[0], 1);
    mbar_init(&m.s_full[1], 1);
    mbar_init(&m.p_ready, NWG * 128);
    mbar_init(&m.o_full, 1);
    mbar_init(&m.q_full, NWG * 128);
    m.abort = 0;
    m.start_b = -1;
    fence_mbar_init();
  }
  if (warp == W_TMA && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == W_MMA) tmem_alloc(&m.tmem, F::TMEM_COLS);

  // ---- the line of tiles and this CTA's run of it: sequences in contiguous
  // shares per thread, their tile counts scanned over the CTA
  const int per = (a.s.B + F::THREADS - 1) / F::THREADS;
  const int sb0 = min(th * per, a.s.B), sb1 = min(sb0 + per, a.s.B);
  int64_t mine = 0;
  for (int b = sb0; b < sb1; ++b) {
    const TreeSeq t = tree_seq<R>(a, b, reporter);
    mine += (int64_t)t.tiles * t.blocks * a.c.Hkv;
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) m.scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < F::THREADS / 32; ++w) {
    if (w < warp) before += m.scan[w];
    total += m.scan[w];
  }
  const int64_t runs = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  const int cta = blockIdx.x;
  const bool active = cta < runs;
  const int64_t w0 = active ? total * cta / runs : 0;
  const int64_t w1 = active ? total * (cta + 1) / runs : 0;
  if (active && w0 >= before && w0 < before + mine) {
    int64_t at = before;
    for (int b = sb0; b < sb1; ++b) {
      const TreeSeq t = tree_seq<R>(a, b, false);
      const int64_t n = (int64_t)t.tiles * t.blocks * a.c.Hkv;
      if (w0 < at + n) {
        m.start_b = b;
        m.start_off = w0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int64_t n_items = w1 - w0;
  const uint32_t tmem = m.tmem;
  if (!active) {
    if (th == 0) a.heads[cta].follow = 0;
  } else if (warp == W_TMA) {
    // ------------------------------------------------------------ page copies
    Cursor<R> cu;
    cu.at(a, m.start_b, m.start_off);
    const int page = a.c.page, ppt = TILE / page;      // pages per tile
    uint32_t g = 0;
    int64_t left = n_items;
    while (left > 0) {
      const int stop = (int)min((int64_t)cu.t.tiles, (int64_t)cu.tile + left);
      left -= stop - cu.tile;
      bool dead = false;
      for (; cu.tile < stop; ++cu.tile, ++g) {
        const int st = g % STAGES;
        // the tile's pages, one per lane
        const int64_t first = (int64_t)cu.tile * TILE + (int64_t)lane * page;
        int64_t row = -1;
        if (lane < ppt && first < cu.t.end) {
          row = row_of(a.c, a.s, cu.b, first);
          if (row < 0)
            atomicOr(a.err, kErrIndex);
          else
            row += (int64_t)cu.hk * page;
        }
        if (g >= (uint32_t)STAGES &&
            !mbar_wait_warp(&m.empty[st], (g / STAGES - 1) & 1, abort_flag, a.err)) {
          dead = true;
          break;
        }
        uint8_t* e = sE + st * 256;
        if (lane < ppt && row < 0) {                   // no page: nothing held there
          for (int i = 0; i < page; i += 16)
            *reinterpret_cast<uint4*>(e + lane * page + i) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();                    // before a later copy to the same place
        }
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&m.full[st], pages * page * (2 * D + 2));
        __syncwarp();
        if (row >= 0) {
          tma_load_2d(sK + st * F::KV_BYTES + lane * page * D, &map_k, 0, (int)row, &m.full[st]);
          tma_load_2d(sV + st * F::KV_BYTES + lane * page * D, &map_v, 0, (int)row, &m.full[st]);
          bulk_load(e + lane * page, a.c.k_exp + row, page, &m.full[st]);
          bulk_load(e + 128 + lane * page, a.c.v_exp + row, page, &m.full[st]);
        }
        __syncwarp();
      }
      if (dead) {
        // copies in flight land before the CTA's shared memory goes away
        for (uint32_t i = g > (uint32_t)STAGES ? g - STAGES : 0; i < g; ++i) {
          const uint32_t bar = smem_addr(&m.full[i % STAGES]);
          const unsigned long long t0 = global_ns();
          while (!mbar_try_wait(bar, (i / STAGES) & 1) && global_ns() - t0 < kWaitLimitNs) {
          }
        }
        break;
      }
      if (left > 0) cu.next_unit(a);
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issue
    const bool leader = elect_one();
    constexpr uint32_t ID_S = idesc_e4m3(TILE, 2 * R, 0, 0);
    constexpr uint32_t ID_O = idesc_e4m3(D, 2 * R, 1, 1);
    const uint32_t t_o = tmem + 2 * F::S_COLS;
    uint32_t g = 0, unit = 0;
    auto scores = [&](uint32_t i) -> bool {
      const int st = i % STAGES;
      if (!mbar_wait_warp(&m.full[st], (i / STAGES) & 1, abort_flag, a.err)) return false;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          mma_f8_ss(tmem + (i & 1) * F::S_COLS,
                    smem_desc(smem_addr(sK + st * F::KV_BYTES) + 32 * k, 8 * D, sw_mode(D)),
                    smem_desc(smem_addr(sQ) + 32 * k, 8 * D, sw_mode(D)), ID_S, k > 0);
        mma_commit(&m.s_full[i & 1]);
      }
      __syncwarp();
      return true;
    };
    Cursor<R> cu;
    cu.at(a, m.start_b, m.start_off);
    int64_t left = n_items;
    bool dead = false;
    while (left > 0 && !dead) {
      const int tiles = (int)min((int64_t)cu.t.tiles - cu.tile, left);
      left -= tiles;
      if (!mbar_wait_warp(&m.q_full, unit & 1, abort_flag, a.err)) break;
      tc_fence_after();
      if (!scores(g)) break;
      for (int i = 0; i < tiles; ++i, ++g) {
        const int st = g % STAGES;
        if (i + 1 < tiles && !scores(g + 1)) {
          dead = true;
          break;
        }
        if (!mbar_wait_warp(&m.p_ready, g & 1, abort_flag, a.err)) {
          dead = true;
          break;
        }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < TILE / 32; ++k)
            mma_f8_ss(t_o,
                      smem_desc(smem_addr(sV + st * F::KV_BYTES) + 32 * k * D, 8 * D, sw_mode(D)),
                      smem_desc(smem_addr(sP) + 32 * k * 2 * R, 16 * R, sw_mode(2 * R)), ID_O,
                      k > 0);
          mma_commit(&m.o_full);
          mma_commit(&m.empty[st]);
        }
        __syncwarp();
      }
      ++unit;
      if (left > 0 && !dead) cu.next_unit(a);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = warp / 4, wq = warp % 4, lt = th % 128;   // lt: position in the tile
    constexpr uint32_t ALL = NWG * 128;
    const uint32_t lanes_at = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t bar_wg = 2 + wg;
    // the feature whose sums this thread keeps (D = 64: 16 lanes per warp)
    const int feat = D == 128 ? lt : wq * 16 + lane;
    const bool has_feat = D == 128 || lane < 16;
    float acc[C], l[C];
    uint32_t g = 0;
    bool ok = true, dead = false;
    int64_t left = n_items;
    Cursor<R> cu;
    cu.at(a, m.start_b, m.start_off);
    if (th == 0) a.heads[cta].follow = 0;

    // O of tile i (sum of its high and low columns) into acc
    auto add_o = [&](uint32_t i) {
      ok = mbar_wait_warp(&m.o_full, i & 1, abort_flag, a.err) && ok;
      tc_fence_after();
      const float* bo = m.beta_o[wg][i & 1];
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += 16) {
        uint32_t hi[16], lo[16];
        const uint32_t col = lanes_at + 2 * F::S_COLS + wg * C + c0;
        tmem_ld_32x32b_x16(col, hi);
        tmem_ld_32x32b_x16(col + R, lo);
        tmem_ld_wait_regs(hi);
        tmem_ld_wait_regs(lo);
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 b4 = *reinterpret_cast<const float4*>(bo + c0 + c);
          const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[c0 + c + j] = fmaf(__uint_as_float(hi[c + j]) + __uint_as_float(lo[c + j]), bb[j],
                                   acc[c0 + c + j]);
        }
      }
    };

    // The unit's results: rounded to the output when the run holds all of it,
    // its part otherwise.
    auto finish_unit = [&](int first_tile, int stop, bool drafts) {
      unsigned long long nan_nodes = drafts ? m.nan_nodes : 0;
      while (nan_nodes) {
        const int j = __ffsll((long long)nan_nodes) - 1;
        nan_nodes &= nan_nodes - 1;
        const int64_t row = row_of(a.c, a.s, cu.b, (int64_t)cu.t.pos + j) + (int64_t)cu.hk * a.c.page;
        if (has_feat && (a.c.v[row * D + feat] & 0x7F) == 0x7F) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            if ((m.sees[wg * C + c] >> j) & 1) acc[c] = __uint_as_float(0x7FC00000u);
        }
      }
      const bool whole = first_tile == 0 && stop == cu.t.tiles;
      const int slot = first_tile == 0 ? 1 : 0;
      float* part = a.parts + (size_t)(2 * cta + slot) * slot_floats(R, D);
      if (!whole && slot == 1 && th == 0) {
        // the last run that holds a tile of this unit: the unit ends
        // (tiles - stop) tiles behind this run
        const int64_t last = w1 + (cu.t.tiles - stop) - 1;
        Head hd;
        hd.follow = (int)(((last + 1) * runs - 1) / total) - cta;
        hd.b = cu.b;
        hd.hk = cu.hk;
        hd.rb = cu.rb;
        a.heads[cta] = hd;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int r = wg * C + c;
        const float4 l4 = *reinterpret_cast<const float4*>(m.lsum[wg][c]);
        float sum = (l4.x + l4.y) + (l4.z + l4.w);
        if (m.nan_row[r]) sum = __uint_as_float(0x7FC00000u);
        if (whole) {
          const int flat = cu.rb * R + r;
          const int node = flat / a.G, h = cu.hk * a.G + flat % a.G;
          if (node < cu.t.count && has_feat) {
            const float o = sum == 0.f ? 0.f : acc[c] / (sum * WSCALE);
            a.out[(((int64_t)cu.b * a.s.N + node) * a.Hq + h) * D + feat] =
                __bfloat16_as_ushort(__float2bfloat16_rn(o));
          }
        } else {
          if (has_feat) part[r * D + feat] = acc[c];
          if (lt == 0) {
            part[R * D + 2 * r] = m.mref[wg][c];
            part[R * D + 2 * r + 1] = sum;
          }
        }
      }
    };

    for (;;) {
      // ---- a unit begins: its query rows, split and scaled, and what they see
      const int first_tile = cu.tile;
      const int stop = (int)min((int64_t)cu.t.tiles, (int64_t)cu.tile + left);
      left -= stop - first_tile;
      const int pos = cu.t.pos;
      const bool drafts = (int64_t)stop * TILE > pos;        // the run reaches the tree
      if (th < NODES && drafts) {
        int p = -1;
        if (th < cu.t.count) {
          p = a.parent ? a.parent[(int64_t)cu.b * a.s.N + th] : th - 1;
          if (p < -1 || p >= th) {
            atomicOr(a.err, kErrIndex);
            p = -1;
          }
        }
        m.parent[th] = p;
      }
      if (th == 0) m.nan_nodes = 0;
      constexpr int LPR = D / 8;             // lanes per row, 8 values each
      for (int r0 = 0; r0 < R; r0 += ALL / LPR) {
        const int r = r0 + th / LPR, ch = th % LPR;
        if (r0 + ALL / LPR > R && r >= R) continue;
        const int flat = cu.rb * R + r;
        const int node = flat / a.G, h = cu.hk * a.G + flat % a.G;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (node < cu.t.count)
          x = ld_nc_v4(a.q + ((int64_t)cu.b * a.s.N + node) * a.q_stride + (int64_t)h * D + ch * 8);
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
        const float s = nan ? 0.f : pow2i(-e);
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
        if (!nan) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = make_float2(bf16_lo(w[i]) * s, bf16_hi(w[i]) * s);
            const __nv_fp8x2_storage_t c8 = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c8, __NV_E4M3)));
            const __nv_fp8x2_storage_t r8 = __nv_cvt_float2_to_fp8x2(
                make_float2(y.x - back.x, y.y - back.y), __NV_SATFINITE, __NV_E4M3);
            hi[i / 2] |= (uint32_t)c8 << (16 * (i & 1));
            lo[i / 2] |= (uint32_t)r8 << (16 * (i & 1));
          }
        }
        *reinterpret_cast<uint2*>(sQ + sw_off<D>(r, ch * 8)) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(sQ + sw_off<D>(R + r, ch * 8)) = make_uint2(lo[0], lo[1]);
        if (ch == 0) {
          m.qf[r] = a.scale * pow2i(e);
          m.nan_row[r] = nan;
        }
      }
      fence_proxy_async_smem();
      named_barrier_sync(1, ALL);
      if (drafts && th < R) {
        const int node = min((cu.rb * R + th) / a.G, NODES - 1);
        uint64_t see = 0;
        for (int j = node; j >= 0; j = m.parent[j]) see |= 1ull << j;
        m.sees[th] = see;
      }
      named_barrier_sync(1, ALL);
      mbar_arrive(&m.q_full);

      float m_run = -INFINITY;               // of column lt, in threads lt < C
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = l[c] = 0.f;
      for (int tile = first_tile; tile < stop; ++tile, ++g) {
        const int st = g % STAGES;
        ok = mbar_wait_warp(&m.full[st], (g / STAGES) & 1, abort_flag, a.err) && ok;
        const int64_t t = (int64_t)tile * TILE + lt;
        const uint32_t ke = sE[st * 256 + lt], ve = sE[st * 256 + 128 + lt];
        const bool held = t < cu.t.end && ke != 0;
        const bool tree = (int64_t)(tile + 1) * TILE > pos;  // some positions are nodes
        const int node = t >= pos ? (int)(t - pos) : -1;     // >= 0: this one is
        const float kf = __uint_as_float(ke << 23);
        if (wg == 0) {
          // V rows that must not reach the product: nothing held (stale
          // bytes), or a node's NaN, which only the nodes that see it may get
          uint4* vr = reinterpret_cast<uint4*>(sV + st * F::KV_BYTES + lt * D);
          if (!held || ve == 0) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) vr[i] = make_uint4(0, 0, 0, 0);
          } else if (node >= 0) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint4 x = vr[i];
              uint32_t n[4] = {__vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                               __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                               __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                               __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)};
              if (n[0] | n[1] | n[2] | n[3]) {
                any = true;
                vr[i] = make_uint4(x.x & ~n[0], x.y & ~n[1], x.z & ~n[2], x.w & ~n[3]);
              }
            }
            if (any) atomicOr(&m.nan_nodes, 1ull << node);
          }
        }
        ok = mbar_wait_warp(&m.s_full[g & 1], (g >> 1) & 1, abort_flag, a.err) && ok;
        tc_fence_after();
        float s[C];
        float top_mine = -INFINITY;          // the warp's maximum of column `lane`
        uint32_t exp_mine = 0;
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 16) {
          uint32_t hi[16], lo[16];
          const uint32_t col = lanes_at + (g & 1) * F::S_COLS + wg * C + c0;
          tmem_ld_32x32b_x16(col, hi);
          tmem_ld_32x32b_x16(col + R, lo);
          tmem_ld_wait_regs(hi);
          tmem_ld_wait_regs(lo);
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(&m.qf[wg * C + c0 + c]);
            const float ff[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float u = __uint_as_float(hi[c + j]) + __uint_as_float(lo[c + j]);
              s[c0 + c + j] = held ? u * (ff[j] * kf) : -INFINITY;
            }
          }
        }
        tc_fence_before();
        if (tree && node >= 0) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (node >= NODES || !((m.sees[wg * C + c] >> (node & 63)) & 1)) s[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float w = warp_max(s[c]);
          if (lane == c) top_mine = w;
        }
        if (tree) {
          // the largest V exponent among what a row sees: one per row here
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const uint32_t w = __reduce_max_sync(0xffffffffu, s[c] == -INFINITY ? 0u : ve);
            if (lane == c) exp_mine = w;
          }
          if (lane < C) m.wexp[wg][lane][wq] = exp_mine;
        } else {
          const uint32_t w = __reduce_max_sync(0xffffffffu, held ? ve : 0u);
          if (lane == 0) m.wtop[wg][wq] = w;
        }
        if (lane < C) m.wmax[wg][lane][wq] = top_mine;
        dead = named_barrier_or(bar_wg, 128, !ok);
        if (dead) break;
        const uint32_t etop = tree ? 0u
                                   : max(max(m.wtop[wg][0], m.wtop[wg][1]),
                                         max(m.wtop[wg][2], m.wtop[wg][3]));
        bool moved = false;
        if (lt < C) {
          const float4 w4 = *reinterpret_cast<const float4*>(m.wmax[wg][lt]);
          const float top = fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w));
          uint32_t e = etop;
          if (tree) {
            const uint4 e4 = *reinterpret_cast<const uint4*>(m.wexp[wg][lt]);
            e = max(max(e4.x, e4.y), max(e4.z, e4.w));
            m.ecol[wg][lt] = e;
          }
          // a tile without a visible position changes nothing
          const float ref = top == -INFINITY ? (m_run == -INFINITY ? 0.f : m_run) : ceilf(top);
          const float now = top == -INFINITY ? m_run : fmaxf(m_run, ref);
          float al = 1.f;
          if (now != m_run) {
            al = m_run == -INFINITY ? 0.f : pow2i((int)fmaxf(m_run - now, -200.f));
            moved = true;
          }
          const int d = now == -INFINITY ? 0 : (int)fmaxf(ref - now, -200.f);
          m_run = now;
          m.mref[wg][lt] = ref;
          m.alpha[wg][lt] = al;
          m.beta[wg][lt] = pow2i(d);
          m.beta_o[wg][g & 1][lt] = pow2i(d + (int)e - 127);
        }
        const bool rescale = named_barrier_or(bar_wg, 128, moved);
        // weights; their sums per position in l, scaled to the running maximum
        uint32_t ph[C / 2];
        const float vf = tree ? 0.f : pow2i(min((int)ve - (int)etop, 0)) * WSCALE;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 r4 = *reinterpret_cast<const float4*>(&m.mref[wg][c]);
          const float4 b4 = *reinterpret_cast<const float4*>(&m.beta[wg][c]);
          const float rr[4] = {r4.x, r4.y, r4.z, r4.w}, bb[4] = {b4.x, b4.y, b4.z, b4.w};
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ta_exp2(s[c + j] - rr[j]);
            if (rescale) l[c + j] *= m.alpha[wg][c + j];
            l[c + j] = fmaf(p[j], bb[j], l[c + j]);
          }
          if (tree) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              p[j] *= pow2i(min((int)ve - (int)m.ecol[wg][c + j], 0)) * WSCALE;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] *= vf;
          }
          ph[c / 2] = pack_f16x2(p[0], p[1]);
          ph[c / 2 + 1] = pack_f16x2(p[2], p[3]);
        }
        // the tile before: its output, now that its product is done
        if (tile > first_tile) add_o(g - 1);
        if (rescale) {
#pragma unroll
          for (int c = 0; c < C; ++c) acc[c] *= m.alpha[wg][c];
        }
        // the weights' codes, 16 rows a store
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            split4(ph[c0 / 2 + 2 * i], ph[c0 / 2 + 2 * i + 1], &hi[i], &lo[i]);
          *reinterpret_cast<uint4*>(sP + sw_off<2 * R>(lt, wg * C + c0)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sP + sw_off<2 * R>(lt, R + wg * C + c0)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // also orders this thread's reads of the stage before the next copy into it
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&m.p_ready);
      }
      // ---- the unit's last product, and what it leaves
      if (!dead) {
        add_o(g - 1);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float x = l[c];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
          if (lane == 0) m.lsum[wg][c][wq] = x;
        }
        if (lt < C) m.mref[wg][lt] = m_run;
        dead = named_barrier_or(bar_wg, 128, !ok);
      }
      if (!dead) finish_unit(first_tile, stop, drafts);
      // all warpgroups are done with the unit's rows, or stop together
      if (named_barrier_or(1, ALL, dead) || left <= 0) break;
      cu.next_unit(a);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, F::TMEM_COLS);
  }
}

// Joins the parts of the units that lie in more than one run: one warp per
// row, in run order.
template <int D, int R>
__global__ void __launch_bounds__(128) tree_attn_combine_kernel(const TreeArgs a) {
  using namespace ta;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Head hd = a.heads[blockIdx.x];
  if (hd.follow <= 0) return;
  const int lane = threadIdx.x % 32, r = blockIdx.y * 4 + threadIdx.x / 32;
  const int flat = hd.rb * R + r;
  const int node = flat / a.G, h = hd.hk * a.G + flat % a.G;
  bool bad;
  const SeqRange sq = seq_range(a.s, hd.b, &bad);
  if (node >= sq.count) return;
  const int n = hd.follow + 1;
  // part i: slot 1 of this run, then slot 0 of the following ones
  auto part = [&](int i) {
    return a.parts + (size_t)(2 * (blockIdx.x + i) + (i == 0)) * slot_floats(R, D);
  };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, part(i)[R * D + 2 * r]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  constexpr int V = D / 32;
  float o[V], sum = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* p = part(i);
    const float2 ml = *reinterpret_cast<const float2*>(p + R * D + 2 * r);
    const float f = ml.x == -INFINITY ? 0.f : pow2i((int)fmaxf(ml.x - top, -200.f));
    sum = fmaf(ml.y, f, sum);
    float v[V];
    if (V == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + r * D + lane * 4);
      v[0] = x.x; v[1] = x.y; v[2 % V] = x.z; v[3 % V] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(p + r * D + lane * 2);
      v[0] = x.x; v[1] = x.y;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = fmaf(v[j], f, o[j]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / (sum * WSCALE);
  uint16_t* dst = a.out + (((int64_t)hd.b * a.s.N + node) * a.Hq + h) * D + lane * V;
#pragma unroll
  for (int j = 0; j < V; j += 2)
    *reinterpret_cast<uint32_t*>(dst + j) =
        sum == 0.f ? 0u : pack_bf16x2(o[j] * inv, o[j + 1] * inv);
}

static int tree_block_rows(int N, int G) {
  const int rows = N * G;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

size_t tree_attn_scratch(const strata_kv_cache_t& c, const strata_kv_seqs_t& s, int Hq) {
  const int R = tree_block_rows(s.N, Hq / c.Hkv);
  return ((ta::MAX_CTAS * sizeof(ta::Head) + 255) & ~size_t(255)) +
         (size_t)ta::MAX_CTAS * 2 * ta::slot_floats(R, c.D) * sizeof(float);
}

template <int D, int R>
static cudaError_t launch_tree(const TreeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                               cudaStream_t stream) {
  using F = ta::Cfg<D, R>;
  constexpr int SMEM = F::MISC_OFF + (int)sizeof(ta::Misc<R, F::NWG, F::C, F::STAGES>);
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(F::CTAS == 1 || 2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, R>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  int grid = sm_count() * F::CTAS;
  if (grid > ta::MAX_CTAS) grid = ta::MAX_CTAS;
  tree_attn_kernel<D, R><<<grid, F::THREADS, SMEM, stream>>>(mk, mv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, R / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_attn_combine_kernel<D, R>, a);
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
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                     ((ta::MAX_CTAS * sizeof(ta::Head) + 255) & ~size_t(255)));
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
    return R == 16 ? launch_tree<128, 16>(a, mk, mv, stream)
           : R == 32 ? launch_tree<128, 32>(a, mk, mv, stream)
                     : launch_tree<128, 64>(a, mk, mv, stream);
  return R == 16 ? launch_tree<64, 16>(a, mk, mv, stream)
         : R == 32 ? launch_tree<64, 32>(a, mk, mv, stream)
                   : launch_tree<64, 64>(a, mk, mv, stream);
}

}  // namespace strata
