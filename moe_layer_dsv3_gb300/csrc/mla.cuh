// What the latent-attention kernels share: arguments, the split of the work,
// TMEM and barrier helpers, and the join of cut sequences.
#pragma once
#include <cudaTypedefs.h>

#include "gemm.cuh"
#include "mla_split.h"
#include "prof.h"

namespace moe {
namespace mla {

constexpr int kBlock = 64;                // cached tokens a CTA holds of a tile
constexpr int kMaxHeadsCta = 64;          // heads per CTA
constexpr int kChunk = kBlock * 128;      // 64 columns of a block: [64 tokens][128 bytes]
constexpr int kChunkStep = 1024;          // bytes from one 64-column chunk of 8 tokens to the next in a ring slot
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 232448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A tile's scores may exceed the running reference by this many powers of two
// before O is rescaled: P and the sums stay far inside fp32 and bf16 range, and
// their relative precision does not depend on the reference.
constexpr float kSlack = 10.0f;
// Reference of a head that has met no score above it: any such score is far past kSlack, and P of -inf is 0.
constexpr float kNoRef = -3.0e38f;

struct MlaArgs {
  int B, H, latent, rope, page, num_pages, max_pages;
                             // (with drafted tokens: B is sequences times row groups, H the rows of a sequence)
  int G, hg;                 // head groups, heads per group
  int nm, um, nu;            // latent / 128; 128-column tiles per ring slot; slots per token tile
  int nlat, nrope;           // ring slots: latent, rope
  int nts;                   // 64-column chunks of Q held in TMEM; the others stay in shared memory
  int W;                     // workers per head group
  int piece;                 // tokens per TMA box: 64, or as many as every page holds whole
  int piece_log;             // its logarithm
  uint32_t page_mul;         // see page_div
  int page_shift;
  int row8_step;             // bytes from 8 tokens of a ring slot to the next 8
  float scale2;              // scale * log2(e)
  const __nv_bfloat16* q;
  int64_t q_b, q_h;          // strides of q, in elements
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* out;
  float* lse;                // or null
  int* status;
  int4* join;                // [W]: per worker that ends a cut sequence {b, first slot, first worker, pieces}
  // Pieces of cut sequences, two per CTA:
  float* part_o;             // [64 * latent] unnormalised output, in the register order of the epilogue
  float* part_m;             // [64] reference (log2 units)
  float* part_l;             // [64] sum of P as rounded for the product
  float* part_e;             // [64] sum of P in fp32 (for the lse)
  // Drafted tokens. The rows of a sequence are its drafted tokens' heads, token by token, in V groups of hv rows, each of which is
  // walked like a sequence of its own.
  int V, hv, heads, drafts;  // heads of a token; most drafted tokens of a sequence
  const int32_t* draft_lens; // [sequences], or null: `drafts` each
  const uint64_t* tree;      // [sequences][drafts], or null: each sees the ones before it and itself
};

// What a walked item b is: a sequence, or (TREE) a group of a sequence's rows.
struct Item {
  int seq, row0, rows;       // sequence, first row, rows
};
template <bool TREE>
__device__ __forceinline__ Item item_of(const MlaArgs& a, int b) {
  if constexpr (TREE) {
    const int s = b / a.V, r = (b - s * a.V) * a.hv;
    return {s, r, a.H - r < a.hv ? a.H - r : a.hv};
  } else {
    return {b, 0, a.H};
  }
}
// Drafted tokens of a sequence of len tokens: counts outside [0, min(drafts, len)] are clamped (and reported once).
__device__ __forceinline__ int drafts_of(const MlaArgs& a, int seq, int len, bool report) {
  const int n = a.draft_lens != nullptr ? ld_global_s32(a.draft_lens + seq) : (len > 0 ? a.drafts : 0);
  const int most = a.drafts < len ? a.drafts : len;
  if (n < 0 || n > most) {
    if (report) report_error(a.status, kErrBounds, 68);
    return n < 0 ? 0 : most;
  }
  return n;
}
// What a row sees of its sequence: all tokens before `prefix`, and of those from there on the ones whose bit is set; nothing
// if its token is not one of the sequence's drafted ones.
struct Sight {
  uint64_t mask;
  bool live;
};
__device__ __forceinline__ Sight sight_of(const MlaArgs& a, int seq, int row, int drafted) {
  const int i = row / a.heads;
  Sight s{0, i < drafted};
  if (s.live) {
    s.mask = 2ull * (1ull << i) - 1ull;                    // (i = 63: all bits)
    if (a.tree != nullptr) {
      const uint2 m = ld_global_u2(a.tree + static_cast<int64_t>(seq) * a.drafts + i);
      s.mask = (static_cast<uint64_t>(m.y) << 32 | m.x) & (2ull * (1ull << (drafted - 1)) - 1ull);
    }
  }
  return s;
}
// Bit j: the row sees token at + j, for 64 tokens.
__device__ __forceinline__ uint64_t sees(const Sight& s, int prefix, int at) {
  if (!s.live) return 0;
  const int before = prefix - at;                          // tokens of the prefix from `at` on
  if (before >= 64) return ~0ull;
  if (before >= 0) return s.mask << before | ((1ull << before) - 1ull);
  return before > -64 ? s.mask >> -before : 0;
}

// An output's sum times its row's factor, the reciprocal of the row's sum of P. (TREE) A row that sees nothing has a factor of 0 and
// is zero whatever the cache holds: its P are all 0, and the product gave NaN where a cached row is not finite.
template <bool TREE>
__device__ __forceinline__ float normed(float o, float f) {
  if constexpr (TREE) return f == 0.0f ? 0.0f : o * f;
  else return o * f;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Valid cached tokens of sequence b: lengths outside [0, capacity] are clamped (and reported once).
__device__ __forceinline__ int valid_len(const MlaArgs& a, int n, bool report) {
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page;
  if (n < 0 || n > cap) {
    if (report) report_error(a.status, kErrBounds, 60);
    return n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}
template <bool TREE>
__device__ __forceinline__ int given_len(const MlaArgs& a, int b) { return ld_global_s32(a.lens + (TREE ? b / a.V : b)); }
template <bool TREE>
__device__ __forceinline__ int seq_len(const MlaArgs& a, int b, bool report) { return valid_len(a, given_len<TREE>(a, b), report); }
template <int TILE>
__device__ __forceinline__ int tiles_of(int len) { return tiles_of(len, TILE); }

// Work of one worker: contiguous pieces of sequences, walked the same way by every role.
template <int TILE, bool TREE>
struct Walk {
  int b, t, left;            // next sequence, its next tile, tiles left in the range
  int len, nt;               // current piece's sequence: tokens, tiles
  int ahead;                 // length of sequence b as given: read a piece early, looked at when its turn comes
  int t0, n;                 // current piece: first tile, tiles
  bool first;                // the worker's first piece
  __device__ __forceinline__ bool next(const MlaArgs& a, bool& started) {
    if (left <= 0) return false;
#pragma unroll 1
    while (true) {
      if (b >= a.B) return false;
      len = valid_len(a, ahead, false);
      ahead = b + 1 < a.B ? given_len<TREE>(a, b + 1) : 0;
      nt = tiles_of<TILE>(len);
      if (t < nt) break;
      ++b;
      t = 0;
    }
    first = !started;
    started = true;
    t0 = t;
    n = left < nt - t ? left : nt - t;
    left -= n;
    return true;
  }
  __device__ __forceinline__ void done() { ++b; t = 0; }
};

// TMEM loads. 16 lanes x 8 fp32 columns per step: register 4 i + {0, 1} is
// (lane / 4, 8 i + 2 (lane % 4) + {0, 1}), register 4 i + {2, 3} the row 8 below.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Store four 8 x 8 blocks of 16-bit values: lane l gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
// The same, each block transposed.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}

// CTAs of this cluster.
__device__ __forceinline__ uint32_t num_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Stores to shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, const float2& v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// 3-D tiled load (q: columns, heads, sequences).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 4-D tiled load (cached rows: columns, 8 rows, chunks, groups of 8 rows).
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] x B[smem]^T for bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes x 32 columns from the register order of the 16x256b loads: v[2 i + e] is row lane / 4 + 8 e, columns
// 8 i + 2 (lane % 4) + {0, 1}.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint2* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0].x),
      "r"(v[0].y), "r"(v[1].x), "r"(v[1].y), "r"(v[2].x), "r"(v[2].y), "r"(v[3].x), "r"(v[3].y), "r"(v[4].x), "r"(v[4].y),
      "r"(v[5].x), "r"(v[5].y), "r"(v[6].x), "r"(v[6].y), "r"(v[7].x), "r"(v[7].y), "r"(taddr)
      : "memory");
}

// mbar_wait in few instructions. Seven warps run five different loops here, and
// with mbar_wait's unrolled polls at every wait the kernel was 150 KB of code:
// its instruction-cache misses set the pace of every warp.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, int* status, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      report_error(status, kErrTimeout, site);
      return false;
    }
  return true;
}

// bar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, int site) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, status, site));
}

// Barrier over the NT softmax threads that also gives the OR of their flags.
template <int NT>
__device__ __forceinline__ bool barrier_or(int id, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(flag)), "r"(id), "n"(NT)
      : "memory");
  return r != 0;
}

// Cache rows of the TMA boxes that one warp loads of a sequence: those of a block of 64 tokens a tile, `piece` tokens
// each. Lane l holds the first row of the l-th box from tile `tb` on, so one read of the page table serves 32 boxes, and
// the pages of the next 32 are read while these are used.
template <int TILE>
struct BoxRows {
  const int32_t* table;
  int first, len, t1;        // first token of the block in a tile; the sequence's tokens; end of the walked tiles
  int tb, row, page, rest;   // page, rest: the next batch
  __device__ __forceinline__ void fetch(const MlaArgs& a, int t) {
    const int lane = threadIdx.x & 31, box = lane << a.piece_log;   // boxes are 64 tokens of a tile after another
    const int tile = t + (box >> 6);
    const uint32_t tok = static_cast<uint32_t>(tile) * TILE + first + (box & 63);   // 2^31 or more only past the end
    const int at = page_of(tok, a.page_mul, a.page_shift);
    rest = static_cast<int>(tok) - at * a.page;
    page = tile < t1 && tok < static_cast<uint32_t>(len) ? ld_global_s32(table + at) : 0;
  }
  __device__ __forceinline__ void turn(const MlaArgs& a, int t) {
    tb = t;
    if (page >= 0 && page < a.num_pages) {
      row = page * a.page + rest;
    } else {
      report_error(a.status, kErrBounds, 62);
      row = a.num_pages * a.page;                          // past the cache: reads zeros
    }
    fetch(a, t + a.piece / 2);                             // 32 boxes are piece / 2 tiles
  }
  __device__ __forceinline__ void start(const MlaArgs& a, int b, int t0, int t1_, int first_, int len_) {
    table = a.table + static_cast<int64_t>(b) * a.max_pages;
    first = first_;
    len = len_;
    t1 = t1_;
    fetch(a, t0);
  }
  // The rows of tile t's boxes, in every lane: the issuing lane then has them in registers. At 8 boxes of 8 tokens that
  // is faster than a lane per box (83 x 4955 tokens, one head: 84.6 and 87.3 us; a shuffle before each box took 119).
  __device__ __forceinline__ void get(const MlaArgs& a, int t, int (&ys)[8]) {
    if (t - tb == a.piece / 2) turn(a, t);
#pragma unroll
    for (int p = 0; p < 8; ++p) ys[p] = __shfl_sync(0xffffffffu, row, (((t - tb) * kBlock) >> a.piece_log) + p);
  }
};

// Ring position: slot index and the parity of its current use.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) { slot = 0; phase ^= 1u; }
  }
};

// This worker's range of the tiles of all sequences, laid end to end: prefix sums
// with a run of sequences per thread, then the thread whose run holds the first
// tile finds it. Called by all NT threads; ends with a __syncthreads.
struct Range {
  int total, W, f0, f1;      // all tiles, workers that get tiles, this worker's [f0, f1)
};
template <bool TREE, int NT, int TILE, int MIN_TILES, typename Control>
__device__ __forceinline__ Range find_range(const MlaArgs& a, Control& c, int w, bool report) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = tid * per < a.B ? tid * per : a.B;
  const int b1 = b0 + per < a.B ? b0 + per : a.B;
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += tiles_of<TILE>(seq_len<TREE>(a, b, report));
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) c.scan[warp] = incl;
  __syncthreads();
  Range r;
  int before = 0;
  r.total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    if (i < warp) before += c.scan[i];
    r.total += c.scan[i];
  }
  // A piece costs a join, so no more workers than tiles / MIN_TILES (rounded up) get any; ranges differ by a tile at most.
  r.W = workers_of(r.total, a.W, MIN_TILES);
  r.f0 = w < r.W ? range_begin(r.total, w, r.W) : r.total;
  r.f1 = w < r.W ? range_begin(r.total, w + 1, r.W) : r.total;
  int at = before + incl - mine;
  if (r.f0 >= at && r.f0 < at + mine)
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int len = seq_len<TREE>(a, b, false), n = tiles_of<TILE>(len);
      if (r.f0 < at + n) {
        c.start_b = b;
        c.start_t = r.f0 - at;
        c.start_len = len;
        break;
      }
      at += n;
    }
  __syncthreads();
  return r;
}

// The worker that ends a cut sequence names its pieces for the join: {b, first slot, first worker, pieces}.
// Only its first piece can end a sequence that another worker began.
template <int TILE, typename Control>
__device__ __forceinline__ int4 join_entry(const Control& c, const Range& r, int w) {
  if (r.f1 <= r.f0 || c.start_t == 0) return make_int4(0, 0, 0, 0);
  const int s0 = r.f0 - c.start_t;                         // the sequence's first tile in the common count
  if (s0 + tiles_of<TILE>(c.start_len) > r.f1) return make_int4(0, 0, 0, 0);
  const Cut cut = cut_of(r.total, r.W, s0, w);
  return make_int4(c.start_b, cut.slot, cut.worker, cut.pieces);
}

// Joins the pieces of the sequences that the work split cut. An item is 8 heads and
// 128 latent columns of one cut sequence, for 128 threads: a warp takes 32 columns,
// in the register order in which the pieces were stored. Bound by the latency of
// dependent rounds of loads, four pieces each. So half a block takes an item with a
// short list alone, and of a long one the half blocks of a cluster take every group-th
// piece each, and their sums are added in order. What counts as short depends on how
// many items there are: where they fill the grid, two or three rounds in a row cost
// less than meeting (37 x 700 tokens, 20 heads: 22.7 us for the call with 12 pieces,
// 23.7 with 4); where they do not, the halves meet earlier (1500 tokens: 14.1, 14.5).
// The order of additions depends on the lengths only.
// A worker is one CTA of a head group with all latent columns, or (PAIR) a pair of
// CTAs, each with all heads and half of the columns.
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 2;             // blocks an SM
constexpr int kJoinFew = 4, kJoinFewFull = 12;   // pieces that a half block adds alone: in general, and if items fill the grid
// Where a sequence can have many pieces and items are few, a cluster of four blocks shares an item: 46 -> 34 us for
// 100000 tokens of 16 heads. At up to 32 pieces it costs more than it gives (8 pieces of 1500 tokens: 13.8 -> 15.1 us).
constexpr int kJoinCluster = 4;
constexpr int kJoinLong = 32;
struct JoinPart {
  float4 sum[2][128];
  float2 stat[3][4];                       // of the heads of lane % 4
};
// A thread's share of an item with M 128-column tiles: heads h (x, z) and h + 1 (y, w), four columns of a tile.
template <int M>
struct JoinSum {
  float2 top, l, le;                       // reference, sums
  float4 s[M][2];
  __device__ __forceinline__ void clear() {
    top = make_float2(kNoRef, kNoRef);
    l = le = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int m = 0; m < M; ++m) s[m][0] = s[m][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ __forceinline__ void add(float2 mk, float2 lk, float2 ek, const float4 (&v)[M][2]) {
    const float2 up = make_float2(fmaxf(top.x, mk.x), fmaxf(top.y, mk.y));
    const float gx = ex2(top.x - up.x), gy = ex2(top.y - up.y), fx = ex2(mk.x - up.x), fy = ex2(mk.y - up.y);
    top = up;
    l = make_float2(fmaf(fx, lk.x, gx * l.x), fmaf(fy, lk.y, gy * l.y));
    le = make_float2(fmaf(fx, ek.x, gx * le.x), fmaf(fy, ek.y, gy * le.y));
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float4& o = s[m][r];
        const float4& w = v[m][r];
        o = make_float4(fmaf(fx, w.x, gx * o.x), fmaf(fy, w.y, gy * o.y), fmaf(fx, w.z, gx * o.z), fmaf(fy, w.w, gy * o.w));
      }
  }
};
template <int N, bool PAIR, bool TREE>
__global__ void __launch_bounds__(kJoinThreads, 2) mla_join_kernel(const __grid_constant__ MlaArgs a) {
  constexpr int NP = N / 8, kHeads = PAIR ? 2 * kMaxHeadsCta : kMaxHeadsCta;
  __shared__ int4 list[kMaxSms];           // entries with few pieces from the front, the others from the back
  __shared__ int2 counts[kMaxSms / 32];
  extern __shared__ uint8_t smem_raw[];
  JoinPart* parts = reinterpret_cast<JoinPart*>(smem_raw);  // first block of the cluster: the other half blocks' sums
  const int tid = threadIdx.x, lane = tid & 31, half = tid >> 7, t = tid & 127, q = t >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the decode kernel's writes are visible
  // The workers that end a cut sequence: one thread looks at each.
  static_assert(kMaxSms % 32 == 0 && kMaxSms <= kJoinThreads, "one pass over the workers");
  const int4 e = tid < a.W ? a.join[tid] : make_int4(0, 0, 0, 0);
  const int per = PAIR ? 2 : a.G, cols = a.latent / (PAIR ? 256 : 128);
  const int each = per * cols * NP;                         // items of an entry
  const int items = __syncthreads_count(e.w != 0) * each, blocks = static_cast<int>(gridDim.x);
  const int alone = items > blocks ? kJoinFewFull : kJoinFew;
  const uint32_t bf = __ballot_sync(0xffffffffu, e.w != 0 && e.w <= alone);
  const uint32_t bm = __ballot_sync(0xffffffffu, e.w > alone);
  if (lane == 0 && tid < kMaxSms) counts[tid >> 5] = make_int2(__popc(bf), __popc(bm));
  __syncthreads();
  int few = 0, many = 0, few_at = __popc(bf & ((1u << lane) - 1u)), many_at = __popc(bm & ((1u << lane) - 1u));
#pragma unroll
  for (int i = 0; i < kMaxSms / 32; ++i) {
    const int2 c = counts[i];
    if (i < (tid >> 5)) {
      few_at += c.x;
      many_at += c.y;
    }
    few += c.x;
    many += c.y;
  }
  if (e.w != 0) list[e.w <= alone ? few_at : kMaxSms - 1 - many_at] = e;
  __syncthreads();

  // Pieces first, first + step, ... of the entry, several in flight.
  auto gather = [&](auto& acc, const int4& j, int g, int m, int i, int first, int step) {
    constexpr int M = sizeof(acc.s) / sizeof(acc.s[0]), kDeep = 4 / M;
    const int h = 8 * i + 2 * (lane & 3);
    acc.clear();
#pragma unroll 1
    for (int k0 = first; k0 < j.w; k0 += kDeep * step) {
      float2 mk[kDeep], lk[kDeep], ek[kDeep];
      float4 v[kDeep][M][2];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int k = k0 + u * step;
        if (k < j.w) {
          const int slot = (PAIR ? 2 * (j.z + k) : 2 * ((j.z + k) * a.G + g)) + (k == 0 ? j.y : 0);
          const int64_t part = PAIR ? 2 * slot + g : slot;
          const float4* p = reinterpret_cast<const float4*>(a.part_o) + part * (kMaxHeadsCta / 4) * a.latent +
                            (2 * m * NP + i) * 128 + t;
          mk[u] = *reinterpret_cast<const float2*>(a.part_m + slot * kHeads + h);
          lk[u] = *reinterpret_cast<const float2*>(a.part_l + slot * kHeads + h);
          ek[u] = *reinterpret_cast<const float2*>(a.part_e + slot * kHeads + h);
#pragma unroll
          for (int c = 0; c < 2 * M; ++c) v[u][c >> 1][c & 1] = p[c * NP * 128];
        }
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (k0 + u * step < j.w) acc.add(mk[u], lk[u], ek[u], v[u]);
    }
  };
  auto store = [&](const auto& acc, const int4& j, int g, int m, int i) {
    constexpr int M = sizeof(acc.s) / sizeof(acc.s[0]);
    const int h = 8 * i + 2 * (lane & 3);
    const float2 l = acc.l, le = acc.le;
    const float ix = l.x == 0.0f ? 0.0f : 1.0f / l.x, iy = l.y == 0.0f ? 0.0f : 1.0f / l.y;
    const int hg = PAIR ? h >> 6 : g, hl = PAIR ? h & 63 : h;
    const Item item = item_of<TREE>(a, j.x);
    const int head0 = hg * a.hg, nh = item.rows - head0 < a.hg ? item.rows - head0 : a.hg;
    const int64_t row = static_cast<int64_t>(item.seq) * a.H + item.row0 + head0 + hl;
    if (a.lse != nullptr && m == 0 && t < 4 && (!PAIR || g == 0)) {
      if (hl < nh) a.lse[row] = le.x == 0.0f ? -INFINITY : (acc.top.x + log2f(le.x)) * kLn2;
      if (hl + 1 < nh) a.lse[row + 1] = le.y == 0.0f ? -INFINITY : (acc.top.y + log2f(le.y)) * kLn2;
    }
    // Columns c + 8 k of head h (x) and h + 1 (y). Lanes of neighbouring columns swap: the even one
    // then stores two columns of head h, the odd one of head h + 1.
    const int odd = (lane >> 2) & 1;
    __nv_bfloat16* out =
        a.out + (row + odd) * a.latent + (PAIR ? g * (a.latent / 2) : 0) + m * 128 + q * 32 + ((lane >> 2) & ~1);
#pragma unroll
    for (int c = 0; c < M; ++c) {
      const float4 s0 = acc.s[c][0], s1 = acc.s[c][1];
      const float x[4] = {s0.x * ix, s0.z * ix, s1.x * ix, s1.z * ix}, y[4] = {s0.y * iy, s0.w * iy, s1.y * iy, s1.w * iy};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? x[k] : y[k], 4);
        const uint32_t v = odd ? pack_bf16x2(got, y[k]) : pack_bf16x2(x[k], got);
        // (a row that sees nothing: see normed, which took 0.06 us more here than one choice a store)
        if (hl + odd < nh) *reinterpret_cast<uint32_t*>(out + c * 128 + 8 * k) = TREE && (odd ? iy : ix) == 0.0f ? 0u : v;
      }
    }
  };
  // Short lists, an item to half a block; two column tiles to an item, which then reads and weighs the statistics once
  // for both, if that leaves a round of items for every half block (128 x 4096 tokens, 128 heads: 144.0 -> 141.9 us;
  // 37 x 700, 20 heads, with fewer items: 22.9 -> 23.8).
  auto short_lists = [&](auto& acc) {
    constexpr int M = sizeof(acc.s) / sizeof(acc.s[0]);
    const int of = each / M, tiles = cols / M;
    for (int it = blockIdx.x * 2 + half; it < few * of; it += gridDim.x * 2) {
      const int n = it / of, mg = (it - n * of) / NP, i = it % NP;
      const int g = mg >= tiles ? 1 : 0, m = (mg - g * tiles) * M;   // (at most two head groups or column halves)
      const int4 j = list[n];
      gather(acc, j, g, m, i, 0, 1);
      store(acc, j, g, m, i);
    }
  };
  JoinSum<1> one;
  if (items >= 4 * blocks && cols % 2 == 0) {
    JoinSum<2> two;
    short_lists(two);
  } else {
    short_lists(one);
  }
  // Long lists: the half blocks of a cluster take every group-th piece each.
  const int nc = static_cast<int>(num_ctas()), groups = 2 * nc, group = 2 * static_cast<int>(pair::cta_rank()) + half;
#pragma unroll 1
  for (int it = static_cast<int>(pair::cluster_id()); it < many * each; it += static_cast<int>(pair::num_clusters())) {
    const int e = it / each, mg = (it - e * each) / NP, i = it % NP;
    const int g = mg >= cols ? 1 : 0, m = mg - g * cols;
    const int4 j = list[kMaxSms - 1 - e];
    gather(one, j, g, m, i, group, groups);
    if (nc > 1) pair::cluster_sync();                       // the place of the sums is free
    else __syncthreads();
    if (group > 0) {
      const uint32_t to = pair::map_rank(smem_u32(&parts[group - 1]), 0);
      st_cluster(to + t * sizeof(float4), one.s[0][0]);
      st_cluster(to + (128 + t) * sizeof(float4), one.s[0][1]);
      if (t < 4) {
        const uint32_t st = to + offsetof(JoinPart, stat) + t * sizeof(float2);
        st_cluster(st, one.top);
        st_cluster(st + 4 * sizeof(float2), one.l);
        st_cluster(st + 8 * sizeof(float2), one.le);
      }
    }
    if (nc > 1) pair::cluster_sync();
    else __syncthreads();
    if (group == 0) {
      const int n = j.w < groups ? j.w : groups;
#pragma unroll 1
      for (int k = 0; k < n - 1; ++k) {
        const JoinPart& p = parts[k];
        const float4 v[1][2] = {{p.sum[0][t], p.sum[1][t]}};
        one.add(p.stat[0][lane & 3], p.stat[1][lane & 3], p.stat[2][lane & 3], v);
      }
      store(one, j, g, m, i);
    }
  }
}

// The join of a decode launch just made on the same stream. Its blocks start when the last decode CTAs leave room and
// wait for their writes on the device.
template <int N, bool PAIR, bool TREE, int TILE, int MIN_TILES>
void launch_join(const MlaArgs& a, int sms, cudaStream_t s) {
  const int64_t each = (PAIR ? 2 : a.G) * (a.latent / (PAIR ? 256 : 128)) * (N / 8);
  const int64_t most = a.B < a.W ? a.B : a.W;               // sequences that can be cut
  const int64_t tiles = ceil_div(static_cast<int64_t>(a.max_pages) * a.page, TILE);
  const int64_t slots = static_cast<int64_t>(kJoinBlocks) * sms;
  const int64_t pieces = tiles / MIN_TILES < a.W ? tiles / MIN_TILES : a.W;
  const int cluster = pieces > kJoinLong && most * each * kJoinCluster <= slots ? kJoinCluster : 1;
  const int64_t grid = most * each * cluster < slots ? most * each * cluster : slots;
  launch_cluster_after("mla_join", mla_join_kernel<N, PAIR, TREE>, dim3(static_cast<unsigned>(grid)), cluster,
                       dim3(kJoinThreads), (2 * cluster - 1) * sizeof(JoinPart), s, a);
}

// Decode with both head groups on one pair of CTAs (more than 64 heads, an even number of 128-column tiles), and
// its condition. The maps' boxes hold half of a row's latent columns.
bool pair_form(int heads, int latent);
template <bool TREE>
int run_decode_pair(MlaArgs a, const CUtensorMap& tk, const CUtensorMap& tr, const CUtensorMap& tq, int sms, cudaStream_t s);

}  // namespace mla
}  // namespace moe
