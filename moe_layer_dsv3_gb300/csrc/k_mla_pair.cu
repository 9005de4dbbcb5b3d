// Latent decode attention for more than 64 heads: one pair of CTAs (a cluster on
// two SMs) works on all heads with tcgen05 .cta_group::2.
//
// Two CTAs that each take 64 heads would both hold every cached row. The pair
// holds it once. Of a tile of 128 tokens, CTA r keeps tokens 64 r .. 64 r + 63:
//   S [128 heads x 128 tokens] = Q . K^T: CTA r has heads 64 r .. as rows of A and
//     its tokens as rows of B; it gets the scores of its own heads for all tokens.
//   O^T [latent x 128 heads] += V^T . P^T: CTA r has half r of the latent columns as
//     rows of A and P of its own heads as rows of B; it gets all heads for its columns.
// The second product needs, in each CTA, both token blocks of its own columns. One
// half of them is the CTA's own block, in place from the first product. The other
// half (the other block's rows) is loaded over the columns that the CTA held for the
// first product only, as soon as that is done. So both products find their operands
// at the same offsets in both CTAs, as the instruction wants, a tile takes
// 64 x 576 elements of shared memory per CTA, and the tensor cores run at their full
// rate (36 products of 32 clocks and 16 of 64 for 128 tokens at 512 + 64 columns;
// two single CTAs take 1920 clocks for 64 tokens).
//
// Softmax statistics belong to the CTA of the head. Each CTA tells the other, tile
// by tile, whether a reference moved; only then do the two exchange the factors of
// their heads (shared::cluster stores) and both rescale their columns of O^T.
//
// Measured at 512 + 64 columns and 128 heads: 128 sequences of about 4096 tokens
// (646 MB) in 140-144 us, of which this kernel takes 127 (0.75 of the copy rate, the
// tensor pipe 54 % active); 2 sequences of 131072 tokens in 71-73 us. The
// form of 64 heads a CTA took 200 and 106 us. Between the two limits stand the
// hand-offs of a tile: scores, softmax and second product follow one another, with
// one S buffer. In the first build, 159 us a call, leaving out the reload or the
// exponentials changed nothing, leaving out both products gave 142, and without
// products and loads 109 were left.
#include "mla.cuh"

namespace moe {

using namespace mla;

namespace {

constexpr int kThreads = 384;
constexpr int kSoft = 256;                 // softmax threads: eight warps, two per TMEM lane quarter
constexpr int kTile = 2 * kBlock;          // cached tokens per tile, a block per CTA
constexpr int kSlots = 5;                  // ring slots of half a row's latent columns: 2.5 tiles. A slot's barrier is
                                           // waited on within two tiles of its use, which this bound ensures
constexpr int kRopeSlots = 2;
constexpr int kMinTiles = 2;
constexpr int kS = 256, kQ = kS + 64;      // TMEM: O^T (128 columns per 128 of this CTA's latent ones), S, chunks of Q
constexpr int kMaxTs = (512 - kQ) / 32;
constexpr int kFloats = 2 * 128 + 3 * kSoft;   // fac, inv, and a maximum and two sums of each softmax thread

struct Smem {
  uint64_t full[kSlots], empty[kSlots];    // slots: both CTAs' data landed (even CTA) / product done
  uint64_t ropee[kRopeSlots];
  uint64_t qf, qe;                         // Q in shared memory: filled (even CTA) / free
  uint64_t sf, sd[2], se;                  // S: done, for the softmax and (by tile parity) the reload / read (even CTA)
  uint64_t vl[2];                          // reload landed, by tile parity
  uint64_t pf, pe;                         // P and reload ready (even CTA) / product done
  uint64_t of, oe;                         // O: all products of the piece done / read (even CTA)
  uint64_t gx[2], gf[2];                   // "moved" word of the other CTA, by tile parity / both CTAs' factors, alternating
  uint32_t moved[2];
  uint32_t failed;                         // a wait gave up in either CTA
  uint32_t tmem;
  int scan[kThreads / 32];
  int start_b, start_t, start_len;
};
static_assert(sizeof(Smem) <= kBarBytes, "control block");

// bar_wait with acquire at cluster scope, for barriers that the other CTA arrives on.
__device__ __forceinline__ bool bar_wait_cluster(uint64_t* bar, uint32_t parity, int* status, int site) {
  if (pair::mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!pair::mbar_try_wait_cluster(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      report_error(status, kErrTimeout, site);
      return false;
    }
  return true;
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, int* status, int site) {
  return __all_sync(0xffffffffu, bar_wait_cluster(bar, parity, status, site));
}
// Arrive on a barrier of either CTA, ordering only what this CTA's own memory holds: registers that were read from
// TMEM, or operands written here for this SM's tensor core. Each writer has passed its fence to the async proxy, and
// its warp's barrier, before the arrival leaves this SM, and the other CTA reads none of it: it only issues the product.
// A release at cluster scope took about 1000 clocks, twice a tile.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Store a word in the other CTA and count its 4 bytes on a barrier there.
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
               : "memory");
}
// Tiled loads into this CTA whose bytes count on a barrier of either CTA.
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_4d(void* dst, const CUtensorMap* m, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// 64 rows of 16 bytes to four TMEM columns, in both CTAs, each from its own shared memory: rows 0-31 to lanes 0-31
// and 64-95, rows 32-63 to lanes 32-63 and 96-127, as the pair instruction reads its 64 rows of A.
__device__ __forceinline__ void tc_cp_rows64(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.64x128b.warpx2::02_13 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

}  // namespace

// Warps: 0 loads for the first product, 11 reloads for the second; 1 and 10 (even CTA)
// issue the first and second products; 2-9 softmax and epilogue.
template <bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_pair_kernel(const __grid_constant__ CUtensorMap tma_k, const __grid_constant__ CUtensorMap tma_r,
                           const __grid_constant__ CUtensorMap tma_q, const __grid_constant__ MlaArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int hc = a.latent >> 7;                        // 64-column chunks in half of the latent columns
  const int mt = hc >> 1;                              // 128-column tiles of this CTA's half
  const int nchunk = 2 * hc + 1;
  const int nss = nchunk - a.nts;
  const int slot_bytes = hc * kChunk;
  const int nq = (a.nts + hc - 1) / hc;                // ring slots that a piece's TMEM chunks of Q pass through
  uint8_t* sq = smem;                                  // [nss][64 heads][128 bytes]
  uint8_t* sp = sq + nss * kChunk;                     // [2 token blocks][64 heads][128 bytes]: P
  uint8_t* lat = sp + 2 * kChunk;
  uint8_t* ropes = lat + kSlots * slot_bytes;
  Smem& c = *reinterpret_cast<Smem*>(ropes + kRopeSlots * kChunk);
  float* fac = reinterpret_cast<float*>(ropes + kRopeSlots * kChunk + kBarBytes);   // [128 heads] factors of a rescale
  float* inv = fac + 128;                              // [128 heads] 1 / sum
  float* xm = inv + 128;                               // [softmax threads] maxima, sums (rounded, fp32)
  float* xl = xm + kSoft;
  float* xe = xl + kSoft;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = pair::cta_rank();
  const int w = static_cast<int>(pair::cluster_id());

  if (tid == 0) {
    c.failed = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < kRopeSlots; ++i) mbar_init(&c.ropee[i], 1);
    mbar_init(&c.qf, 1);
    mbar_init(&c.qe, 1);
    mbar_init(&c.sf, 1);
    mbar_init(&c.se, 16);
    mbar_init(&c.pf, 16);
    mbar_init(&c.pe, 1);
    mbar_init(&c.of, 1);
    mbar_init(&c.oe, 16);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sd[i], 1);
      mbar_init(&c.vl[i], 1);
      mbar_init(&c.gx[i], 1);
      mbar_init(&c.gf[i], 2);
    }
    fence_barrier_init();
    fence_proxy_async();
    tma_prefetch(&tma_k);
    tma_prefetch(&tma_r);
    tma_prefetch(&tma_q);
  }
  if (warp == 1) {
    pair::tmem_alloc(&c.tmem, 512);
    pair::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");       // inputs and workspace of the stream's earlier kernels
  const Range r = find_range<TREE, kThreads, kTile, kMinTiles>(a, c, w, blockIdx.x == 0);
  tc_fence_before();
  pair::cluster_sync();                                    // both CTAs' barriers are initialised
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;");       // the join's blocks may be placed; they wait for this grid's end
  const uint32_t tmem = c.tmem;
  Walk<kTile, TREE> wk;
  wk.b = c.start_b;
  wk.t = c.start_t;
  wk.ahead = c.start_len;
  wk.left = r.f1 - r.f0;
  bool started = false, ok = true;

  // Loads of one token block (0 or 1) of a tile.
  const int pieces = kBlock >> a.piece_log, piece_step = (a.piece >> 3) * a.row8_step;
  BoxRows<kTile> rows;
  // Pieces of block blk of tile t that hold tokens.
  auto live_of = [&](int t, int blk, int len) {
    const int left = len - t * kTile - blk * kBlock;
    return left <= 0 ? 0 : (left >= kBlock ? pieces : (left + a.piece - 1) >> a.piece_log);
  };

  if (warp == 0) {
    Ring lr, rr;
    int issued = 0;
    const uint32_t full0 = pair::map_rank(smem_u32(c.full), 0);
    while (ok && wk.next(a, started)) {
      const int b = __shfl_sync(0xffffffffu, wk.b, 0), len = __shfl_sync(0xffffffffu, wk.len, 0);
      const int t0 = __shfl_sync(0xffffffffu, wk.t0, 0), t1 = t0 + __shfl_sync(0xffffffffu, wk.n, 0);
      const Item item = item_of<TREE>(a, b);
      rows.start(a, item.seq, t0, t1, rank * kBlock, len);
      // The chunks of Q for TMEM pass through ring slots ahead of the piece's tiles.
#pragma unroll 1
      for (int u = 0; u < nq && ok; ++u) {
        ok = warp_wait(&c.empty[lr.slot], lr.phase ^ 1u, a.status, 161);
        if (!ok) break;
        const int k1 = (u + 1) * hc < a.nts ? (u + 1) * hc : a.nts;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&c.full[lr.slot], 2 * (k1 - u * hc) * kChunk);
#pragma unroll 1
          for (int k = u * hc; k < k1; ++k)
            pair_load_3d(lat + lr.slot * slot_bytes + (k - u * hc) * kChunk, &tma_q, k * 64, item.row0 + rank * a.hg, item.seq, full0 + lr.slot * 8);
        }
        __syncwarp();
        lr.step(kSlots);
        ++issued;
      }
      if (!ok) break;
      rows.turn(a, t0);
#pragma unroll 1
      for (int t = t0; t < t1 && ok; ++t) {
        const int live = live_of(t, rank, len), both = live_of(t, 0, len) + live_of(t, 1, len);
        int ys[8];
        rows.get(a, t, ys);
#pragma unroll 1
        for (int u = 0; u < 2 && ok; ++u) {                // half u of the latent columns, the rope columns with half 0
          if (u == 0) ok = warp_wait(&c.ropee[rr.slot], rr.phase ^ 1u, a.status, 163);
          ok = ok && warp_wait(&c.empty[lr.slot], lr.phase ^ 1u, a.status, 163);
          if (!ok) break;
          uint8_t* dst = lat + lr.slot * slot_bytes;
          uint8_t* rdst = ropes + rr.slot * kChunk;
          const uint32_t bar = full0 + lr.slot * 8;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&c.full[lr.slot], both * a.piece * 128 * (hc + (u == 0 ? 1 : 0)));
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              if (p >= live) break;
              pair_load_4d(dst + p * piece_step, &tma_k, 0, 0, hc * u, ys[p] >> 3, bar);
              if (u == 0) pair::tma_load_2d(rdst + p * a.piece * 128, &tma_r, a.latent, ys[p], bar);
            }
          }
          __syncwarp();
          lr.step(kSlots);
          ++issued;
        }
        rr.step(kRopeSlots);
      }
      wk.done();
    }
    // Every copy into either CTA has landed before the pair may exit (the even CTA's barriers count both CTAs'
    // bytes; the final cluster barrier holds the odd CTA until then).
    if (lane == 0 && rank == 0) {
#pragma unroll 1
      for (int i = 0, n = issued < kSlots ? issued : kSlots; i < n; ++i) {
        if (--lr.slot < 0) { lr.slot = kSlots - 1; lr.phase ^= 1u; }
        ok = bar_wait(&c.full[lr.slot], lr.phase, a.status, 164) && ok;
      }
    }
  } else if (warp == 11) {
    // Reload: rows of the other CTA's block, in this CTA's half of the columns, into the slot of the half that only the
    // first product used.
    const int blk = 1 - static_cast<int>(rank);
    int slot = blk;                                        // slot of half blk of the tile
    uint32_t phase = 0, qphase = 0;                        // phase: by tile parity, bit p
    int tile = 0, issued_q = 0;
    const uint32_t qf0 = pair::map_rank(smem_u32(&c.qf), 0);
    while (ok && wk.next(a, started)) {
      const int b = __shfl_sync(0xffffffffu, wk.b, 0), len = __shfl_sync(0xffffffffu, wk.len, 0);
      const int t0 = __shfl_sync(0xffffffffu, wk.t0, 0), t1 = t0 + __shfl_sync(0xffffffffu, wk.n, 0);
      const Item item = item_of<TREE>(a, b);
      rows.start(a, item.seq, t0, t1, blk * kBlock, len);
      // Chunks of Q in shared memory, once the previous piece's products have read the last ones.
      ok = warp_wait(&c.qe, qphase ^ 1u, a.status, 167);
      if (!ok) break;
      if (elect_one()) {
        if (rank == 0) mbar_arrive_expect_tx(&c.qf, 2 * nss * kChunk);
#pragma unroll 1
        for (int k = 0; k < nss; ++k) pair_load_3d(sq + k * kChunk, &tma_q, (a.nts + k) * 64, item.row0 + rank * a.hg, item.seq, qf0);
      }
      __syncwarp();
      qphase ^= 1u;
      ++issued_q;
      slot = (slot + nq) % kSlots;
      rows.turn(a, t0);
#pragma unroll 1
      for (int t = t0; t < t1 && ok; ++t, ++tile) {
        const int live = live_of(t, blk, len);
        int ys[8];
        rows.get(a, t, ys);
        const int par = tile & 1;
        ok = warp_wait(&c.sd[par], (phase >> par) & 1u, a.status, 165);
        if (!ok) break;
        phase ^= 1u << par;
        uint8_t* dst = lat + slot * slot_bytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&c.vl[par], live * a.piece * 128 * hc);
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            if (p >= live) break;
            tma_load_4d(dst + p * piece_step, &tma_k, 0, 0, hc * rank, ys[p] >> 3, &c.vl[par]);
          }
        }
        __syncwarp();
        slot += 2;
        if (slot >= kSlots) slot -= kSlots;
      }
      wk.done();
    }
    if (lane == 0) {                                       // the last copies have landed
      if (rank == 0 && issued_q > 0) ok = bar_wait(&c.qf, qphase ^ 1u, a.status, 166) && ok;
      for (int i = 1; i <= 2 && i <= tile; ++i) {
        const int par = (tile - i) & 1;
        ok = bar_wait(&c.vl[par], ((tile - i) >> 1) & 1u, a.status, 166) && ok;
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // Issues S. See the single-CTA kernel on why the whole warp walks.
      constexpr uint32_t idesc = idesc_bf16(128, kTile);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dq0 = desc_kmajor_sw128(smem_u32(sq)), dl0 = smem_desc(smem_u32(lat), 16, a.row8_step, 2);
      const uint64_t dr0 = desc_kmajor_sw128(smem_u32(ropes));
      Ring lr, rr;
      uint32_t qphase = 0, sphase = 0;
      int tile = 0;
      while (ok && wk.next(a, started)) {
        const int n = __shfl_sync(0xffffffffu, wk.n, 0);
        // Q to TMEM, after the previous piece's products
        if (tile > 0) ok = warp_wait(&c.sd[(tile - 1) & 1], ((tile - 1) >> 1) & 1u, a.status, 174);
#pragma unroll 1
        for (int u = 0; u < nq && ok; ++u) {
          ok = warp_wait_cluster(&c.full[lr.slot], lr.phase, a.status, 176);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint64_t d0 = desc_kmajor_sw128(smem_u32(lat)) + lr.slot * (slot_bytes >> 4);
#pragma unroll 1
            for (int k = u * hc; k < (u + 1) * hc && k < a.nts; ++k)
#pragma unroll
              for (int j = 0; j < 8; ++j) tc_cp_rows64(tm + kQ + k * 32 + 4 * j, d0 + (k - u * hc) * (kChunk >> 4) + j);
            pair::tc_commit_mc(&c.empty[lr.slot], 0x3);
          }
          __syncwarp();
          lr.step(kSlots);
        }
        ok = ok && warp_wait_cluster(&c.qf, qphase, a.status, 172);
        qphase ^= 1u;
        for (int i = 0; i < n && ok; ++i, ++tile) {
          ok = warp_wait_cluster(&c.se, sphase ^ 1u, a.status, 173);
          sphase ^= 1u;
#pragma unroll 1
          for (int u = 0; u < 2 && ok; ++u) {
            ok = warp_wait_cluster(&c.full[lr.slot], lr.phase, a.status, 175);
            tc_fence_after();
            if (ok && elect_one()) {
              auto chunk = [&](int k, uint64_t dk, bool fresh) {
                if (k < a.nts) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) mma2_ts(tm + kS, tm + kQ + k * 32 + kk * 8, dk + kk * 2, idesc, !fresh || kk > 0);
                } else {
                  const uint64_t dq = dq0 + (k - a.nts) * (kChunk >> 4);
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) mma2_ss(tm + kS, dq + kk * 2, dk + kk * 2, idesc, !fresh || kk > 0);
                }
              };
              const uint64_t dl = dl0 + lr.slot * (slot_bytes >> 4);
#pragma unroll 1
              for (int k = 0; k < hc; ++k) chunk(u * hc + k, dl + k * (kChunkStep >> 4), u + k == 0);
              if (u == 0) {
                chunk(nchunk - 1, dr0 + rr.slot * (kChunk >> 4), false);
                pair::tc_commit_mc(&c.ropee[rr.slot], 0x3);
              } else {
                pair::tc_commit_mc(&c.sf, 0x3);
                pair::tc_commit_mc(&c.sd[tile & 1], 0x3);
                if (i == n - 1) pair::tc_commit_mc(&c.qe, 0x3);
              }
            }
            __syncwarp();
            lr.step(kSlots);
          }
          rr.step(kRopeSlots);
        }
        wk.done();
      }
    }
  } else if (warp == 10) {
    if (rank == 0) {
      // Issues O^T.
      constexpr uint32_t idesc = idesc_bf16(256, 128) | (1u << 15);   // A (V^T) is MN-major
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dp0 = desc_kmajor_sw128(smem_u32(sp)), dv0 = smem_desc(smem_u32(lat), kChunkStep, a.row8_step, 2);
      if (lane == 0) a.join[w] = join_entry<kTile>(c, r, w);
      Ring lr;
      uint32_t pphase = 0, ophase = 0;
      while (ok && wk.next(a, started)) {
        const int n = __shfl_sync(0xffffffffu, wk.n, 0);
        for (int u = 0; u < nq; ++u) lr.step(kSlots);
        ok = warp_wait_cluster(&c.oe, ophase ^ 1u, a.status, 171);    // the previous piece's O has been read
        ophase ^= 1u;
        for (int i = 0; i < n && ok; ++i) {
          ok = warp_wait_cluster(&c.pf, pphase, a.status, 170);
          if (!ok) break;
          pphase ^= 1u;
          tc_fence_after();
          if (elect_one()) {
            int slot = lr.slot;
#pragma unroll 1
            for (int blk = 0; blk < 2; ++blk) {            // token block; half blk's slot holds its rows by now
              uint64_t dv = dv0 + slot * (slot_bytes >> 4);
              uint32_t d = tm;
#pragma unroll 1
              for (int m = 0; m < mt; ++m, dv += kChunkStep >> 3, d += 128)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma2_ss(d, dv + kk * (a.row8_step >> 3), dp0 + blk * (kChunk >> 4) + kk * 2, idesc, i > 0 || blk + kk > 0);
              pair::tc_commit_mc(&c.empty[slot], 0x3);
              if (++slot == kSlots) slot = 0;
            }
            pair::tc_commit_mc(&c.pe, 0x3);
            if (i == n - 1) pair::tc_commit_mc(&c.of, 0x3);
          }
          __syncwarp();
          lr.step(kSlots);
          lr.step(kSlots);
        }
        wk.done();
      }
    }
  } else {
    const int q = warp & 3, sub = (warp - 2) >> 2;
    const int st = tid - 64;                               // softmax thread
    const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
    const int blk = q >> 1;                                // this thread's tokens: 32 sub .. of this block
    const int hl = (q & 1) * 32 + lane;                    // and head of the CTA
    const int head0 = static_cast<int>(rank) * a.hg;       // first head of the CTA
    // heads that a CTA whose first is h0 has of an item (a sequence's last row group may be small)
    auto heads_of = [&](const Item& it, int h0) {
      const int n = it.rows - h0 < a.hg ? it.rows - h0 : a.hg;
      return TREE && n < 0 ? 0 : n;
    };
    const int tl = sub * 128 + q * 32 + lane;              // a head's four threads: tl with bits 6 and 7 free
    const bool first = blk == 0 && sub == 0;               // the one that speaks for the head
    const uint32_t se0 = pair::map_rank(smem_u32(&c.se), 0), pf0 = pair::map_rank(smem_u32(&c.pf), 0);
    const uint32_t oe0 = pair::map_rank(smem_u32(&c.oe), 0);
    const uint32_t other = rank ^ 1u;
    const uint32_t gx_o = pair::map_rank(smem_u32(c.gx), other), gf_o = pair::map_rank(smem_u32(c.gf), other);
    const uint32_t moved_o = pair::map_rank(smem_u32(c.moved), other);
    const uint32_t fac_o = pair::map_rank(smem_u32(fac), other), inv_o = pair::map_rank(smem_u32(inv), other);
    uint32_t pphase = 0, ophase = 0, sphase = 0;
    int swaps = 0;                                         // exchanges so far
    Ring lr;                                               // ring position of the current tile
    int tile = 0;
    // After a wait that gave up, these threads stop waiting but keep walking, so that all of them meet at every
    // CTA barrier and the kernel ends. A thread that gave up may read a word that the other CTA is still to write.
    // So nothing between the CTAs decides whether a CTA barrier is met: only `grow`, which a barrier hands out, and
    // the walk do. A thread that gave up sends nothing and arrives on no memory barrier: no barrier gets more arrivals
    // than it expects, no product starts on what is not there, and the others' waits run out too.
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
      if (ok) ok = bar_wait_cluster(bar, parity, a.status, site);
    };
    // One arrival of this warp on a barrier of the even CTA.
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive_remote(bar);
    };
    // A factor per head into both CTAs' arrays (the same place in both), complete in this CTA at the end. Two warps
    // speak for the 64 heads; each arrives after its own stores and expects 32 words of the other CTA.
    auto exchange = [&](float* arr, uint32_t arr_o, float v) {
      uint64_t* bar = &c.gf[swaps & 1];
      if (first) {
        if (ok) {
          arr[rank * 64 + hl] = v;
          st_async(arr_o + (rank * 64 + hl) * 4, __float_as_uint(v), gf_o + (swaps & 1) * 8);
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive_expect_tx(bar, 32 * 4);
      }
      wait(bar, (swaps >> 1) & 1u, 184);
      ++swaps;
    };
    while (wk.next(a, started)) {
      for (int u = 0; u < nq; ++u) lr.step(kSlots);
      float ref = kNoRef, l = 0.0f, le = 0.0f;
      const Item item = item_of<TREE>(a, wk.b);
      const int nh = heads_of(item, head0);
      Sight sight;                                         // of this thread's row
      int prefix = 0;
      if constexpr (TREE) {
        const int drafted = drafts_of(a, item.seq, wk.len, st == 0);
        prefix = wk.len - drafted;
        sight = sight_of(a, item.seq, item.row0 + head0 + hl, drafted);
      }
      // P of the scores x (a head, 32 tokens), packed, and its sums; the largest score above the reference.
      auto take = [&](const uint32_t* x, uint32_t* p, float& ls, float& les) {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float rs[4] = {}, es[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y0 = fmaf(__uint_as_float(x[2 * i]), a.scale2, -ref), y1 = fmaf(__uint_as_float(x[2 * i + 1]), a.scale2, -ref);
          top[i & 3] = fmaxf(top[i & 3], fmaxf(y0, y1));
          const float p0 = ex2(y0), p1 = ex2(y1);
          es[i & 3] += p0 + p1;
          p[i] = pack_bf16x2(p0, p1);
          rs[i & 3] += __uint_as_float(p[i] << 16) + __uint_as_float(p[i] & 0xFFFF0000u);
        }
        ls = (rs[0] + rs[1]) + (rs[2] + rs[3]);
        les = (es[0] + es[1]) + (es[2] + es[3]);
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      };
#pragma unroll 1
      for (int ti = 0; ti < wk.n; ++ti, ++tile) {
        const int valid = wk.len - (wk.t0 + ti) * kTile;   // tokens of the tile (>= 128: all)
        const int par = tile & 1;
        wait(&c.sf, sphase, 180);
        sphase ^= 1u;
        tc_fence_after();
        uint32_t x[32], p[16];
        tmem_ld32_async(tmem + tlane + kS + sub * 32, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) reg_fence(x[i]);
        tc_fence_before();
        arrive(se0);
        if constexpr (TREE) {
          const int at = (wk.t0 + ti) * kTile + blk * kBlock + sub * 32;
          if (prefix - at < 32 || !sight.live) {
            const uint32_t see = static_cast<uint32_t>(sees(sight, prefix, at));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((see >> i) & 1u)) x[i] = __float_as_uint(-INFINITY);
          }
        } else if (valid < kTile) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (blk * kBlock + sub * 32 + i >= valid) x[i] = __float_as_uint(-INFINITY);
        }
        float ls, les;
        const float over = take(x, p, ls, les);
        const bool grow = barrier_or<kSoft>(2, over > kSlack);
        // O is rescaled only when a score of the tile passes kSlack in either CTA.
        if (st == 0 && ok) {
          mbar_arrive_expect_tx(&c.gx[par], 4);            // the other CTA's word
          st_async(moved_o + par * 4, grow ? 1u : 0u, gx_o + par * 8);
        }
        float corr = 1.0f;
        if (grow) {
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) m = fmaxf(m, __uint_as_float(x[i]));
          xm[tl] = m * a.scale2;
          named_barrier(3, kSoft);
          m = fmaxf(fmaxf(fmaxf(xm[tl], xm[tl ^ 64]), fmaxf(xm[tl ^ 128], xm[tl ^ 192])), ref);
          corr = ex2(ref - m);                             // 0 from kNoRef to a score
          l *= corr;
          le *= corr;
          ref = m;
          take(x, p, ls, les);
        }
        l += ls;
        le += les;
        // The previous tile's product is done: P is free and O stands still.
        if (tile > 0) {
          wait(&c.pe, pphase, 181);
          pphase ^= 1u;
        }
        wait(&c.gx[par], (tile >> 1) & 1u, 185);
        const bool theirs = *reinterpret_cast<volatile uint32_t*>(&c.moved[par]) != 0u;
        if (__any_sync(0xffffffffu, grow || theirs) && ti > 0) {       // one answer a warp, also after a wait that gave up
          exchange(fac, fac_o, corr);
          tc_fence_after();
#pragma unroll 1
          for (int hc16 = sub * 64 * mt; hc16 < (sub + 1) * 64 * mt; hc16 += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(tmem + tlane + hc16, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              reg_fence(o[j]);
              o[j] = __float_as_uint(__uint_as_float(o[j]) * fac[(hc16 & 127) + j]);
            }
            tmem_st_32x32b_x16(tmem + tlane + hc16, o);
          }
          tmem_wait_st();
        }
        uint8_t* prow = sp + blk * kChunk + hl * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(prow + (((4 * sub + k) ^ (hl & 7)) << 4)) =
              make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
        // The reload has landed (its bytes are the second product's operand).
        wait(&c.vl[par], (tile >> 1) & 1u, 182);
        if (valid < kTile) {
          // Rows past the sequence's end have to be 0 for the second product. Block u's rows are in half u's slot.
          int slot = lr.slot;
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const int first = valid - u * kBlock < 0 ? 0 : (valid - u * kBlock > kBlock ? kBlock : valid - u * kBlock);
            const int per = (kBlock - first) * 8;          // 16-byte words to clear in a chunk
            uint8_t* v = lat + slot * slot_bytes;
#pragma unroll 1
            for (int i = st; i < hc * per; i += kSoft) {
              const int k = i / per, row = first + (i - k * per) / 8;
              *reinterpret_cast<uint4*>(v + k * kChunkStep + (row >> 3) * a.row8_step + (row & 7) * 128 + (i & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            if (++slot == kSlots) slot = 0;
          }
        }
        lr.step(kSlots);
        lr.step(kSlots);
        fence_proxy_async();
        tc_fence_before();
        arrive(pf0);
      }
      // ---- epilogue of the piece
      const bool whole = wk.n == wk.nt;
      const int slot = 2 * w + (wk.first ? 0 : 1);
      xl[tl] = l;
      xe[tl] = le;
      named_barrier(3, kSoft);
      float norm = 0.0f;
      if (first) {
        const float v = (l + xl[tl + 64]) + (xl[tl + 128] + xl[tl + 192]);
        const float ve = (le + xe[tl + 64]) + (xe[tl + 128] + xe[tl + 192]);
        const int h = static_cast<int>(rank) * 64 + hl;
        norm = v == 0.0f ? 0.0f : 1.0f / v;
        if (whole) {
          if (a.lse != nullptr && hl < nh)
            a.lse[static_cast<int64_t>(item.seq) * a.H + item.row0 + head0 + hl] = ve == 0.0f ? -INFINITY : (ref + log2f(ve)) * kLn2;
        } else {
          a.part_m[slot * 128 + h] = ref;
          a.part_l[slot * 128 + h] = v;
          a.part_e[slot * 128 + h] = ve;
        }
      }
      if (whole) exchange(inv, inv_o, norm);
      wait(&c.of, ophase, 183);
      ophase ^= 1u;
      tc_fence_after();
      uint8_t* stage = sp + (sub * 4 + q) * 2048;          // [64 heads][16 columns] of this warp, over P
      const int grp = sub;                                 // a warp takes the heads of one CTA, and its lanes' 32 columns
      float4* part = reinterpret_cast<float4*>(a.part_o + static_cast<int64_t>(2 * slot + rank) * kMaxHeadsCta * a.latent) +
                     q * 32 + lane;
#pragma unroll 1
      for (int mh = 0; mh < 2 * mt; ++mh) {
        uint32_t o[32];
        tmem_ld_16x256b_x8(tmem + tlane + (static_cast<uint32_t>(mh & 1) << 20) + (mh >> 1) * 128 + grp * 64, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) reg_fence(o[i]);
        if (whole) {
          const float2* f = reinterpret_cast<const float2*>(inv) + grp * 32 + (lane & 3);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 f0 = f[4 * i], f1 = f[4 * i + 4];
            const int h = 8 * (i + (lane >> 4)) + (lane & 7);
            stmatrix_x4_trans(smem_u32(stage) + h * 32 + ((((lane >> 3) ^ (h >> 2)) & 1) << 4),
                              pack_bf16x2(normed<TREE>(__uint_as_float(o[4 * i]), f0.x), normed<TREE>(__uint_as_float(o[4 * i + 1]), f0.y)),
                              pack_bf16x2(normed<TREE>(__uint_as_float(o[4 * i + 2]), f0.x), normed<TREE>(__uint_as_float(o[4 * i + 3]), f0.y)),
                              pack_bf16x2(normed<TREE>(__uint_as_float(o[4 * i + 4]), f1.x), normed<TREE>(__uint_as_float(o[4 * i + 5]), f1.y)),
                              pack_bf16x2(normed<TREE>(__uint_as_float(o[4 * i + 6]), f1.x), normed<TREE>(__uint_as_float(o[4 * i + 7]), f1.y)));
          }
          __syncwarp();
          const int g0 = grp * a.hg, gn = heads_of(item, g0);
          __nv_bfloat16* out = a.out + (static_cast<int64_t>(item.seq) * a.H + item.row0 + g0) * a.latent + rank * (a.latent / 2) +
                               (mh >> 1) * 128 + q * 32 + (mh & 1) * 16;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int h = 16 * k + (lane >> 1), ch = lane & 1;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + h * 32 + (((ch ^ (h >> 2)) & 1) << 4));
            if (h < gn) *reinterpret_cast<uint4*>(out + h * a.latent + ch * 8) = v;
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part[(mh * 16 + grp * 8 + i) * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                             __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
      tc_fence_before();
      arrive(oe0);
      wk.done();
    }
    // Sequences without tokens: zero rows, lse = -inf.
#pragma unroll 1
    for (int b = w; b < a.B; b += a.W) {
      if (seq_len<TREE>(a, b, false) > 0) continue;
      const Item item = item_of<TREE>(a, b);
      const int nh = heads_of(item, head0);
      const int64_t at = static_cast<int64_t>(item.seq) * a.H + item.row0 + head0;
      __nv_bfloat16* out = a.out + at * a.latent;
#pragma unroll 1
      for (int i = st; i < nh * a.latent / 8; i += kSoft) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse != nullptr)
#pragma unroll 1
        for (int i = st; i < nh; i += kSoft) a.lse[at + i] = -INFINITY;
      if constexpr (TREE) {
        if (st == 0) drafts_of(a, item.seq, 0, true);
      }
    }
  }
  // Neither CTA leaves (or frees TMEM) while the other may still use its shared memory, its TMEM or its barriers. After
  // a wait that gave up, both stay until what was under way without anybody waiting for it has landed.
  if (!ok) {
    st_cluster(pair::map_rank(smem_u32(&c.failed), 0), 1u);
    st_cluster(pair::map_rank(smem_u32(&c.failed), 1), 1u);
  }
  tc_fence_before();
  __syncwarp();
  pair::cluster_sync();
  if (*reinterpret_cast<volatile uint32_t*>(&c.failed) != 0u) {
    drain_pause();
    __syncwarp();
    pair::cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    pair::tmem_dealloc(tmem, 512);
  }
}

namespace mla {

bool pair_form(int heads, int latent) { return heads > kMaxHeadsCta && latent % 256 == 0; }

template <bool TREE>
int run_decode_pair(MlaArgs a, const CUtensorMap& tk, const CUtensorMap& tr, const CUtensorMap& tq, int sms, cudaStream_t s) {
  static DevOnce once;
  if (!once.ready([] {
        return cudaFuncSetAttribute(mla_decode_pair_kernel<TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
      }))
    return MOE_ERR_CUDA;
  const int hc = a.latent / 128, nchunk = 2 * hc + 1;
  a.W = sms / 2;
  a.hg = static_cast<int>(ceil_div(TREE ? a.hv : a.H, 2));
  // a rope part under 64 columns is zero-filled by its TMA box only, so it stays in shared memory
  a.nts = kMaxTs < nchunk - 1 ? kMaxTs : (a.rope == 64 && kMaxTs >= nchunk ? nchunk : nchunk - 1);
  const size_t smem = 1024 + static_cast<size_t>(nchunk - a.nts + 2 + kSlots * hc + kRopeSlots) * kChunk + kBarBytes +
                      kFloats * sizeof(float);
  launch_cluster_after("mla_decode_pair", mla_decode_pair_kernel<TREE>, dim3(static_cast<unsigned>(2 * a.W)), 2, dim3(kThreads),
                       smem, s, tk, tr, tq, a);
  if (call_error() != cudaSuccess) return MOE_ERR_CUDA;
  launch_join<128, true, TREE, kTile, kMinTiles>(a, sms, s);
  return MOE_OK;
}
template int run_decode_pair<false>(MlaArgs, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
template int run_decode_pair<true>(MlaArgs, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

}  // namespace mla

}  // namespace moe
