// Latent attention over a paged cache: the write of new tokens and the
// attention of one new token a sequence (absorbed form).
//
// The cache holds one row a token, [latent | rope], shared by all heads: keys
// are whole rows, values their first `latent` columns.
//
//   s_j = scale q . k_j   (j < len),   out = sum_j softmax(s)_j k_j[0 : latent]
//
// One cached token costs 2 (latent + rope) bytes of HBM and, with H heads,
// 2 H (2 latent + rope) products: at 512 + 64 columns and 128 heads that is
// 242 flop/byte, where HBM and the tensor pipe are both close to their
// limits; with fewer heads HBM alone bounds the kernel. So the cache is read
// once per group of up to 64 heads, straight into the shared memory that both
// products read.
//
//   S [64 heads x 64 tokens]   = Q . K^T    (rows past the group's heads are not used)
//   O^T [latent x N heads]    += V^T . P^T   (N = the group's heads, rounded up to 16)
// The second product runs transposed, with latent columns as its 128-row
// operand and the heads as the narrow one: the output of 64 heads then takes
// half of TMEM, a few heads cost little, and V^T is the K tile itself, read as
// an MN-major operand.
//
// Work is split by tiles of 64 tokens: the tiles of all sequences, one after
// another, are cut into equal contiguous ranges, one per worker (CTA; with two
// head groups, one worker per group). A sequence inside one range is finished
// there; one that is cut leaves a partial (unnormalised O, maximum, sum) per
// piece in the workspace, and the join kernel adds the pieces in order. Every
// worker finds its range from seq_lens on the device, so the host never reads
// lengths and the call can be captured in a graph.
//
// P is rounded to bf16: the product takes operands of one type, and V is the bf16
// cache. A second bf16 part of P would double the second product's time and P's
// place in shared memory. With the sums taken of the rounded values the output's
// error against 64 bits is 0.0018 to 0.0020 (relative norm) where fp32 P gives 0.0016
// to 0.0017, nearly all of it the output's own rounding. The lse takes fp32 sums.
//
// Measured: 64 sequences of about 16384 tokens with 16 heads (1.15 GB) in 175-178 us,
// 0.95 of the copy rate; 37 of about 700 tokens with 20 heads in 21.2 us, of which
// the cache's bytes need 4.4: there the kernels' starts, a piece's Q and output, and
// the join's rounds of loads are what is left. More than 64 heads run here only where
// the pair form does not take them (latent columns not a multiple of 256): each of two
// head groups then reads the cache.
//
// With drafted tokens (TREE) a sequence's rows are the heads of all its drafted tokens, in groups of up to 64 (128 on
// pairs) that are walked like sequences; Q, output and statistics of a group lie one after another, so only the place
// of an item and the scores' masks differ (mla.cuh). 32 x ~4096 tokens with 1024 rows: 229 us for 0.26 TFLOP, 0.59 of the
// measured bf16 rate.
#include <cmath>

#include "mla.cuh"

namespace moe {

using namespace mla;

namespace {

constexpr int kThreads = 224;
constexpr int kTile = kBlock;             // cached tokens per tile
constexpr int kAppendBlocks = 3;          // resident blocks an SM: 32768 tokens in 17.2 us; 4 spill more and take 20.7
constexpr int kMaxLatSlots = 12;
constexpr int kMaxRopeSlots = kMaxLatSlots;
constexpr int kMinTiles = 3;              // fewest tiles of a worker: 1500 tokens, and 37 sequences of about 700, took
                                          // 12.9 and 22.2 us at 2, 13.3 and 21.3 at 3, 14.5 and 21.9 at 4

struct Smem {
  uint64_t latf[kMaxLatSlots], late[kMaxLatSlots];     // latent slots: filled / free
  uint64_t ropee[kMaxRopeSlots];                       // (a tile's rope columns arrive with its first latent slot)
  uint64_t qf, qe;                                      // Q of the piece: filled (both parts) / free
  uint64_t sf[2], se[2];                                // S buffers: products done / read
  uint64_t pf, pe;                                      // P: written / its product done
  uint64_t of, oe;                                      // O: all products of the piece done / read
  uint32_t tmem;
  int scan[kThreads / 32];
  int start_b, start_t, start_len;
};
static_assert(sizeof(Smem) <= kBarBytes, "control block");

// TMEM columns: O^T (a block of N per 128 latent columns), the S buffers, then as
// many chunks of Q (32 columns each) as fit. Q in TMEM leaves shared memory to
// the ring, and the product then reads only the cached rows from there. 64 heads
// leave room for one S buffer: the next product waits until the last scores are
// in registers, while the other product runs.
template <int N>
struct Plan {
  static constexpr int kBufs = N > 48 ? 1 : 2;
  static constexpr int kS = 4 * N;
  static constexpr int kQ = kS + kBufs * kTile;
  static constexpr int kMaxTs = (512 - kQ) / 32 < 9 ? (512 - kQ) / 32 : 9;
};

}  // namespace

// Threads: warp 0 loads (TMA), warps 1 and 6 issue the MMAs of S and O^T, warps
// 2-5 do the softmax and the epilogue (TMEM lane quarter warp % 4).
template <int N, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap tma_k, const __grid_constant__ CUtensorMap tma_r,
                      const __grid_constant__ CUtensorMap tma_q, const __grid_constant__ MlaArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nm = a.nm, nchunk = 2 * nm + 1;            // 64-column chunks of a row: latent, then rope
  const int slot_bytes = a.um * 2 * kChunk;
  const int nss = nchunk - a.nts;                      // chunks of Q in shared memory
  uint8_t* sq = smem;                                  // [nss][N][128 bytes]; the product's 64 rows of a chunk
                                                       // run on into what follows when N is less
  uint8_t* sp = sq + nss * N * 128;                 // [N][128 bytes]: P, 64 tokens a head
  uint8_t* lat = sp + N * 128;
  uint8_t* ropes = lat + a.nlat * slot_bytes;
  Smem& c = *reinterpret_cast<Smem*>(ropes + a.nrope * kChunk);
  float* fac = reinterpret_cast<float*>(ropes + a.nrope * kChunk + kBarBytes);   // [64] a factor per head
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.G, w = blockIdx.x / a.G;
  using P = Plan<N>;

  if (tid == 0) {
    for (int i = 0; i < a.nlat; ++i) {
      mbar_init(&c.latf[i], 1);
      mbar_init(&c.late[i], 1);
    }
    for (int i = 0; i < a.nrope; ++i) mbar_init(&c.ropee[i], 1);
    mbar_init(&c.qf, 129);
    mbar_init(&c.qe, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sf[i], 1);
      mbar_init(&c.se[i], 128);
    }
    mbar_init(&c.pf, 128);
    mbar_init(&c.pe, 1);
    mbar_init(&c.of, 1);
    mbar_init(&c.oe, 128);
    fence_barrier_init();
    fence_proxy_async();
    tma_prefetch(&tma_k);
    tma_prefetch(&tma_r);
    tma_prefetch(&tma_q);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");       // inputs and workspace of the stream's earlier kernels
  tc_fence_before();
  const Range r = find_range<TREE, kThreads, kTile, kMinTiles>(a, c, w, blockIdx.x == 0);
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;");       // the join's blocks may be placed; they wait for this grid's end
  const uint32_t tmem = c.tmem;
  Walk<kTile, TREE> wk;
  wk.b = c.start_b;
  wk.t = c.start_t;
  wk.ahead = c.start_len;
  wk.left = r.f1 - r.f0;
  bool started = false, ok = true;

  if (warp == 0) {
    // Loads. Like the MMA warps, the whole warp walks and one elected lane issues
    // from warp-uniform registers (a box took about 250 clocks to issue from a
    // divergent lane, and this warp then set the pace).
    Ring lr, rr;
    uint32_t qphase = 0;
    int issued = 0, issued_q = 0;
    BoxRows<kTile> rows;
    const int pieces = kTile >> a.piece_log;
    const int piece_step = (a.piece >> 3) * a.row8_step;
    const int h0 = g * a.hg;
    while (ok && wk.next(a, started)) {
      const int b = __shfl_sync(0xffffffffu, wk.b, 0), len = __shfl_sync(0xffffffffu, wk.len, 0);
      const int t0 = __shfl_sync(0xffffffffu, wk.t0, 0), t1 = t0 + __shfl_sync(0xffffffffu, wk.n, 0);
      const Item item = item_of<TREE>(a, b);
      rows.start(a, item.seq, t0, t1, 0, len);
      // Q of this sequence and head group, once the previous piece's products have read the last one.
      ok = warp_wait(&c.qe, qphase ^ 1u, a.status, 61);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&c.qf, nss * N * 128);
#pragma unroll 1
        for (int k = 0; k < nss; ++k) tma_load_3d(sq + k * N * 128, &tma_q, (a.nts + k) * 64, item.row0 + h0, item.seq, &c.qf);
      }
      __syncwarp();
      qphase ^= 1u;
      ++issued_q;
      rows.turn(a, t0);
#pragma unroll 1
      for (int t = t0; t < t1 && ok; ++t) {
        const int left = len - t * kTile;
        const int live = left >= kTile ? pieces : (left + a.piece - 1) >> a.piece_log;   // pieces with tokens
        int ys[8];
        rows.get(a, t, ys);
#pragma unroll 1
        for (int u = 0; u < a.nu && ok; ++u) {           // a slot of latent columns, the rope columns with the first
          if (u == 0) ok = warp_wait(&c.ropee[rr.slot], rr.phase ^ 1u, a.status, 63);
          ok = ok && warp_wait(&c.late[lr.slot], lr.phase ^ 1u, a.status, 63);
          if (!ok) break;
          uint64_t* full = &c.latf[lr.slot];
          uint8_t* dst = lat + lr.slot * slot_bytes;
          uint8_t* rdst = ropes + rr.slot * kChunk;
          if (elect_one()) {
            mbar_arrive_expect_tx(full, live * a.piece * 128 * (2 * a.um + (u == 0 ? 1 : 0)));
            // A box holds all chunks of the slot for the tokens of one piece.
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              if (p >= live) break;
              tma_load_4d(dst + p * piece_step, &tma_k, 0, 0, 2 * a.um * u, ys[p] >> 3, full);
              if (u == 0) tma_load_2d(rdst + p * a.piece * 128, &tma_r, a.latent, ys[p], full);
            }
          }
          __syncwarp();
          lr.step(a.nlat);
          ++issued;
        }
        rr.step(a.nrope);
      }
      wk.done();
    }
    // Every copy this CTA started has landed before its shared memory is released.
    if (lane == 0) {
#pragma unroll 1
      for (int i = 0, n = issued < a.nlat ? issued : a.nlat; i < n; ++i) {
        if (--lr.slot < 0) { lr.slot = a.nlat - 1; lr.phase ^= 1u; }
        ok = bar_wait(&c.latf[lr.slot], lr.phase, a.status, 64) && ok;
      }
      if (issued_q > 0) ok = bar_wait(&c.qf, qphase ^ 1u, a.status, 64) && ok;
    }
  } else if (warp == 1) {
    // Issues S. The whole warp walks the tiles and waits, and one elected lane
    // issues; with every wait's result and every length taken warp-wide, the
    // descriptors stay in uniform registers. That counts: an MMA of these sizes
    // takes 23 to 48 clocks, and issuing one from a divergent branch took 100.
    constexpr uint32_t idesc_s = idesc_bf16(64, kTile);
    constexpr uint32_t kChunkUnits = kChunk >> 4;         // descriptor address units
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq0 = desc_kmajor_sw128(smem_u32(sq)), dl0 = smem_desc(smem_u32(lat), 16, a.row8_step, 2);
    const uint64_t dr0 = desc_kmajor_sw128(smem_u32(ropes));
    Ring lr, rr;
    uint32_t qphase = 0, sbuf = 0, sphase = 0;
    while (ok && wk.next(a, started)) {
      const int n = __shfl_sync(0xffffffffu, wk.n, 0);
      ok = warp_wait(&c.qf, qphase, a.status, 72);
      qphase ^= 1u;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        ok = warp_wait(&c.se[sbuf], sphase ^ 1u, a.status, 73);
        const uint32_t d = tm + P::kS + sbuf * kTile;
#pragma unroll 1
        for (int u = 0; u < a.nu && ok; ++u) {
          ok = warp_wait(&c.latf[lr.slot], lr.phase, a.status, 75);
          tc_fence_after();
          if (ok && elect_one()) {
            // one chunk of 64 columns: A from TMEM or shared memory
            auto chunk = [&](int k, uint64_t dk, bool fresh) {
              if (k < a.nts) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) tc_mma_bf16_ts(d, tm + P::kQ + k * 32 + kk * 8, dk + kk * 2, idesc_s, !fresh || kk > 0);
              } else {
                const uint64_t dq = dq0 + (k - a.nts) * (N * 8);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) tc_mma_bf16(d, dq + kk * 2, dk + kk * 2, idesc_s, !fresh || kk > 0);
              }
            };
            const uint64_t dl = dl0 + lr.slot * (a.um * 2 * kChunkUnits);
#pragma unroll 1
            for (int k = 0; k < 2 * a.um; ++k) chunk(u * a.um * 2 + k, dl + k * (kChunkStep >> 4), u + k == 0);
            if (u == 0) {
              chunk(nchunk - 1, dr0 + rr.slot * kChunkUnits, false);
              tc_commit(&c.ropee[rr.slot]);
            }
            if (u == a.nu - 1) {
              tc_commit(&c.sf[sbuf]);
              if (i == n - 1) tc_commit(&c.qe);
            }
          }
          __syncwarp();
          lr.step(a.nlat);
        }
        if (!ok) break;
        rr.step(a.nrope);
        if (++sbuf == P::kBufs) {
          sbuf = 0;
          sphase ^= 1u;
        }
      }
      wk.done();
    }
  } else if (warp == 6) {
    // Issues O^T, in a warp of its own: it then never waits behind the next tile's data.
    constexpr uint32_t idesc_o = idesc_bf16(128, N) | (1u << 15);   // A (V^T) is MN-major
    constexpr uint32_t kChunkUnits = kChunk >> 4;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dp0 = desc_kmajor_sw128(smem_u32(sp)), dv0 = smem_desc(smem_u32(lat), kChunkStep, a.row8_step, 2);
    if (lane == 0 && g == 0) a.join[w] = join_entry<kTile>(c, r, w);
    Ring lr;
    uint32_t pphase = 0, ophase = 0;
    while (ok && wk.next(a, started)) {
      const int n = __shfl_sync(0xffffffffu, wk.n, 0);
      ok = warp_wait(&c.oe, ophase ^ 1u, a.status, 71);             // the previous piece's O has been read
      ophase ^= 1u;
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        ok = warp_wait(&c.pf, pphase, a.status, 70);                // P is written, so the tile's data is there
        if (!ok) break;
        pphase ^= 1u;
        tc_fence_after();
        if (elect_one()) {
          uint32_t d = tm;
          int slot = lr.slot;
#pragma unroll 1
          for (int u = 0; u < a.nu; ++u) {
            uint64_t dv = dv0 + slot * (a.um * 2 * kChunkUnits);
#pragma unroll 1
            for (int m = 0; m < a.um; ++m, dv += kChunkStep >> 3, d += N)
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                tc_mma_bf16(d, dv + kk * (a.row8_step >> 3), dp0 + kk * 2, idesc_o, i > 0 || kk > 0);
            tc_commit(&c.late[slot]);
            if (++slot == a.nlat) slot = 0;
          }
          tc_commit(&c.pe);
          if (i == n - 1) tc_commit(&c.of);
        }
        __syncwarp();
        for (int u = 0; u < a.nu; ++u) lr.step(a.nlat);
      }
      wk.done();
    }
  } else {
    const int q = warp & 3;
    const int st = tid - 64;                               // softmax thread
    const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
    uint32_t pphase = 0, ophase = 0, sphase = 0;
    int sbuf = 0;
    Ring lr;                                               // latent ring position of the current tile
    const int head0 = g * a.hg;                            // first head of the group
    const int nh_all = a.H - head0 < a.hg ? a.H - head0 : a.hg;
    auto heads_of = [&](const Item& it) {
      if constexpr (TREE) return it.rows < a.hg ? it.rows : a.hg;   // (one head group)
      else return nh_all;
    };
    const bool active = 16 * q < N;                        // this warp's 16 rows of S hold heads
    const int hr = 16 * q + (lane >> 2);                   // this thread's heads: rows hr and hr + 8 of S
    bool any_tile = false;                                 // a product into O has been issued before this tile
    // After a wait that gave up, these threads stop waiting but keep walking: all 128 then
    // meet at every CTA barrier, and the kernel ends. They arrive on no memory barrier any more: no barrier
    // gets more arrivals than it expects, and the other warps' waits run out too.
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
      if (ok) ok = bar_wait(bar, parity, a.status, site);
    };
    auto arrive = [&](uint64_t* bar) {
      if (ok) mbar_arrive(bar);
    };
    // Chunks of Q that the TMEM plan holds: row 16 q + r in lane r of the quarter's lanes 0-15, two values a column. A lane
    // loads what the store takes from it: of rows lane / 4 and lane / 4 + 8, the (lane % 4)-th 8 bytes of every 32. All
    // loads are under way together. (16 bytes of a row of its own per lane took twice the sectors, and a start of
    // 3300 clocks with 16 heads, 6600 with 32.)
    auto q_to_tmem = [&](int b) {
      if (active) {
        const Item it = item_of<TREE>(a, b);
        const int nh = heads_of(it);
        const int h = 16 * q + (lane >> 2);
        const uint2* src = reinterpret_cast<const uint2*>(a.q + it.seq * a.q_b + (it.row0 + head0 + h) * a.q_h) + (lane & 3);
        const int64_t down = 8 * a.q_h / 4;                // 8 rows on, in 8-byte words
        uint2 v[P::kMaxTs][4][2];
#pragma unroll
        for (int k = 0; k < P::kMaxTs; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              v[k][j][e] = k < a.nts && h + 8 * e < nh ? ld_global_u2(src + k * 16 + j * 4 + e * down) : make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < P::kMaxTs; ++k)
          if (k < a.nts) tmem_st_16x256b_x4(tmem + tlane + P::kQ + k * 32, &v[k][0][0]);
        tmem_wait_st();
        tc_fence_before();
      }
      arrive(&c.qf);
    };
    // One piece ahead: its Q goes in as soon as the last scores of the piece before are done.
    Walk<kTile, TREE> nx = wk;
    bool nx_started = false;
    bool more = nx.next(a, nx_started);
    if (more) q_to_tmem(nx.b);
    while (wk.next(a, started)) {
      float ref[2] = {kNoRef, kNoRef}, l[2] = {0.0f, 0.0f}, le[2] = {0.0f, 0.0f};
      const Item item = item_of<TREE>(a, wk.b);
      const int nh = heads_of(item);
      Sight sight[2];                                      // of this thread's rows
      int prefix = 0;
      if constexpr (TREE) {
        const int drafted = drafts_of(a, item.seq, wk.len, st == 0);
        prefix = wk.len - drafted;
#pragma unroll
        for (int k = 0; k < 2; ++k) sight[k] = sight_of(a, item.seq, item.row0 + hr + 8 * k, drafted);
      }
      // P of the scores x, packed to bf16, and its row sums (this thread's part): as rounded for the product,
      // which normalise the output, and in fp32 for the lse. Returns the largest score above its head's
      // reference, in powers of two.
      auto take = [&](const uint32_t* x, uint32_t* p, float* ls, float* les) {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float rs[4] = {}, es[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float r = -ref[i & 1];
          const float y0 = fmaf(__uint_as_float(x[2 * i]), a.scale2, r), y1 = fmaf(__uint_as_float(x[2 * i + 1]), a.scale2, r);
          top[i & 3] = fmaxf(top[i & 3], fmaxf(y0, y1));
          const float p0 = ex2(y0), p1 = ex2(y1);
          es[i & 3] += p0 + p1;
          p[i] = pack_bf16x2(p0, p1);
          rs[i & 3] += __uint_as_float(p[i] << 16) + __uint_as_float(p[i] & 0xFFFF0000u);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ls[k] = rs[k] + rs[k + 2];
          les[k] = es[k] + es[k + 2];
        }
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      };
#pragma unroll 1
      for (int ti = 0; ti < wk.n; ++ti) {
        const int valid = wk.len - (wk.t0 + ti) * kTile;   // tokens of the tile (>= 64: all)
        wait(&c.sf[sbuf], sphase, 80);
        // Register 4 i + 2 r + e: head hr + 8 r, token 8 i + 2 (lane % 4) + e.
        float over = -INFINITY, ls[2] = {0.0f, 0.0f}, les[2] = {0.0f, 0.0f};
        uint32_t x[32], p[16];
        if (active) {
          tc_fence_after();
          tmem_ld_16x256b_x8(tmem + tlane + P::kS + sbuf * kTile, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) reg_fence(x[i]);
          tc_fence_before();
        }
        arrive(&c.se[sbuf]);
        if (++sbuf == P::kBufs) {
          sbuf = 0;
          sphase ^= 1u;
        }
        if (active) {
          if constexpr (TREE) {
            const int t64 = (wk.t0 + ti) * kTile;
            if (prefix - t64 < kTile || !sight[0].live || !sight[1].live) {
              uint64_t see[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) see[k] = sees(sight[k], prefix, t64) >> (2 * (lane & 3));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see[(i >> 1) & 1] >> (8 * (i >> 2) + (i & 1))) & 1u)) x[i] = __float_as_uint(-INFINITY);
            }
          } else if (valid < kTile) {
            const int col = 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (8 * (i >> 2) + col + (i & 1) >= valid) x[i] = __float_as_uint(-INFINITY);
          }
          over = take(x, p, ls, les);
        }
        // O is rescaled only when a score of the tile passes kSlack, as in a piece's first tile; P above
        // (formed before the warps meet here) is then formed again.
        const bool grow = barrier_or<128>(2, over > kSlack);
        if (grow && active) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              m = fmaxf(m, fmaxf(__uint_as_float(x[4 * i + 2 * k]), __uint_as_float(x[4 * i + 2 * k + 1])));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            m = fmaxf(m * a.scale2, ref[k]);
            const float corr = ex2(ref[k] - m);            // 0 from kNoRef to a score
            l[k] *= corr;
            le[k] *= corr;
            ref[k] = m;
            if (ti > 0 && (lane & 3) == 0) fac[hr + 8 * k] = corr;
          }
          take(x, p, ls, les);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          l[k] += ls[k];
          le[k] += les[k];
        }
        // The previous tile's product is done: P is free and O stands still.
        if (any_tile) {
          wait(&c.pe, pphase, 81);
          pphase ^= 1u;
        }
        any_tile = true;
        if (grow && ti > 0) {
          named_barrier(3, 128);                           // fac is written
          tc_fence_after();
#pragma unroll 1
          for (int m = 0; m < nm; ++m)
#pragma unroll 1
            for (int hc = 0; hc < N; hc += 16) {
              uint32_t o[16];
              const uint32_t at = tmem + tlane + m * N + hc;
              tmem_ld_32x32b_x16(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                reg_fence(o[j]);
                o[j] = __float_as_uint(__uint_as_float(o[j]) * fac[hc + j]);
              }
              tmem_st_32x32b_x16(at, o);
            }
          tmem_wait_st();
        }
        if (active) {
          const int h = 16 * q + (lane & 15);              // lanes 0-7, 8-15: rows of the first two blocks; 16-31: the next token block
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int ch = i + (lane >> 4);
            stmatrix_x4(smem_u32(sp) + h * 128 + ((ch ^ (h & 7)) << 4), p[2 * i], p[2 * i + 1], p[2 * i + 2], p[2 * i + 3]);
          }
        }
        if (valid < kTile) {
          // Rows past the sequence's end hold whatever the page held (NaN included): their P is 0, and they
          // have to be 0 themselves for the product. Only a sequence's last tile is partial.
          Ring z = lr;
          const int per = (kTile - valid) * 8;             // 16-byte words to clear in a chunk
#pragma unroll 1
          for (int u = 0; u < a.nu; ++u) {
            wait(&c.latf[z.slot], z.phase, 82);
            uint8_t* v = lat + z.slot * slot_bytes;
#pragma unroll 1
            for (int i = st; i < 2 * a.um * per; i += 128) {
              const int k = i / per, r = valid + (i - k * per) / 8;
              *reinterpret_cast<uint4*>(v + k * kChunkStep + (r >> 3) * a.row8_step + (r & 7) * 128 + (i & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            z.step(a.nlat);
          }
        }
        for (int u = 0; u < a.nu; ++u) lr.step(a.nlat);
        fence_proxy_async();
        tc_fence_before();
        arrive(&c.pf);
      }
      // ---- epilogue of the piece, after the next one's Q
      nx.done();
      if (more && (more = nx.next(a, nx_started))) q_to_tmem(nx.b);
      const bool whole = wk.n == wk.nt;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (wk.first ? 0 : 1);
      named_barrier(3, 128);                               // fac is free
      if (active) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // a head's sums lie in the four lanes of its row
          float v = l[k], ve = le[k];
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          ve += __shfl_xor_sync(0xffffffffu, ve, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          ve += __shfl_xor_sync(0xffffffffu, ve, 2);
          const int h = hr + 8 * k;
          if ((lane & 3) == 0) {
            if (whole) {
              fac[h] = v == 0.0f ? 0.0f : 1.0f / v;
              if (a.lse != nullptr && h < nh)
                a.lse[static_cast<int64_t>(item.seq) * a.H + item.row0 + head0 + h] = ve == 0.0f ? -INFINITY : (ref[k] + log2f(ve)) * kLn2;
            } else {
              a.part_m[slot * kMaxHeadsCta + h] = ref[k];
              a.part_l[slot * kMaxHeadsCta + h] = v;
              a.part_e[slot * kMaxHeadsCta + h] = ve;
            }
          }
        }
      }
      named_barrier(3, 128);
      wait(&c.of, ophase, 83);
      ophase ^= 1u;
      tc_fence_after();
      // O^T in blocks of 16 latent columns: register 4 i + 2 r + e is column lane / 4 + 8 r, head 8 i + 2 (lane % 4) + e.
      constexpr int NP = N / 8;
      float2 f[NP];
      if (whole)
#pragma unroll
        for (int i = 0; i < NP; ++i) f[i] = reinterpret_cast<const float2*>(fac)[4 * i + (lane & 3)];
      uint8_t* stage = sp + q * (N * 32);                  // [N heads][16 columns] of this warp, over P
      __nv_bfloat16* out = a.out + (static_cast<int64_t>(item.seq) * a.H + item.row0 + head0) * a.latent;
      float4* part = reinterpret_cast<float4*>(a.part_o + static_cast<int64_t>(slot) * kMaxHeadsCta * a.latent) + q * 32 + lane;
      constexpr int kAtOnce = N <= 32 ? 2 : 1;             // blocks read from TMEM at once
#pragma unroll 1
      for (int mh0 = 0; mh0 < 2 * nm; mh0 += kAtOnce) {
        uint32_t ob[kAtOnce][4 * NP];
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b)
#pragma unroll
          for (int i = 0; i < NP; i += 2)
            tmem_ld_16x256b_x2(tmem + tlane + (static_cast<uint32_t>((mh0 + b) & 1) << 20) + ((mh0 + b) >> 1) * N + 8 * i,
                               ob[b] + 4 * i);
        tmem_wait_ld();
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b) {
          uint32_t (&o)[4 * NP] = ob[b];
          const int mh = mh0 + b;
#pragma unroll
          for (int i = 0; i < 4 * NP; ++i) reg_fence(o[i]);
          if (whole) {
            // Normalised, rounded and turned through shared memory: two lanes then store 32 bytes of a head.
#pragma unroll
            for (int i = 0; i < NP; i += 2) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(normed<TREE>(__uint_as_float(o[4 * i + 2 * k]), f[i + (k >> 1)].x),
                                   normed<TREE>(__uint_as_float(o[4 * i + 2 * k + 1]), f[i + (k >> 1)].y));
              const int h = 8 * (i + (lane >> 4)) + (lane & 7);
              stmatrix_x4_trans(smem_u32(stage) + h * 32 + ((((lane >> 3) ^ (h >> 2)) & 1) << 4), w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
              const int h = 16 * k + (lane >> 1), ch = lane & 1;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + h * 32 + (((ch ^ (h >> 2)) & 1) << 4));
              if (h < nh)
                *reinterpret_cast<uint4*>(out + h * a.latent + (mh >> 1) * 128 + q * 32 + (mh & 1) * 16 + ch * 8) = v;
            }
            __syncwarp();
          } else {
            // A partial keeps this register order: every store is 512 bytes in a row.
#pragma unroll
            for (int i = 0; i < NP; ++i)
              part[(mh * NP + i) * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                      __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
      }
      tc_fence_before();
      arrive(&c.oe);
      wk.done();
    }
    // Sequences without tokens: zero rows, lse = -inf.
#pragma unroll 1
    for (int b = w; b < a.B; b += a.W) {
      if (seq_len<TREE>(a, b, false) > 0) continue;
      const Item item = item_of<TREE>(a, b);
      const int nh = heads_of(item);
      const int64_t at = static_cast<int64_t>(item.seq) * a.H + item.row0 + head0;
      __nv_bfloat16* out = a.out + at * a.latent;
#pragma unroll 1
      for (int i = st; i < nh * a.latent / 8; i += 128) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse != nullptr)
#pragma unroll 1
        for (int i = st; i < nh; i += 128) a.lse[at + i] = -INFINITY;
      if constexpr (TREE) {
        if (st == 0) drafts_of(a, item.seq, 0, true);
      }
    }
  }
  tc_fence_before();
  // After a wait that gave up, products may be under way that nobody waits for.
  if (__syncthreads_or(!ok)) drain_pause();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// New tokens into the cache: one warp a token. The latent part is normalised
// (gamma given) in fp32 and rounded once; neighbouring rope columns (2 i, 2 i + 1)
// are rotated by the position's angle i (cos_sin given).
struct AppendArgs {
  int n, B, latent, rope, page, num_pages, max_pages, ld, max_pos;
  const __nv_bfloat16* kv;
  const __nv_bfloat16* gamma;    // or null
  float eps;
  const float* cos_sin;          // [max_pos][rope]: cos, then sin; or null
  const int32_t* seq;
  const int32_t* pos;
  const int32_t* table;
  __nv_bfloat16* cache;
  int* status;
};

// HBM bounds it: a row in, a row out (75 MB and 11 us for 32768 tokens of 512 + 64
// columns, measured 17.2 us of which 3 are launch and ramp). A token's place takes
// two dependent reads (position, then page): each warp walks tokens warp,
// warp + warps, ... with the position read two tokens ahead, and page, row and
// rotation one ahead.
__global__ void __launch_bounds__(256, kAppendBlocks) mla_append_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int step = static_cast<int>(gridDim.x) * 8;
  const int nlat = a.latent >> 3, nrope = a.rope >> 3;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  struct Token {
    uint4 c[2], u;               // latent vectors lane and lane + 32, rope vector lane
    float4 co, si;
    int page, row;               // page and row in it (row < 0: nothing to write)
  };
  auto read = [&](int64_t i, int p, int b, Token& t) {
    t.page = 0;
    t.row = -1;
    t.c[0] = t.c[1] = t.u = make_uint4(0, 0, 0, 0);
    t.co = t.si = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= a.n || p < 0) return;                         // past the end, or padding
    if (b < 0 || b >= a.B || p >= cap || (a.cos_sin != nullptr && p >= a.max_pos)) {
      if (lane == 0) report_error(a.status, kErrBounds, 65);
      return;
    }
    const int pg = p / a.page;
    t.row = p - pg * a.page;
    t.page = ld_global_s32(a.table + static_cast<int64_t>(b) * a.max_pages + pg);
    const __nv_bfloat16* src = a.kv + i * a.ld;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lane + 32 * h < nlat) t.c[h] = ld_global_u4(src + (lane + 32 * h) * 8);
    if (lane < nrope) {
      t.u = ld_global_u4(src + a.latent + lane * 8);
      if (a.cos_sin != nullptr) {
        const float* cs = a.cos_sin + static_cast<int64_t>(p) * a.rope + lane * 4;
        t.co = ld_global_f4(cs);
        t.si = ld_global_f4(cs + a.rope / 2);
      }
    }
  };
  int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= a.n) return;
  auto place = [&](int64_t k, int& p, int& b) {
    p = k < a.n ? ld_global_s32(a.pos + k) : -1;
    b = k < a.n ? ld_global_s32(a.seq + k) : 0;
  };
  int p0, b0, p1, b1;
  place(i, p0, b0);
  place(i + step, p1, b1);
  uint4 ug[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    ug[h] = a.gamma != nullptr && lane + 32 * h < nlat ? ld_global_u4(a.gamma + (lane + 32 * h) * 8)
                                                       : make_uint4(0, 0, 0, 0);
  Token t;
  read(i, p0, b0, t);
  for (; i < a.n; i += step) {
    Token nt;
    read(i + step, p1, b1, nt);
    place(i + 2 * step, p1, b1);
    if (t.page < 0 || t.page >= a.num_pages) {
      if (lane == 0) report_error(a.status, kErrBounds, 66);
      t.row = -1;
    }
    if (t.row >= 0) {                                      // the same in every lane
      __nv_bfloat16* dst = a.cache + (static_cast<int64_t>(t.page) * a.page + t.row) * (a.latent + a.rope);
      if (a.gamma != nullptr) {
        float v[2][8], ss = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          unpack_bf16x8(t.c[h], v[h]);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(v[h][e], v[h][e], ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rstd = rsqrtf(ss / static_cast<float>(a.latent) + a.eps);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float g[8];
          unpack_bf16x8(ug[h], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = v[h][e] * rstd * g[e];
          t.c[h] = pack_bf16x8(g);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < nlat) reinterpret_cast<uint4*>(dst)[lane + 32 * h] = t.c[h];
      if (lane < nrope) {
        if (a.cos_sin != nullptr) {
          const float cc[4] = {t.co.x, t.co.y, t.co.z, t.co.w}, sn[4] = {t.si.x, t.si.y, t.si.z, t.si.w};
          float v[8];
          unpack_bf16x8(t.u, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = v[2 * e], y = v[2 * e + 1];
            v[2 * e] = x * cc[e] - y * sn[e];
            v[2 * e + 1] = x * sn[e] + y * cc[e];
          }
          t.u = pack_bf16x8(v);
        }
        reinterpret_cast<uint4*>(dst + a.latent)[lane] = t.u;
      }
    }
    t = nt;
  }
}

namespace {

// The cache's latent columns as [rows / 8][latent / 64][8 rows][64]: a box is `piece` rows of the `chunks` chunks of a
// ring slot, 8 rows of every chunk after another.
bool make_tmap_latent(CUtensorMap* m, const void* base, int64_t rows, const moe_mla_config_t* c, int piece, int chunks) {
  const uint64_t pitch = static_cast<uint64_t>(c->latent + c->rope) * 2;
  return make_tmap_strided(m, base, {64, 8, static_cast<uint64_t>(c->latent / 64), static_cast<uint64_t>(rows / 8)},
                           {pitch, 128, 8 * pitch},
                           {64, 8, static_cast<uint32_t>(chunks), static_cast<uint32_t>(piece / 8)}, 4);
}
// Whole cache rows; the rope columns are one box of 64, zero past the row's end.
bool make_tmap_rope(CUtensorMap* m, const void* base, int64_t rows, const moe_mla_config_t* c, int piece) {
  const uint64_t cols = static_cast<uint64_t>(c->latent + c->rope);
  return make_tmap_strided(m, base, {cols, static_cast<uint64_t>(rows), 1, 1}, {cols * 2, 0, 0},
                           {64, static_cast<uint32_t>(piece), 1, 1}, 2);
}

int validate_mla(const moe_mla_config_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->batch < 0 || c->heads < 1 || c->heads > 128) return MOE_ERR_INVALID_ARG;
  if (c->latent < 128 || c->latent > 512 || c->latent % 128) return MOE_ERR_INVALID_ARG;
  if (c->rope < 8 || c->rope > 64 || c->rope % 8) return MOE_ERR_INVALID_ARG;
  if (c->page_size < 8 || c->page_size % 8 || c->num_pages < 1 || c->max_pages < 1) return MOE_ERR_INVALID_ARG;
  // the kernels work in powers of two: with a factor past fp32's range a score of 0 would be NaN
  if (!(c->softmax_scale > 0.0f) || !std::isfinite(c->softmax_scale * kLog2e)) return MOE_ERR_INVALID_ARG;
  const int64_t lim = (1LL << 31) - 1;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  // row coordinates and token positions are 32-bit, and so is the count of tiles of all sequences
  if (static_cast<int64_t>(c->num_pages) * c->page_size >= lim || cap >= lim) return MOE_ERR_INVALID_ARG;
  if (c->batch > 0 && ceil_div(cap, kTile) > lim / c->batch) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct MlaLayout {
  size_t status, join, m, l, e, o, total;
};
MlaLayout mla_layout(const moe_mla_config_t* c) {
  MlaLayout L{};
  const size_t slots = 2 * static_cast<size_t>(kMaxSms);
  size_t cur = 0;
  auto add = [&](size_t n) {
    const size_t at = cur;
    cur += (n + 255) / 256 * 256;
    return at;
  };
  L.status = add(16);
  L.join = add(sizeof(int4) * kMaxSms);
  L.m = add(sizeof(float) * slots * kMaxHeadsCta);
  L.l = add(sizeof(float) * slots * kMaxHeadsCta);
  L.e = add(sizeof(float) * slots * kMaxHeadsCta);
  L.o = add(sizeof(float) * slots * kMaxHeadsCta * c->latent);
  L.total = cur;
  return L;
}

template <int N, bool TREE>
int run_decode(MlaArgs a, const CUtensorMap& tk, const CUtensorMap& tr, const CUtensorMap& tq, int sms,
               cudaStream_t s) {
  static DevOnce once;
  if (!once.ready([] {
        return cudaFuncSetAttribute(mla_decode_kernel<N, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
      }))
    return MOE_ERR_CUDA;
  const int nchunk = 2 * a.nm + 1;
  // a row past 64 * nchunk columns does not exist: a rope part under 64 columns is zero-filled by its TMA box only
  a.nts = Plan<N>::kMaxTs < nchunk - 1 ? Plan<N>::kMaxTs : (a.rope == 64 && Plan<N>::kMaxTs >= nchunk ? nchunk : nchunk - 1);
  const int fixed = 1024 + kBarBytes + kMaxHeadsCta * 4 + (nchunk - a.nts) * N * 128 + N * 128;
  // The ring: rope slots for as many whole tiles as fit, latent slots in the rest (3 and 6 at 512 + 64 columns and few
  // heads, 9 and 9 at 128 + 64).
  const int slot_bytes = a.um * 2 * kChunk, ring = kSmemMax - fixed;
  a.nrope = ring / (a.nu * slot_bytes + kChunk);
  if (a.nrope > kMaxRopeSlots) a.nrope = kMaxRopeSlots;
  a.nlat = (ring - a.nrope * kChunk) / slot_bytes;
  if (a.nlat > kMaxLatSlots) a.nlat = kMaxLatSlots;
  const int smem = fixed + a.nrope * kChunk + a.nlat * slot_bytes;
  launch_kernel_after("mla_decode", mla_decode_kernel<N, TREE>, dim3(static_cast<unsigned>(a.W * a.G)), dim3(kThreads), smem, s, tk, tr, tq,
                a);
  if (int e = call_error() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA) return e;
  launch_join<N, false, TREE, kTile, kMinTiles>(a, sms, s);
  return MOE_OK;
}

inline bool mis(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The launches of moe_mla_decode and (TREE) moe_mla_decode_tree: `a` comes with what is the tree's own.
template <bool TREE>
int decode(const moe_mla_config_t* cfg, MlaArgs a, const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* cache,
           const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse, void* ws, cudaStream_t s) {
  CallScope call;
  if (!get_encode()) return MOE_ERR_CUDA;
  const MlaLayout L = mla_layout(cfg);
  char* base = static_cast<char*>(ws);
  const int row = cfg->latent + cfg->rope;
  const int rows_walked = TREE ? a.hv : cfg->heads;        // rows of a walked item
  a.B = cfg->batch * a.V;
  a.latent = cfg->latent;
  a.rope = cfg->rope;
  a.page = cfg->page_size;
  a.num_pages = cfg->num_pages;
  a.max_pages = cfg->max_pages;
  a.G = static_cast<int>(ceil_div(rows_walked, kMaxHeadsCta));
  a.hg = static_cast<int>(ceil_div(rows_walked, a.G));
  a.nm = cfg->latent / 128;
  a.um = a.nm % 2 ? 1 : 2;
  a.nu = a.nm / a.um;
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  a.W = sms / a.G;
  // A box takes as many tokens as every page holds whole: 8 to 64, a power of two. Groups of 8 rows, the swizzle's
  // period, lie one after another in a slot, each with its chunks side by side, so a slot looks alike for every box.
  a.piece = cfg->page_size & -cfg->page_size;
  if (a.piece > kTile) a.piece = kTile;
  for (a.piece_log = 3; 1 << a.piece_log < a.piece;) ++a.piece_log;
  const PageDiv pd = page_div(a.page);
  a.page_mul = pd.mul;
  a.page_shift = pd.shift;
  const bool pair = pair_form(rows_walked, cfg->latent);
  const int chunks = pair ? a.nm : 2 * a.um;               // 64-column chunks of a ring slot
  a.row8_step = chunks * kChunkStep;
  a.scale2 = cfg->softmax_scale * kLog2e;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_b = q_stride_b;
  a.q_h = q_stride_h;
  a.table = block_table;
  a.lens = seq_lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = reinterpret_cast<int*>(base + L.status);
  a.join = reinterpret_cast<int4*>(base + L.join);
  a.part_m = reinterpret_cast<float*>(base + L.m);
  a.part_l = reinterpret_cast<float*>(base + L.l);
  a.part_e = reinterpret_cast<float*>(base + L.e);
  a.part_o = reinterpret_cast<float*>(base + L.o);
  const int N = pair ? kMaxHeadsCta : static_cast<int>(round_up(a.hg, 16));
  CUtensorMap tk, tr, tq;
  const int64_t rows = static_cast<int64_t>(cfg->num_pages) * cfg->page_size;
  if (!make_tmap_latent(&tk, cache, rows, cfg, a.piece, chunks) || !make_tmap_rope(&tr, cache, rows, cfg, a.piece))
    return MOE_ERR_CUDA;
  if (!make_tmap_strided(&tq, q,
                         {static_cast<uint64_t>(row), static_cast<uint64_t>(a.H), static_cast<uint64_t>(cfg->batch), 1},
                         {static_cast<uint64_t>(q_stride_h) * 2, static_cast<uint64_t>(q_stride_b) * 2, 0},
                         {64, static_cast<uint32_t>(N), 1, 1}, 3))
    return MOE_ERR_CUDA;
  if (pair) {
    if (int r = run_decode_pair<TREE>(a, tk, tr, tq, sms, s)) return r;
    return call.status();
  }
  int r;
  switch (N) {
    case 16: r = run_decode<16, TREE>(a, tk, tr, tq, sms, s); break;
    case 32: r = run_decode<32, TREE>(a, tk, tr, tq, sms, s); break;
    case 48: r = run_decode<48, TREE>(a, tk, tr, tq, sms, s); break;
    default: r = run_decode<64, TREE>(a, tk, tr, tq, sms, s); break;
  }
  if (r) return r;
  return call.status();
}

// What the two calls refuse alike.
int refuse_decode(const moe_mla_config_t* cfg, const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* cache,
                  const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse, void* ws) {
  const int row = cfg->latent + cfg->rope;
  if (cache == nullptr || ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (cfg->batch > 0 && (q == nullptr || block_table == nullptr || seq_lens == nullptr || out == nullptr))
    return MOE_ERR_INVALID_ARG;
  // strides in elements; a TMA dimension's pitch is below 2^40 bytes. (Sequences may share rows of q: it is only read.)
  if (q_stride_h < row || q_stride_b < row || q_stride_h % 8 || q_stride_b % 8 || q_stride_h >= (1LL << 38) ||
      q_stride_b >= (1LL << 38))
    return MOE_ERR_INVALID_ARG;
  if (mis(q, 16) || mis(cache, 16) || mis(out, 16) || mis(ws, 16) || mis(lse, 4) || mis(block_table, 4) || mis(seq_lens, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_mla_workspace_size(const moe_mla_config_t* cfg, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  if (int r = validate_mla(cfg)) return r;
  *bytes = mla_layout(cfg).total;
  return MOE_OK;
}

extern "C" int moe_mla_append(const moe_mla_config_t* cfg, int n, const void* kv, int ld_kv, const void* gamma,
                              float eps, const float* cos_sin, int max_pos, const int32_t* seq, const int32_t* pos,
                              const int32_t* block_table, void* cache, void* ws, moe_stream_t stream) {
  if (int r = validate_mla(cfg)) return r;
  if (n < 0 || ld_kv < cfg->latent + cfg->rope || ld_kv % 8 || cache == nullptr || ws == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (n > 0 && (kv == nullptr || seq == nullptr || pos == nullptr || block_table == nullptr)) return MOE_ERR_INVALID_ARG;
  if (gamma != nullptr && !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (cos_sin != nullptr && max_pos < 1) return MOE_ERR_INVALID_ARG;
  if (mis(kv, 16) || mis(gamma, 16) || mis(cos_sin, 16) || mis(cache, 16) || mis(ws, 16) || mis(seq, 4) || mis(pos, 4) ||
      mis(block_table, 4))
    return MOE_ERR_INVALID_ARG;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  CallScope call;
  if (n == 0) return MOE_OK;
  AppendArgs a{};
  a.n = n;
  a.B = cfg->batch;
  a.latent = cfg->latent;
  a.rope = cfg->rope;
  a.page = cfg->page_size;
  a.num_pages = cfg->num_pages;
  a.max_pages = cfg->max_pages;
  a.ld = ld_kv;
  a.max_pos = max_pos;
  a.kv = static_cast<const __nv_bfloat16*>(kv);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.seq = seq;
  a.pos = pos;
  a.table = block_table;
  a.cache = static_cast<__nv_bfloat16*>(cache);
  a.status = reinterpret_cast<int*>(static_cast<char*>(ws) + mla_layout(cfg).status);
  const int64_t blocks = ceil_div(n, 8), most = static_cast<int64_t>(kAppendBlocks) * num_sms();
  launch_kernel_after("mla_append", mla_append_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256),
                      0, static_cast<cudaStream_t>(stream), a);
  return call.status();
}

extern "C" int moe_mla_decode(const moe_mla_config_t* cfg, const void* q, int64_t q_stride_b, int64_t q_stride_h,
                              const void* cache, const int32_t* block_table, const int32_t* seq_lens, void* out,
                              float* lse, void* ws, moe_stream_t stream) {
  if (int r = validate_mla(cfg)) return r;
  if (int r = refuse_decode(cfg, q, q_stride_b, q_stride_h, cache, block_table, seq_lens, out, lse, ws))
    return r;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (cfg->batch == 0) return MOE_OK;
  MlaArgs a{};
  a.H = cfg->heads;
  a.V = 1;
  return decode<false>(cfg, a, q, q_stride_b, q_stride_h, cache, block_table, seq_lens, out, lse, ws,
                       static_cast<cudaStream_t>(stream));
}

extern "C" int moe_mla_decode_tree(const moe_mla_config_t* cfg, int drafts, const void* q, int64_t q_stride_b,
                                   int64_t q_stride_h, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                   const int32_t* draft_lens, const uint64_t* tree, void* out, float* lse, void* ws,
                                   moe_stream_t stream) {
  if (int r = validate_mla(cfg)) return r;
  if (drafts < 1 || drafts > MOE_MLA_MAX_DRAFTS || mis(draft_lens, 4) || mis(tree, 8)) return MOE_ERR_INVALID_ARG;
  if (int r = refuse_decode(cfg, q, q_stride_b, q_stride_h, cache, block_table, seq_lens, out, lse, ws))
    return r;
  // A sequence's rows in groups that one worker takes: up to 128 where the pair form does, else up to 64. Pairs also where they are
  // not full. In us, after a flushed L2, on pairs and in groups of up to 64 on single CTAs: 48 x ~8192 tokens with 80 rows 108 and
  // 156, 64 x ~1000 with 80 44 and 56, 4 x ~1500 with 80 27 and 31, 16 x ~4000 with 160 53 and 58. Of ten sizes one is the other
  // way round: 23 x ~700 with 140 rows, two groups of 70 or three of 47, 37.5 and 36.
  MlaArgs a{};
  a.H = drafts * cfg->heads;
  a.V = static_cast<int>(ceil_div(a.H, cfg->latent % 256 == 0 ? 2 * kMaxHeadsCta : kMaxHeadsCta));
  a.hv = static_cast<int>(ceil_div(a.H, a.V));
  // the count of tiles of all groups is 32-bit
  const int64_t tiles = ceil_div(static_cast<int64_t>(cfg->max_pages) * cfg->page_size, kTile);
  if (cfg->batch > 0 && tiles > ((1LL << 31) - 1) / (static_cast<int64_t>(cfg->batch) * a.V)) return MOE_ERR_INVALID_ARG;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (cfg->batch == 0) return MOE_OK;
  a.heads = cfg->heads;
  a.drafts = drafts;
  a.draft_lens = draft_lens;
  a.tree = tree;
  return decode<true>(cfg, a, q, q_stride_b, q_stride_h, cache, block_table, seq_lens, out, lse, ws,
                      static_cast<cudaStream_t>(stream));
}

extern "C" int moe_mla_status(const moe_mla_config_t* cfg, void* ws, int* code, int* site, int clear,
                              moe_stream_t stream) {
  if (int r = validate_mla(cfg)) return r;
  if (!ws || !code || !site) return MOE_ERR_INVALID_ARG;
  return read_status(static_cast<char*>(ws) + mla_layout(cfg).status, code, site, clear, static_cast<cudaStream_t>(stream));
}
