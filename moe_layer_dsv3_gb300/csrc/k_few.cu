// The whole layer for up to 64 tokens: router, experts and combine in three
// launches, each placed while the one before still runs.
//
//   route   logits = x Wr^T, the choice of every token (route.cuh), MX(x)
//   up      [g | u] = Wgu MX(x)^T, h = silu(g) u, MX(h)
//   down    o = Wd MX(h)^T, y = sum over a token's experts of w o
//
// Few tokens read many weights: one token of 9 experts with 7168 x 2048 matrices
// reads 410 MB for 0.8 GFLOP, and HBM bounds it (0.4 us of products, 60 us of
// copies). So the weights are the 128-row operand of the tensor cores and the
// tokens the narrow one (16 to 64 columns): a tile of weights goes from HBM
// through shared memory once, for all tokens, and nothing has to be converted,
// gathered or padded to 128 rows.
//
// Each of the two expert kernels streams the weight tiles of all experts in use,
// laid end to end, cut into equal contiguous ranges, one per CTA. A range may begin and end
// inside a reduction: the pieces of a cut one are left in the workspace, and the
// CTA that arrives last adds them in the order of the ranges, so the result does
// not depend on who that is. No CTA waits for another.
//
//   up    unit: 128 gate rows and their 128 up rows of one expert (K = d). All T
//         tokens are columns, also those that did not choose the expert: a
//         product of 16 columns takes the tensor pipe a tenth of the time its
//         weights take to arrive, and X needs no gather.
//   down  unit: 128 rows of one expert (K = I), the tokens of the expert as columns.
//         Units of the same rows follow one another, expert by expert, so that
//         their weighted sum stays in shared memory and only rows that a range cuts pass
//         through the workspace.
// `down` starts on its weights before `up` is done: they do not depend on it.
#include <cudaTypedefs.h>

#include "gemm.cuh"
#include "mla_split.h"
#include "prof.h"
#include "route.cuh"

namespace moe {

namespace {

using mla::cut_of;
using mla::owner_of;
using mla::range_begin;
using mla::workers_of;

constexpr int kMaxT = MOE_FEW_MAX_T;
constexpr int kMaxEp = 513;                // experts, a shared one included
constexpr int kMaxRows = kMaxT * 9;        // (token, expert) pairs
constexpr int kThreads = 192;
constexpr int kMaxStages = 12;
constexpr int kTileBytes = 128 * 128;      // a weight tile: 128 rows x 128 values
constexpr int kSmemMax = 232448;
constexpr int kSfCol = 256;                // TMEM: accumulators below, scales of the ring's stages from here on
constexpr int kMinSteps = 4;               // fewest steps of a CTA
static_assert(kMaxT == 64, "a token is a bit of an expert's 64-bit mask");

struct FewArgs {
  int T, d, E, k, G, gtop, I, S, Ep;
  int N;                                   // T, rounded up to 16
  int nst, stage_bytes;                    // ring of the kernel: stages, operand bytes of one (the scales lie behind the ring)
  const __nv_bfloat16* x;
  const __nv_bfloat16* w_router;
  const float* bias;
  int32_t* idx;
  float* w;
  float* logits;                           // [T][E]
  uint8_t* xq;                             // [64][d]
  uint8_t* xsf;                            // [d / 128] atoms
  const uint8_t* wsf;                      // scales of the kernel's weights
  uint8_t* hq;                             // [rows][I], an expert's tokens one after another
  uint8_t* hsf;                            // [experts in use][I / 128] atoms
  float* part;                             // pieces of cut units, two per CTA
  int* cnt_route;                          // per token group: CTAs done
  int* cnt_up;                             // per unit: pieces done
  int* cnt_down;                           // per 128 rows: pieces done
  int ncnt;                                // of the last two, which lie together
  __nv_bfloat16* y;
  int* status;
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, site));
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// After a wait that gave up, products and copies that nobody waits for may be under way.
__device__ __forceinline__ void drain_pause() {
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (global_timer_ns() - t0 < 100000) {
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ---------------------------------------------------------------- route
// Logits: four warps share an expert's row, ER rows at once for TG tokens, in fp32
// on the CUDA cores (a row of Wr is read once per token group; the tensor cores
// would wait for one CTA's chain of 7168 / 64 stages). The CTA that finishes a group of tokens last
// chooses for them. Further CTAs quantise x and clear the counters of the kernels that follow.
constexpr int kRouteThreads = 256;
constexpr int kRowWarps = 4;

template <int TG, int ER>
__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kSets = 8 / kRowWarps;
  constexpr int kDeep = TG == 1 ? 4 : 1;                   // chunks whose loads are under way together
  __shared__ float red[kSets][kRowWarps][ER * TG];
  __shared__ int last;
  extern __shared__ float sv_all[];                        // [8][E]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NE = (a.E + kSets * ER - 1) / (kSets * ER), NG = (a.T + TG - 1) / TG;
  grid_wait();
  grid_launch();
  const int bid = static_cast<int>(blockIdx.x);
  if (bid >= NE * NG) {
    const int kb = a.d >> 5, step = static_cast<int>(gridDim.x - NE * NG) * kRouteThreads;
    for (int i = (bid - NE * NG) * kRouteThreads + tid; i < a.T * kb; i += step) {
      const int t = i / kb, b = i - t * kb;
      float v[32];
      const int64_t at = static_cast<int64_t>(t) * a.d + b * 32;
#pragma unroll
      for (int q = 0; q < 4; ++q) unpack_bf16x8(ld_global_u4(a.x + at + 8 * q), v + 8 * q);
      emit_rowq(v, a.xq + at, a.xsf + sf_off(t, b, a.d >> 7));
    }
    for (int i = (bid - NE * NG) * kRouteThreads + tid; i < a.ncnt; i += step) a.cnt_up[i] = 0;
    return;
  }
  const int g = bid / NE, set = warp / kRowWarps, part = warp % kRowWarps;
  const int e0 = ((bid - g * NE) * kSets + set) * ER;
  float acc[ER][TG];
#pragma unroll
  for (int r = 0; r < ER; ++r)
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[r][t] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c0 = part * 256; c0 < a.d; c0 += kDeep * kRowWarps * 256) {
    uint4 uw[kDeep][ER], ux[kDeep][TG];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int col = c0 + u * kRowWarps * 256 + lane * 8;
#pragma unroll
      for (int r = 0; r < ER; ++r)
        uw[u][r] = col < a.d && e0 + r < a.E ? ld_global_u4(a.w_router + static_cast<int64_t>(e0 + r) * a.d + col) : zero;
#pragma unroll
      for (int t = 0; t < TG; ++t)
        ux[u][t] = col < a.d && g * TG + t < a.T ? ld_global_u4(a.x + static_cast<int64_t>(g * TG + t) * a.d + col) : zero;
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      float w[ER][8];
#pragma unroll
      for (int r = 0; r < ER; ++r) unpack_bf16x8(uw[u][r], w[r]);
#pragma unroll
      for (int t = 0; t < TG; ++t) {
        float v[8];
        unpack_bf16x8(ux[u][t], v);
#pragma unroll
        for (int r = 0; r < ER; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[r][t] = fmaf(w[r][i], v[i], acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ER; ++r)
#pragma unroll
    for (int t = 0; t < TG; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (lane == 0) red[set][part][r * TG + t] = acc[r][t];
    }
  __syncthreads();
  if (tid < kSets * ER * TG) {
    const int s = tid / (ER * TG), i = tid - s * (ER * TG);
    const int e = ((bid - g * NE) * kSets + s) * ER + i / TG, t = g * TG + i % TG;
    float v = red[s][0][i];
#pragma unroll
    for (int p = 1; p < kRowWarps; ++p) v += red[s][p][i];
    if (e < a.E && t < a.T) a.logits[static_cast<int64_t>(t) * a.E + e] = v;
    __threadfence();
  }
  __syncthreads();
  if (tid == 0) last = atomicAdd(a.cnt_route + g, 1) == NE - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (tid == 0) a.cnt_route[g] = 0;
#pragma unroll 1
  for (int i = warp; i < TG; i += 8) {
    const int t = g * TG + i;
    if (t >= a.T) break;
    int e;
    float s, tot;
    choose_experts<16>([&](int n) { return __ldcg(a.logits + static_cast<int64_t>(t) * a.E + n); },
                       [&](int n) { return __int_as_float(ld_global_s32(reinterpret_cast<const int*>(a.bias + n))); }, a.E, a.k,
                       a.G, a.gtop, sv_all + warp * a.E, lane, e, s, tot);
    if (lane < a.k) {
      a.idx[t * a.k + lane] = e;
      a.w[t * a.k + lane] = __fdiv_rn(s, tot);
    }
  }
}

// ---------------------------------------------------------------- the experts in use
// Which tokens chose which expert, made by every CTA for itself from the router's choice: a 64-bit mask of tokens per
// expert, the experts in use in ascending order, and their tokens' rows one after another.
struct FewPlan {
  uint32_t mask[kMaxEp][2];
  uint16_t expert[kMaxEp];                 // of a slot
  uint16_t slot[kMaxEp];                   // of an expert in use
  uint16_t first[kMaxEp + 1];              // row of a slot's first token
  uint8_t token[kMaxRows];                 // of a row
  float gate[kMaxRows];
  uint32_t bad[2];                         // tokens without a valid choice: their scores are NaN
  uint32_t scan[kThreads / 32];
  int slots;
};

__device__ __forceinline__ void make_plan(const FewArgs& a, FewPlan& p, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < a.Ep; i += kThreads) p.mask[i][0] = p.mask[i][1] = 0;
  if (tid < 2) p.bad[tid] = 0;
  __syncthreads();
  const int n = a.T * a.k;
  for (int i = tid; i < n; i += kThreads) {
    const int e = ld_global_s32(a.idx + i), t = i / a.k;
    const bool ok = e >= 0 && e < a.E;
    atomicOr(ok ? &p.mask[e][t >> 5] : &p.bad[t >> 5], 1u << (t & 31));
    if (!ok && report) report_error(a.status, kErrBounds, 200);
  }
  if (a.S > 0 && tid < 2) p.mask[a.E][tid] = tid * 32 >= a.T ? 0u : (a.T - tid * 32 >= 32 ? 0xffffffffu : (1u << (a.T - tid * 32)) - 1u);
  __syncthreads();
  const int per = (a.Ep + kThreads - 1) / kThreads;
  uint32_t mine = 0;                       // experts in use << 16 | their tokens
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.Ep) break;
    const uint32_t c = __popc(p.mask[e][0]) + __popc(p.mask[e][1]);
    mine += c > 0 ? 0x10000u + c : 0u;
  }
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) p.scan[warp] = incl;
  __syncthreads();
  uint32_t at = incl - mine, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) at += p.scan[i];
    all += p.scan[i];
  }
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.Ep) break;
    const uint32_t c = __popc(p.mask[e][0]) + __popc(p.mask[e][1]);
    if (c == 0) continue;
    p.expert[at >> 16] = static_cast<uint16_t>(e);
    p.first[at >> 16] = static_cast<uint16_t>(at & 0xffffu);
    p.slot[e] = static_cast<uint16_t>(at >> 16);
    at += 0x10000u + c;
  }
  if (tid == 0) {
    p.slots = static_cast<int>(all >> 16);
    p.first[all >> 16] = static_cast<uint16_t>(all & 0xffffu);
  }
  __syncthreads();
  auto place = [&](int e, int t, float w) {
    const uint32_t below = t < 32 ? __popc(p.mask[e][0] & ((1u << t) - 1u))
                                  : __popc(p.mask[e][0]) + __popc(p.mask[e][1] & ((1u << (t - 32)) - 1u));
    const int row = p.first[p.slot[e]] + static_cast<int>(below);
    p.token[row] = static_cast<uint8_t>(t);
    p.gate[row] = w;
  };
  for (int i = tid; i < n; i += kThreads) {
    const int e = ld_global_s32(a.idx + i);
    if (e >= 0 && e < a.E) place(e, i / a.k, __int_as_float(ld_global_s32(reinterpret_cast<const int*>(a.w + i))));
  }
  if (a.S > 0)
    for (int t = tid; t < a.T; t += kThreads) place(a.E, t, 1.0f);
  __syncthreads();
}

struct FewSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t accf[4], acce[4];
  uint32_t tmem;
  int last;
  FewPlan plan;
};
constexpr int kControl = (sizeof(FewSmem) + 1023) / 1024 * 1024;

// Place in the ring of stages.
struct Stage {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// The steps of a range, unit by unit. A step is one 128-wide piece of K of a unit with K / 128 = len steps.
struct Walk {
  int unit, at, left, len;
  __device__ __forceinline__ Walk(int f0, int f1, int len_) : unit(f0 / len_), at(f0 - f0 / len_ * len_), left(f1 - f0), len(len_) {}
  __device__ __forceinline__ int steps() const { return left < len - at ? left : len - at; }   // in the current unit
  __device__ __forceinline__ void next() {
    left -= steps();
    ++unit;
    at = 0;
  }
};

// The worker that arrives last at a cut sum adds its pieces. Called by the 128 epilogue threads after their piece is stored;
// true in all of them if every piece is there.
__device__ __forceinline__ bool last_piece(FewSmem& c, int* cnt, int pieces) {
  __threadfence();
  named_barrier(1, 128);
  if (threadIdx.x == 64) c.last = atomicAdd(cnt, 1) == pieces - 1;
  named_barrier(1, 128);
  if (c.last == 0) return false;
  __threadfence();
  return true;
}

__device__ __forceinline__ void few_setup(FewSmem& c, int nst, const CUtensorMap* a, const CUtensorMap* b) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < nst; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c.accf[i], 1);
      mbar_init(&c.acce[i], 128);
    }
    fence_barrier_init();
    fence_proxy_async();
    tma_prefetch(a);
    tma_prefetch(b);
  }
  if (threadIdx.x >> 5 == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
}
__device__ __forceinline__ void few_finish(uint32_t tmem, bool ok) {
  tc_fence_before();
  if (__syncthreads_or(!ok)) drain_pause();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// The copies of the last stages that were issued have landed.
__device__ __forceinline__ bool land(FewSmem& c, Stage st, int issued, int nst, int* status, int site) {
  bool ok = true;
  for (int i = 0, n = issued < nst ? issued : nst; i < n; ++i) {
    if (--st.i < 0) {
      st.i = nst - 1;
      st.phase ^= 1u;
    }
    ok = warp_wait(&c.full[st.i], st.phase, status, site) && ok;
  }
  return ok;
}

// ---------------------------------------------------------------- gate and up projections
// Warps: 0 loads, 1 issues the products, 2-5 epilogue (row = TMEM lane).
// Stage: [256 rows of weights][N rows of X], and the scale atoms of gate, up and X.
__global__ void __launch_bounds__(kThreads, 1)
    few_up_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ CUtensorMap tma_x,
                  const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewSmem& c = *reinterpret_cast<FewSmem*>(smem);
  uint8_t* ring = smem + kControl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  few_setup(c, a.nst, &tma_w, &tma_x);
  grid_wait();
  grid_launch();
  tc_fence_before();
  make_plan(a, c.plan, blockIdx.x == 0);                   // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const int KA = a.d >> 7, NB = a.I >> 7;
  const int total = c.plan.slots * NB * KA;
  const int W = workers_of(total, static_cast<int>(gridDim.x), kMinSteps), w = static_cast<int>(blockIdx.x);
  const int f0 = w < W ? range_begin(total, w, W) : total, f1 = w < W ? range_begin(total, w + 1, W) : total;
  bool ok = true;
  uint8_t* scales = ring + a.nst * a.stage_bytes;          // three atoms a stage
  if (warp == 0) {
    Stage st;
    int issued = 0;
    for (Walk wk(f0, f1, KA); wk.left > 0 && ok; wk.next()) {
      const int s = wk.unit / NB, b = wk.unit - s * NB, e = c.plan.expert[s];
      const int row = __shfl_sync(0xffffffffu, e * 2 * a.I + b * 256, 0);
      const uint8_t* sf = a.wsf + static_cast<int64_t>(row >> 7) * KA * 512;
      const int k1 = __shfl_sync(0xffffffffu, wk.at + wk.steps(), 0);
#pragma unroll 1
      for (int k = __shfl_sync(0xffffffffu, wk.at, 0); k < k1; ++k) {
        ok = warp_wait(&c.empty[st.i], st.phase ^ 1u, a.status, 201);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* dst = ring + st.i * a.stage_bytes;
          uint64_t* bar = &c.full[st.i];
          mbar_arrive_expect_tx(bar, 2 * kTileBytes + a.N * 128 + 3 * 512);
          tma_load_2d(dst, &tma_w, k * 128, row, bar);
          tma_load_2d(dst + 2 * kTileBytes, &tma_x, k * 128, 0, bar);
          uint8_t* sfd = scales + st.i * (3 * 512);
          bulk_load(sfd, sf + static_cast<int64_t>(k) * 512, 512, bar);
          bulk_load(sfd + 512, sf + static_cast<int64_t>(KA + k) * 512, 512, bar);
          bulk_load(sfd + 1024, a.xsf + static_cast<int64_t>(k) * 512, 512, bar);
        }
        __syncwarp();
        st.step(a.nst);
        ++issued;
      }
    }
    ok = land(c, st, issued, a.nst, a.status, 202) && ok;
  } else if (warp == 1) {
    Stage st, acc;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t idesc = idesc_mxf8(128, a.N), sf0 = smem_u32(scales);
    for (Walk wk(f0, f1, KA); wk.left > 0 && ok; wk.next()) {
      ok = warp_wait(&c.acce[acc.i], acc.phase ^ 1u, a.status, 203);
      const int n = __shfl_sync(0xffffffffu, wk.steps(), 0);
      const uint32_t d = tm + acc.i * 128;
#pragma unroll 1
      for (int k = 0; k < n && ok; ++k) {
        ok = warp_wait(&c.full[st.i], st.phase, a.status, 204);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t base = smem_u32(ring + st.i * a.stage_bytes), sf = tm + kSfCol + st.i * 12;
#pragma unroll
          for (int j = 0; j < 3; ++j) tc_cp_sf(sf + 4 * j, desc_sf_chunk(sf0 + st.i * (3 * 512) + 512 * j));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tc_mma_mxf8(d + 64 * j, desc_kmajor_sw128(base + j * kTileBytes + kk * 32),
                          desc_kmajor_sw128(base + 2 * kTileBytes + kk * 32), idesc_mxf8_sf(idesc, kk, kk), sf + 4 * j, sf + 8,
                          (k | kk) != 0);
          tc_commit(&c.empty[st.i]);
          if (k == n - 1) tc_commit(&c.accf[acc.i]);
        }
        __syncwarp();
        st.step(a.nst);
      }
      acc.step(2);
    }
  } else {
    const int q = warp & 3, row = q * 32 + lane;
    Stage acc;
    // MX(h) of a token: its 32 values lie in the warp's lanes.
    auto emit = [&](int s, int r, int b, float g, float u) {
      const float h = __fdividef(g, 1.0f + __expf(-g)) * u;
      const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h)));
      const int sb = mx_scale_byte(__uint_as_float(top));
      const uint32_t code = e4m3x2(h * mx_inv_scale(sb), 0.0f) & 0xffu;
      a.hq[static_cast<int64_t>(c.plan.first[s] + r) * a.I + b * 128 + row] = static_cast<uint8_t>(code);
      if (lane == 0) a.hsf[(static_cast<int64_t>(s) * NB + b) * 512 + (r & 31) * 16 + (r >> 5) * 4 + q] = static_cast<uint8_t>(sb);
    };
    for (Walk wk(f0, f1, KA); wk.left > 0 && ok; wk.next()) {
      const int s = wk.unit / NB, b = wk.unit - s * NB, e = c.plan.expert[s];
      const bool whole = wk.steps() == KA;
      const int u0 = wk.unit * KA;
      float* mine = a.part + static_cast<int64_t>(2 * w + (u0 < f0 || wk.left == f1 - f0 ? 0 : 1)) * a.T * 256 + row;
      ok = __all_sync(0xffffffffu, mbar_wait(&c.accf[acc.i], acc.phase, a.status, 205));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.i * 128;
      int r = 0;
#pragma unroll 1
      for (int t0 = 0; t0 < a.T; t0 += 16) {
        const uint32_t m = (c.plan.mask[e][t0 >> 5] >> (t0 & 31)) & 0xffffu;
        if (m == 0) continue;
        uint32_t g[16], u[16];
        tmem_ld16(tacc + t0, g);
        tmem_ld16(tacc + 64 + t0, u);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          reg_fence(g[i]);
          reg_fence(u[i]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((m >> i) & 1u) {
            if (whole) {
              emit(s, r, b, __uint_as_float(g[i]), __uint_as_float(u[i]));
            } else {
              mine[r * 256] = __uint_as_float(g[i]);
              mine[r * 256 + 128] = __uint_as_float(u[i]);
            }
            ++r;
          }
      }
      tc_fence_before();
      mbar_arrive(&c.acce[acc.i]);
      acc.step(2);
      if (whole) continue;
      const int last = owner_of(total, u0 + KA - 1, W);
      const mla::Cut cut = cut_of(total, W, u0, last);
      if (!last_piece(c, a.cnt_up + wk.unit, cut.pieces)) continue;
#pragma unroll 1
      for (int i = 0; i < r; ++i) {
        float g = 0.0f, u = 0.0f;
        for (int p = 0; p < cut.pieces; ++p) {
          const float* src = a.part + static_cast<int64_t>(2 * (cut.worker + p) + (p == 0 ? cut.slot : 0)) * a.T * 256 + row + i * 256;
          g += __ldcg(src);
          u += __ldcg(src + 128);
        }
        emit(s, i, b, g, u);
      }
    }
  }
  few_finish(tmem, ok);
}

// ---------------------------------------------------------------- down projection and combine
// Stage: [128 rows of weights][up to N rows of H], and the scale atoms of both.
__global__ void __launch_bounds__(kThreads, 1)
    few_down_kernel(const __grid_constant__ CUtensorMap tma_w, const __grid_constant__ CUtensorMap tma_h,
                    const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewSmem& c = *reinterpret_cast<FewSmem*>(smem);
  uint8_t* ring = smem + kControl;
  uint8_t* scales = ring + a.nst * a.stage_bytes;          // two atoms a stage
  float* sum = reinterpret_cast<float*>(scales + a.nst * 2 * 512);   // [T][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  few_setup(c, a.nst, &tma_w, &tma_h);
  grid_launch();
  tc_fence_before();
  // The router's choice is complete: the kernel before this one let it start after its own wait for the router.
  make_plan(a, c.plan, false);
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  const int KI = a.I >> 7, RT = a.d >> 7, ns = c.plan.slots;
  const int row_steps = ns * KI;                           // steps of 128 output rows
  const int total = RT * row_steps;
  const int W = workers_of(total, static_cast<int>(gridDim.x), kMinSteps), w = static_cast<int>(blockIdx.x);
  const int f0 = w < W ? range_begin(total, w, W) : total, f1 = w < W ? range_begin(total, w + 1, W) : total;
  bool ok = true;
  if (warp == 0) {
    // Where a step is: expert slot s, rows r, piece k of K.
    struct Step {
      int r, s, k, boxes;
    };
    auto boxes_of = [&](int s) { return (c.plan.first[s + 1] - c.plan.first[s] + 15) >> 4; };
    auto start = [&](int f) {
      const int u = f / KI;
      Step p;
      p.k = f - u * KI;
      p.r = u / ns;
      p.s = u - p.r * ns;
      p.boxes = boxes_of(p.s);
      return p;
    };
    auto next = [&](Step& p) {
      if (++p.k < KI) return;
      p.k = 0;
      if (++p.s == ns) {
        p.s = 0;
        ++p.r;
      }
      p.boxes = boxes_of(p.s);
    };
    auto load_w = [&](const Step& p, int i) {
      uint8_t* dst = ring + i * a.stage_bytes;
      uint64_t* bar = &c.full[i];
      const int row = c.plan.expert[p.s] * a.d + p.r * 128;
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, kTileBytes + p.boxes * 2048 + 2 * 512);
        tma_load_2d(dst, &tma_w, p.k * 128, row, bar);
        bulk_load(scales + i * 1024, a.wsf + (static_cast<int64_t>(row >> 7) * KI + p.k) * 512, 512, bar);
      }
      __syncwarp();
    };
    auto load_h = [&](const Step& p, int i) {
      uint8_t* dst = ring + i * a.stage_bytes + kTileBytes;
      uint64_t* bar = &c.full[i];
      const int row = c.plan.first[p.s];
      if (elect_one()) {
#pragma unroll 1
        for (int j = 0; j < p.boxes; ++j) tma_load_2d(dst + j * 2048, &tma_h, p.k * 128, row + j * 16, bar);
        bulk_load(scales + i * 1024 + 512, a.hsf + (static_cast<int64_t>(p.s) * KI + p.k) * 512, 512, bar);
      }
      __syncwarp();
    };
    const int n = f1 - f0;
    if (n > 0) {
      const int ahead = n < a.nst ? n : a.nst;
      Step p = start(f0), h = p;
      for (int i = 0; i < ahead; ++i) {
        load_w(p, i);
        if (i + 1 < n) next(p);
      }
      grid_wait();
      fence_proxy_async_global();
      for (int i = 0; i < ahead; ++i) {
        load_h(h, i);
        if (i + 1 < n) next(h);
      }
      Stage st;
      st.i = ahead == a.nst ? 0 : ahead;
      st.phase = ahead == a.nst ? 1u : 0u;
      int issued = ahead;
#pragma unroll 1
      for (int i = ahead; i < n; ++i) {
        ok = warp_wait(&c.empty[st.i], st.phase ^ 1u, a.status, 211);
        if (!ok) break;
        load_w(p, st.i);
        load_h(p, st.i);
        if (i + 1 < n) next(p);
        st.step(a.nst);
        ++issued;
      }
      ok = land(c, st, issued, a.nst, a.status, 212) && ok;
    }
  } else if (warp == 1) {
    Stage st, acc;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sf0 = smem_u32(scales);
    for (Walk wk(f0, f1, KI); wk.left > 0 && ok; wk.next()) {
      const int s = wk.unit % ns;
      const int rows = __shfl_sync(0xffffffffu, (c.plan.first[s + 1] - c.plan.first[s] + 15) & ~15, 0);
      const uint32_t idesc = idesc_mxf8(128, 0) | (static_cast<uint32_t>(rows >> 3) << 17);
      ok = warp_wait(&c.acce[acc.i], acc.phase ^ 1u, a.status, 213);
      const int n = __shfl_sync(0xffffffffu, wk.steps(), 0);
      const uint32_t d = tm + acc.i * 64;
#pragma unroll 1
      for (int k = 0; k < n && ok; ++k) {
        ok = warp_wait(&c.full[st.i], st.phase, a.status, 214);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t base = smem_u32(ring + st.i * a.stage_bytes), sf = tm + kSfCol + st.i * 8;
#pragma unroll
          for (int j = 0; j < 2; ++j) tc_cp_sf(sf + 4 * j, desc_sf_chunk(sf0 + st.i * 1024 + 512 * j));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mxf8(d, desc_kmajor_sw128(base + kk * 32), desc_kmajor_sw128(base + kTileBytes + kk * 32),
                        idesc_mxf8_sf(idesc, kk, kk), sf, sf + 4, (k | kk) != 0);
          tc_commit(&c.empty[st.i]);
          if (k == n - 1) tc_commit(&c.accf[acc.i]);
        }
        __syncwarp();
        st.step(a.nst);
      }
      acc.step(4);
    }
  } else {
    const int q = warp & 3, row = q * 32 + lane;
    Stage acc;
    // A token without a valid choice has NaN scores, and so has its sum.
    auto fresh = [&](int t) { return (c.plan.bad[t >> 5] >> (t & 31)) & 1u ? __int_as_float(0x7fffffff) : 0.0f; };
    auto put = [&](int r, int t, float v) { a.y[static_cast<int64_t>(t) * a.d + r * 128 + row] = __float2bfloat16(v); };
    int r = -1;                                            // rows whose sum is under way
    for (Walk wk(f0, f1, KI); wk.left > 0 && ok; wk.next()) {
      const int ur = wk.unit / ns, s = wk.unit - ur * ns;
      if (ur != r) {
        r = ur;
        for (int t = 0; t < a.T; ++t) sum[t * 128 + row] = fresh(t);
      }
      const int row0 = c.plan.first[s], n = c.plan.first[s + 1] - row0;
      ok = __all_sync(0xffffffffu, mbar_wait(&c.accf[acc.i], acc.phase, a.status, 215));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc.i * 64;
#pragma unroll 1
      for (int c0 = 0; c0 < n; c0 += 16) {
        uint32_t o[16];
        tmem_ld16(tacc + c0, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          reg_fence(o[i]);
          if (c0 + i < n) {
            float& v = sum[c.plan.token[row0 + c0 + i] * 128 + row];
            v = fmaf(c.plan.gate[row0 + c0 + i], __uint_as_float(o[i]), v);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&c.acce[acc.i]);
      acc.step(4);
      const int r0 = r * row_steps, at = f1 - wk.left + wk.steps();   // steps done so far
      if (at < f1 && at < r0 + row_steps) continue;        // more of these rows to come
      if (f0 <= r0 && at == r0 + row_steps) {
        for (int t = 0; t < a.T; ++t) put(r, t, sum[t * 128 + row]);
        continue;
      }
      const int last = owner_of(total, r0 + row_steps - 1, W);
      const mla::Cut cut = cut_of(total, W, r0, last);
      float* mine = a.part + static_cast<int64_t>(2 * w + (r0 <= f0 ? 0 : 1)) * a.T * 128 + row;
      for (int t = 0; t < a.T; ++t) mine[t * 128] = sum[t * 128 + row];
      if (!last_piece(c, a.cnt_down + r, cut.pieces)) continue;
#pragma unroll 4
      for (int t = 0; t < a.T; ++t) {
        float v = 0.0f;
        for (int p = 0; p < cut.pieces; ++p)
          v += __ldcg(a.part + static_cast<int64_t>(2 * (cut.worker + p) + (p == 0 ? cut.slot : 0)) * a.T * 128 + t * 128 + row);
        put(r, t, v);
      }
    }
    // No expert at all: every token's scores are NaN.
    if (total == 0) {
      grid_wait();
      for (int u = w; u < RT; u += static_cast<int>(gridDim.x))
        for (int t = 0; t < a.T; ++t) put(u, t, fresh(t));
    }
  }
  few_finish(tmem, ok);
}

struct FewLayout {
  size_t status, cnt_route, cnt_up, cnt_down, logits, xq, xsf, hq, hsf, part, total;
  int64_t ncnt;
};

int64_t slots_of(const moe_config_t* c) {
  const int64_t chosen = static_cast<int64_t>(c->T) * c->k;
  return (chosen < c->E ? chosen : c->E) + c->n_shared;
}

FewLayout few_layout(const moe_config_t* c) {
  FewLayout L{};
  size_t cur = 0;
  auto add = [&](size_t n) {
    const size_t at = cur;
    cur += (n + 1023) / 1024 * 1024;
    return at;
  };
  const size_t T = c->T, slots = slots_of(c);
  L.ncnt = static_cast<int64_t>(slots) * (c->I / 128) + c->d / 128;
  L.status = add(16 + sizeof(int) * kMaxT);
  L.cnt_route = L.status + 16;
  L.cnt_up = add(sizeof(int) * L.ncnt);
  L.cnt_down = L.cnt_up + sizeof(int) * slots * (c->I / 128);
  L.logits = add(sizeof(float) * T * c->E);
  L.xq = add(static_cast<size_t>(kMaxT) * c->d);
  L.xsf = add(static_cast<size_t>(c->d / 128) * 512);
  L.hq = add((T * (c->k + c->n_shared) + 16) * c->I);
  L.hsf = add(slots * (c->I / 128) * 512);
  L.part = add(2 * sizeof(float) * kMaxSms * T * 256);
  L.total = cur;
  return L;
}

int validate_few(const moe_config_t* c) {
  if (int r = validate(c)) return r;
  if (c->T > kMaxT || (c->flags & MOE_FLAG_X_QUANTIZED)) return MOE_ERR_INVALID_ARG;
  // rows of the weights and steps of an expert kernel are counted in 32 bits
  const int64_t lim = (1LL << 31) - 1, Ep = c->E + c->n_shared;
  if (Ep * 2 * c->I > lim || Ep * c->d > lim || Ep * (c->I / 128) * (c->d / 128) > lim) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

inline bool mis(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_few_workspace_size(const moe_config_t* cfg, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  if (int r = validate_few(cfg)) return r;
  *bytes = few_layout(cfg).total;
  return MOE_OK;
}

extern "C" int moe_few_forward(const moe_config_t* cfg, const void* x, const void* w_router, const float* bias, const void* wq,
                               int32_t* topk_idx, float* topk_w, void* y, void* ws, moe_stream_t stream) {
  if (int r = validate_few(cfg)) return r;
  const bool none = cfg->T == 0;
  if (!w_router || !bias || !wq || !ws || (!none && (!x || !topk_idx || !topk_w || !y))) return MOE_ERR_INVALID_ARG;
  if (mis(x, 16) || mis(w_router, 16) || mis(wq, 16) || mis(y, 16) || mis(ws, 16) || mis(bias, 4) || mis(topk_idx, 4) ||
      mis(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  CallScope call;
  if (none) return MOE_OK;
  if (!get_encode()) return MOE_ERR_CUDA;
  static DevOnce once;
  if (!once.ready([] {
        const cudaError_t e = cudaFuncSetAttribute(few_up_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        return e != cudaSuccess ? e : cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
      }))
    return MOE_ERR_CUDA;
  const FewLayout L = few_layout(cfg);
  const WLayout WL = make_wlayout(cfg);
  char* base = static_cast<char*>(ws);
  uint8_t* w = static_cast<uint8_t*>(const_cast<void*>(wq));
  FewArgs a{};
  a.T = cfg->T;
  a.d = cfg->d;
  a.E = cfg->E;
  a.k = cfg->k;
  a.G = cfg->n_groups;
  a.gtop = cfg->topk_groups;
  a.I = cfg->I;
  a.S = cfg->n_shared;
  a.Ep = a.E + a.S;
  a.N = static_cast<int>(round_up(a.T, 16));
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w_router = static_cast<const __nv_bfloat16*>(w_router);
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  a.logits = reinterpret_cast<float*>(base + L.logits);
  a.xq = reinterpret_cast<uint8_t*>(base + L.xq);
  a.xsf = reinterpret_cast<uint8_t*>(base + L.xsf);
  a.hq = reinterpret_cast<uint8_t*>(base + L.hq);
  a.hsf = reinterpret_cast<uint8_t*>(base + L.hsf);
  a.part = reinterpret_cast<float*>(base + L.part);
  a.cnt_route = reinterpret_cast<int*>(base + L.cnt_route);
  a.cnt_up = reinterpret_cast<int*>(base + L.cnt_up);
  a.cnt_down = reinterpret_cast<int*>(base + L.cnt_down);
  a.ncnt = static_cast<int>(L.ncnt);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.status = reinterpret_cast<int*>(base + L.status);
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  CUtensorMap tw1, tw2, tx, th;
  if (!make_tmap(&tw1, wq_ptr<uint8_t>(WL, w, MOE_WQ_W1F), static_cast<int64_t>(a.Ep) * 2 * a.I, a.d, 256, false) ||
      !make_tmap(&tw2, wq_ptr<uint8_t>(WL, w, MOE_WQ_W2F), static_cast<int64_t>(a.Ep) * a.d, a.I, 128, false) ||
      !make_tmap(&tx, a.xq, kMaxT, a.d, a.N, false) ||
      !make_tmap(&th, a.hq, static_cast<int64_t>(a.T) * (a.k + a.S) + 16, a.I, 16, false))
    return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int quant = static_cast<int>(ceil_div(static_cast<int64_t>(a.T) * (a.d / 32), kRouteThreads));
  auto route = [&](auto kern, int tg, int er) {
    const int blocks = static_cast<int>(ceil_div(a.E, 2 * er) * ceil_div(a.T, tg)) + quant;
    launch_kernel_after("few_route", kern, dim3(static_cast<unsigned>(blocks)), dim3(kRouteThreads), 8 * a.E * sizeof(float), s, a);
  };
  if (a.T == 1)
    route(few_route_kernel<1, 1>, 1, 1);
  else
    route(few_route_kernel<8, 2>, 8, 2);
  if (int r = call.status()) return r;
  const int room = kSmemMax - 1024 - kControl;
  auto ring = [&](int tiles, int atoms, int more) {
    a.stage_bytes = tiles * kTileBytes + a.N * 128;
    a.nst = (room - more) / (a.stage_bytes + atoms * 512);
    if (a.nst > kMaxStages) a.nst = kMaxStages;
    return 1024 + kControl + a.nst * (a.stage_bytes + atoms * 512) + more;
  };
  int smem = ring(2, 3, 0);
  a.wsf = wq_ptr<uint8_t>(WL, w, MOE_WQ_W1F_SF);
  launch_kernel_after("few_up", few_up_kernel, dim3(static_cast<unsigned>(sms)), dim3(kThreads), smem, s, tw1, tx, a);
  if (int r = call.status()) return r;
  smem = ring(1, 2, a.T * 128 * static_cast<int>(sizeof(float)));
  a.wsf = wq_ptr<uint8_t>(WL, w, MOE_WQ_W2F_SF);
  launch_kernel_after("few_down", few_down_kernel, dim3(static_cast<unsigned>(sms)), dim3(kThreads), smem, s, tw2, th, a);
  return call.status();
}

extern "C" int moe_few_status(const moe_config_t* cfg, void* ws, int* code, int* site, int clear, moe_stream_t stream) {
  if (int r = validate_few(cfg)) return r;
  if (!ws || !code || !site) return MOE_ERR_INVALID_ARG;
  return read_status(static_cast<char*>(ws) + few_layout(cfg).status, code, site, clear, static_cast<cudaStream_t>(stream));
}
