// The whole layer for up to 64 tokens: router, experts and combine in two
// launches, the second placed while the first still runs.
//
//   route    logits = x Wr^T, the choice of every token (route.cuh), MX(x)
//   experts  [g | u] = Wgu MX(x)^T, h = silu(g) u, o = Wd MX(h)^T, y = sum over a token's experts of w o
//
// Few tokens read many weights: one token of 9 experts with 7168 x 2048 matrices
// reads 410 MB for 0.8 GFLOP, and HBM bounds it (0.4 us of products, 60 us of
// copies). So the weights are the 128-row operand of the tensor cores and the
// tokens the narrow one (16 to 64 columns): a tile of weights goes from HBM
// through shared memory once, for all tokens, and nothing has to be converted,
// gathered or padded to 128 rows.
//
// The work is a list of pieces, which CTAs take from its front one after another:
//   up    256 interleaved gate and up rows of one expert, all of K = d or a part of it.
//         All T tokens are columns, also those that did not choose the expert: a product of
//         16 columns takes the tensor pipe a tenth of the time its weights take to arrive,
//         and X needs no gather. Parts leave g and u in the workspace, and the CTA that
//         stores the last part adds them in their order, forms h and quantises it.
//   down  256 rows of one expert, all of K = I or a part; the expert's tokens are columns.
//         The rows of o go to the workspace in fp32.
// All up pieces come first, and down pieces of an expert wait until its h is
// complete; their weights are loaded without waiting. At the end every CTA waits for the last
// piece and sums a share of y. What a CTA waits for was taken before by a
// CTA that runs and waits for nothing later, so no wait needs all CTAs to be resident. Which CTA
// takes a piece changes no result: parts and sums have a fixed order.
//
// Taken from a list, pieces keep every SM loading to the end: 75 us for one token of 9 such
// experts, 312 to 340 for 16 tokens and 47 experts, 413 to 426 for 64 and 61 (5.5, 6.6 and 6.6 TB/s of the
// weights read). Behind a router of 256 experts: 81 us for one token, 448 for 16 and 67 experts, 748 for 64 and 110.
// The first build of this file, equal ranges fixed in advance in a kernel for each projection, left some SMs
// 15 % behind the others (HBM does not serve all alike) and HBM idle for 9 us between the kernels: 106, 403 and 544 us.
#include <cudaTypedefs.h>

#include "few_pieces.h"
#include "gemm.cuh"
#include "prof.h"
#include "route.cuh"

namespace moe {

namespace {

using few::Piece;
using few::Work;

constexpr int kMaxT = MOE_FEW_MAX_T;
constexpr int kMaxEp = 513;                // experts, a shared one included
constexpr int kMaxPicks = kMaxT * 8;       // routed (token, expert) pairs
constexpr int kThreads = 224;
constexpr int kMaxStages = 6;             // of the ring: 6 fit at 16 tokens, 5 at 64 (4 cost 1 to 2 %, 2 cost 10)
constexpr int kTileBytes = 128 * 128;      // a weight tile: 128 rows x 128 values
constexpr int kSmemMax = 232448;
constexpr int kSfCol = few::kAccCols;      // TMEM: accumulators below, scales of the ring's stages from here on
static_assert(kSfCol + 12 * kMaxStages <= 512, "TMEM columns");
constexpr int kQueue = 4;                  // pieces on their way from the warp that takes them to the others
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
  const uint8_t* w1sf;                     // scales of the weights
  const uint8_t* w2sf;
  uint8_t* hq;                             // [rows][I], an expert's tokens one after another
  uint8_t* hsf;                            // [experts in use][I / 128] atoms
  float* gu;                               // [rows][I / 128][parts][256]: parts of g and u
  float* o;                                // [rows][parts][d]
  int* cnt_route;                          // per token group: CTAs done
  int* cnt;                                // counters of `experts`, cleared by `route`: pieces taken, pieces of down done,
  int ncnt;                                // then per expert slot its blocks of h done, then per block its parts done
  __nv_bfloat16* y;
  int* status;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, site));
}
// Barrier over the epilogue's 128 threads that also gives the OR of their flags.
__device__ __forceinline__ bool epilogue_or(bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(flag))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One column of two accumulators, and four.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
// Counts an arrival after a CTA barrier: what the CTA's threads wrote before the barrier is released with it, and what earlier
// arrivals released is acquired. (A fence by every thread before the barrier took 4 to 8 us while the rings are loading.)
__device__ __forceinline__ int atom_add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// ---------------------------------------------------------------- route
// Logits: the eight warps of a CTA share the columns of ER rows of Wr, for TG tokens, in
// fp32 on the CUDA cores: one round of loads at 7168 columns for one token, two for eight, where the tensor cores would wait
// for one CTA's chain of 112 stages. One token, 64 experts: logits after 2.0 us, the last CTA found after 3.2, the choice
// written after 5.3. The CTA that finishes a group of tokens last
// chooses for them. Further CTAs quantise x and clear the counters of the kernel that follows.
constexpr int kRouteThreads = 256;
constexpr int kRowWarps = kRouteThreads / 32;

template <int TG, int ER, int PER>
__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kDeep = TG == 1 ? 4 : 2;                   // chunks of 256 columns whose loads are under way together
  __shared__ float red[kRowWarps][ER * TG];
  __shared__ int last;
  extern __shared__ float sv_all[];                        // [8][E] for the choosing warps, [E] bias
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NE = (a.E + ER - 1) / ER, NG = (a.T + TG - 1) / TG;
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
    for (int i = (bid - NE * NG) * kRouteThreads + tid; i < a.ncnt; i += step) a.cnt[i] = 0;
    return;
  }
  const int g = bid / NE, e0 = (bid - g * NE) * ER;
  float* bias = sv_all + 8 * a.E;                          // read ahead: the choice then waits for the logits alone
  for (int e = tid; e < a.E; e += kRouteThreads) bias[e] = __int_as_float(ld_global_s32(reinterpret_cast<const int*>(a.bias + e)));
  float acc[ER][TG];
#pragma unroll
  for (int r = 0; r < ER; ++r)
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[r][t] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c0 = warp * 256; c0 < a.d; c0 += kDeep * kRowWarps * 256) {
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
      if (lane == 0) red[warp][r * TG + t] = acc[r][t];
    }
  __syncthreads();
  if (tid < ER * TG) {
    const int e = e0 + tid / TG, t = g * TG + tid % TG;
    float v = red[0][tid];
#pragma unroll
    for (int p = 1; p < kRowWarps; ++p) v += red[p][tid];
    if (e < a.E && t < a.T) a.logits[static_cast<int64_t>(t) * a.E + e] = v;
  }
  __syncthreads();
  if (tid == 0) last = atom_add_acq_rel(a.cnt_route + g, 1) == NE - 1;
  __syncthreads();
  if (!last) return;
  if (tid == 0) a.cnt_route[g] = 0;
#pragma unroll 1
  for (int i = warp; i < TG; i += 8) {
    const int t = g * TG + i;
    if (t >= a.T) break;
    int e;
    float s, tot;
    choose_experts<PER, BestByRedux>([&](int n) { return __ldcg(a.logits + static_cast<int64_t>(t) * a.E + n); },
                       [&](int n) { return bias[n]; }, a.E, a.k, a.G, a.gtop, sv_all + warp * a.E, lane, e, s, tot);
    if (lane < a.k) {
      a.idx[t * a.k + lane] = e;
      a.w[t * a.k + lane] = __fdiv_rn(s, tot);
    }
  }
}

// ---------------------------------------------------------------- the experts in use
// Which tokens chose which expert, made by every CTA for itself from the router's choice: a 64-bit mask of tokens per
// expert, the experts in use in ascending order, and their tokens' rows one after another. A shared expert is number 0, and
// expert e number e + n_shared.
struct FewPlan {
  uint32_t mask[kMaxEp][2];
  uint16_t expert[kMaxEp];                 // of a slot
  uint16_t slot[kMaxEp];                   // of an expert in use
  uint16_t first[kMaxEp + 1];              // row of a slot's first token
  uint16_t row[kMaxPicks];                 // of a token's pick
  float gate[kMaxPicks];
  uint32_t bad[2];                         // tokens without a valid choice (biases of NaN)
  uint32_t scan[kThreads / 32];
  int slots;
};

__device__ __forceinline__ void make_plan(const FewArgs& a, FewPlan& p, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // This thread's picks: expert and gate, read together.
  constexpr int kPicks = (kMaxPicks + kThreads - 1) / kThreads;
  const int n = a.T * a.k;
  int pick[kPicks];
  float gate[kPicks];
#pragma unroll
  for (int j = 0; j < kPicks; ++j) {
    const int i = tid + j * kThreads;
    pick[j] = i < n ? ld_global_s32(a.idx + i) : 0;
    gate[j] = i < n ? __int_as_float(ld_global_s32(reinterpret_cast<const int*>(a.w + i))) : 0.0f;
  }
  for (int i = tid; i < a.Ep; i += kThreads) p.mask[i][0] = p.mask[i][1] = 0;
  if (tid < 2) p.bad[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPicks; ++j) {
    const int i = tid + j * kThreads;
    if (i >= n) break;
    const int e = pick[j], t = i / a.k;
    const bool ok = e >= 0 && e < a.E;
    atomicOr(ok ? &p.mask[e + a.S][t >> 5] : &p.bad[t >> 5], 1u << (t & 31));
    if (!ok && report) report_error(a.status, kErrBounds, 200);
  }
  if (a.S > 0 && tid < 2) p.mask[0][tid] = tid * 32 >= a.T ? 0u : (a.T - tid * 32 >= 32 ? 0xffffffffu : (1u << (a.T - tid * 32)) - 1u);
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
#pragma unroll
  for (int j = 0; j < kPicks; ++j) {
    const int i = tid + j * kThreads;
    if (i >= n) break;
    const int e = pick[j], t = i / a.k;
    if (e < 0 || e >= a.E) continue;
    const uint32_t* m = p.mask[e + a.S];
    const uint32_t below = t < 32 ? __popc(m[0] & ((1u << t) - 1u)) : __popc(m[0]) + __popc(m[1] & ((1u << (t - 32)) - 1u));
    p.row[i] = static_cast<uint16_t>(p.first[p.slot[e + a.S]] + below);
    p.gate[i] = gate[j];
  }
  __syncthreads();
}

struct FewSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t accf[few::kMaxSlots], acce[few::kMaxSlots];   // of accumulator slots: a piece that ends there is done; read
  uint64_t qf[kQueue], qe[kQueue];
  int queue[kQueue];                       // pieces, -1 after the last
  uint32_t tmem;
  int last;
  FewPlan plan;
};
constexpr int kControl = (sizeof(FewSmem) + 1023) / 1024 * 1024;

// Place in a ring.
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

// y from the rows of o, by the epilogue's four warps: blocks of 128 columns of a token, IT at once. A warp adds every fourth of the
// token's experts, and the four sums (in `sums`, shared memory) are added in order.
// Not inlined, so that a first call which only goes through it (`real` false: it reads and writes no global memory) fetches
// the code while the router works: at the end of the list, one miss after another, that took 6 of 54 us at 5 tokens (in the
// build before this).
template <int IT>
__device__ __noinline__ void sum_blocks(const FewArgs& a, const FewPlan& p, float4* sums_, int PD, bool real) {
  float4 (*sums)[4][32] = reinterpret_cast<float4 (*)[4][32]>(sums_);
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  // (copies: a reference into the kernel's parameters would be read again after every barrier)
  const int d = a.d, k0 = a.k, picks = a.k + a.S;
  const float* o = a.o;
  __nv_bfloat16* out = a.y;
  const int cols = d >> 7, ctas = static_cast<int>(gridDim.x);
  const int begin = static_cast<int>(blockIdx.x), units = real ? a.T * cols : begin + 1;
#pragma unroll 1
  for (int u0 = begin; u0 < units; u0 += IT * ctas) {
    const float4* src[IT][3];
    float gate[IT][3];
    float4 v[IT][3];
#pragma unroll
    for (int n = 0; n < IT; ++n) {
      const bool some = real && u0 + n * ctas < units;
      const int u = some ? u0 + n * ctas : 0, t = u / cols, col = (u - t * cols) * 128 + lane * 4;
      const bool bad = (p.bad[t >> 5] >> (t & 31)) & 1u;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int j = warp + 4 * i;
        const bool has = some && (j < k0 ? !bad : j < picks);
        const int r = !has ? 0 : (j < k0 ? p.row[t * k0 + j] : t);                 // (the shared expert's rows are the first)
        gate[n][i] = !has ? 0.0f : (j < k0 ? p.gate[t * k0 + j] : 1.0f);
        src[n][i] = has ? reinterpret_cast<const float4*>(o + static_cast<int64_t>(r) * PD * d + col) : nullptr;
        v[n][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
#pragma unroll 1
    for (int k = 0; k < PD; ++k) {
      float4 x[IT][3];
#pragma unroll
      for (int n = 0; n < IT; ++n)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          x[n][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (src[n][i] != nullptr) x[n][i] = ld_global_f4(src[n][i] + static_cast<int64_t>(k) * (d >> 2));
        }
      __syncwarp();                                        // all of them are issued before the first is added
#pragma unroll
      for (int n = 0; n < IT; ++n)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          v[n][i] = make_float4(v[n][i].x + x[n][i].x, v[n][i].y + x[n][i].y, v[n][i].z + x[n][i].z, v[n][i].w + x[n][i].w);
    }
#pragma unroll
    for (int n = 0; n < IT; ++n) {
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (src[n][i] != nullptr)
          y = make_float4(fmaf(gate[n][i], v[n][i].x, y.x), fmaf(gate[n][i], v[n][i].y, y.y), fmaf(gate[n][i], v[n][i].z, y.z),
                          fmaf(gate[n][i], v[n][i].w, y.w));
      sums[n][warp][lane] = y;
    }
    named_barrier(1, 128);
    if (warp < IT) {                                       // a warp finishes a block
      const int u = u0 + warp * ctas, t = u / cols, col = (u - t * cols) * 128 + lane * 4;
      // A token without a valid choice: NaN.
      const float zero = u < units && (p.bad[(t >> 5) & 1] >> (t & 31)) & 1u ? __int_as_float(0x7fffffff) : 0.0f;
      float4 y = make_float4(zero, zero, zero, zero);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = sums[warp][i][lane];
        y = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
      }
      if (real && u < units)
        *reinterpret_cast<uint2*>(out + static_cast<int64_t>(t) * d + col) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    }
    named_barrier(1, 128);
  }
}
// One block at once where there is no more than one a CTA. With four throughout (more code to fetch) one token takes 75.7 us
// instead of 74.9 and five of narrow experts 49.4 instead of 47.1; with one throughout 64 tokens take 431 instead of 417. Between
// them one would do a little better (4 tokens 173 instead of 175, 16 of narrow experts 75.4 instead of 77.0).
__device__ __forceinline__ void sum_y(const FewArgs& a, const FewPlan& p, float4* sums, int PD, bool real) {
  if (a.T * (a.d >> 7) <= static_cast<int>(gridDim.x)) sum_blocks<1>(a, p, sums, PD, real);
  else sum_blocks<4>(a, p, sums, PD, real);
}

// Warps: 0 takes pieces and loads weights, 6 loads X and H, 1 issues the products, 2-5 epilogue (row = TMEM lane).
// Stage: [256 rows of weights][N rows of X or H], and three scale atoms.
__global__ void __launch_bounds__(kThreads, 1)
    few_experts_kernel(const __grid_constant__ CUtensorMap tma_w1, const __grid_constant__ CUtensorMap tma_w2,
                       const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_h,
                       const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewSmem& c = *reinterpret_cast<FewSmem*>(smem);
  uint8_t* ring = smem + kControl;
  uint8_t* scales = ring + a.nst * a.stage_bytes;          // three atoms a stage
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < a.nst; ++i) {
      mbar_init(&c.full[i], 2);                            // the two loading warps
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < few::kMaxSlots; ++i) {
      mbar_init(&c.accf[i], 1);
      mbar_init(&c.acce[i], 128);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&c.qf[i], 1);
      mbar_init(&c.qe[i], 6);                              // the other warps
    }
    fence_barrier_init();
    fence_proxy_async();
    tma_prefetch(&tma_w1);
    tma_prefetch(&tma_w2);
    tma_prefetch(&tma_x);
    tma_prefetch(&tma_h);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  if (warp >= 2 && warp < 6) {
    sum_y(a, c.plan, reinterpret_cast<float4*>(ring), 1, false);
    fence_proxy_async();                                   // (copies into the ring come after its stores)
  }
  grid_wait();
  grid_launch();
  // The first piece, on its way while the plan is made. It is taken like all others: given by a CTA's number it could be one
  // that others wait for while its CTA has no SM (two such kernels at once).
  int first = 0;
  if (tid == 0) first = atomicAdd(a.cnt, 1);
  tc_fence_before();
  make_plan(a, c.plan, blockIdx.x == 0);                   // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  Work w;
  few::work_of(w, a, c.plan, static_cast<int>(gridDim.x));
  int* done = a.cnt + 1;
  int* ready = a.cnt + 2;
  int* parts = ready + w.slots;
  const int slots = few::acc_slots(a.N);                   // of accumulators
  bool ok = true;
  // The next piece, for the warps that follow warp 0.
  Stage q;
  auto next_piece = [&]() {
    ok = warp_wait(&c.qf[q.i], q.phase, a.status, 201);
    if (!ok) return -1;
    const int id = *reinterpret_cast<volatile int*>(&c.queue[q.i]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.qe[q.i]);
    q.step(kQueue);
    return __shfl_sync(0xffffffffu, id, 0);
  };
  // Every copy that this warp issued has landed.
  auto land = [&](Stage st, int issued) {
    for (int i = 0, n = issued < a.nst ? issued : a.nst; i < n; ++i) {
      if (--st.i < 0) {
        st.i = a.nst - 1;
        st.phase ^= 1u;
      }
      ok = ok && warp_wait(&c.full[st.i], st.phase, a.status, 202);   // (the CTA stays a while after a wait that gave up)
    }
  };
  if (warp == 0) {
    Stage st;
    int issued = 0;
    int id = __shfl_sync(0xffffffffu, first, 0);
    while (ok) {
      const bool more = id < w.total;
      ok = warp_wait(&c.qe[q.i], q.phase ^ 1u, a.status, 203);
      if (!ok) break;
      int ahead = 0;
      if (lane == 0) {
        *reinterpret_cast<volatile int*>(&c.queue[q.i]) = more ? id : -1;
        mbar_arrive(&c.qf[q.i]);
        if (more) ahead = atomicAdd(a.cnt, 1);             // its latency passes behind this piece's loads
      }
      __syncwarp();
      q.step(kQueue);
      if (!more) break;
      const Piece p = few::piece_of(w, id);
      const int n = c.plan.expert[p.s], e = n < a.S ? a.E : n - a.S, K = p.up ? w.KA : w.KI;   // (e: its place in the weights)
      const int row = __shfl_sync(0xffffffffu, p.up ? e * 2 * a.I + p.b * 256 : e * a.d + p.b * 256, 0);
      const int tiles = p.up || 2 * p.b + 1 < w.KA ? 2 : 1;
      const CUtensorMap* map = p.up ? &tma_w1 : &tma_w2;
      const uint8_t* sf = (p.up ? a.w1sf : a.w2sf) + static_cast<int64_t>(row >> 7) * K * 512;
#pragma unroll 1
      for (int k = p.k0; k < p.k1; ++k) {
        ok = warp_wait(&c.empty[st.i], st.phase ^ 1u, a.status, 204);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* dst = ring + st.i * a.stage_bytes;
          uint8_t* sfd = scales + st.i * (3 * 512);
          uint64_t* bar = &c.full[st.i];
          mbar_arrive_expect_tx(bar, tiles * (kTileBytes + 512));
          tma_load_2d(dst, map, k * 128, row, bar);
          if (tiles == 2) tma_load_2d(dst + kTileBytes, map, k * 128, row + 128, bar);
          bulk_load(sfd, sf + static_cast<int64_t>(k) * 512, 512, bar);
          if (tiles == 2) bulk_load(sfd + 512, sf + static_cast<int64_t>(K + k) * 512, 512, bar);
        }
        __syncwarp();
        st.step(a.nst);
        ++issued;
      }
      id = __shfl_sync(0xffffffffu, ahead, 0);
    }
    land(st, issued);
  } else if (warp == 6) {
    Stage st;
    int issued = 0;
    int have = -1;                                         // the last expert whose h was found complete
    for (int id; ok && (id = next_piece()) >= 0;) {
      const Piece p = few::piece_of(w, id);
      const int row = p.up ? 0 : c.plan.first[p.s];
      const int boxes = p.up ? a.N >> 4 : (c.plan.first[p.s + 1] - row + 15) >> 4;
      const CUtensorMap* map = p.up ? &tma_x : &tma_h;
      const uint8_t* sf = p.up ? a.xsf : a.hsf + static_cast<int64_t>(p.s) * w.KI * 512;
      if (!p.up && p.s != have) {
        ok = __all_sync(0xffffffffu, wait_counter(ready + p.s, w.NB, a.status, 205));
        if (!ok) break;
        fence_proxy_async_global();
        have = p.s;
      }
#pragma unroll 1
      for (int k = p.k0; k < p.k1; ++k) {
        ok = warp_wait(&c.empty[st.i], st.phase ^ 1u, a.status, 206);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* dst = ring + st.i * a.stage_bytes + 2 * kTileBytes;
          uint64_t* bar = &c.full[st.i];
          mbar_arrive_expect_tx(bar, boxes * 2048 + 512);
#pragma unroll 1
          for (int j = 0; j < boxes; ++j) tma_load_2d(dst + j * 2048, map, k * 128, row + j * 16, bar);
          bulk_load(scales + st.i * (3 * 512) + 1024, sf + static_cast<int64_t>(k) * 512, 512, bar);
        }
        __syncwarp();
        st.step(a.nst);
        ++issued;
      }
    }
    land(st, issued);
  } else if (warp == 1) {
    Stage st;
    int slot = 0;                                          // of the next chunk
    uint32_t used = 0;                                     // bit s: parity of slot s's uses
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sf0 = smem_u32(scales);
    for (int id; ok && (id = next_piece()) >= 0;) {
      const Piece p = few::piece_of(w, id);
      const int tiles = p.up || 2 * p.b + 1 < w.KA ? 2 : 1;
      const int cols = __shfl_sync(0xffffffffu, p.up ? a.N : (c.plan.first[p.s + 1] - c.plan.first[p.s] + 15) & ~15, 0);
      const uint32_t idesc = idesc_mxf8(128, 0) | (static_cast<uint32_t>(cols >> 3) << 17);
      const int chunks = few::chunks_of(p, a.N);
      int k = p.k0;
#pragma unroll 1
      for (int chunk = 0; chunk < chunks && ok; ++chunk) {
        ok = warp_wait(&c.acce[slot], (used >> slot & 1u) ^ 1u, a.status, 207);
        used ^= 1u << slot;
        const uint32_t d = tm + slot * 2 * a.N;
        const int end = few::chunk_at(p, chunk + 1, chunks);
        uint32_t more = 0;                                 // the chunk's first product starts its sums
#pragma unroll 1
        for (; k < end && ok; ++k) {
          ok = warp_wait(&c.full[st.i], st.phase, a.status, 208);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t base = smem_u32(ring + st.i * a.stage_bytes), sf = tm + kSfCol + st.i * 12, sfs = sf0 + st.i * (3 * 512);
            tc_cp_sf(sf + 8, desc_sf_chunk(sfs + 1024));
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (j < tiles) {
                tc_cp_sf(sf + 4 * j, desc_sf_chunk(sfs + 512 * j));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_mxf8(d + a.N * j, desc_kmajor_sw128(base + j * kTileBytes + kk * 32),
                              desc_kmajor_sw128(base + 2 * kTileBytes + kk * 32), idesc_mxf8_sf(idesc, kk, kk), sf + 4 * j, sf + 8,
                              more | (kk > 0));
              }
            tc_commit(&c.empty[st.i]);
            if (k == p.k1 - 1) tc_commit(&c.accf[slot]);
          }
          __syncwarp();
          st.step(a.nst);
          more = 1;
        }
        if (++slot == slots) slot = 0;
      }
    }
  } else {
    const int lq = warp & 3, row = lq * 32 + lane;
    int slot = 0;                                          // of the next piece's first chunk
    uint32_t seen = 0;                                     // bit s: parity of the pieces that ended in slot s
    // MX(h) of a token: its 32 values lie in the warp's lanes. silu by the fast exponential and quotient, as in the layer's own
    // epilogue: off by about (6 + 1.2 |g|) 2^-23 of itself, where the E4M3 code that h is rounded to has a half step of 2^-4.
    auto emit = [&](int s, int r, int b, float g, float u) {
      const float h = __fdividef(g, 1.0f + __expf(-g)) * u;
      const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h)));
      const int sb = mx_scale_byte(__uint_as_float(top));
      const uint32_t code = e4m3x2(h * mx_inv_scale(sb), 0.0f) & 0xffu;
      a.hq[static_cast<int64_t>(c.plan.first[s] + r) * a.I + b * 128 + row] = static_cast<uint8_t>(code);
      if (lane == 0) a.hsf[(static_cast<int64_t>(s) * w.KI + b) * 512 + (r & 31) * 16 + (r >> 5) * 4 + lq] = static_cast<uint8_t>(sb);
    };
    while (true) {
      const int id = next_piece();
      const Piece p = few::piece_of(w, id >= 0 ? id : 0);
      const int chunks = few::chunks_of(p, a.N);
      const int first = slot;
      slot += chunks;
      const int last = slot - 1 < slots ? slot - 1 : slot - 1 - slots;
      if (slot >= slots) slot -= slots;
      if (id >= 0) ok = mbar_wait(&c.accf[last], seen >> last & 1u, a.status, 209);
      seen ^= 1u << last;
      // Whether a wait gave up is the answer of all four warps, which meet at barriers below.
      ok = !epilogue_or(!ok);
      if (!ok || id < 0) break;
      tc_fence_after();
      const int row0 = c.plan.first[p.s], n = c.plan.first[p.s + 1] - row0;
      // The piece's accumulators have been read.
      auto give_back = [&]() {
        tc_fence_before();
#pragma unroll 1
        for (int j = 0, s = first; j < chunks; ++j) {
          mbar_arrive(&c.acce[s]);
          if (++s == slots) s = 0;
        }
      };
      const uint32_t tacc = tmem + (static_cast<uint32_t>(lq * 32) << 16) + first * 2 * a.N;
      if (p.up) {
        const int e = c.plan.expert[p.s];
        const bool whole = w.PU == 1;
        // parts of row r: gu + r * gu_step, the next part 256 floats on
        const int64_t gu_step = static_cast<int64_t>(w.NB) * w.PU * 256;
        float* gu = a.gu + (static_cast<int64_t>(row0) * w.NB + p.b) * w.PU * 256 + row;
        // A token at a time, in a loop: its code is fetched while the rings are loading, 5 us a miss, and unrolled it took 15 us.
        uint64_t m = static_cast<uint64_t>(c.plan.mask[e][1]) << 32 | c.plan.mask[e][0];
#pragma unroll 1
        for (int r = 0; m != 0; ++r, m &= m - 1) {
          const int t = __ffsll(static_cast<long long>(m)) - 1;
          float g = 0.0f, u = 0.0f;
#pragma unroll 1
          for (int j = 0; j < chunks; ++j) {
            const int back = first + j < slots ? j : j - slots;
            uint32_t x[2];
            tmem_ld1(tacc + back * 2 * a.N + t, x[0]);
            tmem_ld1(tacc + (back * 2 + 1) * a.N + t, x[1]);
            tmem_wait_ld();
            reg_fence(x[0]);
            reg_fence(x[1]);
            g += __uint_as_float(x[0]);
            u += __uint_as_float(x[1]);
          }
          if (whole) {
            emit(p.s, r, p.b, g, u);
          } else {
            float* to = gu + r * gu_step + p.part * 256;
            to[0] = g;
            to[128] = u;
          }
        }
        give_back();
        if (!whole) {
          // The CTA that stores a block's last part adds all of them.
          named_barrier(1, 128);
          if (tid == 64) c.last = atom_add_acq_rel(parts + p.s * w.NB + p.b, 1) == w.PU - 1;
          named_barrier(1, 128);
          if (c.last == 0) continue;
#pragma unroll 1
          for (int i = 0; i < n; i += 2) {
            float g[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
            const float* src = gu + i * gu_step;
            const int64_t two = i + 1 < n ? gu_step : 0;
#pragma unroll 4
            for (int k = 0; k < w.PU; ++k) {
              g[0] += __ldcg(src + k * 256);
              u[0] += __ldcg(src + k * 256 + 128);
              g[1] += __ldcg(src + two + k * 256);
              u[1] += __ldcg(src + two + k * 256 + 128);
            }
            emit(p.s, i, p.b, g[0], u[0]);
            if (i + 1 < n) emit(p.s, i + 1, p.b, g[1], u[1]);
          }
        }
        // h is read by copies of other CTAs.
        fence_proxy_async_global();
        named_barrier(1, 128);
        if (tid == 64) red_release_add(ready + p.s, 1);
      } else {
        const int tiles = 2 * p.b + 1 < w.KA ? 2 : 1;
        float* o = a.o + (static_cast<int64_t>(row0) * w.PD + p.part) * a.d + p.b * 256 + row;
        const int64_t o_step = static_cast<int64_t>(w.PD) * a.d;
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += 4) {
          uint32_t v[2][4];
          tmem_ld4(tacc + c0, v[0]);
          tmem_ld4(tacc + a.N + c0, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              reg_fence(v[j][i]);
              if (j < tiles && c0 + i < n) o[(c0 + i) * o_step + j * 128] = __uint_as_float(v[j][i]);
            }
        }
        give_back();
        named_barrier(1, 128);
        if (tid == 64) red_release_add(done, 1);
      }
    }
    // ---- y, when all rows of o are there: every CTA takes a share
    if (ok) {
      if (tid == 64) c.last = wait_counter(done, w.total - w.nup, a.status, 210);
      named_barrier(1, 128);
      ok = c.last != 0;
    }
    if (ok) sum_y(a, c.plan, reinterpret_cast<float4*>(ring), w.PD, true);   // (every copy into the ring has been used)
  }
  tc_fence_before();
  if (__syncthreads_or(!ok)) drain_pause();
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

struct FewLayout {
  size_t status, cnt_route, cnt, logits, xq, xsf, hq, hsf, gu, o, total;
  int64_t ncnt;
};

// Most experts in use.
int64_t most_slots(const moe_config_t* c) {
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
  const size_t T = c->T, slots = most_slots(c), rows = T * (c->k + c->n_shared), d = c->d, I = c->I;
  L.ncnt = static_cast<int64_t>(2 + slots + slots * (I / 128));
  L.status = add(16 + sizeof(int) * kMaxT);
  L.cnt_route = L.status + 16;
  L.cnt = add(sizeof(int) * L.ncnt);
  L.logits = add(sizeof(float) * T * c->E);
  L.xq = add(kMaxT * d);
  L.xsf = add(d / 128 * 512);
  L.hq = add((rows + 16) * I);
  L.hsf = add(slots * (I / 128) * 512);
  const int64_t I128 = c->I / 128, d128 = c->d / 128, picks = c->k + c->n_shared;
  const size_t gu = few::parts_room(c->T, picks, kMaxSms, d128, I128, few::kUpPieces);
  const size_t o = few::parts_room(c->T, picks, kMaxSms, I128, (d128 + 1) / 2, few::kDownPieces);
  L.gu = add(gu * I128 * 256 * sizeof(float));
  L.o = add(o * d * sizeof(float));
  L.total = cur;
  return L;
}

int validate_few(const moe_config_t* c) {
  if (int r = validate(c)) return r;
  if (c->T > kMaxT || (c->flags & MOE_FLAG_X_QUANTIZED)) return MOE_ERR_INVALID_ARG;
  // rows of the weights and steps of an expert kernel are counted in 32 bits
  const int64_t lim = (1LL << 31) - 1, Ep = c->E + c->n_shared;
  if (Ep * 2 * c->I > lim || Ep * c->d > lim || 4 * Ep * (c->I / 128) * (c->d / 128) > lim) return MOE_ERR_INVALID_ARG;
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
  if (!once.ready([] { return cudaFuncSetAttribute(few_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax); }))
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
  a.gu = reinterpret_cast<float*>(base + L.gu);
  a.o = reinterpret_cast<float*>(base + L.o);
  a.cnt_route = reinterpret_cast<int*>(base + L.cnt_route);
  a.cnt = reinterpret_cast<int*>(base + L.cnt);
  a.ncnt = static_cast<int>(L.ncnt);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.status = reinterpret_cast<int*>(base + L.status);
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  a.w1sf = wq_ptr<uint8_t>(WL, w, MOE_WQ_W1F_SF);
  a.w2sf = wq_ptr<uint8_t>(WL, w, MOE_WQ_W2F_SF);
  CUtensorMap tw1, tw2, tx, th;
  if (!make_tmap(&tw1, wq_ptr<uint8_t>(WL, w, MOE_WQ_W1F), static_cast<int64_t>(a.Ep) * 2 * a.I, a.d, 128, false) ||
      !make_tmap(&tw2, wq_ptr<uint8_t>(WL, w, MOE_WQ_W2F), static_cast<int64_t>(a.Ep) * a.d, a.I, 128, false) ||
      !make_tmap(&tx, a.xq, kMaxT, a.d, 16, false) ||
      !make_tmap(&th, a.hq, static_cast<int64_t>(a.T) * (a.k + a.S) + 16, a.I, 16, false))
    return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int quant = static_cast<int>(ceil_div(static_cast<int64_t>(a.T) * (a.d / 32), kRouteThreads));
  auto route = [&](auto kern, int tg, int er) {
    const int blocks = static_cast<int>(ceil_div(a.E, er) * ceil_div(a.T, tg)) + quant;
    launch_kernel_after("few_route", kern, dim3(static_cast<unsigned>(blocks)), dim3(kRouteThreads), 9 * a.E * sizeof(float), s, a);
  };
  const int per = static_cast<int>(ceil_div(a.E, 32));     // experts a lane of the choosing warp
  // A row of Wr for one token, or two rows for eight. Whole calls of 7168 columns, in us: with 64 experts 75 and 77 for 1 token,
  // 120 and 122 for 2, 171 and 175 for 4, 327 and 330 for 16, 425 and 417 for 64; with 256 experts 80 and 84, 127 and 130, 194
  // and 197, 452 and 447, 773 and 748. (So the border could lie a little higher, at 4 to 16 tokens as the experts are.)
  if (a.T <= 2) {
    if (per <= 2) route(few_route_kernel<1, 1, 2>, 1, 1);
    else if (per <= 4) route(few_route_kernel<1, 1, 4>, 1, 1);
    else if (per <= 8) route(few_route_kernel<1, 1, 8>, 1, 1);
    else route(few_route_kernel<1, 1, 16>, 1, 1);
  } else {
    if (per <= 2) route(few_route_kernel<8, 2, 2>, 8, 2);
    else if (per <= 4) route(few_route_kernel<8, 2, 4>, 8, 2);
    else if (per <= 8) route(few_route_kernel<8, 2, 8>, 8, 2);
    else route(few_route_kernel<8, 2, 16>, 8, 2);
  }
  if (int r = call.status()) return r;
  a.stage_bytes = 2 * kTileBytes + a.N * 128;
  a.nst = (kSmemMax - 1024 - kControl) / (a.stage_bytes + 3 * 512);
  if (a.nst > kMaxStages) a.nst = kMaxStages;
  launch_kernel_after("few_experts", few_experts_kernel, dim3(static_cast<unsigned>(sms)), dim3(kThreads),
                      1024 + kControl + a.nst * (a.stage_bytes + 3 * 512), s, tw1, tw2, tx, th, a);
  return call.status();
}

extern "C" int moe_few_status(const moe_config_t* cfg, void* ws, int* code, int* site, int clear, moe_stream_t stream) {
  if (int r = validate_few(cfg)) return r;
  if (!ws || !code || !site) return MOE_ERR_INVALID_ARG;
  return read_status(static_cast<char*>(ws) + few_layout(cfg).status, code, site, clear, static_cast<cudaStream_t>(stream));
}
