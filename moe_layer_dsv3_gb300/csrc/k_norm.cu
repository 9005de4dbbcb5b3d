// Residual add + RMSNorm with the MX quantisation of its output, and its
// gradient.
//
//   h = x + r,  rstd = (mean(h^2) + eps)^(-1/2),  y = h rstd gamma
//   dx = dr = rstd (g - xhat mean(g xhat)) + dres,  g = dy gamma, xhat = h rstd
//   dgamma = sum over rows of dy xhat
//
// Both directions move each element once and compute a dozen operations on
// it, so HBM bounds them: a row stays on chip (in registers forward, in shared
// memory backward, where rows arrive ahead of their turn) between its reduction
// and its outputs. Measured at 16384 x 7168: forward with residual and codes 151 us
// (1.06 GB, 1.04 of the copy rate), backward 135 us (0.94 GB, 1.03); one row forward
// takes 2.5 us on the device. Sums, rstd and dgamma are held in fp32; h, y and dx are
// rounded to bf16 once, at the store. The codes are MX of the rounded y: the layer's
// experts then read the same bytes as if they had quantised the bf16 rows.
#include "moe_internal.h"
#include "mx.cuh"
#include "prof.h"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads that share a row: a warp (kWarpRow), or the CTA. `red`
// holds 32 floats per parity; the caller alternates parity so that a fast warp
// cannot overwrite sums that a slow one still reads.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (!kWarpRow) {
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum((threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f);
  }
  return v;
}

}  // namespace

struct NormArgs {
  int T, d, rows;            // rows: T, or ceil128(T) when the tiled scales' padding rows are written too
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;    // or null
  const __nv_bfloat16* gamma;
  float eps;
  __nv_bfloat16* h;          // or null
  __nv_bfloat16* y;
  float* rstd;               // or null
  uint8_t* codes;            // or null
  uint8_t* sf;               // row-major scales [T][d / 32], or null
  uint8_t* sf_tiled;         // tiled scales, or null
};

// Thread i of the row's group holds vectors (8 bf16) i, i + n, ..., V in all.
// Four neighbouring lanes hold one MX block, so its maximum takes two shuffles.
template <int V, bool kWarpRow>
__global__ void add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[32];
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int i0 = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= a.rows) return;   // whole warp, or whole CTA
  const int nvec = a.d >> 3;
  const int64_t base = row * a.d;
  if (row >= a.T) {            // padding rows of the tiled layout: zero codes, zero scale bytes
    const int64_t kt = a.d >> 7;
    for (int i = i0; i < nvec; i += nt) {
      *reinterpret_cast<uint2*>(a.codes + base + i * 8) = make_uint2(0, 0);
      if ((i & 3) == 0) a.sf_tiled[sf_off(row, i >> 2, kt)] = 0;
    }
    return;
  }
  uint4 ux[V], ur[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = i0 + j * nt;
    ux[j] = i < nvec ? ld_global_u4(a.x + base + i * 8) : make_uint4(0, 0, 0, 0);
  }
  if (a.r != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = i0 + j * nt;
      ur[j] = i < nvec ? ld_global_u4(a.r + base + i * 8) : make_uint4(0, 0, 0, 0);
    }
  }
  uint4 ug[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = i0 + j * nt;
    ug[j] = i < nvec ? ld_global_u4(a.gamma + i * 8) : make_uint4(0, 0, 0, 0);
  }
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    unpack_bf16x8(ux[j], h[j]);
    if (a.r != nullptr) {
      float rr[8];
      unpack_bf16x8(ur[j], rr);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] += rr[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
  }
  ss = row_sum<kWarpRow>(ss, red);
  const float rstd = rsqrtf(ss / static_cast<float>(a.d) + a.eps);
  if (a.rstd != nullptr && i0 == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = i0 + j * nt;
    const bool in = i < nvec;
    if (in && a.h != nullptr) *reinterpret_cast<uint4*>(a.h + base + i * 8) = pack_bf16x8(h[j]);
    float g[8];
    unpack_bf16x8(ug[j], g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = h[j][e] * rstd * g[e];
    const uint4 uy = pack_bf16x8(g);
    if (in) *reinterpret_cast<uint4*>(a.y + base + i * 8) = uy;
    if (a.codes != nullptr) {
      unpack_bf16x8(uy, g);          // the rounded y is what is quantised
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(g[e]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int b = mx_scale_byte(m);
      const float inv = mx_inv_scale(b);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + base + i * 8) =
            make_uint2(e4m3x2(g[0] * inv, g[1] * inv) | (e4m3x2(g[2] * inv, g[3] * inv) << 16),
                       e4m3x2(g[4] * inv, g[5] * inv) | (e4m3x2(g[6] * inv, g[7] * inv) << 16));
        if ((i & 3) == 0) {
          if (a.sf != nullptr) a.sf[row * (a.d >> 5) + (i >> 2)] = static_cast<uint8_t>(b);
          if (a.sf_tiled != nullptr) a.sf_tiled[sf_off(row, i >> 2, a.d >> 7)] = static_cast<uint8_t>(b);
        }
      }
    }
  }
}

struct NormBwdArgs {
  int T, d;
  const __nv_bfloat16* dy;
  const __nv_bfloat16* dres;   // or null
  const __nv_bfloat16* h;
  const __nv_bfloat16* gamma;
  const float* rstd;
  __nv_bfloat16* dx;
  float* part;                 // [CTAs][d] partial sums of dgamma
};

// Asynchronous 16-byte copies into shared memory; each thread copies what it
// alone reads, so waiting for its own groups is all the synchronisation needed.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Each row group (a warp, or the CTA) walks rows group, group + groups, ...; a
// thread's columns stay the same, so its share of dgamma accumulates in
// registers. The CTA's sums (over its warps in warp order when a warp has a
// row) go to part, and norm_dgamma_kernel adds the CTAs in order: no float
// atomics, same bytes every run. The next S - 1 rows are on their way into
// shared memory while one is worked on.
template <int V, bool kWarpRow, int S>
__global__ void __launch_bounds__(512, 1) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) uint8_t smem[];
  const int nt = kWarpRow ? 32 : blockDim.x;
  const int i0 = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int per_cta = kWarpRow ? blockDim.x >> 5 : 1;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * per_cta + (kWarpRow ? threadIdx.x >> 5 : 0);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * per_cta;
  const int nvec = a.d >> 3;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool res = a.dres != nullptr;
  constexpr bool kKeep = V <= 2;   // h and dy stay in registers over the reduction; 4 vectors of each would spill
  // [stage][h, dy, dres][vector][thread of the CTA]
  uint4* mine = reinterpret_cast<uint4*>(smem) + threadIdx.x;
  const int pitch = blockDim.x;
  auto at = [&](int st, int k, int j) -> uint4* { return mine + ((st * 3 + k) * V + j) * pitch; };
  auto fetch = [&](int64_t row, int st) {
    if (row < a.T) {
      const int64_t base = row * a.d;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = i0 + j * nt;
        if (i < nvec) {
          cp_async16(at(st, 0, j), a.h + base + i * 8);
          cp_async16(at(st, 1, j), a.dy + base + i * 8);
          if (res) cp_async16(at(st, 2, j), a.dres + base + i * 8);
        }
      }
    }
    cp_async_commit();
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint4 ug[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = i0 + j * nt;
    ug[j] = i < nvec ? ld_global_u4(a.gamma + i * 8) : make_uint4(0, 0, 0, 0);
  }
  float acc[V][8] = {};
#pragma unroll
  for (int st = 0; st < S - 1; ++st) fetch(group + st * groups, st);
  float rnext = group < a.T ? a.rstd[group] : 0.0f;
  int par = 0, st = 0;
  for (int64_t row = group; row < a.T; row += groups, par ^= 1) {
    const float rstd = rnext;
    if (row + groups < a.T) rnext = a.rstd[row + groups];
    fetch(row + (S - 1) * groups, st == 0 ? S - 1 : st - 1);   // the stage of the row before
    cp_async_wait<S - 1>();
    float dot = 0.0f;
    uint4 uh[V], uy[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = i0 + j * nt < nvec;
      uh[j] = in ? *at(st, 0, j) : make_uint4(0, 0, 0, 0);
      uy[j] = in ? *at(st, 1, j) : make_uint4(0, 0, 0, 0);
      float h[8], y[8], g[8];
      unpack_bf16x8(uh[j], h);
      unpack_bf16x8(uy[j], y);
      unpack_bf16x8(ug[j], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = y[e] * (h[e] * rstd);
        acc[j][e] += t;
        dot = fmaf(t, g[e], dot);
      }
    }
    dot = row_sum<kWarpRow>(dot, red[par]) * inv_d;
    const int64_t base = row * a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = i0 + j * nt;
      if (i < nvec) {
        float h[8], y[8], g[8], r[8] = {};
        unpack_bf16x8(kKeep ? uh[j] : *at(st, 0, j), h);
        unpack_bf16x8(kKeep ? uy[j] : *at(st, 1, j), y);
        unpack_bf16x8(ug[j], g);
        if (res) unpack_bf16x8(*at(st, 2, j), r);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = fmaf(fmaf(-h[e] * rstd, dot, y[e] * g[e]), rstd, r[e]);
        *reinterpret_cast<uint4*>(a.dx + base + i * 8) = pack_bf16x8(g);
      }
    }
    st = st == S - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.d;
  asm volatile("griddepcontrol.launch_dependents;");         // norm_dgamma may be placed; it waits for this grid's end
  if constexpr (kWarpRow) {
    __syncthreads();   // the stages are free: the warps' sums meet there
    float* sums = reinterpret_cast<float*>(smem);
    float* w = sums + (threadIdx.x >> 5) * a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = i0 + j * nt;
      if (i < nvec)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i * 8 + e] = acc[j][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      float s = sums[c];
      for (int k = 1; k < per_cta; ++k) s += sums[k * a.d + c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = i0 + j * nt;
      if (i < nvec) {
        float4* o = reinterpret_cast<float4*>(out + i * 8);
        o[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        o[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
      }
    }
  }
}

// dgamma[c] = sum over n partial rows, in a fixed order: 32 columns a CTA,
// 32 threads a column.
__global__ void __launch_bounds__(1024) norm_dgamma_kernel(const float* part, int n, int d, float* dgamma) {
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the partial sums are visible
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < d)
    for (int r = threadIdx.y; r < n; r += 32) v += part[static_cast<int64_t>(r) * d + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int oc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && oc < d) dgamma[oc] = v;
}

namespace {

constexpr int kWarpRowMax = 1024;   // widest row that one warp holds (4 vectors of 8 a lane)
constexpr int kWarpsPerCta = 8;
constexpr int bwd_smem(int stages, int vectors, int threads) { return stages * 3 * vectors * threads * 16; }

// Launch shape of the gradient. A row of up to 1024 columns takes a warp (16 rows a
// CTA: 16384 x 1024 took 41 us with 8 and takes 27), a wider one a CTA with 2 vectors a
// thread up to 8192 columns and 4 beyond. With 4, h and dy are read again from shared
// memory after the reduction (2000 x 16384: 62 us with them in registers, 48 without);
// with 2 they stay in registers (11982 x 4480: 79 us read again, 74 kept).
// Rows in flight and CTAs an SM fill its shared memory, but no more CTAs than keep
// about 8192 columns in work: each leaves a partial of dgamma, and 2 CTAs of 4480
// columns took 82 us where 1 takes 74 (11982 rows).
struct BwdShape {
  int threads, ctas_per_sm, rows_per_cta;
};
BwdShape bwd_shape(int d) {
  if (d <= kWarpRowMax) return {512, d <= 512 ? 512 / (d < 256 ? 256 : d) : 1, 16};
  const int per = 8192 / d;
  return {static_cast<int>(round_up(ceil_div(d / 8, d <= 8192 ? 2 : 4), 32)), per < 1 ? 1 : (per > 4 ? 4 : per), 1};
}
int norm_bwd_ctas(int T, int d, int sms) {
  const BwdShape b = bwd_shape(d);
  const int64_t rows = ceil_div(T, b.rows_per_cta), most = static_cast<int64_t>(b.ctas_per_sm) * sms;
  return static_cast<int>(rows < most ? rows : most);
}

template <int V, bool kWarpRow>
void fwd(const NormArgs& a, cudaStream_t s) {
  const int threads = kWarpRow ? 32 * kWarpsPerCta : static_cast<int>(round_up(ceil_div(a.d / 8, V), 32));
  launch_kernel_after("add_rmsnorm", add_rmsnorm_kernel<V, kWarpRow>,
                dim3(static_cast<unsigned>(ceil_div(a.rows, kWarpRow ? kWarpsPerCta : 1))), dim3(threads), 0, s, a);
}

template <int V, bool kWarpRow, int S>
void bwd(const NormBwdArgs& a, const BwdShape& b, int ctas, cudaStream_t s) {
  static DevOnce once;
  if (!once.ready([] {
        return cudaFuncSetAttribute(rmsnorm_bwd_kernel<V, kWarpRow, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    bwd_smem(S, V, 512));
      })) {
    note(cudaErrorUnknown);
    return;
  }
  launch_kernel_after("rmsnorm_bwd", rmsnorm_bwd_kernel<V, kWarpRow, S>, dim3(static_cast<unsigned>(ctas)),
                      dim3(static_cast<unsigned>(b.threads)), bwd_smem(S, V, b.threads), s, a);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool norm_shape_ok(int T, int d) { return T >= 0 && d >= 8 && d % 8 == 0 && d <= MOE_NORM_MAX_D; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_add_rmsnorm(int T, int d, const void* x, const void* residual, const void* gamma, float eps,
                               void* h, void* y, float* rstd, void* codes, void* scales, void* scales_tiled,
                               moe_stream_t stream) {
  if (!norm_shape_ok(T, d) || !(eps >= 0.0f) || gamma == nullptr) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (x == nullptr || y == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(residual) || !al16(gamma) || !al16(h) || !al16(y) || !al16(codes) || !al4(rstd))
    return MOE_ERR_INVALID_ARG;
  if (codes == nullptr && (scales != nullptr || scales_tiled != nullptr)) return MOE_ERR_INVALID_ARG;
  if (codes != nullptr) {
    if (scales == nullptr && scales_tiled == nullptr) return MOE_ERR_INVALID_ARG;
    if (d % 32 || (scales_tiled != nullptr && d % 128)) return MOE_ERR_INVALID_ARG;
  }
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  CallScope call;
  if (T == 0) return MOE_OK;
  NormArgs a{};
  a.T = T;
  a.d = d;
  a.rows = scales_tiled != nullptr ? static_cast<int>(round_up(T, 128)) : T;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.r = static_cast<const __nv_bfloat16*>(residual);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.eps = eps;
  a.h = static_cast<__nv_bfloat16*>(h);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.rstd = rstd;
  a.codes = static_cast<uint8_t*>(codes);
  a.sf = static_cast<uint8_t*>(scales);
  a.sf_tiled = static_cast<uint8_t*>(scales_tiled);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d <= 256) fwd<1, true>(a, s);
  else if (d <= 512) fwd<2, true>(a, s);
  else if (d <= kWarpRowMax) fwd<4, true>(a, s);
  else fwd<4, false>(a, s);
  return call.status();
}

extern "C" int moe_add_rmsnorm_backward_workspace(int T, int d, size_t* bytes) {
  if (bytes == nullptr || !norm_shape_ok(T, d)) return MOE_ERR_INVALID_ARG;
  *bytes = sizeof(float) * static_cast<size_t>(norm_bwd_ctas(T, d, kMaxSms)) * d;
  return MOE_OK;
}

extern "C" int moe_add_rmsnorm_backward(int T, int d, const void* dy, const void* dres, const void* h,
                                        const void* gamma, const float* rstd, void* dx, float* dgamma, void* ws,
                                        moe_stream_t stream) {
  if (!norm_shape_ok(T, d) || gamma == nullptr || dgamma == nullptr) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr || ws == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(dres) || !al16(h) || !al16(gamma) || !al16(dx) || !al16(ws) || !al4(rstd) || !al4(dgamma))
    return MOE_ERR_INVALID_ARG;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  CallScope call;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    note(cudaMemsetAsync(dgamma, 0, sizeof(float) * d, s));
    return call.status();
  }
  NormBwdArgs a{};
  a.T = T;
  a.d = d;
  a.dy = static_cast<const __nv_bfloat16*>(dy);
  a.dres = static_cast<const __nv_bfloat16*>(dres);
  a.h = static_cast<const __nv_bfloat16*>(h);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.rstd = rstd;
  a.dx = static_cast<__nv_bfloat16*>(dx);
  a.part = static_cast<float*>(ws);
  const int sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  const int ctas = norm_bwd_ctas(T, d, sms);
  const BwdShape b = bwd_shape(d);
  if (d <= 256) bwd<1, true, 4>(a, b, ctas, s);
  else if (d <= 512) bwd<2, true, 4>(a, b, ctas, s);
  else if (d <= kWarpRowMax) bwd<4, true, 2>(a, b, ctas, s);
  else if (d <= 8192) bwd<2, false, 4>(a, b, ctas, s);
  else bwd<4, false, 2>(a, b, ctas, s);
  if (call_error() != cudaSuccess) return call.status();      // no partial sums to add
  launch_kernel_after("norm_dgamma", norm_dgamma_kernel, dim3(static_cast<unsigned>(ceil_div(d, 32))), dim3(32, 32), 0, s,
                static_cast<const float*>(a.part), ctas, d, dgamma);
  return call.status();
}
