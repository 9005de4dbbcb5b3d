// Router: logits on the tensor cores, then sigmoid + bias + group-limited
// top-k + gate normalisation as warp-shuffle reductions (one warp per token,
// route.cuh).
#include <cudaTypedefs.h>

#include <mutex>

#include "moe_internal.h"
#include "gemm.cuh"
#include "prof.h"
#include "route.cuh"

namespace moe {

template <int kMaxPerLane>
__global__ void router_topk_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T, int E,
                                   int k, int G, int gtop, int32_t* __restrict__ idx_out,
                                   float* __restrict__ w_out, float* __restrict__ s_out) {
  extern __shared__ float sv_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  float* sv = sv_all + warp * E;
  if (t >= T) return;
  int my_e;
  float my_s, tot;
  choose_experts<kMaxPerLane, BestByShuffles>([&](int e) { return logits[static_cast<int64_t>(t) * E + e]; }, [&](int e) { return bias[e]; }, E, k,
                              G, gtop, sv, lane, my_e, my_s, tot);
  if (lane < k) {
    const int64_t o = static_cast<int64_t>(t) * k + lane;
    idx_out[o] = my_e;
    w_out[o] = __fdiv_rn(my_s, tot);
    if (s_out != nullptr) s_out[o] = my_s;
  }
}

int launch_router_logits(const Dims& m, const void* x, const void* w_router, float* logits, cudaStream_t s) {
  GemmOperands op{};
  op.a = static_cast<const uint8_t*>(x);
  op.a_rows = m.T;
  op.a_cols = m.d;
  op.b = static_cast<const uint8_t*>(w_router);
  op.b_rows = m.E;
  op.b_cols = m.d;
  GemmEpilogue ep{};
  ep.out = logits;
  ep.ldo = m.E;
  return gemm_dispatch("router_gemm", kRouterMode, m, 0, m.E, m.d, m.T, op, ep, nullptr, nullptr, nullptr, nullptr,
                       nullptr, s);
}

void launch_router_topk(const Dims& m, const float* logits, const float* bias, int32_t* idx, float* w, float* s_sel,
                        cudaStream_t s) {
  if (m.T == 0) return;
  const int warps = 4;
  const int per = (m.E + 31) / 32;   // E <= 512
  auto kern = per <= 4 ? router_topk_kernel<4> : per <= 8 ? router_topk_kernel<8> : per <= 12 ? router_topk_kernel<12>
                                                                                    : router_topk_kernel<16>;
  launch_kernel("router_topk", kern, dim3(static_cast<unsigned>(ceil_div(m.T, warps))), dim3(warps * 32),
                warps * m.E * sizeof(float), s, logits, bias, m.T, m.E, m.k, m.G, m.gtop, idx, w, s_sel);
}

// ---------------------------------------------------------------- router without allocation
// Scratch of moe_route_noalloc: the fp32 logits of one call, in a fixed
// file-scope device array (every GPU that loads the library holds it until
// the process exits). Host code must not pass the array's name to a kernel:
// on the host it is only a stand-in symbol, so its device address is looked
// up with cudaGetSymbolAddress, once per CUDA context of a device.
constexpr int64_t kRouteScratchFloats = int64_t(1) << 22;   // 16 MiB: T * E <= 4,194,304
static __device__ __align__(256) float g_route_scratch[kRouteScratchFloats];

namespace {
std::mutex g_scratch_mu;
struct ScratchSlot {
  unsigned long long ctx_id = 0;   // context the address belongs to (0 = none yet)
  float* addr = nullptr;
};
ScratchSlot g_scratch[kMaxDev];

PFN_cuCtxGetCurrent_v4000 g_ctx_current = nullptr;
PFN_cuCtxGetId_v12000 g_ctx_id = nullptr;

// Unique id of the calling thread's current context (ids are never reused in a
// process, so a context created after cudaDeviceReset gets a new one); 0 if
// it cannot be read.
unsigned long long current_ctx_id() {
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_ctx_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(f);
    f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_ctx_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(f);
  });
  if (g_ctx_current == nullptr || g_ctx_id == nullptr) return 0;
  CUcontext c = nullptr;
  unsigned long long id = 0;
  if (g_ctx_current(&c) != CUDA_SUCCESS || c == nullptr || g_ctx_id(c, &id) != CUDA_SUCCESS) return 0;
  return id;
}

// Device address of the scratch in the current context (looked up on the
// first call in each context).
int route_scratch(float** out) {
  const int dev = current_device();
  if (dev < 0) return MOE_ERR_CUDA;
  const unsigned long long id = current_ctx_id();
  if (id == 0) return MOE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_scratch_mu);
  ScratchSlot& slot = g_scratch[dev];
  if (slot.ctx_id != id) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_route_scratch) != cudaSuccess || p == nullptr) {
      (void)cudaGetLastError();   // the failed lookup's own error: not left for the caller to find
      return MOE_ERR_CUDA;
    }
    slot.addr = static_cast<float*>(p);
    slot.ctx_id = id;
  }
  *out = slot.addr;
  return MOE_OK;
}
}  // namespace

}  // namespace moe

extern "C" int moe_route_noalloc(const moe_config_t* cfg, const void* x, const void* w_router, const float* bias,
                                 int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  if (int r = moe::validate(cfg)) return r;
  const bool no_tokens = cfg->T == 0;   // per-token arrays may be null then
  if ((!x && !no_tokens) || !w_router || !bias || (!topk_idx && !no_tokens) || (!topk_w && !no_tokens))
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_router)) & 15u) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(cfg->T) * cfg->E > moe::kRouteScratchFloats) return MOE_ERR_SCRATCH;
  if (!moe::arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  if (cfg->T == 0) return MOE_OK;
  float* logits = nullptr;
  if (int r = moe::route_scratch(&logits)) return r;
  const moe::Dims m = moe::make_dims(cfg);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  moe::CallScope call;
  if (int r = moe::launch_router_logits(m, x, w_router, logits, s)) return r;
  moe::launch_router_topk(m, logits, bias, topk_idx, topk_w, nullptr, s);
  return call.status();
}
