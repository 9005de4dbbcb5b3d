// Block tables and slot maps from request lengths: the pages that sequences gain or
// leave in a step, and where each new token goes.
//
// Free pages are a stack, `count` of them in free[0 .. count). With F pages left
// and G taken in a step, the left ones are pushed in order (sequence by sequence,
// page by page) and the taken ones popped in order after that, so the taken page
// number i is entry count + F - 1 - i of the stack: one of the left pages while
// i < F, an old entry after that. Every thread can therefore work out each page that it needs
// from the prefix sums over the sequences, and nothing has to be pushed before
// it is popped: the free stack is only read below count and only written at and above it, and
// entries of the block table that are left are read but not changed.
//
// Latency bounds it (96 sequences read and write 3 KB; half a million tokens write
// 6 MB, 1 us at the copy rate). So it is one launch, in which every CTA makes
// the prefix sums for itself; lengths and count are stored by the CTA that
// arrives last, when every other has read them, so that they may be updated in place.
// Measured in a graph of such calls: 4.5 to 5.7 us a call for 96 sequences with a token each, 7.1 to 8.8
// for 512 of which some grow and some shrink, 8.0 for 37 prompts of 524288 tokens; called from
// Python the host's 8 to 9 us bound it.
#include "moe_internal.h"
#include "pages_sums.h"
#include "prof.h"
#include "ptx.cuh"

namespace moe {

namespace {

using pages::Sums;

constexpr int kThreads = 256;
constexpr int kTokens = 4;                 // consecutive tokens of a thread: their stores are 16 bytes wide

struct PagesArgs {
  int B, page, num_pages, max_pages, max_new;
  int page_ctas;                           // CTAs, the first ones, that write pages; the others write tokens
  const int32_t* lens;
  const int32_t* target;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* count;
  int32_t* lens_out;
  int32_t* count_out;
  int32_t* seq;
  int32_t* pos;
  int32_t* slot;
  int32_t* starts;
  int* ws;                                 // {code, site, -, CTAs done}
};

// Index of the sequence that holds number i: the largest b with first[b] <= i (first[n] > i).
__device__ __forceinline__ int owner(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) pages_update_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ int sm[];
  int* starts = sm;                        // [B + 1] new tokens before a sequence
  int* taken = starts + a.B + 1;           // [B + 1] pages taken before it
  int* left = taken + a.B + 1;             // [B + 1] pages left before it
  int* len = left + a.B + 1;               // [B]
  int* want = len + a.B;                   // [B]
  __shared__ Sums scan[kThreads / 32];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const int count = ld_global_s32(a.count);
  bool bad = count < 0 || count > a.num_pages;
  for (int b = tid; b < a.B; b += kThreads) {
    const int n = ld_global_s32(a.lens + b), m = ld_global_s32(a.target + b);
    bad = bad || n < 0 || n > cap || m < 0 || m > cap;
    len[b] = n;
    want[b] = m;
  }
  auto pages_of = [&](int n) { return pages::pages_of(n, a.page); };
  bad = __syncthreads_or(bad);
  Sums mine{0, 0, 0};
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  if (!bad)
    for (int b = b0; b < b1; ++b) mine += pages::sums_of(len[b], want[b], a.page);
  Sums at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v{__shfl_up_sync(0xffffffffu, at.add, o), __shfl_up_sync(0xffffffffu, at.grow, o),
                 __shfl_up_sync(0xffffffffu, at.drop, o)};
    if (lane >= o) at += v;
  }
  if (lane == 31) scan[warp] = at;
  // (before this thread's run, within its warp; only used when no sum was cut)
  at = Sums{at.add - mine.add, at.grow - mine.grow, at.drop - mine.drop};
  __syncthreads();
  Sums all{0, 0, 0};
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) at += scan[i];
    all += scan[i];
  }
  // A step that cannot be made as a whole is not made at all.
  const int code = bad ? MOE_ERR_BOUNDS : pages::step_code(all, count, a.num_pages, a.max_new);
  if (code != MOE_OK) {
    if (blockIdx.x == 0 && tid == 0) report_error(a.ws, code, 220);
    at = all = Sums{0, 0, 0};
  }
  for (int b = b0; b < b1; ++b) {
    starts[b] = static_cast<int>(at.add);
    taken[b] = static_cast<int>(at.grow);
    left[b] = static_cast<int>(at.drop);
    if (code == MOE_OK) at += pages::sums_of(len[b], want[b], a.page);
  }
  const int N = static_cast<int>(all.add), G = static_cast<int>(all.grow), F = static_cast<int>(all.drop);
  if (tid == 0) {
    starts[a.B] = N;
    taken[a.B] = G;
    left[a.B] = F;
  }
  __syncthreads();

  auto checked = [&](int page) {
    if (page < 0 || page >= a.num_pages) report_error(a.ws, MOE_ERR_BOUNDS, 221);
    return page;
  };
  // Where the i-th page that is left, and the i-th that is taken, is written.
  auto left_at = [&](int i) {
    const int b = owner(left, a.B, i);
    return a.table + static_cast<int64_t>(b) * a.max_pages + pages_of(want[b]) + i - left[b];
  };
  auto taken_at = [&](int i) { return i < F ? left_at(F - 1 - i) : a.free_pages + count + F - 1 - i; };
  const int bid = static_cast<int>(blockIdx.x);
  if (bid < a.page_ctas) {
    const int step = a.page_ctas * kThreads, me = bid * kThreads + tid;
    for (int i = me; i < G; i += step) {
      const int b = owner(taken, a.B, i);
      a.table[static_cast<int64_t>(b) * a.max_pages + pages_of(len[b]) + i - taken[b]] = checked(ld_global_s32(taken_at(i)));
    }
    for (int i = me; i < F - G; i += step) a.free_pages[count + i] = checked(ld_global_s32(left_at(i)));
    for (int b = me; b <= a.B; b += step) a.starts[b] = starts[b];
  } else {
    const int64_t step = static_cast<int64_t>(gridDim.x - a.page_ctas) * kThreads * kTokens;
    for (int64_t i0 = (static_cast<int64_t>(bid - a.page_ctas) * kThreads + tid) * kTokens; i0 < a.max_new; i0 += step) {
      int s[kTokens], p[kTokens], w[kTokens], in[kTokens];
      const int32_t* at_page[kTokens];
      int b = i0 < N ? owner(starts, a.B, static_cast<int>(i0)) : 0;
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        const int i = static_cast<int>(i0) + k;
        s[k] = 0;
        p[k] = w[k] = -1;
        at_page[k] = nullptr;
        if (i0 + k >= N) continue;
        while (starts[b + 1] <= i) ++b;    // (sequences without new tokens lie between)
        s[k] = b;
        p[k] = pages::nth(len[b], i, starts[b]);
        const int j = p[k] / a.page, old = pages_of(len[b]);
        in[k] = p[k] - j * a.page;
        at_page[k] = j < old ? a.table + static_cast<int64_t>(b) * a.max_pages + j : taken_at(pages::nth(taken[b], j, old));
      }
      int page[kTokens];
#pragma unroll
      for (int k = 0; k < kTokens; ++k) page[k] = at_page[k] != nullptr ? ld_global_s32(at_page[k]) : -1;
#pragma unroll
      for (int k = 0; k < kTokens; ++k)
        if (at_page[k] != nullptr && checked(page[k]) >= 0 && page[k] < a.num_pages) w[k] = page[k] * a.page + in[k];
      if (i0 + kTokens <= a.max_new) {
        *reinterpret_cast<int4*>(a.seq + i0) = make_int4(s[0], s[1], s[2], s[3]);
        *reinterpret_cast<int4*>(a.pos + i0) = make_int4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<int4*>(a.slot + i0) = make_int4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
          if (i0 + k < a.max_new) {
            a.seq[i0 + k] = s[k];
            a.pos[i0 + k] = p[k];
            a.slot[i0 + k] = w[k];
          }
      }
    }
  }
  // Every thread of this CTA has read lengths and count.
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(a.ws + 3, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  for (int b = tid; b < a.B; b += kThreads) a.lens_out[b] = code == MOE_OK ? want[b] : len[b];
  if (tid == 0) {
    *a.count_out = count + F - G;
    a.ws[3] = 0;
  }
}

inline bool mis(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_pages_update(int batch, int page_size, int num_pages, int max_pages, int max_new, const int32_t* seq_lens,
                                const int32_t* target, int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                                int32_t* lens_out, int32_t* count_out, int32_t* seq, int32_t* pos, int32_t* slot,
                                int32_t* starts, void* ws, moe_stream_t stream) {
  const int64_t lim = (1LL << 31) - 1;
  if (batch < 0 || batch > MOE_PAGES_MAX_BATCH || page_size < 1 || num_pages < 1 || max_pages < 1 || max_new < 0 ||
      static_cast<uint32_t>(max_new) >= pages::kMost || static_cast<uint32_t>(num_pages) >= pages::kMost)
    return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_pages) * page_size >= lim || static_cast<int64_t>(max_pages + 1LL) * page_size >= lim)
    return MOE_ERR_INVALID_ARG;
  if (!free_pages || !free_count || !count_out || !starts || !ws || (batch > 0 && (!seq_lens || !target || !block_table || !lens_out)) ||
      (max_new > 0 && (!seq || !pos || !slot)))
    return MOE_ERR_INVALID_ARG;
  if (mis(seq, 16) || mis(pos, 16) || mis(slot, 16) || mis(ws, 16) || mis(seq_lens, 4) || mis(target, 4) || mis(block_table, 4) ||
      mis(free_pages, 4) || mis(free_count, 4) || mis(lens_out, 4) || mis(count_out, 4) || mis(starts, 4))
    return MOE_ERR_INVALID_ARG;
  if (!arch_ok()) return MOE_ERR_UNSUPPORTED_ARCH;
  CallScope call;
  static DevOnce once;
  constexpr int kSmemMost = (5 * MOE_PAGES_MAX_BATCH + 3) * static_cast<int>(sizeof(int));
  if (!once.ready([] { return cudaFuncSetAttribute(pages_update_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost); }))
    return MOE_ERR_CUDA;
  PagesArgs a{};
  a.B = batch;
  a.page = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.max_new = max_new;
  a.lens = seq_lens;
  a.target = target;
  a.table = block_table;
  a.free_pages = free_pages;
  a.count = free_count;
  a.lens_out = lens_out;
  a.count_out = count_out;
  a.seq = seq;
  a.pos = pos;
  a.slot = slot;
  a.starts = starts;
  a.ws = static_cast<int*>(ws);
  // Pages and tokens by CTAs of their own: one after the other in the same threads cost 2 us of 8 (512 sequences).
  const int64_t most = num_sms(), pages = ceil_div(max_new / page_size + batch + 1, kThreads);
  const int64_t tokens = ceil_div(max_new, kThreads * kTokens);
  a.page_ctas = static_cast<int>(pages < most ? pages : most);
  const int grid = a.page_ctas + static_cast<int>(tokens < 4 * most ? tokens : 4 * most);
  launch_kernel_after("pages_update", pages_update_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                      (5 * batch + 3) * sizeof(int), static_cast<cudaStream_t>(stream), a);
  return call.status();
}

extern "C" int moe_pages_status(void* ws, int* code, int* site, int clear, moe_stream_t stream) {
  if (!ws || !code || !site) return MOE_ERR_INVALID_ARG;
  return read_status(ws, code, site, clear, static_cast<cudaStream_t>(stream));
}
