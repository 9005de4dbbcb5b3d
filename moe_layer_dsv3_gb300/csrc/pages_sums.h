// Integer arithmetic of the page plans, the same on the device and the host: sums
// over sequences, and whether a step can be made.
#pragma once
#include <cstdint>

#include "../../include/moe.h"

#ifndef MOE_HD
#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif
#endif

namespace moe {
namespace pages {

// Sums over sequences. Lengths may be anything up to 2^31 - 1, so every term is cut to kMost and a sum stays there once it
// gets there: past every buffer (the library takes fewer than kMost pages and new tokens), and two of them fit in 32 bits
// without a sign.
constexpr uint32_t kMost = 1u << 30;
MOE_HD uint32_t cut(uint32_t n) { return n < kMost ? n : kMost; }
struct Sums {
  uint32_t add, grow, drop;                // new tokens, pages taken, pages left
  MOE_HD void operator+=(const Sums& o) {
    add = cut(add + o.add);
    grow = cut(grow + o.grow);
    drop = cut(drop + o.drop);
  }
};

MOE_HD int pages_of(int tokens, int page) { return (tokens + page - 1) / page; }   // (capacity + page is below 2^31)

// Number i of a list whose number `first` is `base`. (base + i may pass 2^31, the result does not.)
MOE_HD int nth(int base, int i, int first) { return base + (i - first); }

// What a sequence that goes from n to m tokens, both in [0, capacity], adds to them.
MOE_HD Sums sums_of(int n, int m, int page) {
  const int o = pages_of(n, page), w = pages_of(m, page);
  return {cut(static_cast<uint32_t>(m > n ? m - n : 0)), cut(static_cast<uint32_t>(w > o ? w - o : 0)),
          cut(static_cast<uint32_t>(o > w ? o - w : 0))};
}

// Whether a step with these sums over all sequences can be made with `count` of num_pages pages free (0 <= count <= num_pages).
// A sum that was cut is refused: it is past max_new, past the room num_pages - count, or past count + drop <= num_pages.
MOE_HD int step_code(const Sums& all, int count, int num_pages, int max_new) {
  if (all.add > static_cast<uint32_t>(max_new) || all.drop > static_cast<uint32_t>(num_pages - count)) return MOE_ERR_BOUNDS;
  return all.grow > static_cast<uint32_t>(count) + all.drop ? MOE_ERR_PAGES : MOE_OK;
}

}  // namespace pages
}  // namespace moe
