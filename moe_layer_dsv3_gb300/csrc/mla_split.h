// Integer arithmetic of the latent decode's work split, the same on the device
// and the host: tiles, workers and their ranges, and the page of a token.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {
namespace mla {

MOE_HD int tiles_of(int len, int tile) {                   // (len may end within a tile of 2^31)
  return static_cast<int>((static_cast<uint32_t>(len) + static_cast<uint32_t>(tile) - 1) / static_cast<uint32_t>(tile));
}

// Workers of W that get tiles: no more than total / min_tiles, rounded up, and one at least. total may be 2^31 - 1.
MOE_HD int workers_of(int total, int W, int min_tiles) {
  const int most = total / min_tiles + (total % min_tiles != 0);
  return W < most ? W : (most > 0 ? most : 1);
}

// First tile of worker w of W over `total` tiles: total * w / W rounded down, in 32 bits (the remainder times w stays
// below W * W; two 64-bit divisions here were part of every worker's start).
MOE_HD int range_begin(int total, int w, int W) {
  const unsigned q = static_cast<unsigned>(total) / static_cast<unsigned>(W), rest = total - q * W;
  return static_cast<int>(q * w + rest * static_cast<unsigned>(w) / static_cast<unsigned>(W));
}

// The worker that owns tile t.
MOE_HD int owner_of(int total, int t, int W) {
  return static_cast<int>((static_cast<int64_t>(t + 1) * W - 1) / total);
}

// Pieces of a sequence whose first tile is s0 and that worker w ends.
struct Cut {
  int slot, worker, pieces;  // slot of the first piece, its worker, pieces in all
};
MOE_HD Cut cut_of(int total, int W, int s0, int w) {
  const int w0 = owner_of(total, s0, W);
  return {range_begin(total, w0, W) == s0 ? 0 : 1, w0, w - w0 + 1};   // it opened w0's range, or came after another piece there
}

// Division by the page size as a multiplication (T. Granlund and P. L. Montgomery, 1994): with L = ceil(log2 page) and
// m = floor(2^(31 + L) / page) + 1, n m / 2^(31 + L) rounded down is n / page for every n below 2^31.
struct PageDiv {
  uint32_t mul;
  int shift;                 // n / page = n * mul / 2^(32 + shift)
};
MOE_HD PageDiv page_div(int page) {                        // 8 or more
  int log = 3;
  while ((int64_t{1} << log) < page) ++log;
  return {static_cast<uint32_t>((uint64_t{1} << (31 + log)) / page + 1), log - 1};
}
MOE_HD int page_of(uint32_t tok, uint32_t mul, int shift) {
#ifdef __CUDA_ARCH__
  return static_cast<int>(__umulhi(tok, mul) >> shift);
#else
  return static_cast<int>(static_cast<uint32_t>((static_cast<uint64_t>(tok) * mul) >> 32) >> shift);
#endif
}

}  // namespace mla
}  // namespace moe
