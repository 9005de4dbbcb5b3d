// The few-token layer's list of pieces and the room for their parts, in integer
// arithmetic that is the same on the device and the host.
#pragma once
#include <cstdint>

#ifndef MOE_HD
#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif
#endif

namespace moe {
namespace few {

// Pieces of a CTA that K is cut for, where there are fewer, up and down. More of them balance better and cost the joining of
// parts. One token of 9 wide experts: 74.9 us with 1 and 2, 78.4 with 1 and 1, 76.4 with 1 and 4, 77.5 with 2 and 4, 79.1 with 4
// and 8. Five tokens of 37 narrow ones: 47.1, 47.2, 47.0, 49.2, 50.7. From 16 tokens on within 1 %, but for narrow experts with 4
// and 8 (80 instead of 77).
constexpr int kUpPieces = 1, kDownPieces = 2;
constexpr int kMinSteps = 2;               // fewest 128-wide steps of a part

// Parts that K (`steps` steps) of `units` units is cut into, so that each of `ctas` CTAs gets `want` pieces.
MOE_HD int parts_of(int units, int steps, int ctas, int want) {
  const int most = steps / kMinSteps > 1 ? steps / kMinSteps : 1;
  const int n = (ctas * want + units - 1) / units;
  return n < most ? n : most;
}

// First step of part i of n: an even one, since two steps of a row (256 bytes) come from HBM together.
MOE_HD int cut_at(int steps, int i, int n) {
  const int at = ((steps + 1) >> 1) * i / n * 2;
  return at < steps ? at : steps;
}

// The list of a layer's d and I columns, the `slots` experts in use and `ctas` CTAs.
struct Work {
  int KA, KI, NB, RP, slots;               // steps of d and of I, blocks of 256 up and of 256 down rows, experts in use
  int PU, PD, nup, total;                  // parts, pieces
};
// (Filled in place from the kernel's own arguments and plan: with numbers for arguments the compiler makes 2.7 KB more code of the
// kernel, and every call takes 0.2 to 0.8 % longer.)
template <typename Args, typename Plan>
MOE_HD void work_of(Work& w, const Args& a, const Plan& p, int ctas) {
  w.KA = a.d >> 7;
  w.KI = a.I >> 7;
  w.NB = a.I >> 7;
  w.RP = ((a.d >> 7) + 1) >> 1;
  w.slots = p.slots;
  w.PU = w.slots > 0 ? parts_of(w.slots * w.NB, w.KA, ctas, kUpPieces) : 1;
  w.PD = w.slots > 0 ? parts_of(w.slots * w.RP, w.KI, ctas, kDownPieces) : 1;
  w.nup = w.slots * w.NB * w.PU;
  w.total = w.nup + w.slots * w.RP * w.PD;
}
struct Piece {
  bool up;
  int s, b, part, k0, k1;                  // expert slot, block of rows, part of K, its steps
};
MOE_HD Piece piece_of(const Work& w, int id) {
  Piece p;
  p.up = id < w.nup;
  if (p.up) {
    const int u = id / w.PU;
    p.part = id - u * w.PU;
    p.s = u / w.NB;
    p.b = u - p.s * w.NB;
    p.k0 = cut_at(w.KA, p.part, w.PU);
    p.k1 = cut_at(w.KA, p.part + 1, w.PU);
  } else {
    // (parts of the same rows side by side: with all CTAs on the same quarter of every 2 KB row HBM gave 4.3 TB/s)
    const int q = id - w.nup, u = q / w.PD;
    p.part = q - u * w.PD;
    p.s = u / w.RP;
    p.b = u - p.s * w.RP;
    p.k0 = cut_at(w.KI, p.part, w.PD);
    p.k1 = cut_at(w.KI, p.part + 1, w.PD);
  }
  return p;
}

// Accumulators. The tensor core truncates when it adds into TMEM: with products of one sign the sums of 448 additions (14336 columns)
// were 67 x 2^-23 of themselves too small, and with random ones over 7168 columns 5 of 295000 values of h took the neighbouring code
// of MX(h), or a block's scale the neighbouring power of two (which moved a token's y by up to 2 %), where sums rounded to nearest
// give 1. So K of an up piece is cut into chunks with accumulators of their own, which the epilogue adds: up to four, as TMEM has room
// for them and for the next piece's first. That leaves 7 x 2^-23, and 2 values of 295000. It costs 0.3 to 0.6 us for one token and for
// five of narrow experts, 0.7 of 317 for 16 and 0.3 of 416 for 64. (A down piece's sums are rounded, not quantised.)
constexpr int kAccCols = 440;              // TMEM columns of accumulators, two tiles of N columns each
constexpr int kMaxChunks = 4;
constexpr int kMinChunkSteps = 14;
MOE_HD int acc_slots(int N) { return kAccCols / (2 * N); }   // 13, 6, 4 and 3 for 16 to 64 columns
constexpr int kMaxSlots = kAccCols / 32;
MOE_HD int chunks_of(const Piece& p, int N) {
  if (!p.up) return 1;
  const int fit = acc_slots(N) - 1, most = fit < kMaxChunks ? fit : kMaxChunks, n = (p.k1 - p.k0) / kMinChunkSteps;
  return n < 1 ? 1 : n < most ? n : most;
}
// First step of chunk i of n.
MOE_HD int chunk_at(const Piece& p, int i, int n) { return p.k0 + (p.k1 - p.k0) * i / n; }

// Rows times parts of a product of `steps` steps over `blocks` blocks of rows an expert, whatever T tokens choose of `picks` experts
// each (a shared one among them) on up to `ctas` CTAs: with s experts in use rows are at most T min(s, picks), and parts at
// most ctas want / (s blocks) + 1.
MOE_HD int64_t parts_room(int64_t T, int64_t picks, int64_t ctas, int64_t steps, int64_t blocks, int64_t want) {
  const int64_t most = steps / kMinSteps > 1 ? steps / kMinSteps : 1;
  const int64_t all = T * ((ctas * want + blocks - 1) / blocks + picks);
  return all < T * picks * most ? all : T * picks * most;
}

}  // namespace few
}  // namespace moe
