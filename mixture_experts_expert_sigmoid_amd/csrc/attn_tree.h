// The ancestors of drafted tokens, which form a tree behind a sequence's
// context, as bits: bit b of token t's row is set iff t sees token b of the same
// tree, that is b is t or an ancestor of t and, with a window, near enough.
//
// A token's row is found by one thread that walks up the parents in LDS. A
// parent comes before its children, so every walk ends, after as many steps as
// the tree is deep. With a window a row needs its depth first: it walks twice. A
// walk of 10 steps is 10 LDS latencies, under 1 us, beside the first keys' loads;
// only tiles that not all rows see in full ask for it.
#pragma once
#include "attn_dev.h"

namespace moe {
namespace {

// of the tokens of a tile of at most N rows
template <int N>
struct TreeRows {
  static constexpr int W = kTreeMax / 32;
  static_assert(kTreeMax <= 256, "a depth fits a byte");
  short par[kTreeMax];                           // kTreeMax: none that there can be
  uint8_t deep[N];
  uint32_t row[N][W];

  // The parents of the sequence's m <= kTreeMax tokens, by the whole
  // workgroup; a barrier before build().
  __device__ void fetch(const int* parent, int m) {
    for (int i = threadIdx.x; i < min(m, kTreeMax); i += blockDim.x) {
      const int p = parent[i];
      par[i] = (short)(p < -1 || p > kTreeMax ? kTreeMax : p);
    }
  }
  // Rows of tokens t0 .. t1 - 1 behind C tokens of context, a thread each; a
  // barrier before their use.
  __device__ void build(int t0, int t1, int C, int window, int first, int* err) {
    const int t = t0 + (int)threadIdx.x;
    if ((int)threadIdx.x >= N || t >= t1) return;
    uint32_t* const r = row[threadIdx.x];
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = 0;
    auto up = [&](int a) {
      const int p = par[a];
      if (p >= -1 && p < a) return p;
      atomicOr(err, kErrTree);                   // taken as a child of the context
      return -1;
    };
    int depth = -1;
    for (int a = t; a >= 0; a = up(a)) ++depth;
    deep[threadIdx.x] = (uint8_t)depth;
    int d = depth;
    for (int a = t; a >= 0; a = up(a), --d)
      if (!window || depth - d < window || C + d < first) r[a >> 5] |= 1u << (a & 31);
  }
  // token t0 + i's bits from b on (outside the tree: 0), 64 of them
  __device__ uint64_t bits(int i, int b) const {
    const int k = b >> 5, sh = b & 31;
    auto word = [&](int j) -> uint64_t { return (unsigned)j < (unsigned)W ? row[i][j] : 0u; };
    const uint64_t lo = word(k) | word(k + 1) << 32, hi = word(k + 2);
    return lo >> sh | (sh ? hi << (64 - sh) : 0);
  }
  __device__ int depth(int i) const { return deep[i]; }
};
template <>
struct TreeRows<0> {};

}  // namespace
}  // namespace moe
