// Attention of the newest tokens of each sequence (a prompt, or the next
// chunk of one) over a paged key-value cache.
//
// Mathematics. One pass over the keys with the running maximum and sum of a
// softmax: S^T = K Q^T, P = 2^(S - m), O^T = V^T P^T, all in fp32 but the
// 16-bit operands. P is one of them (the matrix instructions take no wider one
// at their rate): that rounding is of the size of the result's own, and results
// stand 13-35 % further from the 64-bit values than with P of 32 bits. The rows
// of a tile are (token, query head) pairs of one key-value head, token-major, so
// the heads that share keys share the tile: a tile spans few positions, and a
// short chunk still fills it.
//
// Layout. Four waves of 32 rows, v_mfma_*_32x32x16. A row lies in a lane's
// column of S^T (lane l: row l % 32, 16 of 32 keys), so the softmax
// is a loop in the lane and one exchange with lane l ^ 32, and P is the B
// operand of the second product as it stands when each lane half's 8-key
// slice of a 16-key step is taken as keys 4h..4h+3 and 8+4h..8+4h+3 of it.
// K and V tiles go through LDS, 16-byte units swizzled by key; V is read
// transposed (ds_read_b64_tr_b16), in that key order.
//
// Rescaling. O and the sum follow the maximum only when it has grown by more
// than a factor of 2^8 of P (f16: 2^3.9), which neither type nor sum minds: rare
// after the first tiles, and exact all the same.
//
// Masked places. Scores are replaced, not added to. V rows that no row of the
// tile sees are staged as zeros; in tiles where some rows see a key and some
// do not, V values that are not finite are staged as zero and their products
// added to the rows that see them one by one.
//
// Bound: the matrix cores and the exponentials for long prompts; latency for
// short ones. Few tiles: the keys of each are split over workgroups and the
// parts joined in order. Measured: a causal prompt of 11999 tokens, 32 heads
// of 128 over 8 (bf16) 1.07-1.10 ms, 1.08-1.10 PFLOP/s (a large library
// product: 1.25); 6000 tokens of head_dim 64 860, of 256 760 TFLOP/s; two
// chunks of 500 tokens over 16..24 k e4m3 keys 406-411 us, 0.9 PFLOP/s; seven
// prompts of 130..3001 tokens, window 512, head_dim 64 (f16) 85 us; a prompt of
// 37 tokens 8.1 us. A wave by itself on its SIMD takes 1.15 us for 64 keys of
// head_dim 128, two 1.1 us for both: loads further ahead (four buffers) gained
// nothing, so that is the wave's own chain of reads, products and softmax.
#pragma once
#include <type_traits>

#include "attn_dev.h"
#include "attn_tree.h"

namespace moe {
namespace {

// What the newest tokens of a sequence see of each other: those before them, or
// their ancestors in a tree. kDense: those before them, and keys and values in
// rows instead of pages, a head of them for each query head; behind a key's D
// values come kLatRope that all heads share.
enum { kCausal, kTree, kDense };

// Trees (kTree): the tile, its products and its loop are the prompt's; a key among
// the drafted tokens is seen by a bit of the row's ancestors, and all tiles before
// them are whole, so that the tree costs a mask in the last ones. The keys are
// split further than a prompt's (tree_splits). Bound by HBM for a batch, by the
// matrix cores and the codes' expansion for long contexts. Measured: 48 trees of
// 9..33 tokens over 201..4001 keys, 32 heads over 8 of 128, bf16 (436 MB) 108-118 us,
// 3.7-4.0 TB/s; two of 41 and 61, 64 heads, over 50..60 k e4m3 keys (217 GFLOP) 260-277
// us, 0.79-0.84 PFLOP/s; one of 8 tokens over 777 keys 14.2-14.7 us, latency.
// Dense rows (kDense): a group's place is its row, and the loads' own bounds end
// each sequence, so a ragged batch needs no pages; a key's rotary values are a tile
// of 64 beside it, read for all heads alike. Two workgroups fill a CU's LDS (2 x 80
// KB). Bound by the matrix cores: 6001 tokens of 32 heads (369 GFLOP) 372-397 us from
// one card to the next, 0.93-0.99 PFLOP/s; three prompts of 17..130 tokens of 16 heads
// 11.5-11.8 us, latency. Dealt out by tiles, all at once: where they are few and long, a
// CU with a long one and its part has twice the average (1689 tokens of 16 heads 44 us,
// ten prompts of 553..1574 of 3 heads 52).

// keys of a tile, rows of a workgroup's tile
template <int D>
struct PreShape {
  static constexpr int BN = D == 256 ? 32 : 64;
  static constexpr int ROWS = kPreRows;
};

// what a workgroup works on
struct PreTile {
  int seq, slot, L, m, q0;     // sequence; its slot, length, new tokens, first row of q
  long k0;                     // first row of keys (kDense)
  int tile, rows;              // tile of PreShape::ROWS rows, rows of the sequence
  int p_min, p_max;            // positions of its first and last row
  int lo_min, lo_max;          // first key of the window at those
  int ng1, b2, nb;             // 16-key groups: 0..ng1-1, then b2 and on; tiles of them
};

__device__ __forceinline__ int pre_cu(const AttnArgs& a, int i) {
  const int c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? (int)a.T : c);
}

// The last sequence i whose ok(i, cu[i]) holds (ok holds up to some i >= 0 and
// not after): a search with 64 candidates a step, one to a lane.
template <typename Ok>
__device__ __forceinline__ int pre_last(const AttnArgs& a, Ok ok) {
  const int lane = lane_id();
  int lo = 0, n = a.n;
  while (true) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    const bool yes = lane * step < n && ok(i, pre_cu(a, i));
    const int last = 63 - __builtin_clzll(__ballot(yes) | 1);
    lo += last * step;
    if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
    n = min(step, n - last * step);
  }
}

template <int D, int MODE>
__device__ __forceinline__ bool pre_span(const AttnArgs& a, PreTile& t) {
  constexpr int BN = PreShape<D>::BN, ROWS = PreShape<D>::ROWS;
  const int g = a.g;
  t.q0 = pre_cu(a, t.seq);
  t.m = max(0, pre_cu(a, t.seq + 1) - t.q0);
  t.rows = t.m * g;
  // (below 0 where rows of q come before the first sequence's)
  if (t.tile < 0 || t.tile * ROWS >= t.rows) return false;
  // (uniform, told so: loads behind the error word's atomic are not taken for it)
  if constexpr (MODE == kDense) {
    auto row = [&](int i) { return max(0L, min((long)a.cu_k[i], a.S)); };
    t.slot = 0;
    t.k0 = row(t.seq);
    t.L = (int)max(0L, row(t.seq + 1) - t.k0);
  } else {
    t.slot = __builtin_amdgcn_readfirstlane(kv_slot(a.slots, t.seq, a.t.n_slots, a.err));
    t.L = __builtin_amdgcn_readfirstlane(kv_len(a.t, t.slot));
  }
  const int r1 = min(t.rows, (t.tile + 1) * ROWS) - 1;
  if constexpr (MODE == kTree) {
    // any row may see any drafted token; all see those before (p_min), from the
    // shallowest one's window on
    if (t.m > kTreeMax) {
      atomicOr(a.err, kErrTree);
      t.L = 0;
    }
    if (t.L < t.m) t.L = 0;
    t.p_min = max(0, t.L - t.m) - 1;
    t.p_max = t.L - 1;
    t.lo_min = a.window ? max(0, t.p_min - a.window + 2) : 0;
  } else {
    t.p_min = t.L - t.m + t.tile * ROWS / g;
    t.p_max = t.L - t.m + r1 / g;
    t.lo_min = a.window ? max(0, t.p_min - a.window + 1) : 0;
  }
  t.lo_max = a.window ? max(0, t.p_max - a.window + 1) : 0;
  // the groups of the first keys and those of the window lie end to end, so
  // that the few first keys do not take a tile of their own
  t.b2 = t.lo_min / 16;
  t.ng1 = min(t.b2, (min(a.first, t.lo_min) + 15) / 16);
  const int end = (max(0, t.p_max + 1) + 15) / 16;
  t.nb = (t.ng1 + max(0, end - t.b2) + BN / 16 - 1) / (BN / 16);
  return true;
}

// Parts that a tile's keys are split into: at least four key tiles each (trees:
// two), and no more than pay. With nb tiles of a time t, nb t / p + p c is least at p =
// sqrt(nb t / c); the cost c of a part is that of its fp32 rows written and
// read back, so t / c is split_gain, a constant over the rows of the call.
template <int MODE>
__device__ __forceinline__ int pre_parts(const AttnArgs& a, int nb) {
  if (a.n_split == 1) return 1;
  constexpr int least = MODE == kTree ? kTreePartMin : kPartMin;
  return max(1, min(min(a.n_split, nb / least), (int)sqrtf((float)nb * a.split_gain)));
}

// what a workgroup's waves tell each other
struct PreNotes {
  int gone;                                      // last tile with a group that has no page
  int miss[2][4];                                // the same for each wave's group, by buffer
  int bad;                                       // values of V not finite were taken out
};

template <bool BF, bool F8, int D, int MODE>
__global__ __launch_bounds__(256, D == 256 ? 1 : D == 128 ? 2 : 3) void attn_prefill_kernel(AttnArgs a) {
  constexpr int BN = PreShape<D>::BN, ROWS = PreShape<D>::ROWS;
  constexpr int NA = BN / 32;                    // 32-key score tiles
  constexpr bool PAGED = MODE != kDense;
  constexpr int DR = PAGED ? 0 : kLatRope;       // shared values of a key
  constexpr int NC = (D + DR) / 16;              // steps of the first product
  constexpr int ND = D / 32;                     // 32-row tiles of O^T
  constexpr int UPR = D / 8;                     // 16-byte units of a row in LDS
  constexpr int WR = BN / 4;                     // rows of a tile that a wave brings
  constexpr int GPR = F8 ? D / 16 : UPR;         // 16-byte units of a row in memory
  constexpr int NL = WR * GPR / 64;              // loads per lane and array
  constexpr int TB = BN * D * 2;                 // bytes of a tile in LDS
  constexpr int KB = TB + BN * DR * 2;           // with the keys' shared values
  static_assert(NL >= 1, "tile");

  __shared__ __align__(16) char s_k0[KB], s_k1[KB], s_v0[TB], s_v1[TB];
  // (dense tiles of two workgroups fill a CU's LDS; of the notes they need bad
  // alone, and find room for it in the end)
  __shared__ PreNotes s_note;
  bool bad = false;
  __shared__ TreeRows<MODE == kTree ? ROWS : 0> s_tree;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l31 = lane & 31;

  PreTile t;
  const int block = a.block0 + (int)blockIdx.x, kvh = block % a.c.hkv;
  // longest tiles first; sequence i's tiles start at cu[i] g / ROWS + i
  const int tt = a.n_tiles - 1 - block / a.c.hkv;
  t.seq = pre_last(a, [&](int i, int cu) { return (int)((long)cu * a.g / ROWS) + i <= tt; });
  t.tile = tt - (int)((long)pre_cu(a, t.seq) * a.g / ROWS) - t.seq;
  if (!pre_span<D, MODE>(a, t)) return;
  const int parts = pre_parts<MODE>(a, t.nb);
  if ((int)blockIdx.y >= parts) return;
  const int x0 = (int)((long)blockIdx.y * t.nb / parts);
  const int x1 = (int)((long)(blockIdx.y + 1) * t.nb / parts);
  if constexpr (PAGED) {
    if (tid < 8) s_note.miss[tid >> 2][tid & 3] = -1;
    if (tid == 0) {
      s_note.gone = -1;
      s_note.bad = 0;
    }
  }


  // scores are compared unscaled: the sign of the scale goes into q
  float sc = F8 ? a.scale * a.c.ks[kvh] : a.scale;
  const uint32_t flip = sc < 0.0f ? 0x80008000u : 0u;
  const bool flat = sc == 0.0f;
  sc = flat ? 1.0f : fabsf(sc);
  const float thr = fminf(kDefer<BF> / sc, 1e30f);

  constexpr int GT = BN / 16;                    // groups of a tile
  auto group_key = [&](int i) { return 16 * (i < t.ng1 ? i : t.b2 + i - t.ng1); };
  // tiles of which every row sees every key (the first keys' may be such too,
  // and are treated as if not)
  const int whole0 =
      (t.ng1 + max(0, (t.lo_max + 15) / 16 - t.b2) + GT - 1) / GT;
  const int whole1 = (t.ng1 - t.b2 + (t.p_min + 1) / 16) / GT;
  auto whole = [&](int x) { return x >= whole0 && x < whole1; };
  // the rows' ancestors, for the parts that have tiles that are not whole
  const bool masked = MODE == kTree && (x0 < whole0 || x1 > whole1);
  if constexpr (MODE == kTree)
    if (masked) s_tree.fetch(a.parent + t.q0, t.m);

  // this lane's row
  struct Row {
    bool have;
    int head;
    long q;                                      // of q and out
  };
  const int row_of = t.tile * ROWS + w * 32;
  int tok = row_of + l31 < t.rows ? (row_of + l31) / a.g : -1;
  auto row_at = [&] {
    asm volatile("" : "+v"(tok));                // not kept in registers beside it
    const int k = max(tok, 0);
    return Row{tok >= 0, kvh * a.g + (tok >= 0 ? row_of + l31 - k * a.g : 0), (long)t.q0 + k};
  };
  const int tok0 = t.tile * ROWS / a.g;          // the tile's first token
  auto pos_of = [&] {
    asm volatile("" : "+v"(tok));
    if constexpr (MODE == kTree)
      return tok >= 0 ? t.L - t.m + (masked ? s_tree.depth(tok - tok0) : 0) : -1;
    return tok >= 0 ? t.L - t.m + tok : -1;
  };
  u32x4 q[NC];
  {
    const Row y0 = row_at();
    const char* p = a.q + y0.q * a.q_row + y0.head * a.q_head + 16 * half;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const u32x4 y = *(const u32x4*)(p + 32 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[c][e] = flat ? 0u : y[e] ^ flip;
    }
  }

  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNegInf, l = 0.0f;

  const int* row = a.t.table + (long)max(0, t.slot) * a.t.ld;
  const char* kb = a.c.k + kvh * a.c.sh + (PAGED ? 0L : t.k0 * a.c.st);
  const char* vb = a.c.v + (PAGED ? kvh * a.c.sh : kvh * a.v_head + t.k0 * a.v_row);
  const char* rb = PAGED ? nullptr : a.kr + t.k0 * a.kr_row;
  const int grp = w * WR / 16;                   // 16-key group that this wave brings from

  // Byte offset in the cache (dense: the key) of the wave's group of the next 64
  // tiles, a tile a lane; kMissing: no page, kUnseen: nothing of it is visible. One
  // lookup a tile is then two lane reads.
  constexpr long kMissing = -(1L << 32), kUnseen = -(2L << 32);
  struct Group {
    long off;                                    // 0 without a page
    int state;                                   // < 0 without one: high word of the above
  };
  int at0 = x0;
  auto lookup = [&](int x) {
    const int key = group_key(GT * x + grp);
    if (x >= x1 || key > t.p_max || !(key + 16 > t.lo_min || key < a.first)) return kUnseen;
    if constexpr (!PAGED) return (long)key;
    const int i = kv_entry(a.t, key), e = row[i];
    return e >= 0 && e < a.t.n_pages ? e * a.c.sp + (key - i * a.t.ps) * a.c.st : kMissing;
  };
  long offs = lookup(x0 + lane);
  auto group_of = [&](int x) {                   // x one after another
    if (x - at0 == 64) {
      at0 = x;
      offs = lookup(x + lane);
    }
    const uint32_t lo32 = __builtin_amdgcn_readlane((int)offs, x - at0);
    const int hi32 = __builtin_amdgcn_readlane((int)(offs >> 32), x - at0);
    return Group{(long)(((uint64_t)(uint32_t)max(hi32, 0) << 32) | lo32), hi32};
  };
  // Swizzle of 16-byte units by row (of the tile). Half a wave reads one unit of
  // 32 rows of K in turn, and 64 bytes of four rows of V, which have to lie in
  // different banks.
  auto k_swz = [](int kr) { return kr & (UPR < 16 ? UPR - 1 : 15); };
  auto v_swz = [](int kr) { return UPR == 8 ? ((kr >> 1) & 1) << 2 : (kr & 3) << 2; };
  // This lane's places in a tile. Rows are a multiple of 128 bytes and the
  // swizzle is the same for rows 16 (K: 32) apart, so units 2 c + half of K
  // are at k_at ^ 32 c, values 32 d.. of V at v_at ^ 64 d, and the row blocks
  // at constant distances: one address register each, turned by an exclusive
  // or where it is used.
  int k_at = l31 * (2 * D) + 16 * (half ^ k_swz(l31));
  const int v_row = 4 * half + ((lane & 15) >> 2), v_d = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  int v_at = v_row * (2 * D) + (16 * ((v_d >> 3) ^ v_swz(v_row)) + 2 * (v_d & 7));
  // unit 2 c + half of the shared values is at r_at ^ 32 c
  const int r_at = TB + l31 * 128 + 16 * (half ^ (l31 >> 1 & 7));
  const uint32_t kExp = BF ? 0x7F80u : 0x7C00u;
  // either value of a pair infinite or NaN: the exponent's carry
  auto carry = [&](uint32_t x) { return (x & 0x7FFF7FFFu) + (BF ? 0x00800080u : 0x04000400u); };
  auto clean16 = [&](uint32_t x) {
    if ((x & kExp) == kExp) x &= 0xFFFF0000u;
    if (((x >> 16) & kExp) == kExp) x &= 0x0000FFFFu;
    return x;
  };
  // a unit of V of a tile that is not whole, as it is to be staged
  auto clean = [&](u32x4 v, int j, bool ok) {      // of key j
    if (!ok || j > t.p_max || !(j >= t.lo_min || j < a.first)) return u32x4{0, 0, 0, 0};
    if ((carry(v[0]) | carry(v[1]) | carry(v[2]) | carry(v[3])) & 0x80008000u) {
      if constexpr (PAGED) s_note.bad = 1; else bad = true;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = clean16(v[e]);
    }
    return v;
  };

  // The wave's rows of a tile: load i takes RPL of them, row i RPL + lane /
  // GPR of the wave. 16-bit caches load straight into LDS, so the swizzle is
  // applied to the units read. e4m3 ones go through registers, expanded on
  // arrival. A lane's offset stays below 2^31 (16 stride_tok < 2^30).
  constexpr int RPL = 64 / GPR;
  const int l_row = ((w * WR) & 15) + lane / GPR;
  // the lane's unit in load 0; the swizzles are exclusive ors of row bits
  const uint32_t k_unit = 16 * (lane % GPR ^ (F8 ? 0 : k_swz(l_row)));
  const uint32_t v_unit = 16 * (lane % GPR ^ (F8 ? 0 : v_swz(l_row)));
  u32x4 rk[F8 ? NL : 1], rv[F8 ? NL : 1];
  // from rows that lie st bytes apart, of which those from `bytes` on are not there
  auto issue = [&](const char* p, uint32_t bytes, long st, uint32_t unit, auto swz, char* to,
                   u32x4* raw) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint32_t f = (uint32_t)l_row * (uint32_t)st + (unit ^ (F8 ? 0 : 16 * swz(i * RPL)));
      asm volatile("" : "+v"(f));                // added by the load, not ahead of it
      if constexpr (F8)
        raw[i] = *(const u32x4*)(p + i * RPL * st + f);
      else
        load_to_lds(p, bytes, (int)(f + i * RPL * (uint32_t)st),
                    lds_of(to) + (w * WR * UPR + i * 64) * 16);
    }
  };
  // bytes that a group's rows of st bytes have: those of keys before the end
  auto bytes_of = [&](const Group& gr, long st) {
    if (gr.state < 0) return 0u;
    return PAGED ? 0x7FFFFFFFu : (uint32_t)(min(16, t.L - (int)gr.off) * st);
  };
  auto issue_k = [&](int x, const Group& gr, char* to, int* miss) {
    if constexpr (PAGED) {
      if (gr.state == (int)(kMissing >> 32) && lane == 0) {
        atomicOr(a.err, kErrPage);
        s_note.gone = x;
        miss[w] = x;
      }
      issue(kb + gr.off, bytes_of(gr, a.c.st), a.c.st, k_unit, k_swz, to, rk);
    } else {
      issue(kb + gr.off * a.c.st, bytes_of(gr, a.c.st), a.c.st, k_unit, k_swz, to, rk);
      const char* p = rb + gr.off * a.kr_row;
      const uint32_t f = lane / 8 * (uint32_t)a.kr_row;
#pragma unroll
      for (int i = 0; i < 2; ++i)                // eight rows of the wave's 16 each
        load_to_lds(p, bytes_of(gr, a.kr_row),
                    (int)(f + 8 * i * (uint32_t)a.kr_row +
                          16 * (lane % 8 ^ (lane / 16) ^ 4 * i)),
                    lds_of(to) + TB + (w * WR + 8 * i) * 128);
    }
  };
  auto issue_v = [&](const Group& gr, char* to) {
    const long st = PAGED ? a.c.st : a.v_row;
    issue(vb + (PAGED ? gr.off : gr.off * st), bytes_of(gr, st), st, v_unit, v_swz, to, rv);
  };
  auto expand = [&](const u32x4& raw, u32x4 (&y)[2]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e >> 1][2 * (e & 1)] = from_e4m3<BF, false>(raw[e]);
      y[e >> 1][2 * (e & 1) + 1] = from_e4m3<BF, true>(raw[e]);
    }
  };
  auto arrived = [&] {
    if constexpr (!F8) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  auto finish_k = [&](char* to) {
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int up = i * 64 + lane, kr = w * WR + up / GPR, u = up % GPR;
        u32x4 y[2];
        expand(rk[i], y);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *(u32x4*)(to + kr * (2 * D) + 16 * ((2 * u + h) ^ k_swz(kr))) = y[h];
      }
    }
  };
  // takes masked values out of V
  auto finish_v = [&](int x, const Group& gr, char* to) {
    const int key = group_key(GT * x + grp) - 16 * grp;
    const bool as_is = whole(x) && gr.state >= 0;
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int up = i * 64 + lane, kr = w * WR + up / GPR, u = up % GPR;
        u32x4 y[2];
        expand(rv[i], y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!as_is) y[h] = clean(y[h], key + kr, gr.state >= 0);
          *(u32x4*)(to + kr * (2 * D) + 16 * ((2 * u + h) ^ v_swz(kr))) = y[h];
        }
      }
    } else if (!as_is) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int up = i * 64 + lane, kr = w * WR + up / GPR;
        u32x4* p = (u32x4*)(to + (w * WR * UPR + up) * 16);
        *p = clean(*p, key + kr, gr.state >= 0);
      }
    }
  };

  // Operand c, aa of the first product: 8 values of D of 32 keys
  auto read_k = [&](const char* from, int c, int aa) {
    if (c >= D / 16)
      return *(const u32x4*)(from + 32 * aa * 128 + (r_at ^ (32 * (c - D / 16))));
    return *(const u32x4*)(from + 32 * aa * (2 * D) + (k_at ^ (32 * c)));
  };
  // Operand of the second product: keys 4 half + 0..3 of the gth 16-key step,
  // then the same + 8; lane i of 16 reads row i / 4, 4 values from 4 (i % 4),
  // and gets column i
  auto read_v = [&](const char* from, int g, int d) {
    u32x4 va;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* p = from + (16 * g + 8 * h) * (2 * D) + (v_at ^ (64 * d));
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)const_cast<char*>(p));
      const u32x2 z = __builtin_bit_cast(u32x2, y);
      va[2 * h] = z[0];
      va[2 * h + 1] = z[1];
    }
    return va;
  };
  // S^T of a tile, unscaled
  auto scores = [&](f32x16 (&s)[NA], const char* from) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int aa = 0; aa < NA; ++aa) {
        const f32x16 zero = {};
        s[aa] = mfma32<BF>(read_k(from, c, aa), q[c], c == 0 ? zero : s[aa]);
      }
  };
  // masks them, and lets m, l and O follow the maximum
  auto settle = [&](f32x16 (&s)[NA], int x, int gone_tile, const int* miss) {
    const bool miss_any = __builtin_amdgcn_readfirstlane(gone_tile) >= x;
    if (miss_any || !whole(x)) {
      uint32_t gone = 0;                         // 16-key groups without a page
      if (miss_any) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (miss[i] == x) gone |= 1u << (i * WR / 16);
        gone = __builtin_amdgcn_readfirstlane(gone);
      }
      // Bit n of `see`: element n of the lane, key 8 (n / 4) + n % 4 of those
      // from `at` on. Elements ascend by key, so each bound is a run of ones.
      // (Selects without branches: a branch per element would copy the tile.)
      auto below = [&](int c) {                  // elements of keys < c
        const int k = min(max(c, 0), 64), cnt = 4 * (k >> 3) + min(k & 7, 4);
        return (uint32_t)((1ull << cnt) - 1);
      };
      const int pos = pos_of(), lo = a.window ? pos - a.window + 1 : 0;
      const int end = MODE == kTree ? (tok >= 0 ? t.L - t.m : 0) : pos + 1;
      const int at = 16 * (t.b2 - t.ng1 + GT * x) + 4 * half;
      uint32_t see = below(end - at) & (~below(lo - at) | below(a.first - at));
      if constexpr (MODE == kTree) {
        // the row's own key and its ancestors': 64 keys from `at` on, of which
        // the lane has four of each eight
        if (masked && tok >= 0) {
          uint64_t f = s_tree.bits(tok - tok0, at - (t.L - t.m)) & 0x0F0F0F0F0F0F0F0Full;
          f = (f | f >> 4) & 0x00FF00FF00FF00FFull;
          f = (f | f >> 8) & 0x0000FFFF0000FFFFull;
          see |= (uint32_t)(f | f >> 16);
        }
      }
      if (GT * x < t.ng1) {                      // groups of the first keys
        const uint32_t own = below(16 * (t.ng1 - GT * x));
        see = (see & ~own) | (own & below(min(end, a.first) - 16 * GT * x - 4 * half));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) see &= (gone >> i) & 1 ? ~(0xFFu << (8 * i)) : ~0u;
#pragma unroll
      for (int n = 0; n < 16 * NA; ++n) {
        const uint32_t keep = (uint32_t)((int)(see << (31 - n)) >> 31);
        const uint32_t v = __float_as_uint(s[n >> 4][n & 15]);
        s[n >> 4][n & 15] = __uint_as_float((v & keep) | (0xFF800000u & ~keep));
      }
    }
    float bm = s[0][0];
#pragma unroll
    for (int aa = 0; aa < NA; ++aa)
#pragma unroll
      for (int i = 0; i < 16; ++i) bm = fmaxf(bm, s[aa][i]);
    bm = xor32_reduce(bm, OpMax{});
    if (__any(bm > m + thr)) {
      const float mn = fmaxf(m, bm);
      float df = (m - (mn == kNegInf ? 0.0f : mn)) * sc;
      if constexpr (!BF) df += pre_lift<BF>(mn * sc) - pre_lift<BF>(m * sc);
      const float f = exp2_fast(df);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
  };
  // the exponent of P less s sc
  auto neg_of = [&] {
    const float ms = m * sc;
    return m == kNegInf ? 0.0f : BF ? -ms : pre_lift<BF>(ms) - ms;
  };
  // P of a tile (s), its sum and its product with V (vx), and beside them, if
  // NEXT, S^T of the next tile (sn) from its K (kn). One matrix instruction
  // after another, each with the read of the operand that is due kAhead of
  // them later and a share of the exponentials behind it: the order is kept
  // as written, since the reads' latency (some 130 cycles) and the vector
  // work both have to go under matrix instructions of 32 cycles. kAhead: as
  // far as the registers reach (6000 tokens, TFLOP/s at 2 / 3 / 4 / 5:
  // head_dim 64 e4m3 743 709 650; 256 711 734 750 751; 128 e4m3, two long
  // chunks, 3 against 4: 906 872).
  // kLag: an exponential's result is taken up so many of them later, so that
  // the wave does not stand still for it (head_dim 128 0 / 2: 924 / 942
  // TFLOP/s; 64, with three waves a SIMD: 843 / 831; chunks over e4m3: 866 / 853).
  constexpr int kLag = D == 64 || F8 ? 0 : 2;
  constexpr int kAhead = D == 64 ? (F8 ? 2 : 3) : (F8 ? 3 : 5);
  auto products = [&](auto next, f32x16 (&s)[NA], f32x16 (&sn)[NA], const char* kn,
                      const char* vx) {
    constexpr bool NEXT = decltype(next)::value;
    constexpr int MQ = NEXT ? NA * NC : 0, MV = 2 * NA * ND, NE = 16 * NA;
    asm volatile("" : "+v"(k_at), "+v"(v_at));   // not 2 x NC addresses kept in registers
    const float neg = neg_of();
    u32x4 op[MQ + MV], pb[2 * NA];
    float pend[kLag + 1], p0 = 0.0f;
    auto read = [&](int i) {
      op[i] = i < MQ ? read_k(kn, i / NA, i % NA) : read_v(vx, (i - MQ) / ND, (i - MQ) % ND);
    };
    // probabilities come before the step that needs them: 8 for each ND of MV
    auto add = [&](int e) {
      const float pe = pend[e % (kLag + 1)];
      l += pe;
      asm volatile("" : "+v"(l));                // added here: sunk below, all P would stay
      if (e & 1) pb[e >> 3][(e & 7) >> 1] = pack16<BF>(p0, pe);
      p0 = pe;
    };
    constexpr int LAG = NEXT ? kLag : 0;
    auto element = [&](int e) {
      pend[e % (kLag + 1)] = exp2_fast(__builtin_fmaf(s[e >> 4][e & 15], sc, neg));
      if (e >= LAG) add(e - LAG);
      if (e == NE - 1)
#pragma unroll
        for (int i = NE - LAG; i < NE; ++i) add(i);
    };
    if (!NEXT) {
#pragma unroll
      for (int e = 0; e < 8; ++e) element(e);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) read(i);
#pragma unroll
    for (int i = 0; i < MQ + MV; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i + kAhead < MQ + MV) read(i + kAhead);
      if (i < MQ) {
        const f32x16 zero = {};
        sn[i % NA] = mfma32<BF>(op[i], q[i / NA], i < NA ? zero : sn[i % NA]);
      } else {
        const int j = i - MQ;
        o[j % ND] = mfma32<BF>(op[i], pb[j / ND], o[j % ND]);
      }
#pragma unroll
      for (int e = NEXT ? 0 : 8; e < NE; ++e) {
        const int at = NEXT ? e * (MQ + MV - ND) / NE : (e - 8) * (MV - ND) / (NE - 8);
        if (at == i) element(e);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // Tile x's second product runs with tile x + 1's first, so that one's
  // exponentials fill the other's matrix instructions. Iteration x waits for
  // K of x + 1 and V of x and starts the loads of K of x + 2 and V of x + 1,
  // into the buffers that iteration x - 1 read last.
  f32x16 sa[NA], sb[NA];
  Group g0{0, -2}, g1{0, -2};                    // of tiles x and x + 1
  int x = x0;
  // kx, vx: tile x's K and V; kn, vn: tile x + 1's. Distinct buffers, told so
  // that reads do not wait for the loads in flight into the others.
  auto step = [&](f32x16 (&s)[NA], f32x16 (&sn)[NA], char* __restrict kx, char* __restrict kn,
                  char* __restrict vx, char* __restrict vn, int* missx, int* missn) {
    arrived();
    finish_k(kn);
    if (x > x0) finish_v(x, g0, vx);
    __syncthreads();
    const int gone_tile = PAGED ? s_note.gone : -1;
    g0 = g1;
    if (x + 2 < x1) {
      g1 = group_of(x + 2);
      issue_k(x + 2, g1, kx, missx);
    }
    issue_v(g0, vn);
    products(std::true_type{}, s, sn, kn, vx);
    settle(sn, x + 1, gone_tile, missn);
    ++x;
  };
  auto last = [&](f32x16 (&s)[NA], char* vx) {
    if (x > x0) {
      arrived();
      finish_v(x, g0, vx);
      __syncthreads();
    }
    products(std::false_type{}, s, s, nullptr, vx);
  };
  if (x0 < x1) {
    g0 = group_of(x0);
    __syncthreads();                             // s_note is set
    issue_k(x0, g0, s_k0, s_note.miss[0]);
    issue_v(g0, s_v0);
    if constexpr (MODE == kTree)
      if (masked)
        s_tree.build(tok0, min(t.m, (t.tile * ROWS + ROWS - 1) / a.g + 1), t.L - t.m, a.window,
                     a.first, a.err);
    if (x0 + 1 < x1) g1 = group_of(x0 + 1);
    arrived();
    finish_k(s_k0);
    finish_v(x0, g0, s_v0);
    __syncthreads();
    const int gone_tile = PAGED ? s_note.gone : -1;
    if (x0 + 1 < x1) issue_k(x0 + 1, g1, s_k1, s_note.miss[1]);
    scores(sa, s_k0);
    settle(sa, x0, gone_tile, s_note.miss[0]);
    while (x + 2 < x1) {
      step(sa, sb, s_k0, s_k1, s_v0, s_v1, s_note.miss[0], s_note.miss[1]);
      step(sb, sa, s_k1, s_k0, s_v1, s_v0, s_note.miss[1], s_note.miss[0]);
    }
    if (x + 1 < x1) {
      step(sa, sb, s_k0, s_k1, s_v0, s_v1, s_note.miss[0], s_note.miss[1]);
      last(sb, s_v1);
    } else {
      last(sa, s_v0);
    }
  }

  // values of V that are not finite and were staged as zeros: their products,
  // for the rows that see their key
  __syncthreads();
  if constexpr (!PAGED) {
    if (lane == 0) ((int*)s_k0)[w] = 0;
    if (bad) ((int*)s_k0)[w] = 1;
    __syncthreads();
    bad = ((int*)s_k0)[0] | ((int*)s_k0)[1] | ((int*)s_k0)[2] | ((int*)s_k0)[3];
    __syncthreads();
  } else {
    bad = s_note.bad;
  }
  if (bad) {
    const int pos = pos_of(), lo = a.window ? pos - a.window + 1 : 0;
    for (int xx = x0; xx < x1; ++xx) {
      if (whole(xx)) continue;
      for (int i = 0; i < BN; ++i) {
        const int j = group_key(GT * xx + i / 16) + i % 16;
        if (j > t.p_max || !(j >= t.lo_min || j < a.first)) continue;
        long off = 0;
        if constexpr (PAGED) {
          const int e = kv_entry(a.t, j), p = row[e];
          if (p < 0 || p >= a.t.n_pages) continue;
          off = p * a.c.sp + (long)(j - e * a.t.ps) * a.c.st;
        }
        auto value = [&](const char* base, int dd) {
          uint32_t x16;
          if constexpr (F8)
            x16 = from_e4m3<BF, false>(*(const uint8_t*)(base + dd)) & 0xFFFF;
          else
            x16 = *(const uint16_t*)(base + 2 * dd);
          return BF ? bf16_bits_to_f32(x16)
                    : (float)__builtin_bit_cast(_Float16, (uint16_t)x16);
        };
        const char* vj = vb + (PAGED ? off : j * a.v_row);
        const char* kj = kb + (PAGED ? off : j * a.c.st);
        auto finite = [](float f) { return fabsf(f) < __builtin_huge_valf(); };
        bool any = false;
#pragma unroll 1
        for (int dd = lane; dd < D; dd += 64) any |= !finite(value(vj, dd));
        if (!__any(any)) continue;
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t q16 = (q[c][i >> 1] >> (16 * (i & 1))) & 0xFFFF;
            const int dd = 16 * c + 8 * half + i;
            dot += (c < D / 16 ? value(kj, dd) : value(rb + j * a.kr_row, dd - D)) *
                   (BF ? bf16_bits_to_f32(q16)
                       : (float)__builtin_bit_cast(_Float16, (uint16_t)q16));
          }
        dot = xor32_reduce(dot, OpSum{});
        bool sees = j <= pos && (j >= lo || j < a.first);
        if constexpr (MODE == kTree) {
          const int b = j - (t.L - t.m);         // a drafted token
          if (b >= 0) sees = tok >= 0 && (s_tree.bits(tok - tok0, b) & 1);
        }
        const float pv = exp2_fast(__builtin_fmaf(dot, sc, neg_of()));
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = value(vj, 32 * d + 8 * (i >> 2) + 4 * half + (i & 3));
            if (sees && !finite(f)) o[d][i] += pv * f;
            if (i == 15) __builtin_amdgcn_sched_barrier(0);
          }
      }
    }
  }

  l = xor32_reduce(l, OpSum{});
  const Row me = row_at();
  if (parts == 1) {
    // turned round through the wave's share of LDS, so that stores take whole
    // rows; the 16-byte units of a row are swizzled by its number
    const float inv = l == 0.0f ? 0.0f : (F8 ? a.c.vs[kvh] : 1.0f) / l;
    if (__any(me.have && l == 0.0f)) {           // see of_sum; rare, so not a select in all rows
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = of_sum(o[d][i], 1.0f, l);
    }
    constexpr int RB = 2 * D, WB = 32 * RB;
    static_assert(TB >= WB && TB <= 2 * WB, "a buffer holds one or two waves' rows");
    char* const mine =
        TB == WB ? (w < 2 ? (w ? s_k1 : s_k0) : (w == 2 ? s_v0 : s_v1))
                 : (w < 2 ? s_k0 : s_k1) + (w & 1) * WB;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const u32x2 y = {pack16<BF>(o[d][i] * inv, o[d][i + 1] * inv),
                         pack16<BF>(o[d][i + 2] * inv, o[d][i + 3] * inv)};
        *(u32x2*)(mine + l31 * RB + 16 * ((4 * d + (i >> 2)) ^ (l31 & (UPR - 1))) + 8 * half) = y;
      }
#pragma unroll
    for (int i = 0; i < UPR / 2; ++i) {
      const int rr = i * (64 / UPR) + lane / UPR, u = lane % UPR;
      const int tk = __shfl(tok, rr);
      const u32x4 y = *(const u32x4*)(mine + rr * RB + 16 * (u ^ (rr & (UPR - 1))));
      if (tk >= 0)
        *(u32x4*)(a.out + ((long)t.q0 + tk) * a.o_row +
                  (kvh * a.g + row_of + rr - tk * a.g) * a.o_head + 16 * u) = y;
    }
    if (a.lse && half == 0 && me.have)
      a.lse[me.q * a.hq + me.head] =
          (m * sc + (__builtin_amdgcn_logf(l) - pre_lift<BF>(m * sc))) * kLn2;
  } else if (me.have) {
    const long rows = a.T * a.hq, ri = me.q * a.hq + me.head;
    float* dst = a.part + ((long)blockIdx.y * rows + ri) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(f32x4*)(dst + 32 * d + 2 * i + 4 * half) =
            f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (half == 0) {
      float* ml = a.part + (long)a.n_split * rows * D + ((long)blockIdx.y * rows + ri) * 2;
      ml[0] = m * sc - pre_lift<BF>(m * sc);
      ml[1] = l;
    }
  }
}

// Joins the parts of split tiles, the parts in order: 16 lanes a row, or Q times as
// many, every Q-th part to each. Four for trees of more than 16 parts, which are few
// rows, bound by the chain of their loads (three of 64 parts, 10 heads of 256: the
// call 44 us against 52); with few parts of many rows they cost (trees of 52..121
// tokens in two parts 167 us against 151).
template <bool BF, bool F8, int D, int MODE, int Q>
__global__ __launch_bounds__(256) void prefill_join_kernel(AttnArgs a) {
  constexpr int ROWS = PreShape<D>::ROWS, V = D / 16;
  PreTile t;
  const int block = a.block0 + (int)blockIdx.x;
  const int kvh = block % a.c.hkv, tt = block / a.c.hkv;
  t.seq = pre_last(a, [&](int i, int cu) { return (int)((long)cu * a.g / ROWS) + i <= tt; });
  t.tile = tt - (int)((long)pre_cu(a, t.seq) * a.g / ROWS) - t.seq;
  if (!pre_span<D, MODE>(a, t)) return;
  const int parts = pre_parts<MODE>(a, t.nb);
  if (parts == 1) return;
  const int r = t.tile * ROWS + ((int)blockIdx.y * 16 + (int)(threadIdx.x >> 4)) / Q;
  if (r >= t.rows) return;
  const int q = (int)(threadIdx.x >> 4) % Q;
  const int d0 = (int)(threadIdx.x & 15) * V, tok = r / a.g, head = kvh * a.g + r - tok * a.g;
  const long rows = a.T * a.hq, ri = ((long)t.q0 + tok) * a.hq + head;
  const float* ml = a.part + (long)a.n_split * rows * D + ri * 2;
  // maxima and sums: part 16 i + lane of the 16; factor i for those parts
  const int l16 = threadIdx.x & 15;
  constexpr int MP = kPreMaxParts / 16;
  float pm[MP], pl[MP], m = kNegInf, l = 0.0f;
#pragma unroll
  for (int i = 0; i < MP; ++i) {
    const int at = 16 * i + l16;
    pm[i] = at < parts ? ml[(long)at * rows * 2] : kNegInf;
    pl[i] = at < parts ? ml[(long)at * rows * 2 + 1] : 0.0f;
    m = fmaxf(m, pm[i]);
  }
  for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float mu = m == kNegInf ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < MP; ++i) {
    pm[i] = exp2_fast(pm[i] - mu);
    l += pm[i] * pl[i];
  }
  for (int d = 1; d < 16; d <<= 1) l += __shfl_xor(l, d);
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < MP; ++i) {
    const int end = min(16, parts - 16 * i);
#pragma unroll 4
    for (int j = q; j < end; j += Q) {
      const float f = __shfl(pm[i], j, 16);
      const float* p = a.part + ((long)(16 * i + j) * rows + ri) * D + d0;
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const f32x4 y = *(const f32x4*)(p + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[e + k] += f * y[k];
      }
    }
  }
  if constexpr (Q > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = xor32_reduce(xor16_reduce(acc[e], OpSum{}), OpSum{});
    if (q) return;
  }
  const float inv = (F8 ? a.c.vs[kvh] : 1.0f) / l;
  char* dst = a.out + ((long)t.q0 + tok) * a.o_row + head * a.o_head + 2 * d0;
#pragma unroll
  for (int e = 0; e < V; e += 4) {
    const u32x2 y = {pack16<BF>(of_sum(acc[e], inv, l), of_sum(acc[e + 1], inv, l)),
                     pack16<BF>(of_sum(acc[e + 2], inv, l), of_sum(acc[e + 3], inv, l))};
    *(u32x2*)(dst + 2 * e) = y;
  }
  if (a.lse && d0 == 0) a.lse[ri] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool BF, bool F8, int D, int MODE>
hipError_t run_prefill(const AttnArgs& all, hipStream_t s) {
  AttnArgs a = all;
  a.n_tiles = (int)prefill_tiles(a.n, a.T, a.g);
  const long blocks = (long)a.n_tiles * a.c.hkv;
  for (long b = 0; b < blocks; b += kMaxGrid) {
    const unsigned grid = (unsigned)(blocks - b < kMaxGrid ? blocks - b : kMaxGrid);
    a.block0 = (int)b;
    attn_prefill_kernel<BF, F8, D, MODE><<<dim3(grid, a.n_split), 256, 0, s>>>(a);
    constexpr int Q = MODE == kTree ? 4 : 1;
    if (Q > 1 && a.n_split > 16)
      prefill_join_kernel<BF, F8, D, MODE, Q>
          <<<dim3(grid, PreShape<D>::ROWS / 16 * Q), 256, 0, s>>>(a);
    else if (a.n_split > 1)
      prefill_join_kernel<BF, F8, D, MODE, 1>
          <<<dim3(grid, PreShape<D>::ROWS / 16), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int D, int MODE>
hipError_t run_prefill_d(const AttnArgs& a, int fmt, hipStream_t s) {
  const bool f8 = a.c.fmt == KV_E4M3;
  if (fmt == KV_BF16)
    return f8 ? run_prefill<true, true, D, MODE>(a, s) : run_prefill<true, false, D, MODE>(a, s);
  return f8 ? run_prefill<false, true, D, MODE>(a, s) : run_prefill<false, false, D, MODE>(a, s);
}

}  // namespace
}  // namespace moe
