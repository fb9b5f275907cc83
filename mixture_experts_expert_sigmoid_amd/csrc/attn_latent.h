// Attention over a paged cache of latent vectors: keys are a token's latent
// vector and rotary key, values its latent vector, all query heads share them.
//
// Mathematics. As for prompts (one pass with the running maximum and sum, S^T =
// K Q^T, P = 2^(S - m), O^T = V^T P^T, fp32 but for the 16-bit operands, m
// followed only when it has grown by 2^kDefer), with one key head of 576 or 320
// values and g = all query heads: a tile of 64 rows, (token, head) pairs
// token-major, uses each latent vector 64 times in both products, and reads it once,
// as key and as value. (With more rows a sequence has more tiles, and each reads the
// vectors: see Work.) P is rounded to the 16 bits of q, which the matrix instructions
// take at their rate; results stand up to a third further from the 64-bit values than
// with P of 32 bits. Codes of e4m3 caches are multiplied as they are; the scale goes
// into the softmax's and the result's.
//
// Layout. O of 64 rows is 128 KB, a quarter of a CU's registers, so a CU holds one
// workgroup of eight waves: in the second product each has 64 of the 512 values
// for all rows, in the first 16 keys and 16 rows, of which it multiplies half the
// depth for 32 rows (an operand of K, read from LDS, then serves twice) and
// trades the other rows' half with the wave next to it. Q lives in registers, K
// in four LDS buffers of 32 keys, written by DMA three tiles ahead and waited for
// by count, never emptied; V is the same bytes read transposed
// (ds_read_b64_tr_b16, _b8 for codes). The scores and P of tile x + 1 are
// computed among the products of tile x, in written order; two barriers a tile.
// What is rare (masks, a maximum that grew, values that are not finite) stands
// outside the loop: within, it made the compiler copy O in each step.
//
// Work. The keys of all tiles, end to end, are dealt out evenly to at most 256
// workgroups, whatever the lengths; a tile's start (places, queries, an empty
// pipeline: 5 us) counts as kLatStart units of 32 keys. Parts of a tile are
// joined in order by a second launch. The counts are computed by every workgroup
// from the lengths, up to kLatSeqs sequences a launch. The units of a tile come
// after all of the tile before, so that the tiles of a sequence read the same keys at
// different times: 128 heads, two tiles a token, miss the L2 for 356 MB of a cache of
// 177 MB, trees of 64 heads for 571 MB of 60.
//
// Bound. A step (32 keys, 64 rows, 4.5 MFLOP) takes 1.25 us, 0.91 PFLOP/s over 256
// CUs: 37 % of its cycles issue matrix instructions and as many move LDS (28-30 % of
// them in bank conflicts), and eight waves in step overlap the two no better. Reading further ahead, K across the barrier, other places for the loads:
// no change. Beside the steps there are 2 us of prologue, 5 a piece of start and
// the parts, 131 KB each, written and read. Measured: a token of 64 sequences of
// 201..4001 keys, 128 heads (177 MB, 38 GFLOP) 79-80 us, 66-68 of it this kernel
// and 13 the join; trees over e4m3 (142 GFLOP) 176-180 us, 0.79-0.80 PFLOP/s; one
// token of 16 heads over 777 keys 17.7 us, latency. The first form (four waves, O
// in the accumulators' half of the registers, waits by the compiler) took 173 us
// and 294.
#pragma once
#include <type_traits>

#include "attn_dev.h"
#include "attn_tree.h"

namespace moe {
namespace {

// a sequence of the launch, and its rows and keys as tiles
struct LatSeq {
  int q0, m, slot, L, C;       // first row of q, new tokens; slot, tokens, those before
  int ng1, b2, nb;             // 16-key groups 0..ng1-1, then b2 and on; 32-key tiles of them
  int tiles;                   // of kLatRows rows
  int lo_min;
};

__device__ __forceinline__ int lat_cu(const AttnArgs& a, int i) {
  if (!a.cu) return i;
  const int c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? (int)a.T : c);
}

__device__ __forceinline__ LatSeq lat_seq(const AttnArgs& a, int i) {
  LatSeq s;
  s.q0 = lat_cu(a, i);
  s.m = max(0, lat_cu(a, i + 1) - s.q0);
  s.slot = kv_slot(a.slots, i, a.t.n_slots, a.err);
  s.L = kv_len(a.t, s.slot);
  if (a.parent) {
    if (s.m > kTreeMax) {
      atomicOr(a.err, kErrTree);
      s.L = 0;
    }
    if (s.L < s.m) s.L = 0;
  }
  s.C = s.L - s.m;
  s.lo_min = a.window ? max(0, s.C - a.window + 1) : 0;
  s.b2 = s.lo_min / 16;
  s.ng1 = min(s.b2, (min(a.first, s.lo_min) + 15) / 16);
  s.nb = max(1, (s.ng1 + max(0, (s.L + 15) / 16 - s.b2) + 1) / 2);
  s.tiles = (int)(((long)s.m * a.hq + kLatRows - 1) / kLatRows);
  return s;
}

// x / hq for x < hq + kLatRows by the reciprocal h_inv = ceil(2^22 / hq): its excess
// over 2^22 / hq is below 1, so that of x h_inv below x <= 1087, less than 2^22 / hq
__device__ __forceinline__ int lat_token(const AttnArgs& a, int x) {
  return (int)((uint32_t)x * a.h_inv >> 22);
}

// workgroups that share U units (32 keys of a tile of rows)
__device__ __forceinline__ long lat_teams(long U, long grid) {
  const long w = (U + kLatMinUnits - 1) / kLatMinUnits;
  return w < grid ? w : grid;
}

// A value that is to be computed with here: what follows from it is not found
// ahead of the loops around and kept in registers, of which there are none left.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Waits until at most VM of the wave's vector memory operations and LGKM of its
// reads and writes of LDS are in flight (63 and 15: however many).
template <int VM, int LGKM>
__device__ __forceinline__ void wait_counts() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | LGKM << 8 | (VM >> 4) << 14);
  asm volatile("" ::: "memory");
}

// A barrier for LDS alone: loads stay in flight (__syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() {
  wait_counts<63, 0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <bool BF, bool F8, int DC>
__global__ __launch_bounds__(64 * kLatWaves, 2) void attn_latent_kernel(AttnArgs a) {
  constexpr int R = kLatRows, NW = kLatWaves;
  constexpr int ES = F8 ? 1 : 2;
  constexpr int RB = DC * ES, UPR = RB / 16;              // bytes and units of a latent row
  constexpr int RRB = kLatRope * ES, URR = RRB / 16;      // of a rotary one
  constexpr int TB = 32 * (RB + RRB);                     // a tile of 32 keys
  constexpr int RPW = 32 / NW;                            // rows of it that a wave brings
  constexpr int RPL = 64 / UPR, NLD = RPW / RPL;          // rows of a load; loads
  constexpr int LOADS = NLD + 1;
  constexpr int NK = (DC + kLatRope) / 32;                // steps of the first product
  constexpr int QR = 2 * R / NW;                          // a wave's rows of scores
  constexpr int RT = R / 32;                              // 32-row tiles in the second
  constexpr int ND = DC / 32 / NW;                        // a wave's 32-row tiles of O^T
  constexpr int QB = R * (DC + kLatRope) * 2;             // the queries
  static_assert(QR == 16 && ND >= 1 && NLD >= 1, "a wave's shares");

  __shared__ __align__(16) char s_t[4][TB];               // tile x in (x - first) % 4
  __shared__ __align__(16) char s_q[F8 ? QB : 16];        // the queries, or in the last two tiles
  __shared__ __align__(16) char s_p[R * 64];              // P of the tile before the one whose
                                                          // scores are computed
  // halves of scores for the wave next to each; between steps, and in the end,
  // what the rows' waves tell each other
  __shared__ __align__(16) union {
    char half[NW][1024];
    struct { float f[R], top[2][R], l[2][R]; } row;
  } s_x;
  static_assert(F8 || 2 * TB == QB, "two tiles hold the queries");
  __shared__ long s_pref[kLatSeqs + 1];
  __shared__ TreeRows<R> s_tree;
  __shared__ float s_m[R];
  __shared__ long s_scan[NW];
  __shared__ int s_tell[8];                               // by x % 8: tile x if its P is to be
                                                          // done again
  __shared__ int s_again;                                 // a result is not finite

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Its 16 keys (kq) and 16 rows (rq) of scores. The wave next to it has the
  // same keys and the next rows; one of them (dq) multiplies the first half of
  // the depth for both, the other the second, so that an operand of K is read
  // from LDS for 32 rows.
  const int kq = w / (NW / 2), rq = w % (NW / 2), dq = w & 1;
  const int lc = lane & 15, g4 = lane >> 4, half = lane >> 5, l31 = lane & 31;
  const int H = a.hq;

  // prefix sums of the sequences' units
  {
    long v = 0;
    if (tid < a.n) {
      const LatSeq s = lat_seq(a, tid);
      v = (long)s.tiles * (s.nb + kLatStart);
    }
    for (int d = 1; d < 64; d <<= 1) {
      const long o = __shfl_up(v, d);
      if (lane >= d) v += o;
    }
    if (lane == 63) s_scan[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v += s_scan[i];
    if (tid < a.n) s_pref[tid + 1] = v;
    if (tid == 0) s_pref[0] = 0;
    __syncthreads();
  }
  const long U = s_pref[a.n], W = lat_teams(U, gridDim.x);
  // workgroups next to each other go on along a tile or have the next one of the same
  // sequence, which reads the same keys, if later: they go to one XCD (L2 hits of 18-20 %)
  const int wg = W > 128 && gridDim.x % 8 == 0
                     ? (int)(blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8)
                     : (int)blockIdx.x;
  int* const meta = a.meta + 4 * wg;
  if (tid == 0) meta[3] = 0;
  if (wg >= W) return;
  // workgroup v starts at unit v U / W, whole and rest by themselves
  const uint32_t w32 = (uint32_t)W;
  const long each = U >> 32 ? U / W : (uint32_t)U / w32;
  const uint32_t rest = (uint32_t)(U - each * W);
  auto start_of = [&](int v) { return v * each + v * rest / w32; };
  long u = start_of(wg);
  const long u_end = start_of(wg + 1);
  // the sequence of unit u
  if (tid < a.n && s_pref[tid] <= u && s_pref[tid + 1] > u) s_scan[0] = tid;
  __syncthreads();
  int seq = __builtin_amdgcn_readfirstlane((int)s_scan[0]);

  const float sc = F8 ? a.scale * a.c.ks[0] : a.scale;

  // Swizzles: the 16-byte units of a row lie turned by its number, so that what is
  // read at a time -- the same unit of 16 rows (K, P), the next four units of four
  // rows or the next two of eight (V, transposed) -- lies in different places of 256
  // bytes. Not so of 128: rows r and r + 2 of K (codes: r + 4) are that far apart, and
  // 28-30 % of the active cycles of LDS go to conflicts, where the prompts' kernels,
  // whose turn is the row's number, have 1-2 %.
  auto swz = [](int r) {
    return F8 ? (r & 7) << 1 | (r >> 3 & 1) : (r & 3) << 2 | (r >> 2 & 3);
  };
  auto swz_r = [](int r) { return F8 ? r >> 2 & 3 : r >> 1 & 7; };
  auto p_swz = [](int r) { return r >> 2 & 3; };
  // Operands' places in a tile, of which one turn of the swizzle takes 256 bytes:
  // a register for each place within those, the rest by constant distances
  const int k_row = 16 * kq + lc, v_row = 8 * half + (F8 ? lc >> 1 : lc >> 2);
  constexpr int KS = F8 ? 2 : 1, MK = NK / KS;            // reads of K that the depth takes
  constexpr int MR = kLatRope / 32 / KS, ML = MK - MR;    // of rotary values, of latent ones
  constexpr int MW = (MK + 1) / 2;                        // of a wave (the second half: MK - MW)
  int k_at[4], kr_at[MR], v_at[ND][2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = dq * MW + j;
    k_at[j] = k_row * RB + 256 * (g >> 2) + 16 * ((4 * (g & 3) + g4) ^ swz(k_row));
  }
  // the second half's last reads; the first half's of the same number
#pragma unroll
  for (int n = 0; n < MR; ++n) {
    constexpr int first = MK - MW - MR;
    kr_at[n] = dq ? 32 * RB + k_row * RRB + 16 * ((4 * n + g4) ^ swz_r(k_row))
                  : k_at[(first + n) & 3] + 256 * ((first + n) >> 2);
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (w * ND + d) * 32 * ES;
      const int un = F8 ? g4 & 1 : 2 * (g4 & 1) + (lc >> 1 & 1);
      const int r = v_row + 4 * h;
      v_at[d][h] = r * RB + at / 256 * 256 + 16 * ((at % 256 / 16 + un) ^ swz(r)) + 8 * (lc & 1);
    }
  // this lane's unit in a wave's loads of RPW rows: load i takes RPL of them (the
  // swizzles are exclusive ors of row bits)
  const int l_from = w % (NW / 2) * RPW;                  // row of the group
  const int l_row = lane / UPR * (int)a.c.st;
  const int l_unit = 16 * (lane % UPR ^ swz(l_from + lane / UPR));
  const int l_rope = lane / URR * (int)a.c.st + RB + 16 * (lane % URR ^ swz_r(l_from + lane / URR));
  const int p_to = (rq * QR + lc) * 64 + 16 * ((2 * kq + (g4 >> 1)) ^ p_swz(lc)) + 8 * (g4 & 1);
  const int p_from = l31 * 64 + 16 * (half ^ p_swz(l31));

  bool careful = false;                          // the piece is being done again, see s_again
  while (u < u_end) {
    while (s_pref[seq + 1] <= u) ++seq;
    seq = __builtin_amdgcn_readfirstlane(seq);   // (alike in all lanes: told so)
    const LatSeq s = lat_seq(a, seq);
    const long rel = u - s_pref[seq];
    const int units = s.nb + kLatStart;          // of a tile; the first ones stand for its start
    const int tile = __builtin_amdgcn_readfirstlane(
        rel >> 32 ? (int)(rel / units) : (int)((uint32_t)rel / (uint32_t)units));
    const int v0 = __builtin_amdgcn_readfirstlane((int)(rel - (long)tile * units));
    const int v1 = (int)min((long)units, v0 + (u_end - u));
    u += v1 - v0;
    const int b0 = max(0, v0 - kLatStart), b1 = v1 - kLatStart;
    if (b1 <= b0) continue;
    const int rows = s.m * H, r0 = tile * R;
    const int have = min(R, rows - r0);          // rows of the tile
    const int tok0 = r0 / H, head0 = r0 - tok0 * H;          // of the first
    const int tok1 = tok0 + lat_token(a, head0 + have - 1);
    const bool tree = a.parent != nullptr;
    const int p_min = tree ? max(0, s.C) - 1 : s.C + tok0;
    const int p_max = tree ? s.L - 1 : s.C + tok1;
    const int lo_max = a.window ? max(0, p_max - a.window + 1) : 0;
    auto group_key = [&](int i) { return 16 * (i < s.ng1 ? i : s.b2 + i - s.ng1); };
    const int end_g = s.ng1 + max(0, (max(0, p_max + 1) + 15) / 16 - s.b2);
    const int x_end = __builtin_amdgcn_readfirstlane(min(b1, (end_g + 1) / 2));
    const int whole0 = (s.ng1 + max(0, (lo_max + 15) / 16 - s.b2) + 1) / 2;
    const int whole1 = careful ? 0 : (s.ng1 - s.b2 + max(0, p_min + 1) / 16) / 2;
    auto whole = [&](int x) { return x >= whole0 && x < whole1; };
    const bool masked = tree && (b0 < whole0 || x_end > whole1);

    lds_barrier();                               // of the piece before, whose stores may go on
    if (masked) s_tree.fetch(a.parent + s.q0, s.m);
    if (tid < R) s_m[tid] = kNegInf;
    if (tid < 8) s_tell[tid] = -1;
    if (tid == 0) s_again = 0;

    // this lane's row in the first product
    const int my_row = rq * QR + lc;
    const int tok = my_row < have ? tok0 + lat_token(a, head0 + my_row) : -1;
    f32x16 o[ND][RT];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][t][i] = 0.0f;
    float m = kNegInf, l = 0.0f, pend = 0.0f;

    // Byte offset in the cache of the wave's group (the one it brings rows of
    // and has the scores of) in the next 64 tiles, a tile a lane
    constexpr long kMissing = -(1L << 32), kUnseen = -(2L << 32);
    const int* row = a.t.table + (long)max(0, s.slot) * a.t.ld;
    int at0 = b0;
    auto lookup = [&](int x) {
      const int key = group_key(2 * x + kq);
      if (x >= x_end || key > p_max || !(key + 16 > s.lo_min || key < a.first)) return kUnseen;
      const int i = kv_entry(a.t, key), e = row[i];
      return e >= 0 && e < a.t.n_pages ? e * a.c.sp + (key - i * a.t.ps) * a.c.st : kMissing;
    };
    long offs = lookup(b0 + lane);
    int state1 = 0, state2 = 0, state3 = 0;      // of tiles x + 1 and on: < 0 without a page

    // The place of tile x (ascending) and its state; load i of LOADS of it
    const char* src = a.c.k;
    uint32_t bytes = 0;
    auto place = [&](int x) __attribute__((always_inline)) {
      if (x - at0 >= 64) {
        at0 = x;
        offs = lookup(x + lane);
      }
      const uint32_t lo32 = __builtin_amdgcn_readlane((int)offs, x - at0);
      const int hi32 = __builtin_amdgcn_readlane((int)(offs >> 32), x - at0);
      const long off = (long)(((uint64_t)(uint32_t)max(hi32, 0) << 32) | lo32);
      src = a.c.k + (hi32 < 0 ? 0L : off) + l_from * a.c.st;
      bytes = hi32 < 0 ? 0 : 0x7FFFFFFF;         // (without a place: nothing, and zeros in LDS)
      if (hi32 == (int)(kMissing >> 32) && lane == 0) atomicOr(a.err, kErrPage);
      return hi32;
    };
    auto load = [&](int x, int i) __attribute__((always_inline)) {
      const uint32_t to = lds_of(s_t) + ((x - b0) & 3) * TB;
      if (i < NLD)
        load_to_lds(src, bytes,
                    here(l_row + (l_unit ^ 16 * swz(i * RPL)) + i * RPL * (int)a.c.st),
                    to + (RPW * w + i * RPL) * RB);
      else if (lane < RPW * URR)
        load_to_lds(src, bytes, l_rope, to + 32 * RB + RPW * w * RRB);
    };
    auto issue = [&](int x) __attribute__((always_inline)) {
      const int state = place(x);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) load(x, i);
      return state;
    };
    auto arrived = [&](auto left) __attribute__((always_inline)) {              // all but the newest `left` tiles
      wait_counts<decltype(left)::value * LOADS, 15>();
    };

    // The queries, loaded as rows into LDS, turned as keys are in a 16-bit tile
    auto q_swz = [](int r) { return (r & 3) << 2 | (r >> 2 & 3); };
    char* const qa = F8 ? s_q : s_t[2];
    auto issue_q = [&] {
      const int lane = here(tid & 63);
      constexpr int QU = DC / 8, QL = 64 / QU, QW = R / NW;        // units, rows of a load, of a wave
      auto from = [&](int r, int un) {
        const int g = head0 + min(r, have - 1), tk = lat_token(a, g);
        return a.q + (long)(s.q0 + tok0 + tk) * a.q_row + (g - tk * H) * a.q_head + 16 * un;
      };
#pragma unroll
      for (int i = 0; i < QW / QL; ++i) {
        const int r = w * QW + i * QL + lane / QU;
        load_lanes_to_lds(from(r, lane % QU ^ q_swz(r)), lds_of(qa) + (w * QW + i * QL) * DC * 2);
      }
      const int r = w * QW + lane / 8;
      static_assert(QW == 8, "a load for a wave's rotary rows");
      load_lanes_to_lds(from(r, QU + (lane % 8 ^ (r >> 1 & 7))),
                        lds_of(qa) + R * DC * 2 + w * QW * 128);
    };
    u32x4 q[2][MW * KS];                         // of 32 rows, half of the depth
    auto take_q = [&] {
      const int ln = here(lane), lc = ln & 15, g4 = ln >> 4;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < MW * KS; ++i) {
          // values from 32 c + 8 g4 on; e4m3: as a unit of 16 keeps them for two steps
          const int r = (rq & 2) * QR + t * QR + lc, c = min(dq * MW * KS + i, NK - 1);
          const int un = F8 ? 8 * (c >> 1) + 2 * g4 + (c & 1) : 4 * c + g4;
          q[t][i] = *(const u32x4*)(qa + (32 * c < DC
                                              ? r * DC * 2 + 16 * (un ^ q_swz(r))
                                              : R * DC * 2 + r * 128 +
                                                    16 * ((un & 7) ^ (r >> 1 & 7))));
        }
    };

    // Operands of S^T = K Q^T: this wave's 16 keys. Read i is step i of its half, or
    // for e4m3 steps 2 i and 2 i + 1.
    auto read_k = [&](const char* kt, int i) __attribute__((always_inline)) {
      constexpr int first = MK - MW - MR;
      return *(const u32x4*)(kt + (i >= first && i < first + MR ? kr_at[i - first]
                                                                : k_at[i & 3] + 256 * (i >> 2)));
    };
    auto use_k = [&](f32x4 (&sv)[2], const u32x4& raw, int i) __attribute__((always_inline)) {
      if (MK % 2 && i == MW - 1 && dq) return;   // the second half is shorter
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        u32x4 ka = raw;
        if constexpr (F8)
          ka = u32x4{from_e4m3<BF, false>(raw[2 * e]), from_e4m3<BF, true>(raw[2 * e]),
                     from_e4m3<BF, false>(raw[2 * e + 1]), from_e4m3<BF, true>(raw[2 * e + 1])};
#pragma unroll
        for (int t = 0; t < 2; ++t)
          sv[t] = mfma16<BF>(ka, q[t][KS * i + e], i + e == 0 ? f32x4{0, 0, 0, 0} : sv[t]);
      }
    };
    // this wave's scores from both halves, with a barrier between give and take
    auto give = [&](const f32x4 (&sv)[2]) {
      *(f32x4*)(s_x.half[w ^ 1] + 16 * lane) = dq ? sv[0] : sv[1];
    };
    auto take = [&](const f32x4 (&sv)[2]) {
      return (dq ? sv[1] : sv[0]) + *(const f32x4*)(s_x.half[w] + 16 * lane);
    };
    // masks the scores of a tile that is not whole
    auto mask = [&](f32x4& sv, int x, int state) __attribute__((always_inline)) {
      const int key = group_key(2 * x + kq) + 4 * g4;
      uint32_t bits = 0;                         // the lane's four keys among the drafted tokens
      int end = s.C + tok + 1, pos = end - 1;
      if (tree) {
        end = s.C;
        pos = end;
        if (masked && tok >= 0) {
          pos += s_tree.depth(tok - tok0);
          bits = (uint32_t)s_tree.bits(tok - tok0, key - s.C) & 15;
        }
      }
      const int lo = a.window ? pos - a.window + 1 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = key + i;
        const bool ok = ((j < end) & ((j >= lo) | (j < a.first))) | (bits >> i & 1);
        sv[i] = ok & (tok >= 0) & (state >= 0) ? sv[i] : kNegInf;
      }
    };
    auto top_of = [&](const f32x4& sv) {
      return max_across_rows(fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3])));
    };
    // P of tile x from the scores and the row's maximum m, and its sum
    auto probs = [&](const f32x4& sv, int x) __attribute__((always_inline)) {
      const float neg = m == kNegInf ? 0.0f : pre_lift<BF>(m) - m;
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = exp2_fast(sv[i] + neg);
      pend = (p[0] + p[1]) + (p[2] + p[3]);
      *(u32x2*)(s_p + p_to) = u32x2{pack16<BF>(p[0], p[1]), pack16<BF>(p[2], p[3])};
    };
    // lets m, l and O follow the maximum, after a barrier behind soft(); ends in
    // a barrier
    auto follow = [&](const f32x4& sv, int x) __attribute__((always_inline)) {
      const int r = rq * QR + lc;
      const float top = top_of(sv);
      if (g4 == 0) s_x.row.top[kq][r] = top;
      lds_barrier();
      if (tid < R) {
        const float old = s_m[tid], now = fmaxf(old, fmaxf(s_x.row.top[0][tid], s_x.row.top[1][tid]));
        float df = old - (now == kNegInf ? 0.0f : now);
        if constexpr (!BF) df += pre_lift<BF>(now) - pre_lift<BF>(old);
        s_x.row.f[tid] = exp2_fast(df);
        s_m[tid] = now;
      }
      lds_barrier();
      m = s_m[r];
      l *= s_x.row.f[r];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float f = s_x.row.f[32 * t + l31];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][t][i] *= f;
      }
      probs(sv, x);
      lds_barrier();
    };
    // Operand of O^T += V^T P^T: 16 keys (ks) of 32 values
    auto read_v = [&](const char* vt, int ks, int d) __attribute__((always_inline)) {
      const char* p = vt + 16 * ks * RB;
      u32x4 va = {0, 0, 0, 0};
      if constexpr (F8) {
        const auto y = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(p + v_at[d][0]));
        va[0] = y[0];
        va[1] = y[1];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(p + v_at[d][h]));
          const u32x2 z = __builtin_bit_cast(u32x2, y);
          va[2 * h] = z[0];
          va[2 * h + 1] = z[1];
        }
      }
      return va;
    };
    // S^T of tile x if QK, the product of the tile before with its P if PV. One
    // operand after another, each with the read of the one that is due kAhead
    // later and a share of the rest: beside(i) behind the first product's operand
    // i, the steps of soft() behind those of the second, with the barrier that P's
    // room and the scores' halves ask for. The order is kept as written. False if
    // beside() was: nothing has changed, and there was no barrier.
    constexpr int kAhead = 4, kSoft = 3;
    auto products = [&](auto qk, auto pv, f32x4& sum, int x, auto beside, auto soft)
        __attribute__((always_inline)) {
      constexpr int MQ = decltype(qk)::value ? MW : 0, MV = decltype(pv)::value ? 2 * ND : 0;
      const char *kt = s_t[(x - b0) & 3], *vt = s_t[(x - b0 - 1) & 3];
      u32x4 op[MQ + MV], pb[2][RT];
      f32x4 sn[2];
      auto read = [&](int i) __attribute__((always_inline)) {
        op[i] = i < MQ ? read_k(kt, i) : read_v(vt, (i - MQ) / ND, (i - MQ) % ND);
      };
#pragma unroll
      for (int i = 0; i < kAhead && i < MQ + MV; ++i) read(i);
#pragma unroll
      for (int i = 0; i < MQ + MV; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i + kAhead < MQ + MV) read(i + kAhead);
        if (MV && i == (MQ ? MQ - 2 : 0)) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              pb[ks][t] = *(const u32x4*)(s_p + ((p_from + 32 * 64 * t) ^ (32 * ks)));
        }
        if (i < MQ) {
          use_k(sn, op[i], i);
          if (!beside(i)) return false;
          if (i == MQ - 1) give(sn);
        } else {
          const int ks = (i - MQ) / ND, d = (i - MQ) % ND;
          u32x4 va = op[i];
          if constexpr (F8)
            va = u32x4{from_e4m3<BF, false>(op[i][0]), from_e4m3<BF, true>(op[i][0]),
                       from_e4m3<BF, false>(op[i][1]), from_e4m3<BF, true>(op[i][1])};
#pragma unroll
          for (int t = 0; t < RT; ++t) o[d][t] = mfma32<BF>(va, pb[ks][t], o[d][t]);
          if (MQ && i == MQ) {
            lds_barrier();
            sum = take(sn);
          }
          if (MQ && i > MQ) soft(i - MQ - 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (MQ && !MV) {
        lds_barrier();
        sum = take(sn);
      }
      if (MQ) {
#pragma unroll
        for (int i = MV ? MV - 1 : 0; i < kSoft; ++i) soft(i);
      }
      return true;
    };
    // P of tile x from its scores and the rows' maxima of before, in three steps; if
    // one has grown too much that is told, and follow() does it again
    auto soft = [&](f32x4& sv, int x, bool tell, int i) __attribute__((always_inline)) {
      if (i == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sv[e] *= sc;
      }
      if (i == 1) {
        const bool more = top_of(sv) > m + kDefer<BF>;
        if (tell & __any(more) && lane == 0) s_tell[x & 7] = x;
      }
      if (i == 2) probs(sv, x);
    };
    // the last two of them again for a tile that is not whole
    auto soft_masked = [&](f32x4& sv, int x, int state) __attribute__((always_inline)) {
      mask(sv, x, state);
      soft(sv, x, true, 1);
      soft(sv, x, true, 2);
    };

    // Values that are not finite are taken out of a tile that not every row sees.
    // Those that do see one have a score that is not finite either: NaN or
    // infinity, and so have the row's sum and all of its result, or -infinity,
    // and the key does not enter. A tile that every row sees is multiplied as it is:
    // if what comes of it is not finite, the piece is done again with all tiles
    // taken for such as are not whole (codes are finite or NaN: there it would be
    // the same). Looking for scores of -infinity in each tile instead took 1 % of
    // the time, with vectors of 256 3.
    auto bad16 = [](uint32_t x) {
      constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
      return (x & e) == e;
    };
    auto clean = [&](char* vt) {
      for (int i = lane; i < RPW * UPR; i += 64) {
        u32x4* at = (u32x4*)(vt + RPW * w * RB + 16 * i);
        const u32x4 y = *at;
        u32x4 z = y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F8) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if ((y[e] >> (8 * b) & 0x7F) == 0x7F) z[e] &= ~(0xFFu << (8 * b));
          } else {
            if (bad16(y[e])) z[e] &= 0xFFFF0000u;
            if (bad16(y[e] >> 16)) z[e] &= 0x0000FFFFu;
          }
        }
        if (((y[0] ^ z[0]) | (y[1] ^ z[1])) | ((y[2] ^ z[2]) | (y[3] ^ z[3]))) *at = z;
      }
      lds_barrier();
    };

    f32x4 sa = {0, 0, 0, 0};                     // scores of tile x
    int x = b0;
    if (b0 < x_end) {
      int st = issue(b0);
      issue_q();
      state1 = issue(b0 + 1);
      arrived(std::integral_constant<int, 1>{});
      lds_barrier();                             // the first tile, the queries, parents, s_tell
      take_q();
      if (masked) s_tree.build(tok0, min(s.m, tok1 + 1), s.C, a.window, a.first, a.err);
      lds_barrier();                             // all queries taken
      state2 = issue(b0 + 2);
      state3 = place(b0 + 3);
      bool plain = whole(x) && st >= 0;
      products(std::true_type{}, std::false_type{}, sa, x, [](int) { return true; },
               [&](int i) { soft(sa, x, plain, i); });
      if (!plain) soft_masked(sa, x, st);
      // Tile x: its P stands in LDS, computed with the maxima of before unless told
      // otherwise. A step computes the scores and P of tile x + 1 and the product
      // of tile x, and starts the loads of tile x + 3 into the room of tile x - 1
      // (behind the last tile, loads of nothing, so that the count stays the same).
      // (A loop of its own, left where something rare is to be done about tile x
      // first: with that in it, O would be copied from registers to registers in
      // each step.)
      auto told_of = [&](int x) {
        return *(const volatile __attribute__((address_space(3))) int*)
            (const __attribute__((address_space(3))) int*)&s_tell[x & 7];
      };
      int ready = b0 - 1;                        // the tile that it has been done for
      while (true) {
        while (true) {
          if (ready != x) {
            arrived(std::integral_constant<int, 1>{});
            lds_barrier();
          }
          if (x + 1 >= x_end || (ready != x && !whole(x))) break;
          const int tell = told_of(x);
          f32x4 sn = {0, 0, 0, 0};
          int next = 0;
          plain = whole(x + 1) && state1 >= 0;
          // what has been told is looked at behind operand kTold of the first product,
          // the loads are spread over those that follow
          constexpr int kTold = MW / 3, PER = (LOADS + MW - kTold - 2) / (MW - kTold - 1);
          const bool went = products(
              std::true_type{}, std::true_type{}, sn, x + 1,
              [&](int i) __attribute__((always_inline)) {
                if (i == kTold) {
                  if (ready != x && __builtin_amdgcn_readfirstlane(tell) == x)
                    return false;
                  l += pend;
                }
#pragma unroll
                for (int k = 0; k < PER; ++k)
                  if (i > kTold && (i - kTold - 1) * PER + k < LOADS)
                    load(x + 3, (i - kTold - 1) * PER + k);
                return true;
              },
              [&](int i) __attribute__((always_inline)) {
                soft(sn, x + 1, plain, i);
                if (i == 2) next = place(x + 4);
              });
          if (!went) break;
          ++x;
          if (!plain) soft_masked(sn, x, state1);
          state1 = state2;
          state2 = state3;
          state3 = next;
          sa = sn;
        }
        if (ready != x) {
          if (__builtin_amdgcn_readfirstlane(told_of(x)) == x) follow(sa, x);
          if (!whole(x)) clean(s_t[(x - b0) & 3]);
          ready = x;
        }
        if (x + 1 >= x_end) break;
      }
      l += pend;
      products(std::false_type{}, std::true_type{}, sa, x + 1, [](int) { return true; },
               [](int) {});
      arrived(std::integral_constant<int, 0>{});
    }

    // sums of the rows
    l = xor32_reduce(xor16_reduce(l, OpSum{}), OpSum{});
    if (g4 == 0) s_x.row.l[kq][rq * QR + lc] = l;
    if constexpr (!F8) {
      // such a value makes its place NaN in all rows, whatever their scores: those of
      // the first 32 show it
      float z[4] = {};
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i & 3] = __builtin_fmaf(o[d][0][i], 0.0f, z[i & 3]);
      if (__any((z[0] + z[1]) + (z[2] + z[3]) != 0.0f)) s_again = 1;
    }
    lds_barrier();
    if constexpr (!F8) {
      careful = !careful && __builtin_amdgcn_readfirstlane(s_again);
      if (careful) {
        u -= v1 - v0;
        continue;
      }
    }
    const bool all = b0 == 0 && b1 == s.nb;
    if (all) {
      // turned round through LDS, 64-byte runs of a wave's rows
      constexpr int WB = ND * 64;                // bytes of a row that a wave has
      char* const mine = s_t[0] + w * R * WB;
      static_assert(NW * R * WB <= 4 * TB, "the rows fit the tiles");
      constexpr int WU = WB / 16;                // units of it
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int r = here(32 * t + l31), half = here(lane) >> 5;
        const float lr = s_x.row.l[0][r] + s_x.row.l[1][r];
        const float inv = (F8 ? a.c.ks[0] : 1.0f) / lr;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const u32x2 y = {pack16<BF>(of_sum(o[d][t][i], inv, lr), of_sum(o[d][t][i + 1], inv, lr)),
                             pack16<BF>(of_sum(o[d][t][i + 2], inv, lr),
                                        of_sum(o[d][t][i + 3], inv, lr))};
            *(u32x2*)(mine + r * WB + 16 * ((4 * d + (i >> 2)) ^ (r & (WU - 1))) + 8 * half) = y;
          }
      }
#pragma unroll
      for (int i = 0; i < R * WU / 64; ++i) {
        const int ln = here(lane), r = i * (64 / WU) + ln / WU, un = ln % WU;
        const u32x4 y = *(const u32x4*)(mine + r * WB + 16 * (un ^ (r & (WU - 1))));
        if (r < have) {
          const int g = head0 + r, tk = lat_token(a, g);
          *(u32x4*)(a.out + (long)(s.q0 + tok0 + tk) * a.o_row + (g - tk * H) * a.o_head +
                    w * WB + 16 * un) = y;
        }
      }
      if (a.lse && tid < have) {
        const float lr = s_x.row.l[0][tid] + s_x.row.l[1][tid];
        a.lse[(long)s.q0 * H + r0 + tid] =
            (s_m[tid] + (__builtin_amdgcn_logf(lr) - pre_lift<BF>(s_m[tid]))) * kLn2;
      }
    } else {
      // this workgroup's part: the tile that it goes on with, or leaves open
      float* const part = a.part + (long)(2 * wg + (b0 == 0)) * lat_part_floats(DC);
      const int ln = here(lane);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (32 * t + (ln & 31) < have)
              *(f32x4*)(part + 2 * R + ((((w * ND + d) * RT + t) * 4 + (i >> 2)) * 64 + ln) * 4) =
                  f32x4{o[d][t][i], o[d][t][i + 1], o[d][t][i + 2], o[d][t][i + 3]};
      if (tid < R) {
        part[tid] = s_m[tid] - pre_lift<BF>(s_m[tid]);
        part[R + tid] = s_x.row.l[0][tid] + s_x.row.l[1][tid];
      }
      if (b0 == 0 && tid == 0) {
        // the workgroup of the tile's last unit: the largest v that starts before its end
        const long end = s_pref[seq] + (long)(tile + 1) * units;
        int v = min((int)W - 1, (int)((double)end * (double)W / (double)U));
        while (start_of(v) >= end) --v;
        while (v + 1 < (int)W && start_of(v + 1) < end) ++v;
        meta[0] = s.q0;
        meta[1] = rows;
        meta[2] = r0;
        meta[3] = v - wg + 1;
      }
    }
  }
}

// Joins the parts of the tile that workgroup wg of the kernel above left open, in
// their order. A run is 32 values of 32 rows, 16 values a lane. A wave has one to
// itself, or, SPREAD, for few tiles of many parts, a workgroup has, every kLatJoin-th
// part to each wave. Bound by the parts' bytes for batches (50 MB in 13 us), by
// latency else.
constexpr int kLatJoin = 8;
template <bool BF, bool F8, int DC, bool SPREAD>
__device__ __forceinline__ void latent_join(const AttnArgs& a, int wg) {
  constexpr int R = kLatRows, RT = R / 32, NW = SPREAD ? kLatJoin : 1;
  __shared__ f32x4 s_o[NW][4][64];
  __shared__ float s_ml[NW][2][32];
  const i32x4 meta = *(const i32x4*)(a.meta + 4 * wg);     // q0, rows, first row, parts
  const int cnt = meta[3];
  const int lane = lane_id(), w = threadIdx.x >> 6, l31 = lane & 31, half = lane >> 5;
  const int run = SPREAD ? (int)blockIdx.y : 4 * (int)blockIdx.y + w;
  const int t = run % RT, g = meta[2] + 32 * t + l31;      // of the sequence's rows
  if (cnt == 0 || meta[2] + 32 * t >= meta[1]) return;
  const bool there = g < meta[1];
  const long pf = lat_part_floats(DC);
  // part k: of the workgroup that opened the tile, then those that went on
  auto part = [&](int k) { return a.part + (long)(2 * (wg + k) + (k == 0)) * pf; };
  float m = kNegInf, l = 0.0f;
  f32x4 o[4] = {};
  auto scale = [&](float f) {
    l *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= f;
  };
  auto add = [&](float f, float pl, const f32x4 (&y)[4]) {
    l += f * pl;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] += f * y[i][e];
  };
  const int step = SPREAD ? NW : 1;
  for (int k0 = SPREAD ? w : 0; k0 < cnt; k0 += 4 * step) {
    f32x4 y[4][4];
    float pm[4], pl[4];
    if (there) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * step;
        const float* p = part(k < cnt ? k : k0);
        pm[j] = k < cnt ? p[32 * t + l31] : kNegInf;
        pl[j] = p[R + 32 * t + l31];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[j][i] = *(const f32x4*)(p + 2 * R + ((run * 4 + i) * 64 + lane) * 4);
      }
      float mn = m;
#pragma unroll
      for (int j = 0; j < 4; ++j) mn = fmaxf(mn, pm[j]);
      const float mu = mn == kNegInf ? 0.0f : mn;
      scale(exp2_fast(m - mu));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + j * step < cnt) add(exp2_fast(pm[j] - mu), pl[j], y[j]);
      m = mn;
    }
  }
  if constexpr (SPREAD) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[w][i][lane] = o[i];
    if (half == 0) {
      s_ml[w][0][l31] = m;
      s_ml[w][1][l31] = l;
    }
    __syncthreads();
    if (w) return;
    const int n = min(cnt, NW);
    float mn = m;
    for (int k = 1; k < n; ++k) mn = fmaxf(mn, s_ml[k][0][l31]);
    const float mu = mn == kNegInf ? 0.0f : mn;
    scale(exp2_fast(m - mu));
    m = mn;
    for (int k = 1; k < n; ++k) {
      const f32x4 y[4] = {s_o[k][0][lane], s_o[k][1][lane], s_o[k][2][lane], s_o[k][3][lane]};
      add(exp2_fast(s_ml[k][0][l31] - mu), s_ml[k][1][l31], y);
    }
  }
  if (!there) return;
  const int H = a.hq, tk = g / H, dt = run / RT;
  const float inv = (F8 ? a.c.ks[0] : 1.0f) / l;
  char* dst = a.out + (long)(meta[0] + tk) * a.o_row + (g - tk * H) * a.o_head + 64 * dt + 8 * half;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *(u32x2*)(dst + 16 * i) = u32x2{pack16<BF>(of_sum(o[i][0], inv, l), of_sum(o[i][1], inv, l)),
                                    pack16<BF>(of_sum(o[i][2], inv, l), of_sum(o[i][3], inv, l))};
  if (a.lse && dt == 0 && half == 0)
    a.lse[(long)meta[0] * H + g] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Tiles left open: one for each workgroup of the first launch, or, SPREAD, the few
// that there are shared out to blockIdx.x. (Of a workgroup for each of 256 that might
// have left one, times 32 runs, the launch alone took 20 us: one token of 128 heads
// over 16,812 keys, 45 us of joining then.)
template <bool BF, bool F8, int DC, bool SPREAD>
__global__ __launch_bounds__(SPREAD ? 64 * kLatJoin : 256) void latent_join_kernel(AttnArgs a) {
  if constexpr (!SPREAD) {
    latent_join<BF, F8, DC, SPREAD>(a, blockIdx.x);
  } else {
    constexpr int W = kLatGrid / 64;
    static_assert(kLatJoin >= W, "a thread for each workgroup of the first launch");
    __shared__ uint64_t s_open[W];
    const int tid = threadIdx.x;
    if (tid < kLatGrid) {
      const uint64_t open = __ballot(tid < a.teams && a.meta[4 * tid + 3] != 0);
      if (tid % 64 == 0) s_open[tid / 64] = open;
    }
    __syncthreads();
    int i = 0;
    for (int k = 0; k < W; ++k)
      for (uint64_t open = s_open[k]; open; open &= open - 1, ++i)
        if (i % (int)gridDim.x == (int)blockIdx.x) {
          latent_join<BF, F8, DC, SPREAD>(a, 64 * k + __builtin_ctzll(open));
          __syncthreads();                       // its LDS is free again
        }
  }
}

template <bool BF, bool F8, int DC>
hipError_t run_latent(const AttnArgs& a, int grid, hipStream_t s) {
  attn_latent_kernel<BF, F8, DC><<<grid, 64 * kLatWaves, 0, s>>>(a);
  constexpr unsigned runs = DC / 32 * (kLatRows / 32);
  if (a.spread)
    latent_join_kernel<BF, F8, DC, true><<<dim3(a.spread, runs), 64 * kLatJoin, 0, s>>>(a);
  else
    latent_join_kernel<BF, F8, DC, false><<<dim3(grid, runs / 4), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int DC>
hipError_t run_latent_d(const AttnArgs& a, int fmt, int grid, hipStream_t s) {
  const bool f8 = a.c.fmt == KV_E4M3;
  if (fmt == KV_BF16)
    return f8 ? run_latent<true, true, DC>(a, grid, s) : run_latent<true, false, DC>(a, grid, s);
  return f8 ? run_latent<false, true, DC>(a, grid, s) : run_latent<false, false, DC>(a, grid, s);
}

}  // namespace
}  // namespace moe
