// Attention over a paged cache of latent vectors: keys are a token's latent
// vector and rotary key, values its latent vector, all query heads share them.
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
  int tiles;                   // of R rows
  int lo_min;
};

__device__ __forceinline__ int lat_cu(const AttnArgs& a, int i) {
  if (!a.cu) return i;
  const int c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? (int)a.T : c);
}

template <int R>
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
  s.tiles = (int)(((long)s.m * a.hq + R - 1) / R);
  return s;
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

template <bool BF, bool F8, int DC, int R>
__global__ __launch_bounds__(256, 1) void attn_latent_kernel(AttnArgs a) {
  constexpr int ES = F8 ? 1 : 2;
  constexpr int RB = DC * ES, UPR = RB / 16;              // bytes and units of a latent row
  constexpr int RRB = kLatRope * ES, URR = RRB / 16;      // of a rotary one
  constexpr int TB = 32 * (RB + RRB);                     // a tile of 32 keys
  constexpr int RPL = 64 / UPR, NLD = 8 / RPL;            // rows of a load; loads of 8 rows
  constexpr int NK = (DC + kLatRope) / 32;                // steps of the first product
  constexpr int RQ = R / 32;                              // a wave's 16-row tiles in it
  constexpr int RT = R / 32;                              // 32-row tiles in the second
  constexpr int ND = DC / 128;                            // a wave's 32-row tiles of O^T
  constexpr int LOADS = NLD + 1;

  __shared__ __align__(16) char s_t0[TB], s_t1[TB], s_t2[TB], s_t3[TB];
  __shared__ __align__(16) char s_p0[R * 64], s_p1[R * 64];
  __shared__ long s_pref[kLatSeqs + 1];
  __shared__ TreeRows<R> s_tree;
  __shared__ float s_m[R], s_f[R], s_lm[2][R], s_l[2][R];
  __shared__ long s_scan[4];
  __shared__ int s_flag[2];                      // the tile whose P is to be done again
  __shared__ int s_bad;                          // values that are not finite were taken out
  __shared__ int s_gone[4];                      // tile x with a group that has no page, by x % 4

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kq = w >> 1, rq = w & 1;
  const int lc = lane & 15, g4 = lane >> 4, half = lane >> 5, l31 = lane & 31;
  const int H = a.hq;

  // prefix sums of the sequences' units
  {
    long v = 0;
    if (tid < a.n) {
      const LatSeq s = lat_seq<R>(a, tid);
      v = (long)s.tiles * s.nb;
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
  // workgroups next to each other read the same keys: they go to one XCD
  const int wg = W > 128 && gridDim.x % 8 == 0
                     ? (int)(blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8)
                     : (int)blockIdx.x;
  int* const meta = a.meta + 4 * wg;
  if (tid == 0) meta[2] = 0;
  if (wg >= W) return;
  long u = wg * U / W;
  const long u_end = (wg + 1) * U / W;
  int seq = 0;
  for (int hi = a.n - 1; seq < hi;) {
    const int mid = (seq + hi + 1) >> 1;
    if (s_pref[mid] <= u) seq = mid; else hi = mid - 1;
  }
  seq = __builtin_amdgcn_readfirstlane(seq);

  const float sc = F8 ? a.scale * a.c.ks[0] : a.scale;

  // Swizzles: the 16-byte units of a row lie turned by its number, so that the
  // reads of 8 rows' same unit (K), and those of four rows' next two units, or
  // eight rows' one (V, transposed), fall into different banks.
  auto swz = [](int r) { return F8 ? r & 7 : (r & 3) << 1 | (r >> 2 & 1); };
  auto swz_r = [&](int r) { return F8 ? r >> 1 & 3 : swz(r); };
  const int k_row = 16 * kq + lc;
  int k_at = k_row * RB + 16 * (g4 ^ swz(k_row));
  int kr_at = 32 * RB + k_row * RRB + 16 * (g4 ^ swz_r(k_row));
  const int v_row = 8 * half + (F8 ? lc >> 1 : lc >> 2);
  const int v_u = F8 ? g4 & 1 : 2 * (g4 & 1) + (lc >> 1 & 1);
  int v_at = (v_row * RB + 16 * (v_u ^ swz(v_row)) + 8 * (lc & 1)) ^ (w * ND * 32 * ES);
  auto p_swz = [](int r) { return r >> 1 & 3; };
  const int p_to = (rq * (R / 2) + lc) * 64 + 16 * ((2 * kq + (g4 >> 1)) ^ p_swz(lc)) + 8 * (g4 & 1);
  const int p_from = l31 * 64 + 16 * (half ^ p_swz(l31));

  while (u < u_end) {
    while (s_pref[seq + 1] <= u) ++seq;
    const LatSeq s = lat_seq<R>(a, seq);
    const long rel = u - s_pref[seq];
    const int tile = (int)(rel / s.nb), b0 = (int)(rel - (long)tile * s.nb);
    const int b1 = (int)min((long)s.nb, b0 + (u_end - u));
    const int rows = s.m * H, r0 = tile * R;
    const int tok0 = r0 / H, tok1 = (min(rows, r0 + R) - 1) / H;
    const bool tree = a.parent != nullptr;
    const int p_min = tree ? max(0, s.C) - 1 : s.C + tok0;
    const int p_max = tree ? s.L - 1 : s.C + tok1;
    const int lo_max = a.window ? max(0, p_max - a.window + 1) : 0;
    auto group_key = [&](int i) { return 16 * (i < s.ng1 ? i : s.b2 + i - s.ng1); };
    const int end_g = s.ng1 + max(0, (max(0, p_max + 1) + 15) / 16 - s.b2);
    const int x_end = __builtin_amdgcn_readfirstlane(min(b1, (end_g + 1) / 2));
    const int whole0 = (s.ng1 + max(0, (lo_max + 15) / 16 - s.b2) + 1) / 2;
    const int whole1 = (s.ng1 - s.b2 + max(0, p_min + 1) / 16) / 2;
    auto whole = [&](int x) { return x >= whole0 && x < whole1; };
    const bool masked = tree && (b0 < whole0 || x_end > whole1);

    __syncthreads();                             // of the piece before
    if (masked) s_tree.fetch(a.parent + s.q0, s.m);
    if (tid < R) s_m[tid] = kNegInf;
    if (tid < 2) s_flag[tid] = -1;
    if (tid < 4) s_gone[tid] = -1;
    if (tid == 0) s_bad = 0;

    // this lane's rows in the first product
    int tok[RQ];
    u32x4 q[RQ][NK];
#pragma unroll
    for (int t = 0; t < RQ; ++t) {
      const int r = r0 + rq * (R / 2) + 16 * t + lc;
      tok[t] = r < rows ? r / H : -1;
    }
    auto read_q = [&](int t, auto put) __attribute__((always_inline)) {
      const int r = here(r0 + rq * (R / 2) + 16 * t + lc);
      const char* src = a.q + (long)(s.q0 + max(0, tok[t])) * a.q_row +
                        (r < rows ? r - tok[t] * H : 0) * a.q_head;
#pragma unroll
      for (int c = 0; c < NK; ++c) {
        const int d = F8 ? 64 * (c >> 1) + 16 * g4 + 8 * (c & 1) : 32 * c + 8 * g4;
        put(c, *(const u32x4*)(src + 2 * d));
      }
    };
#pragma unroll
    for (int t = 0; t < RQ; ++t) read_q(t, [&](int c, const u32x4& y) { q[t][c] = y; });
    f32x16 o[ND][RT];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][t][i] = 0.0f;
    float m[RQ], l[RQ], pend[RQ];
#pragma unroll
    for (int t = 0; t < RQ; ++t) {
      m[t] = kNegInf;
      l[t] = pend[t] = 0.0f;
    }

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
    int state1 = 0, state2 = 0;                  // of tiles x + 1, x + 2: < 0 without a page

    auto issue = [&](int x, char* to) __attribute__((always_inline)) {          // x ascending
      if (x - at0 >= 64) {
        at0 = x;
        offs = lookup(x + lane);
      }
      const uint32_t lo32 = __builtin_amdgcn_readlane((int)offs, x - at0);
      const int hi32 = __builtin_amdgcn_readlane((int)(offs >> 32), x - at0);
      const long off = (long)(((uint64_t)(uint32_t)max(hi32, 0) << 32) | lo32);
      const char* src = a.c.k + (hi32 < 0 ? 0L : off) + (w & 1) * 8 * a.c.st;
      if (hi32 == (int)(kMissing >> 32) && lane == 0) {
        atomicOr(a.err, kErrPage);
        s_gone[x & 3] = x;
      }
      const int ln = here(lane);
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int r = i * RPL + ln / UPR;
        const uint32_t f = (uint32_t)(ln / UPR) * (uint32_t)a.c.st + 16 * (ln % UPR ^ swz(r));
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(src + i * RPL * a.c.st + f),
            (__attribute__((address_space(3))) void*)(to + (8 * w + i * RPL) * RB), 16, 0, 0);
      }
      if (lane < 8 * URR) {
        const int r = ln / URR;
        const uint32_t f = (uint32_t)r * (uint32_t)a.c.st + RB + 16 * (ln % URR ^ swz_r(r));
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(src + f),
            (__attribute__((address_space(3))) void*)(to + 32 * RB + 8 * w * RRB), 16, 0, 0);
      }
      return hi32;
    };
    auto arrived = [&](auto left) __attribute__((always_inline)) {              // all but the newest `left` tiles
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(left)::value * LOADS) : "memory");
    };

    // Operands of S^T = K Q^T: this wave's 16 keys. Read i is step i, or for e4m3
    // steps 2 i and 2 i + 1.
    constexpr int KS = F8 ? 2 : 1, MK = NK / KS, ML = DC / 32 / KS;
    auto read_k = [&](const char* kt, int i) __attribute__((always_inline)) {
      return *(const u32x4*)(kt + (i < ML ? k_at ^ (64 * i) : kr_at ^ (64 * (i - ML))));
    };
    auto step_k = [&](const u32x4& raw, int e) __attribute__((always_inline)) {
      if constexpr (F8)
        return u32x4{from_e4m3<BF, false>(raw[2 * e]), from_e4m3<BF, true>(raw[2 * e]),
                     from_e4m3<BF, false>(raw[2 * e + 1]), from_e4m3<BF, true>(raw[2 * e + 1])};
      else
        return raw;
    };
    auto use_k = [&](f32x4 (&sv)[RQ], const u32x4& raw, int i) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const u32x4 ka = step_k(raw, e);
#pragma unroll
        for (int t = 0; t < RQ; ++t)
          sv[t] = mfma16<BF>(ka, q[t][KS * i + e], i + e == 0 ? f32x4{0, 0, 0, 0} : sv[t]);
      }
    };
    // scales and masks them
    auto mask = [&](f32x4 (&sv)[RQ], int x, int state) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < RQ; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[t][i] *= sc;
      if (whole(x) && state >= 0) return;
      const int key = group_key(2 * x + kq) + 4 * g4;
#pragma unroll
      for (int t = 0; t < RQ; ++t) {
        uint32_t bits = 0;                       // the lane's four keys among the drafted tokens
        int end = s.C + tok[t] + 1, pos = end - 1;
        if (tree) {
          end = s.C;
          pos = end;
          if (masked && tok[t] >= 0) {
            pos += s_tree.depth(tok[t] - tok0);
            bits = (uint32_t)s_tree.bits(tok[t] - tok0, key - s.C) & 15;
          }
        }
        const int lo = a.window ? pos - a.window + 1 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = key + i;
          const bool ok = ((j < end) & ((j >= lo) | (j < a.first))) | (bits >> i & 1);
          sv[t][i] = ok & (tok[t] >= 0) & (state >= 0) ? sv[t][i] : kNegInf;
        }
      }
    };
    auto tops = [&](const f32x4& sv) {
      return max_across_rows(fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3])));
    };
    // P from the scores and the row's maximum m, and its sum
    auto probs = [&](const f32x4 (&sv)[RQ], char* to) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < RQ; ++t) {
        const float neg = m[t] == kNegInf ? 0.0f : pre_lift<BF>(m[t]) - m[t];
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = exp2_fast(sv[t][i] + neg);
        pend[t] = (p[0] + p[1]) + (p[2] + p[3]);
        *(u32x2*)(to + (p_to + 16 * 64 * t)) = u32x2{pack16<BF>(p[0], p[1]), pack16<BF>(p[2], p[3])};
      }
    };
    // lets m, l and O follow the maximum, after a barrier behind soft(); ends in
    // a barrier
    auto follow = [&](const f32x4 (&sv)[RQ], char* to) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < RQ; ++t) {
        const float top = tops(sv[t]);
        if (g4 == 0) s_lm[kq][rq * (R / 2) + 16 * t + lc] = top;
      }
      __syncthreads();
      if (tid < R) {
        const float old = s_m[tid], now = fmaxf(old, fmaxf(s_lm[0][tid], s_lm[1][tid]));
        float df = old - (now == kNegInf ? 0.0f : now);
        if constexpr (!BF) df += pre_lift<BF>(now) - pre_lift<BF>(old);
        s_f[tid] = exp2_fast(df);
        s_m[tid] = now;
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < RQ; ++t) {
        const int r = rq * (R / 2) + 16 * t + lc;
        m[t] = s_m[r];
        l[t] *= s_f[r];
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float f = s_f[32 * t + l31];
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][t][i] *= f;
      }
      probs(sv, to);
      __syncthreads();
    };
    // Operand of O^T += V^T P^T: 16 keys (ks) of 32 values
    auto read_v = [&](const char* vt, int ks, int d) __attribute__((always_inline)) {
      const char* p = vt + 16 * ks * RB;
      u32x4 va = {0, 0, 0, 0};
      if constexpr (F8) {
        const auto y = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(p + (v_at ^ (32 * d))));
        va[0] = y[0];
        va[1] = y[1];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(p + 4 * h * RB +
                                                         ((v_at ^ (64 * d)) ^ (16 * h))));
          const u32x2 z = __builtin_bit_cast(u32x2, y);
          va[2 * h] = z[0];
          va[2 * h + 1] = z[1];
        }
      }
      return va;
    };
    // S^T of tile x (sn, from kt) if QK, the product of the tile before (vt) with
    // its P (pt) if PV, and then P of tile x (to pn), computed with the rows'
    // maxima of before: if one has grown too much the flag is set, and follow()
    // does it again. One operand after another, each with the read of the one that
    // is due kAhead later and a share of the softmax; the order is kept as written.
    constexpr int kAhead = 4;
    auto products = [&](auto qk, auto pv, f32x4 (&sn)[RQ], int x, int state, const char* kt,
                        const char* vt, const char* pt, char* pn, int* flag)
        __attribute__((always_inline)) {
      constexpr int MQ = decltype(qk)::value ? MK : 0, MV = decltype(pv)::value ? 2 * ND : 0;
      asm volatile("" : "+v"(k_at), "+v"(kr_at), "+v"(v_at));   // not kept for every step
      u32x4 op[MQ + MV], pb[2][RT];
      auto read = [&](int i) __attribute__((always_inline)) {
        op[i] = i < MQ ? read_k(kt, i) : read_v(vt, (i - MQ) / ND, (i - MQ) % ND);
      };
      auto soft = [&](int i) __attribute__((always_inline)) {
        if (i == 0) mask(sn, x, state);
        if (i == 1) {
          bool more = false;
#pragma unroll
          for (int t = 0; t < RQ; ++t) more |= tops(sn[t]) > m[t] + kDefer<BF>;
          if (__any(more) && lane == 0) *flag = x;
        }
        if (i == 2) probs(sn, pn);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) read(i);
#pragma unroll
      for (int i = 0; i < MQ + MV; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if (i + kAhead < MQ + MV) read(i + kAhead);
        if (MV && i == (MQ ? MQ - 2 : 0)) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              pb[ks][t] = *(const u32x4*)(pt + ((p_from + 32 * 64 * t) ^ (32 * ks)));
        }
        if (i < MQ) {
          use_k(sn, op[i], i);
        } else {
          const int ks = (i - MQ) / ND, d = (i - MQ) % ND;
          u32x4 va = op[i];
          if constexpr (F8)
            va = u32x4{from_e4m3<BF, false>(op[i][0]), from_e4m3<BF, true>(op[i][0]),
                       from_e4m3<BF, false>(op[i][1]), from_e4m3<BF, true>(op[i][1])};
#pragma unroll
          for (int t = 0; t < RT; ++t) o[d][t] = mfma32<BF>(va, pb[ks][t], o[d][t]);
          if (MQ) soft(i - MQ);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (MQ && !MV) {
#pragma unroll
        for (int i = 0; i < 3; ++i) soft(i);
      }
    };

    // Values that are not finite, of a tile that not every row sees, are taken out
    // and brought back after the loop, for the rows that see them.
    auto bad16 = [](uint32_t x) {
      constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
      return (x & e) == e;
    };
    auto clean = [&](char* vt) {
      for (int i = here(lane); i < 8 * UPR; i += 64) {
        u32x4* at = (u32x4*)(vt + 8 * w * RB + 16 * i);
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
        if (((y[0] ^ z[0]) | (y[1] ^ z[1])) | ((y[2] ^ z[2]) | (y[3] ^ z[3]))) {
          *at = z;
          s_bad = 1;
        }
      }
      __syncthreads();
    };

    f32x4 sa[RQ];
    int x = b0;
    // Tile x: its P stands in px, computed with the maxima of before unless
    // flagged. Scores and P (pn) of tile x + 1, the product of tile x, and the
    // loads of tile x + 3 into the room of tile x - 1.
    auto settle = [&](char* vt, char* px, const int* flag) __attribute__((always_inline)) {
      const bool again = *(volatile const int*)flag == x;
      const bool gone = *(volatile const int*)&s_gone[x & 3] == x;
      if (__builtin_amdgcn_readfirstlane(again)) follow(sa, px);
#pragma unroll
      for (int t = 0; t < RQ; ++t) l[t] += pend[t];
      if (__builtin_amdgcn_readfirstlane(gone || !whole(x))) clean(vt);
    };
    auto step = [&](char* __restrict vt, char* __restrict kt, char* __restrict to,
                    char* __restrict px, char* __restrict pn, const int* fx, int* fn) __attribute__((always_inline)) {
      if (x + 2 < x_end) arrived(std::integral_constant<int, 1>{});
      else arrived(std::integral_constant<int, 0>{});
      __syncthreads();
      const int st = state1;
      state1 = state2;
      settle(vt, px, fx);
      if (x + 3 < x_end) state2 = issue(x + 3, to);
      products(std::true_type{}, std::true_type{}, sa, x + 1, st, kt, vt, px, pn, fn);
      ++x;
    };
    auto last = [&](char* vt, char* px, const int* fx) __attribute__((always_inline)) {
      __syncthreads();
      settle(vt, px, fx);
      products(std::false_type{}, std::true_type{}, sa, x, 0, nullptr, vt, px, nullptr, nullptr);
    };
    if (b0 < x_end) {
      const int st = issue(b0, s_t0);
      if (b0 + 1 < x_end) state1 = issue(b0 + 1, s_t1);
      if (b0 + 2 < x_end) state2 = issue(b0 + 2, s_t2);
      __syncthreads();                           // the parents; s_gone
      if (masked)
        s_tree.build(tok0, min(s.m, tok1 + 1), s.C, a.window, a.first, a.err);
      arrived(std::integral_constant<int, 0>{});
      __syncthreads();
      products(std::true_type{}, std::false_type{}, sa, b0, st, s_t0, nullptr, nullptr, s_p0,
               &s_flag[0]);
      char *vt = s_t0, *px = s_p0;
      const int* fx = &s_flag[0];
      while (x + 1 < x_end) {
        step(s_t0, s_t1, s_t3, s_p0, s_p1, &s_flag[0], &s_flag[1]);
        vt = s_t1, px = s_p1, fx = &s_flag[1];
        if (x + 1 >= x_end) break;
        step(s_t1, s_t2, s_t0, s_p1, s_p0, &s_flag[1], &s_flag[0]);
        vt = s_t2, px = s_p0, fx = &s_flag[0];
        if (x + 1 >= x_end) break;
        step(s_t2, s_t3, s_t1, s_p0, s_p1, &s_flag[0], &s_flag[1]);
        vt = s_t3, px = s_p1, fx = &s_flag[1];
        if (x + 1 >= x_end) break;
        step(s_t3, s_t0, s_t2, s_p1, s_p0, &s_flag[1], &s_flag[0]);
        vt = s_t0, px = s_p0, fx = &s_flag[0];
      }
      last(vt, px, fx);
    }

    // The values taken out: the scores and P of their tiles once more, and their
    // products with the probabilities that are not zero one by one.
    __syncthreads();
    if (s_bad) {
      auto to_f32 = [](uint32_t x) {
        return BF ? bf16_bits_to_f32(x) : (float)__builtin_bit_cast(_Float16, (uint16_t)x);
      };
      at0 = b0;
      offs = lookup(b0 + lane);
      for (int xx = b0; xx < x_end; ++xx) {
        if (whole(xx)) continue;                 // (of one without a page: nothing is seen)
        const int st = issue(xx, s_t0);
        arrived(std::integral_constant<int, 0>{});
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RQ; ++t) {
          sa[t] = f32x4{0, 0, 0, 0};
          read_q(t, [&](int c, const u32x4& y) {          // (not kept beside O here)
            sa[t] = mfma16<BF>(step_k(read_k(s_t0, c / KS), c % KS), y, sa[t]);
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        mask(sa, xx, st);
        probs(sa, s_p0);
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int r = here(32 * t + l31);
            const float p = to_f32(
                *(const uint16_t*)(s_p0 + r * 64 + 16 * ((k >> 3) ^ p_swz(r)) + 2 * (k & 7)));
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              const int h = here(4 * half), some = p != 0.0f ? -1 : 0;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int at = (32 * (w * ND + d) + 8 * (i >> 2) + h + (i & 3)) * ES;
                const char* v = s_t0 + k * RB + (16 * ((at >> 4) ^ swz(k)) + (at & 15));
                uint32_t y;
                if constexpr (F8) y = from_e4m3<BF, false>(*(const uint8_t*)v) & 0xFFFF;
                else y = *(const uint16_t*)v;
                constexpr int e = BF ? 0x7F80 : 0x7C00;
                const int fine = ((int)(y & e) - e) >> 31;           // all ones if finite
                o[d][t][i] += p * __uint_as_float(__float_as_uint(to_f32(y)) & ~fine & some);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
        __syncthreads();
      }
    }

    // sums of the rows
#pragma unroll
    for (int t = 0; t < RQ; ++t) {
      const float y = xor32_reduce(xor16_reduce(l[t], OpSum{}), OpSum{});
      if (g4 == 0) s_l[kq][rq * (R / 2) + 16 * t + lc] = y;
    }
    __syncthreads();
    const bool all = b0 == 0 && b1 == s.nb;
    if (all) {
      // turned round through LDS, 64-byte runs of a wave's rows
      constexpr int WB = ND * 64;                // bytes of a row that a wave has
      char* const mine = w == 0 ? s_t0 : w == 1 ? s_t1 : w == 2 ? s_t2 : s_t3;
      static_assert(R * WB <= TB, "a wave's rows fit a tile");
      constexpr int WU = WB / 16;                // units of it
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int r = here(32 * t + l31), half = here(lane) >> 5;
        const float lr = s_l[0][r] + s_l[1][r];
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
        const int ln = here(lane), r = i * (64 / WU) + ln / WU, un = ln % WU, g = r0 + r;
        const u32x4 y = *(const u32x4*)(mine + r * WB + 16 * (un ^ (r & (WU - 1))));
        if (g < rows) {
          const int tk = g / H;
          *(u32x4*)(a.out + (long)(s.q0 + tk) * a.o_row + (g - tk * H) * a.o_head + w * WB +
                    16 * un) = y;
        }
      }
      if (a.lse && tid < R && r0 + tid < rows) {
        const float lr = s_l[0][tid] + s_l[1][tid];
        a.lse[(long)s.q0 * H + r0 + tid] =
            (s_m[tid] + (__builtin_amdgcn_logf(lr) - pre_lift<BF>(s_m[tid]))) * kLn2;
      }
    } else {
      // this workgroup's part: the tile that it goes on with, or leaves open
      float* const part = a.part + (long)(2 * wg + (b0 == 0)) * lat_part_floats(DC, R);
      const int ln = here(lane);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *(f32x4*)(part + 2 * R + ((((w * ND + d) * RT + t) * 4 + (i >> 2)) * 64 + ln) * 4) =
                f32x4{o[d][t][i], o[d][t][i + 1], o[d][t][i + 2], o[d][t][i + 3]};
      if (tid < R) {
        part[tid] = s_m[tid] - pre_lift<BF>(s_m[tid]);
        part[R + tid] = s_l[0][tid] + s_l[1][tid];
      }
      if (b0 == 0 && tid == 0) {
        // the workgroup of the tile's last unit: the largest v with v U / W <= unit
        const long end = s_pref[seq] + (long)(tile + 1) * s.nb - 1;
        meta[0] = seq;
        meta[1] = tile;
        meta[2] = (int)(((end + 1) * W - 1) / U - wg) + 1;
      }
    }
    u += b1 - b0;
  }
}

// Joins the parts of the tile that workgroup blockIdx.x of the kernel above left
// open, in their order: four runs of 64 lanes' four values (blockIdx.y), four
// waves with every fourth part each.
template <bool BF, bool F8, int DC, int R>
__global__ __launch_bounds__(256) void latent_join_kernel(AttnArgs a) {
  constexpr int RT = R / 32;
  __shared__ f32x4 s_o[3][4][64];
  __shared__ float s_ml[3][2][32];
  const int wg = blockIdx.x;
  const int cnt = a.meta[4 * wg + 2];
  if (cnt == 0) return;
  const LatSeq s = lat_seq<R>(a, a.meta[4 * wg]);
  const int lane = lane_id(), w = threadIdx.x >> 6, l31 = lane & 31, half = lane >> 5;
  const int run = blockIdx.y, t = run % RT, dt = run / RT;   // rows 32 t.., values 32 dt..
  const long pf = lat_part_floats(DC, R);
  // part k: of the workgroup that opened the tile, then those that went on
  auto part = [&](int k) { return a.part + (long)(2 * (wg + k) + (k == 0)) * pf; };
  float mx = kNegInf, l = 0.0f;
  f32x4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
  for (int k0 = w; k0 < cnt; k0 += 16) {
    f32x4 y[4][4];
    float pm[4], pl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + 4 * j;
      const float* p = part(k < cnt ? k : k0);
      pm[j] = k < cnt ? p[32 * t + l31] : kNegInf;
      pl[j] = p[R + 32 * t + l31];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[j][i] = *(const f32x4*)(p + 2 * R + ((run * 4 + i) * 64 + lane) * 4);
    }
    float mn = mx;
#pragma unroll
    for (int j = 0; j < 4; ++j) mn = fmaxf(mn, pm[j]);
    const float mu = mn == kNegInf ? 0.0f : mn;
    const float f0 = exp2_fast(mx - mu);
    l *= f0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] *= f0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k0 + 4 * j >= cnt) continue;
      const float f = exp2_fast(pm[j] - mu);
      l += f * pl[j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] += f * y[j][i][e];
    }
    mx = mn;
  }
  if (w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[w - 1][i][lane] = acc[i];
    if (half == 0) {
      s_ml[w - 1][0][l31] = mx;
      s_ml[w - 1][1][l31] = l;
    }
  }
  __syncthreads();
  if (w) return;
  float mn = mx;
#pragma unroll
  for (int k = 0; k < 3; ++k) mn = fmaxf(mn, s_ml[k][0][l31]);
  const float mu = mn == kNegInf ? 0.0f : mn;
  const float f0 = exp2_fast(mx - mu);
  l *= f0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] *= f0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const float f = exp2_fast(s_ml[k][0][l31] - mu);
    l += f * s_ml[k][1][l31];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 y = s_o[k][i][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] += f * y[e];
    }
  }
  const int H = a.hq, g = a.meta[4 * wg + 1] * R + 32 * t + l31;
  if (g >= s.m * H) return;
  const int tk = g / H;
  const float inv = (F8 ? a.c.ks[0] : 1.0f) / l;
  char* dst = a.out + (long)(s.q0 + tk) * a.o_row + (g - tk * H) * a.o_head + 64 * dt + 8 * half;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *(u32x2*)(dst + 16 * i) = u32x2{pack16<BF>(of_sum(acc[i][0], inv, l), of_sum(acc[i][1], inv, l)),
                                    pack16<BF>(of_sum(acc[i][2], inv, l), of_sum(acc[i][3], inv, l))};
  if (a.lse && dt == 0 && half == 0)
    a.lse[(long)s.q0 * H + g] = (mn + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool BF, bool F8, int DC, int R>
hipError_t run_latent(const AttnArgs& a, int grid, hipStream_t s) {
  attn_latent_kernel<BF, F8, DC, R><<<grid, 256, 0, s>>>(a);
  latent_join_kernel<BF, F8, DC, R><<<dim3(grid, DC / 32 * (R / 32)), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int DC, int R>
hipError_t run_latent_d(const AttnArgs& a, int fmt, int grid, hipStream_t s) {
  const bool f8 = a.c.fmt == KV_E4M3;
  if (fmt == KV_BF16)
    return f8 ? run_latent<true, true, DC, R>(a, grid, s) : run_latent<true, false, DC, R>(a, grid, s);
  return f8 ? run_latent<false, true, DC, R>(a, grid, s) : run_latent<false, false, DC, R>(a, grid, s);
}

}  // namespace
}  // namespace moe
