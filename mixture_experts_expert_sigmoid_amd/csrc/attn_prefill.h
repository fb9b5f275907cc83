// Attention of the newest tokens of each sequence (a prompt, or the next
// chunk of one) over a paged key-value cache.
//
// Mathematics. One pass over the keys with the running maximum and sum of a
// softmax: S^T = K Q^T, P = 2^(S - m), O^T = V^T P^T, all in fp32 but the
// 16-bit operands. The rows of a tile are (token, query head) pairs of one
// key-value head, token-major, so the heads that share keys share the tile:
// a tile spans few positions, and a short chunk still fills it.
//
// Layout. Four waves of two 32-row blocks (one for head_dim 256),
// v_mfma_*_32x32x16. A row lies in a lane's column of S^T (lane l: row l % 32, 16 of 32 keys), so the softmax
// is a loop in the lane and one exchange with lane l ^ 32, and P is the B
// operand of the second product as it stands when each lane half's 8-key
// slice of a 16-key step is taken as keys 4h..4h+3 and 8+4h..8+4h+3 of it.
// K and V tiles go through LDS, 16-byte units swizzled by key; V is read
// transposed (ds_read_b64_tr_b16), in that key order.
//
// Rescaling. O and the sum follow the maximum only when it has grown by more
// than 8 (a factor of 2^8 of P, which neither type nor sum minds): rare after
// the first tiles, and exact all the same.
//
// Masked places. Scores are replaced, not added to. V rows that no row of the
// tile sees are staged as zeros; in tiles where some rows see a key and some
// do not, V values that are not finite are staged as zero and their products
// added to the rows that see them one by one.
//
// Bound: the matrix cores and the exponentials for long prompts; latency for
// short ones. Few tiles: the keys of each are split over workgroups and the
// parts joined in order.
#pragma once
#include "attn_dev.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// keys of a tile, 32-row blocks of a wave, rows of a workgroup's tile
template <int D>
struct PreShape {
  static constexpr int BN = D == 256 ? 32 : 64;
  static constexpr int RB = D == 64 ? 2 : 1;
  static constexpr int ROWS = prefill_rows(D);
  static_assert(ROWS == 128 * RB, "four waves");
};

// what a workgroup works on
struct PreTile {
  int seq, slot, L, m, q0;     // sequence; its slot, length, new tokens, first row of q
  int tile, rows;              // tile of PreShape::ROWS rows, rows of the sequence
  int p_min, p_max;            // positions of its first and last row
  int lo_min, lo_max;          // first key of the window at those
  int nb1, b2, nb;             // key tiles: 0..nb1-1, then b2 .. b2 + nb - nb1 - 1
};

__device__ __forceinline__ int pre_cu(const AttnArgs& a, int i) {
  const int c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? (int)a.T : c);
}

template <int D>
__device__ __forceinline__ bool pre_span(const AttnArgs& a, PreTile& t) {
  constexpr int BN = PreShape<D>::BN, ROWS = PreShape<D>::ROWS;
  const int g = a.g;
  t.q0 = pre_cu(a, t.seq);
  t.m = max(0, pre_cu(a, t.seq + 1) - t.q0);
  t.rows = t.m * g;
  if (t.tile * ROWS >= t.rows) return false;
  t.slot = kv_slot(a.slots, t.seq, a.t.n_slots, a.err);
  t.L = kv_len(a.t, t.slot);
  const int r1 = min(t.rows, (t.tile + 1) * ROWS) - 1;
  t.p_min = t.L - t.m + t.tile * ROWS / g;
  t.p_max = t.L - t.m + r1 / g;
  t.lo_min = a.window ? max(0, t.p_min - a.window + 1) : 0;
  t.lo_max = a.window ? max(0, t.p_max - a.window + 1) : 0;
  t.b2 = t.lo_min / BN;
  t.nb1 = min(t.b2, (min(a.first, t.lo_min) + BN - 1) / BN);
  const int end = (max(0, t.p_max + 1) + BN - 1) / BN;
  t.nb = t.nb1 + max(0, end - t.b2);
  return true;
}

// parts that a tile's keys are split into: at least four key tiles each
__device__ __forceinline__ int pre_parts(const AttnArgs& a, int nb) {
  return max(1, min(a.n_split, nb >> 2));
}

template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_prefill_kernel(AttnArgs a) {
  constexpr int BN = PreShape<D>::BN, RB = PreShape<D>::RB, ROWS = PreShape<D>::ROWS;
  constexpr int NA = BN / 32;                    // 32-key score tiles
  constexpr int NC = D / 16;                     // steps of the first product
  constexpr int ND = D / 32;                     // 32-row tiles of O^T
  constexpr int UPR = D / 8;                     // 16-byte units of a row in LDS
  constexpr int WR = BN / 4;                     // rows of a tile that a wave brings
  constexpr int GPR = F8 ? D / 16 : UPR;         // 16-byte units of a row in memory
  constexpr int NL = WR * GPR / 64;              // loads per lane and array
  constexpr int TB = BN * D * 2;                 // bytes of a tile in LDS
  static_assert(NL >= 1, "tile");

  __shared__ __align__(16) char s_k[2][TB];
  __shared__ __align__(16) char s_v[2][TB];
  __shared__ int s_ok[2][4];                     // page there, by bringing wave
  __shared__ int s_bad;                          // values of V not finite were taken out

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l31 = lane & 31;

  PreTile t;
  const int kvh = blockIdx.x % a.c.hkv;
  {
    // longest tiles first; sequence i's tiles start at cu[i] g / ROWS + i
    const int tt = (int)(gridDim.x / a.c.hkv) - 1 - (int)(blockIdx.x / a.c.hkv);
    auto base = [&](int i) { return (int)((long)pre_cu(a, i) * a.g / ROWS) + i; };
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base(mid) <= tt) lo = mid; else hi = mid - 1;
    }
    t.seq = lo;
    t.tile = tt - base(lo);
    if (!pre_span<D>(a, t)) return;
  }
  const int parts = pre_parts(a, t.nb);
  if ((int)blockIdx.y >= parts) return;
  const int x0 = (int)((long)blockIdx.y * t.nb / parts);
  const int x1 = (int)((long)(blockIdx.y + 1) * t.nb / parts);
  if (tid == 0) s_bad = 0;

  // the wave's rows and what they see
  const int r0 = t.tile * ROWS + w * (32 * RB);
  const bool idle = r0 >= t.rows;
  const int wp_min = t.L - t.m + min(r0, t.rows - 1) / a.g;
  const int wp_max = t.L - t.m + (min(r0 + 32 * RB, t.rows) - 1) / a.g;
  const int wlo_min = a.window ? max(0, wp_min - a.window + 1) : 0;
  const int wlo_max = a.window ? max(0, wp_max - a.window + 1) : 0;

  // scores are compared unscaled: the sign of the scale goes into q
  float sc = F8 ? a.scale * a.c.ks[kvh] : a.scale;
  const uint32_t flip = sc < 0.0f ? 0x80008000u : 0u;
  const bool flat = sc == 0.0f;
  sc = flat ? 1.0f : fabsf(sc);
  const float thr = fminf(8.0f / sc, 1e30f);

  // this lane's rows
  bool have[RB];
  int head[RB], pos[RB], lo[RB];
  long qrow[RB];
  u32x4 q[RB][NC];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = r0 + 32 * rb + l31;
    have[rb] = r < t.rows;
    const int tok = have[rb] ? r / a.g : 0;
    head[rb] = kvh * a.g + (have[rb] ? r - tok * a.g : 0);
    pos[rb] = have[rb] ? t.L - t.m + tok : -1;
    lo[rb] = a.window ? pos[rb] - a.window + 1 : 0;
    qrow[rb] = t.q0 + tok;
    const char* p = a.q + qrow[rb] * a.q_row + head[rb] * a.q_head + 16 * half;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const u32x4 y = *(const u32x4*)(p + 32 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[rb][c][e] = flat ? 0u : y[e] ^ flip;
    }
  }

  f32x16 o[RB][ND];
  float m[RB], l[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[rb][d][i] = 0.0f;
    m[rb] = kNegInf;
    l[rb] = 0.0f;
  }

  const int* row = a.t.table + (long)max(0, t.slot) * a.t.ld;
  const char* kb = a.c.k + kvh * a.c.sh;
  const char* vb = a.c.v + kvh * a.c.sh;
  const int grp = w * WR / 16;                   // 16-key group that this wave brings from

  auto key_of = [&](int x) { return BN * (x < t.nb1 ? x : t.b2 + x - t.nb1); };
  auto group_seen = [&](int key) {
    return key <= t.p_max && (key + 16 > t.lo_min || key < a.first);
  };
  // table entry of the wave's group of tile x; -2: nothing of it is visible
  auto fetch = [&](int x) {
    const int key = key_of(x) + 16 * grp;
    return x < x1 && group_seen(key) ? row[kv_entry(a.t, key)] : -2;
  };
  auto whole_of = [&](int key) {
    return key + BN - 1 <= t.p_min && (key >= t.lo_max || key + BN <= a.first);
  };
  // swizzle of 16-byte units by row (of the tile)
  auto k_swz = [&](int kr) { return kr & (UPR < 16 ? UPR - 1 : 15); };
  auto v_swz = [&](int kr) { return UPR == 8 ? ((kr >> 1) & 3) << 1 : (kr & 7) << 1; };
  const uint32_t kExp = BF ? 0x7F80u : 0x7C00u;
  auto bad16 = [&](uint32_t x) {                 // either half infinite or NaN
    return (x & kExp) == kExp || ((x >> 16) & kExp) == kExp;
  };
  auto clean16 = [&](uint32_t x) {
    if ((x & kExp) == kExp) x &= 0xFFFF0000u;
    if (((x >> 16) & kExp) == kExp) x &= 0x0000FFFFu;
    return x;
  };
  // a unit of V of a tile that is not whole, as it is to be staged
  auto clean = [&](u32x4 v, int key, int kr) {
    const int j = key + kr;
    if (j > t.p_max || !(j >= t.lo_min || j < a.first)) return u32x4{0, 0, 0, 0};
    if (bad16(v[0]) || bad16(v[1]) || bad16(v[2]) || bad16(v[3])) {
      s_bad = 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = clean16(v[e]);
    }
    return v;
  };

  u32x4 rk[F8 ? NL : 1], rv[F8 ? NL : 1];        // e4m3: raw units on their way
  // starts the loads of this wave's rows of tile x: 16-bit straight into LDS
  auto issue = [&](int x, int e, int buf) {
    const int key = key_of(x) + 16 * grp;
    const bool ok = e >= 0 && e < a.t.n_pages;
    if (!ok && e != -2 && lane == 0) atomicOr(a.err, kErrPage);
    if (lane == 0) s_ok[buf][w] = ok;
    const int in = ok ? key - kv_entry(a.t, key) * a.t.ps : 0;
    // a uniform base, and an offset of the lane below 2^31 (16 stride_tok < 2^30)
    const long off = (ok ? e : 0) * a.c.sp + in * a.c.st;
    const char* kp = kb + off;
    const char* vp = vb + off;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int up = i * 64 + lane, kr = w * WR + up / GPR, u = up % GPR;
      const uint32_t ro = (uint32_t)(kr & 15) * (uint32_t)a.c.st;
      if constexpr (F8) {
        rk[i] = *(const u32x4*)(kp + (ro + 16 * u));
        rv[i] = *(const u32x4*)(vp + (ro + 16 * u));
      } else {
        const int at = (w * WR * UPR + i * 64) * 16;
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(kp + (ro + 16 * (u ^ k_swz(kr)))),
            (__attribute__((address_space(3))) void*)(s_k[buf] + at), 16, 0, 0);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(vp + (ro + 16 * (u ^ v_swz(kr)))),
            (__attribute__((address_space(3))) void*)(s_v[buf] + at), 16, 0, 0);
      }
    }
  };
  // completes them: waits, expands e4m3, takes masked values out of V
  auto finish = [&](int x, int buf) {
    const int key = key_of(x);
    const bool whole = whole_of(key);
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int up = i * 64 + lane, kr = w * WR + up / GPR, u = up % GPR;
        u32x4 kk[2], vv[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk[e >> 1][2 * (e & 1)] = from_e4m3<BF, false>(rk[i][e]);
          kk[e >> 1][2 * (e & 1) + 1] = from_e4m3<BF, true>(rk[i][e]);
          vv[e >> 1][2 * (e & 1)] = from_e4m3<BF, false>(rv[i][e]);
          vv[e >> 1][2 * (e & 1) + 1] = from_e4m3<BF, true>(rv[i][e]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!whole) vv[h] = clean(vv[h], key, kr);
          *(u32x4*)(s_k[buf] + kr * (2 * D) + 16 * ((2 * u + h) ^ k_swz(kr))) = kk[h];
          *(u32x4*)(s_v[buf] + kr * (2 * D) + 16 * ((2 * u + h) ^ v_swz(kr))) = vv[h];
        }
      }
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (!whole) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int up = i * 64 + lane, kr = w * WR + up / GPR;
          u32x4* p = (u32x4*)(s_v[buf] + (w * WR * UPR + up) * 16);
          *p = clean(*p, key, kr);
        }
      }
    }
  };

  int e_next = 0;
  if (x0 < x1) {
    issue(x0, fetch(x0), 0);
    e_next = fetch(x0 + 1);
  }
  for (int x = x0; x < x1; ++x) {
    const int key = key_of(x), buf = (x - x0) & 1;
    finish(x, buf);
    __syncthreads();
    // the other buffer's tile is done with: every wave has passed the barrier
    if (x + 1 < x1) {
      issue(x + 1, e_next, buf ^ 1);
      e_next = fetch(x + 2);
    }
    if (idle || key > wp_max || (key + BN <= wlo_min && key >= a.first)) continue;
    uint32_t gone = 0;                           // 16-key groups without a page
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!s_ok[buf][i]) gone |= 1u << (i * WR / 16);
    const bool whole = !gone && key + BN - 1 <= wp_min && (key >= wlo_max || key + BN <= a.first);

    f32x16 s[RB][NA];
#pragma unroll
    for (int aa = 0; aa < NA; ++aa) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[rb][aa][i] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int kr = 32 * aa + l31;
        const u32x4 ka =
            *(const u32x4*)(s_k[buf] + kr * (2 * D) + 16 * ((2 * c + half) ^ k_swz(kr)));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb][aa] = mfma32<BF>(ka, q[rb][c], s[rb][aa]);
      }
    }
    if (!whole) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int aa = 0; aa < NA; ++aa)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int kk = 32 * aa + 8 * (i >> 2) + (i & 3), at = key + 4 * half;
            const bool ok = kk <= pos[rb] - at && (kk >= lo[rb] - at || kk < a.first - at) &&
                            !((gone >> (kk >> 4)) & 1);
            if (!ok) s[rb][aa][i] = kNegInf;
          }
    }
    float bm[RB];
    bool grown = false;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      bm[rb] = s[rb][0][0];
#pragma unroll
      for (int aa = 0; aa < NA; ++aa)
#pragma unroll
        for (int i = 0; i < 16; ++i) bm[rb] = fmaxf(bm[rb], s[rb][aa][i]);
      bm[rb] = xor32_reduce(bm[rb], OpMax{});
      grown |= bm[rb] > m[rb] + thr;
    }
    if (__any(grown)) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const float mn = fmaxf(m[rb], bm[rb]);
        const float f = exp2_fast((m[rb] - (mn == kNegInf ? 0.0f : mn)) * sc);
        m[rb] = mn;
        l[rb] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[rb][d][i] *= f;
      }
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const float neg = m[rb] == kNegInf ? 0.0f : -m[rb] * sc;
#pragma unroll
      for (int aa = 0; aa < NA; ++aa)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[rb][aa][i] = exp2_fast(__builtin_fmaf(s[rb][aa][i], sc, neg));
          l[rb] += s[rb][aa][i];
        }
    }

#pragma unroll
    for (int aa = 0; aa < NA; ++aa)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        u32x4 pb[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            pb[rb][j] = pack16<BF>(s[rb][aa][8 * st + 2 * j], s[rb][aa][8 * st + 2 * j + 1]);
        // keys 4 half + 0..3 of the 16-key step, then the same + 8; lane i of
        // 16 reads row i / 4, 4 values from 4 (i % 4), and gets column i
        const int k0 = 32 * aa + 16 * st + 4 * half + ((lane & 15) >> 2);
        const int dc = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          u32x4 va;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kr = k0 + 8 * h;
            const int b = 2 * (32 * d + dc);      // byte in the row
            char* p = s_v[buf] + kr * (2 * D) + (16 * ((b >> 4) ^ v_swz(kr)) + (b & 15));
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)p);
            const u32x2 z = __builtin_bit_cast(u32x2, y);
            va[2 * h] = z[0];
            va[2 * h + 1] = z[1];
          }
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) o[rb][d] = mfma32<BF>(va, pb[rb], o[rb][d]);
        }
      }
  }

  // values of V that are not finite and were staged as zeros: their products,
  // for the rows that see their key
  __syncthreads();
  if (s_bad && !idle) {
    for (int x = x0; x < x1; ++x) {
      const int key = key_of(x);
      if (whole_of(key)) continue;
      for (int j = key; j < key + BN; ++j) {
        if (j > t.p_max || !(j >= t.lo_min || j < a.first)) continue;
        const int e = kv_entry(a.t, j), p = row[e];
        if (p < 0 || p >= a.t.n_pages) continue;
        const long off = p * a.c.sp + (long)(j - e * a.t.ps) * a.c.st;
        auto value = [&](const char* base, int dd) {
          uint32_t x16;
          if constexpr (F8)
            x16 = from_e4m3<BF, false>(*(const uint8_t*)(base + off + dd)) & 0xFFFF;
          else
            x16 = *(const uint16_t*)(base + off + 2 * dd);
          return BF ? bf16_bits_to_f32(x16)
                    : (float)__builtin_bit_cast(_Float16, (uint16_t)x16);
        };
        auto finite = [](float f) { return fabsf(f) < __builtin_huge_valf(); };
        bool any = false;
#pragma unroll 1
        for (int dd = lane; dd < D; dd += 64) any |= !finite(value(vb, dd));
        if (!__any(any)) continue;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          float dot = 0.0f;
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t q16 = (q[rb][c][i >> 1] >> (16 * (i & 1))) & 0xFFFF;
              dot += value(kb, 16 * c + 8 * half + i) *
                     (BF ? bf16_bits_to_f32(q16)
                         : (float)__builtin_bit_cast(_Float16, (uint16_t)q16));
            }
          dot = xor32_reduce(dot, OpSum{});
          const bool sees = j <= pos[rb] && (j >= lo[rb] || j < a.first);
          const float pv = exp2_fast(
              __builtin_fmaf(dot, sc, m[rb] == kNegInf ? 0.0f : -m[rb] * sc));
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float f = value(vb, 32 * d + 8 * (i >> 2) + 4 * half + (i & 3));
              if (sees && !finite(f)) o[rb][d][i] += pv * f;
              if (i == 15) __builtin_amdgcn_sched_barrier(0);
            }
        }
      }
    }
  }

#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    l[rb] = xor32_reduce(l[rb], OpSum{});
    if (!have[rb]) continue;
    if (parts == 1) {
      float inv = l[rb] == 0.0f ? 0.0f : 1.0f / l[rb];      // no visible key: 0
      if (F8 && l[rb] != 0.0f) inv *= a.c.vs[kvh];
      char* dst = a.out + qrow[rb] * a.o_row + head[rb] * a.o_head;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const u32x2 y = {pack16<BF>(o[rb][d][i] * inv, o[rb][d][i + 1] * inv),
                           pack16<BF>(o[rb][d][i + 2] * inv, o[rb][d][i + 3] * inv)};
          *(u32x2*)(dst + 2 * (32 * d + 2 * i + 4 * half)) = y;
        }
      if (a.lse && half == 0)
        a.lse[qrow[rb] * a.hq + head[rb]] = (m[rb] * sc + __builtin_amdgcn_logf(l[rb])) * kLn2;
    } else {
      const long rows = a.T * a.hq, ri = qrow[rb] * a.hq + head[rb];
      float* dst = a.part + ((long)blockIdx.y * rows + ri) * D;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *(f32x4*)(dst + 32 * d + 2 * i + 4 * half) =
              f32x4{o[rb][d][i], o[rb][d][i + 1], o[rb][d][i + 2], o[rb][d][i + 3]};
      if (half == 0) {
        float* ml = a.part + (long)a.n_split * rows * D + ((long)blockIdx.y * rows + ri) * 2;
        ml[0] = m[rb] * sc;
        ml[1] = l[rb];
      }
    }
  }
}

// Joins the parts of split tiles: one wave per (token, query head).
template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256) void prefill_join_kernel(AttnArgs a) {
  constexpr int ROWS = PreShape<D>::ROWS;
  constexpr int E = D / 64;
  const long rows = a.T * a.hq;
  const long ri = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (ri >= rows) return;
  const int tok = (int)(ri / a.hq), head = (int)(ri - (long)tok * a.hq);
  PreTile t;
  {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre_cu(a, mid) <= tok) lo = mid; else hi = mid - 1;
    }
    t.seq = lo;
    t.tile = ((tok - pre_cu(a, lo)) * a.g + head % a.g) / ROWS;
    if (!pre_span<D>(a, t)) return;
  }
  const int parts = pre_parts(a, t.nb);
  if (parts == 1) return;
  const int lane = lane_id();
  const float* ml = a.part + (long)a.n_split * rows * D + ri * 2;
  const float pm = lane < parts ? ml[(long)lane * rows * 2] : kNegInf;
  const float pl = lane < parts ? ml[(long)lane * rows * 2 + 1] : 0.0f;
  const float m = wave_max(pm);
  const float mu = m == kNegInf ? 0.0f : m;
  const float f = exp2_fast(pm - mu);
  const float l = wave_sum(f * pl);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int i = 0; i < parts; ++i) {
    const float fi = __shfl(f, i);
    const float* p = a.part + ((long)i * rows + ri) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += fi * p[e];
  }
  float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (F8 && l != 0.0f) inv *= a.c.vs[head / a.g];
  char* dst = a.out + (long)tok * a.o_row + head * a.o_head;
  if constexpr (E == 1) {
    *(uint16_t*)(dst + 2 * lane) = (uint16_t)pack16<BF>(acc[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *(uint32_t*)(dst + 2 * (lane * E + e)) = pack16<BF>(acc[e] * inv, acc[e + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[ri] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool BF, bool F8, int D>
hipError_t run_prefill(const AttnArgs& a, hipStream_t s) {
  const long tiles = prefill_tiles(a.n, a.T, a.g, D);
  attn_prefill_kernel<BF, F8, D>
      <<<dim3((unsigned)(tiles * a.c.hkv), a.n_split), 256, 0, s>>>(a);
  if (a.n_split > 1)
    prefill_join_kernel<BF, F8, D><<<(unsigned)((a.T * a.hq + 3) / 4), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t run_prefill_d(const AttnArgs& a, int fmt, hipStream_t s) {
  const bool f8 = a.c.fmt == KV_E4M3;
  if (fmt == KV_BF16)
    return f8 ? run_prefill<true, true, D>(a, s) : run_prefill<true, false, D>(a, s);
  return f8 ? run_prefill<false, true, D>(a, s) : run_prefill<false, false, D>(a, s);
}

}  // namespace
}  // namespace moe
