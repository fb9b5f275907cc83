// Attention of the newest tokens of each sequence (a prompt, or the next
// chunk of one) over a paged key-value cache.
//
// Mathematics. One pass over the keys with the running maximum and sum of a
// softmax: S^T = K Q^T, P = 2^(S - m), O^T = V^T P^T, all in fp32 but the
// 16-bit operands. The rows of a tile are (token, query head) pairs of one
// key-value head, token-major, so the heads that share keys share the tile:
// a tile spans few positions, and a short chunk still fills it.
//
// Layout. Four waves of 32 rows, v_mfma_*_32x32x16. A wave's row lies in a
// lane's column of S^T (lane l: row l % 32, 16 of 32 keys), so the softmax
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

// what a workgroup works on
struct PreTile {
  int seq, slot, L, m, q0;     // sequence; its slot, length, new tokens, first row of q
  int tile, rows;              // tile of kPreRows rows, rows of the sequence
  int p_min, p_max;            // positions of its first and last row
  int lo_min, lo_max;          // first key of the window at those
  int nb1, b2, nb;             // key tiles: 0..nb1-1, then b2 .. b2 + nb - nb1 - 1
};

__device__ __forceinline__ int pre_cu(const AttnArgs& a, int i) {
  const int c = a.cu[i];
  return c < 0 ? 0 : (c > a.T ? (int)a.T : c);
}

template <int BN>
__device__ __forceinline__ bool pre_span(const AttnArgs& a, PreTile& t) {
  const int g = a.g;
  t.q0 = pre_cu(a, t.seq);
  t.m = max(0, pre_cu(a, t.seq + 1) - t.q0);
  t.rows = t.m * g;
  if (t.tile * kPreRows >= t.rows) return false;
  t.slot = kv_slot(a.slots, t.seq, a.t.n_slots, a.err);
  t.L = kv_len(a.t, t.slot);
  const int r1 = min(t.rows, (t.tile + 1) * kPreRows) - 1;
  t.p_min = t.L - t.m + t.tile * kPreRows / g;
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
  constexpr int BN = D == 256 ? 32 : 64;         // keys of a tile
  constexpr int NA = BN / 32;                    // 32-key score tiles
  constexpr int NC = D / 16;                     // steps of the first product
  constexpr int ND = D / 32;                     // 32-row tiles of O^T
  constexpr int UPR = D / 8;                     // 16-byte units of a row in LDS
  constexpr int GPR = F8 ? D / 16 : D / 8;       // 16-byte units of a row in memory
  constexpr int RPI = 256 / GPR;                 // rows of one load of the workgroup
  constexpr int NL = BN / RPI;                   // loads per thread and array
  static_assert(NL >= 1 && BN % RPI == 0, "tile");

  __shared__ __align__(16) char s_k[BN * D * 2];
  __shared__ __align__(16) char s_v[BN * D * 2];
  __shared__ int s_bad;                          // tile whose V holds values not finite

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int half = lane >> 5, l31 = lane & 31;

  PreTile t;
  const int kvh = blockIdx.x % a.c.hkv;
  {
    // longest tiles first; sequence i's tiles start at cu[i] g / kPreRows + i
    const int tt = (int)(gridDim.x / a.c.hkv) - 1 - (int)(blockIdx.x / a.c.hkv);
    auto base = [&](int i) { return (int)((long)pre_cu(a, i) * a.g / kPreRows) + i; };
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base(mid) <= tt) lo = mid; else hi = mid - 1;
    }
    t.seq = lo;
    t.tile = tt - base(lo);
    if (!pre_span<BN>(a, t)) return;
  }
  const int parts = pre_parts(a, t.nb);
  if ((int)blockIdx.y >= parts) return;
  const int x0 = (int)((long)blockIdx.y * t.nb / parts);
  const int x1 = (int)((long)(blockIdx.y + 1) * t.nb / parts);
  if (tid == 0) s_bad = -1;

  // this lane's row
  const int r = t.tile * kPreRows + 32 * w + l31;
  const bool have = r < t.rows;
  const int tok = have ? r / a.g : 0;
  const int head = kvh * a.g + (have ? r - tok * a.g : 0);
  const int pos = have ? t.L - t.m + tok : -1;
  const int lo = a.window ? pos - a.window + 1 : 0;

  u32x4 q[NC];
  {
    const char* p = a.q + (long)(t.q0 + tok) * a.q_row + head * a.q_head + 16 * half;
#pragma unroll
    for (int c = 0; c < NC; ++c) q[c] = *(const u32x4*)(p + 32 * c);
  }
  const float sc = F8 ? a.scale * a.c.ks[kvh] : a.scale;

  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNegInf, l = 0.0f;

  const int* row = a.t.table + (long)max(0, t.slot) * a.t.ld;
  const char* kb = a.c.k + kvh * a.c.sh;
  const char* vb = a.c.v + kvh * a.c.sh;
  const int srow = tid / GPR, scol = tid % GPR;  // this thread's unit of a load

  auto key_of = [&](int x) { return BN * (x < t.nb1 ? x : t.b2 + x - t.nb1); };
  // page of a 16-key group, -1 where it is missing or holds no visible key
  auto page_of = [&](int key) {
    if (key > t.p_max || !(key + 16 > t.lo_min || key < a.first)) return -1;
    const int p = row[kv_entry(a.t, key)];
    if (p >= 0 && p < a.t.n_pages) return p;
    atomicOr(a.err, kErrPage);
    return -1;
  };

  u32x4 rk[NL], rv[NL];
  auto load = [&](int x) {
    const int key = key_of(x);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int kr = key + i * RPI + srow;
      const int k16 = __builtin_amdgcn_readfirstlane(kr & ~15);
      const int p = page_of(k16);
      rk[i] = rv[i] = u32x4{0, 0, 0, 0};
      if (p >= 0) {
        const int in = k16 - kv_entry(a.t, k16) * a.t.ps;
        const long off = p * a.c.sp + (long)(in + (kr & 15)) * a.c.st + 16 * scol;
        rk[i] = *(const u32x4*)(kb + off);
        rv[i] = *(const u32x4*)(vb + off);
      }
    }
  };
  auto whole_of = [&](int key) {
    return key + BN - 1 <= t.p_min && (key >= t.lo_max || key + BN <= a.first);
  };
  // 16-byte unit u of key kr in LDS
  auto k_unit = [&](char* b, int kr, int u) {
    return b + kr * (2 * D) + 16 * (u ^ (kr & (UPR < 16 ? UPR - 1 : 15)));
  };
  auto v_swz = [&](int kr) {
    return UPR == 8 ? ((kr >> 1) & 3) << 1 : (kr & 7) << 1;
  };
  auto bad16 = [&](uint32_t x) {       // either half infinite or NaN
    const uint32_t e = BF ? 0x7F80u : 0x7C00u;
    return (x & e) == e || ((x >> 16) & e) == e;
  };
  auto clean16 = [&](uint32_t x) {
    const uint32_t e = BF ? 0x7F80u : 0x7C00u;
    if ((x & e) == e) x &= 0xFFFF0000u;
    if (((x >> 16) & e) == e) x &= 0x0000FFFFu;
    return x;
  };
  auto stage = [&](int x) {
    const int key = key_of(x);
    const bool whole = whole_of(key);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int lr = i * RPI + srow, kr = key + lr;
      const bool dead = kr > t.p_max || !(kr >= t.lo_min || kr < a.first);
      u32x4 kk[2], vv[2];
      if constexpr (F8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk[e >> 1][2 * (e & 1)] = from_e4m3<BF, false>(rk[i][e]);
          kk[e >> 1][2 * (e & 1) + 1] = from_e4m3<BF, true>(rk[i][e]);
          vv[e >> 1][2 * (e & 1)] = from_e4m3<BF, false>(rv[i][e]);
          vv[e >> 1][2 * (e & 1) + 1] = from_e4m3<BF, true>(rv[i][e]);
        }
      } else {
        kk[0] = rk[i];
        vv[0] = rv[i];
      }
      constexpr int H = F8 ? 2 : 1;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (!whole) {
          if (dead) vv[h] = u32x4{0, 0, 0, 0};
          if (bad16(vv[h][0]) || bad16(vv[h][1]) || bad16(vv[h][2]) || bad16(vv[h][3])) {
            s_bad = x;
#pragma unroll
            for (int e = 0; e < 4; ++e) vv[h][e] = clean16(vv[h][e]);
          }
        }
        const int u = H * scol + h;
        *(u32x4*)k_unit(s_k, lr, u) = kk[h];
        *(u32x4*)(s_v + lr * (2 * D) + 16 * (u ^ v_swz(lr))) = vv[h];
      }
    }
  };

  if (x0 < x1) load(x0);
  for (int x = x0; x < x1; ++x) {
    const int key = key_of(x);
    __syncthreads();                   // the tile before is done with
    stage(x);
    __syncthreads();
    uint32_t gone = 0;                 // 16-key groups without a page
    bool whole = whole_of(key);
#pragma unroll
    for (int gi = 0; gi < BN / 16; ++gi)
      if (page_of(key + 16 * gi) < 0) gone |= 1u << gi;
    if (gone) whole = false;
    if (x + 1 < x1) load(x + 1);

    f32x16 s[NA];
#pragma unroll
    for (int aa = 0; aa < NA; ++aa) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[aa][i] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const u32x4 ka = *(const u32x4*)k_unit(s_k, 32 * aa + l31, 2 * c + half);
        s[aa] = mfma32<BF>(ka, q[c], s[aa]);
      }
    }
    float bm = kNegInf;
#pragma unroll
    for (int aa = 0; aa < NA; ++aa)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[aa][i] *= sc;
        if (!whole) {
          const int kk = 32 * aa + 8 * (i >> 2) + 4 * half + (i & 3), j = key + kk;
          const bool ok = j <= pos && (j >= lo || j < a.first) && !((gone >> (kk >> 4)) & 1);
          if (!ok) s[aa][i] = kNegInf;
        }
        bm = fmaxf(bm, s[aa][i]);
      }
    bm = xor32_reduce(bm, OpMax{});
    if (__any(bm > m + 8.0f)) {
      const float mn = fmaxf(m, bm);
      const float f = exp2_fast(m - (mn == kNegInf ? 0.0f : mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    const float mu = m == kNegInf ? 0.0f : m;
#pragma unroll
    for (int aa = 0; aa < NA; ++aa)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[aa][i] = exp2_fast(s[aa][i] - mu);
        l += s[aa][i];
      }

    if (!whole && s_bad == x) {
      // values of V that are not finite, for the rows that see their key
      for (int k = 0; k < BN; ++k) {
        const int kp = page_of((key + k) & ~15);
        if (kp < 0) continue;
        float pv = 0.0f;
#pragma unroll
        for (int aa = 0; aa < NA; ++aa)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (k == 32 * aa + 8 * (i >> 2) + 4 * ((k >> 2) & 1) + (i & 3)) pv = s[aa][i];
        pv = __shfl(pv, l31 + 32 * ((k >> 2) & 1));
        const int j = key + k;
        const bool sees = j <= pos && (j >= lo || j < a.first);
        const int in = j - kv_entry(a.t, j) * a.t.ps;
        const char* vr = vb + kp * a.c.sp + (long)in * a.c.st;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int dd = 32 * d + 8 * (i >> 2) + 4 * half + (i & 3);
            uint32_t x16;
            if constexpr (F8)
              x16 = from_e4m3<BF, false>(*(const uint8_t*)(vr + dd)) & 0xFFFF;
            else
              x16 = *(const uint16_t*)(vr + 2 * dd);
            if (bad16(x16) && sees) {
              const float vf = BF ? bf16_bits_to_f32(x16)
                                  : (float)__builtin_bit_cast(_Float16, (uint16_t)x16);
              o[d][i] += pv * vf;
            }
          }
      }
    }

#pragma unroll
    for (int aa = 0; aa < NA; ++aa)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        u32x4 pb;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          pb[j] = pack16<BF>(s[aa][8 * st + 2 * j], s[aa][8 * st + 2 * j + 1]);
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
            char* p = s_v + kr * (2 * D) + (16 * ((b >> 4) ^ v_swz(kr)) + (b & 15));
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)p);
            const u32x2 z = __builtin_bit_cast(u32x2, y);
            va[2 * h] = z[0];
            va[2 * h + 1] = z[1];
          }
          o[d] = mfma32<BF>(va, pb, o[d]);
        }
      }
  }

  l = xor32_reduce(l, OpSum{});
  if (!have) return;
  if (parts == 1) {
    float inv = l == 0.0f ? 0.0f : 1.0f / l;       // no visible key: 0
    if (F8 && l != 0.0f) inv *= a.c.vs[kvh];
    char* dst = a.out + (long)(t.q0 + tok) * a.o_row + head * a.o_head;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const u32x2 y = {pack16<BF>(o[d][i] * inv, o[d][i + 1] * inv),
                         pack16<BF>(o[d][i + 2] * inv, o[d][i + 3] * inv)};
        *(u32x2*)(dst + 2 * (32 * d + 2 * i + 4 * half)) = y;
      }
    if (a.lse && half == 0)
      a.lse[(long)(t.q0 + tok) * a.hq + head] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  } else {
    const long rows = a.T * a.hq, ri = (long)(t.q0 + tok) * a.hq + head;
    float* dst = a.part + ((long)blockIdx.y * rows + ri) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(f32x4*)(dst + 32 * d + 2 * i + 4 * half) =
            f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (half == 0) {
      float* ml = a.part + (long)a.n_split * rows * D + ((long)blockIdx.y * rows + ri) * 2;
      ml[0] = m;
      ml[1] = l;
    }
  }
}

// Joins the parts of split tiles: one wave per (token, query head).
template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256) void prefill_join_kernel(AttnArgs a) {
  constexpr int BN = D == 256 ? 32 : 64;
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
    t.tile = ((tok - pre_cu(a, lo)) * a.g + head % a.g) / kPreRows;
    if (!pre_span<BN>(a, t)) return;
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
  const long tiles = a.T * a.g / kPreRows + a.n;
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
