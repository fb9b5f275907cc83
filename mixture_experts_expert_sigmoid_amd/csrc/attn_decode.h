// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics. Per sequence and key-value head, with the g query heads that
// share it as the columns of Q^T: S^T = K Q^T, p = 2^(S - m) with the running
// maximum m and sum l of a softmax, O^T = V^T P^T, rescaled when m grows.
// One pass over the keys and values, everything else in registers.
//
// Layout. A wave takes 32 keys at a time with v_mfma_*_16x16x32. K rows go
// from memory straight to the A operand (lane l: key l % 16, 8 values of D).
// The result has a query head in each lane's column (l % 16) and 4 keys in
// its rows, so a lane holds P of 8 keys of one head -- the B operand of the
// second product as it stands, if its 8-key slice of lane group l / 16 is
// taken as keys 4 (l / 16) + 0..3 of both 16-key tiles. V is loaded in that
// order, 8 keys of D / 16 consecutive d a lane, and the 16-bit pairs turned
// round in the lane (one v_perm per pair of values), so row m of output tile
// td is d = (D / 16) m + td. Nothing of K, V, S or P passes through LDS.
//
// Split. The keys that each sequence sees are cut into units of 128 (32 per
// wave); the units of all (sequence, key-value head) pairs, laid end to end,
// are dealt out evenly to the workgroups whatever the lengths. A workgroup
// finishes every pair that lies wholly in its run; of the first and the last
// it leaves fp32 partial results that the join kernel adds in order.
//
// Bound: HBM reads of K and V; short contexts by latency (length -> table ->
// keys -> join).
#pragma once
#include "attn_dev.h"

namespace moe {
namespace {

constexpr int kDecUnit = 4 * kDecKeys;
constexpr int kDecPartRow = 32;       // maxima and sums before the D floats of 16 heads

__device__ __host__ inline size_t dec_slot_floats(int D) { return (size_t)kDecPartRow + 16 * D; }

// what a query at position L - 1 sees, as blocks of 32 keys: blocks 0..nb1-1
// (first keys), then those from b2 on up to the length
struct DecSpan {
  int L, lo, nf, nb1, b2, nb;
};
__device__ __forceinline__ DecSpan dec_span(int L, int window, int first) {
  DecSpan s;
  s.L = L;
  s.lo = window && L > window ? L - window : 0;
  s.nf = first < s.lo ? first : s.lo;
  s.b2 = s.lo / kDecKeys;
  const int nb1 = (s.nf + kDecKeys - 1) / kDecKeys;
  s.nb1 = nb1 < s.b2 ? nb1 : s.b2;
  s.nb = s.nb1 + (L + kDecKeys - 1) / kDecKeys - s.b2;
  return s;
}
__device__ __forceinline__ int dec_units(const DecSpan& s) {
  const int u = (s.nb + 3) >> 2;
  return u > 0 ? u : 1;               // a sequence without keys still gets its row written
}

// Q operand of one lane: head l % 16 of the tile, D values in the order of
// the K loads
template <bool F8, int D>
__device__ __forceinline__ void dec_load_q(u32x4 (&q)[D / 32], const char* row, bool have) {
  const int lg = lane_id() >> 4;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const int d = F8 ? 64 * (c >> 1) + 16 * lg + 8 * (c & 1) : 32 * c + 8 * lg;
    u32x4 z = {0, 0, 0, 0};
    q[c] = have ? *(const u32x4*)(row + 2 * d) : z;
  }
}

// raw bytes of one wave's block: K per 16-key tile, V per key
template <bool F8, int D>
struct DecRaw {
  static constexpr int KL = F8 ? D / 64 : D / 32;          // 16-byte loads per lane and tile
  static constexpr int VB = F8 ? D / 16 : D / 8;           // bytes per lane and key
  u32x4 k[2][KL];
  uint32_t v[8][VB / 4];
};

template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256, dec_waves(D, F8)) void attn_decode_kernel(AttnArgs a) {
  constexpr int NC = D / 32;             // 32-deep steps of the first product
  constexpr int VE = D / 16;             // d values of a lane (rows of V^T it feeds)
  constexpr int VH = F8 ? 1 : (VE > 8 ? 2 : 1);    // 16-byte halves of them
  constexpr int VW = VE / VH;            // d values of one half
  using Raw = DecRaw<F8, D>;

  __shared__ int s_pref[kDecMaxSeqs + 1];
  __shared__ int s_len[kDecMaxSeqs];
  __shared__ int s_scan[4];
  __shared__ float s_ml[4][2][16];
  __shared__ float s_o[4][16][D + 4];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lg = lane >> 4, lc = lane & 15;
  const int n = a.n, ht = (a.g + 15) >> 4;       // 16-head tiles per key-value head
  const int HT = a.c.hkv * ht;

  // lengths and the prefix sums of the units (2 sequences a thread)
  int un[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * tid + k;
    un[k] = 0;
    if (i < n) {
      const int L = kv_len(a.t, kv_slot(a.slots, i, a.t.n_slots, a.err));
      s_len[i] = L;
      un[k] = dec_units(dec_span(L, a.window, a.first));
    }
  }
  int incl = un[0] + un[1];
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) s_scan[w] = incl;
  __syncthreads();
  for (int i = 0; i < w; ++i) incl += s_scan[i];
  if (2 * tid < n) s_pref[2 * tid] = incl - un[0] - un[1];
  if (2 * tid + 1 < n) s_pref[2 * tid + 1] = incl - un[1];
  if (tid == 255) s_pref[n] = incl;
  __syncthreads();

  const long U = (long)s_pref[n] * HT;
  const long W = U < (long)gridDim.x ? U : (long)gridDim.x;
  if ((long)blockIdx.x >= W) return;
  long u = (long)blockIdx.x * U / W;
  const long u_end = ((long)blockIdx.x + 1) * U / W;

  // the sequence of unit u: the last i with pref[i] * HT <= u
  int seq = 0;
  {
    int hi = n - 1;
    while (seq < hi) {
      const int mid = (seq + hi + 1) >> 1;
      if ((long)s_pref[mid] * HT <= u) seq = mid; else hi = mid - 1;
    }
  }

  const long koff = (long)lc * a.c.st + 16 * lg;            // K: key lc, 16 bytes of D
  const long voff = (long)(4 * lg) * a.c.st + lc * (F8 ? VE : 2 * VW);

  while (u < u_end) {
    const int pre = s_pref[seq], ns = s_pref[seq + 1] - pre;
    const long rel = u - (long)pre * HT;
    const int hti = (int)(rel / ns), b0 = (int)(rel - (long)hti * ns);
    const int b1 = (int)min((long)ns, b0 + (u_end - u));
    const int kvh = hti / ht, hbase = (hti - kvh * ht) * 16;
    const int heads = min(16, a.g - hbase);
    const DecSpan sp = dec_span(s_len[seq], a.window, a.first);
    const int slot = a.slots ? a.slots[seq] : seq;
    const int* row = a.t.table + (long)(slot < 0 || slot >= a.t.n_slots ? 0 : slot) * a.t.ld;

    u32x4 q[NC];
    dec_load_q<F8, D>(q, a.q + seq * a.q_row + (long)(kvh * a.g + hbase + lc) * a.q_head,
                      lc < heads);
    const float sc = F8 ? a.scale * a.c.ks[kvh] : a.scale;

    f32x4 o[VE];
#pragma unroll
    for (int t = 0; t < VE; ++t) o[t] = f32x4{0, 0, 0, 0};
    float m = kNegInf, l = 0.0f;

    const char* kb = a.c.k + kvh * a.c.sh;
    const char* vb = a.c.v + kvh * a.c.sh;

    // blocks 4 x + w of units x = b0 .. b1 - 1 are this wave's
    const int x_end = min(b1, (sp.nb - w + 3) >> 2);
    int x = b0;
    while (x < x_end) {
      // page and place of the two 16-key tiles of the next 64 blocks, one
      // block a lane; -1 where a tile has no visible key or no page
      const int xb = x, xe = min(x_end, x + 64);
      int pg[2], in[2];
      {
        const int bi = 4 * (xb + lane) + w;
        const int key = kDecKeys * (bi < sp.nb1 ? bi : sp.b2 + bi - sp.nb1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int kt = key + 16 * t;
          pg[t] = -1;
          in[t] = 0;
          const bool seen = xb + lane < xe && kt < sp.L && (kt + 16 > sp.lo || kt < sp.nf);
          if (seen) {
            const int e = kv_entry(a.t, kt);
            const int p = row[e];
            if (p >= 0 && p < a.t.n_pages) {
              pg[t] = p;
              in[t] = kt - e * a.t.ps;
            } else {
              atomicOr(a.err, kErrPage);
            }
          }
        }
      }
      Raw r;
      auto load_k = [&](int xx) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int p = max(0, __builtin_amdgcn_readlane(pg[t], xx - xb));
          const int i = __builtin_amdgcn_readlane(in[t], xx - xb);
          const char* b = kb + p * a.c.sp + i * a.c.st + koff;
#pragma unroll
          for (int c = 0; c < Raw::KL; ++c) r.k[t][c] = *(const u32x4*)(b + 64 * c);
        }
      };
      auto load_v = [&](int xx) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int p = max(0, __builtin_amdgcn_readlane(pg[t], xx - xb));
          const int i = __builtin_amdgcn_readlane(in[t], xx - xb);
          const char* b = vb + p * a.c.sp + i * a.c.st + voff;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t* dst = r.v[4 * t + j];
            const char* src = b + j * a.c.st;
            if constexpr (Raw::VB == 4) {
              dst[0] = *(const uint32_t*)src;
            } else if constexpr (Raw::VB == 8) {
              const u32x2 y = *(const u32x2*)src;
              dst[0] = y[0];
              dst[1] = y[1];
            } else {
#pragma unroll
              for (int h = 0; h < Raw::VB / 16; ++h) {
                // 16-bit D = 256: the second half of the lane's d lies 256 bytes on
                const u32x4 y = *(const u32x4*)(src + h * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[4 * h + e] = y[e];
              }
            }
          }
        }
      };
      load_k(x);
      load_v(x);
      for (; x < xe; ++x) {
        const int bi = 4 * x + w;
        const int key = kDecKeys * (bi < sp.nb1 ? bi : sp.b2 + bi - sp.nb1);
        const int p0 = __builtin_amdgcn_readlane(pg[0], x - xb);
        const int p1 = __builtin_amdgcn_readlane(pg[1], x - xb);
        // every key of the block visible and there
        const bool whole = p0 >= 0 && p1 >= 0 && key + kDecKeys <= sp.L &&
                           (key >= sp.lo || key + kDecKeys <= sp.nf);
        f32x4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            u32x4 ka;
            if constexpr (F8) {
              const u32x4 raw = r.k[t][c >> 1];
              const uint32_t x0 = raw[2 * (c & 1)], x1 = raw[2 * (c & 1) + 1];
              ka = u32x4{from_e4m3<BF, false>(x0), from_e4m3<BF, true>(x0),
                         from_e4m3<BF, false>(x1), from_e4m3<BF, true>(x1)};
            } else {
              ka = r.k[t][c];
            }
            s[t] = mfma16<BF>(ka, q[c], s[t]);
          }
        }
        if (x + 1 < xe) load_k(x + 1);

        float sv[8];
        uint32_t seen = 0xFF;
#pragma unroll
        for (int j = 0; j < 8; ++j) sv[j] = s[j >> 2][j & 3] * sc;
        if (!whole) {
          seen = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int kj = key + 16 * (j >> 2) + 4 * lg + (j & 3);
            const bool ok = (j < 4 ? p0 : p1) >= 0 && kj < sp.L && (kj >= sp.lo || kj < sp.nf);
            if (ok) seen |= 1u << j;
            else sv[j] = kNegInf;
          }
        }
        float bm = sv[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) bm = fmaxf(bm, sv[j]);
        bm = max_across_rows(bm);
        const float mn = fmaxf(m, bm);
        const float mu = mn == kNegInf ? 0.0f : mn;
        const float alpha = exp2_fast(m - mu);
        m = mn;
        float ps = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sv[j] = exp2_fast(sv[j] - mu);
          ps += sv[j];
        }
        l = l * alpha + ps;
#pragma unroll
        for (int t = 0; t < VE; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][i] *= alpha;
        u32x4 pb;
#pragma unroll
        for (int j = 0; j < 4; ++j) pb[j] = pack16<BF>(sv[2 * j], sv[2 * j + 1]);

        if (!whole) {      // what lies in masked places is not to enter, NaN included
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < Raw::VB / 4; ++e)
              r.v[j][e] = (seen >> j) & 1 ? r.v[j][e] : 0;
        }
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          // dword e: values d, d + 1 of the lane's 8 keys
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if constexpr (F8)
              y[j] = e & 1 ? from_e4m3<BF, true>(r.v[j][e >> 1])
                           : from_e4m3<BF, false>(r.v[j][e >> 1]);
            else
              y[j] = r.v[j][e];
          }
          u32x4 lo, hi;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo[j] = pair_lo(y[2 * j], y[2 * j + 1]);
            hi[j] = pair_hi(y[2 * j], y[2 * j + 1]);
          }
          o[2 * e] = mfma16<BF>(lo, pb, o[2 * e]);
          o[2 * e + 1] = mfma16<BF>(hi, pb, o[2 * e + 1]);
        }
        if (x + 1 < xe) load_v(x + 1);
      }
    }

    // join the four waves
    l = xor32_reduce(xor16_reduce(l, OpSum{}), OpSum{});
    if (lg == 0) {
      s_ml[w][0][lc] = m;
      s_ml[w][1][lc] = l;
    }
    if (lc < heads) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < VH; ++h) {
          float* dst = &s_o[w][lc][h * (D / VH) + VW * (4 * lg + i)];
#pragma unroll
          for (int t = 0; t < VW; t += 4)
            *(f32x4*)(dst + t) = f32x4{o[h * VW + t][i], o[h * VW + t + 1][i],
                                       o[h * VW + t + 2][i], o[h * VW + t + 3][i]};
        }
    }
    __syncthreads();
    {
      // thread: head hh, values d0 .. d0 + D / 16 - 1
      const int hh = tid >> 4, d0 = (tid & 15) * VE;
      const bool whole_pair = b0 == 0 && b1 == ns;
      if (hh < heads) {
        float mm = kNegInf;
#pragma unroll
        for (int i = 0; i < 4; ++i) mm = fmaxf(mm, s_ml[i][0][hh]);
        const float mu = mm == kNegInf ? 0.0f : mm;
        float acc[VE], ll = 0.0f;
#pragma unroll
        for (int t = 0; t < VE; ++t) acc[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = exp2_fast(s_ml[i][0][hh] - mu);
          ll += f * s_ml[i][1][hh];
#pragma unroll
          for (int t = 0; t < VE; t += 4) {
            const f32x4 y = *(const f32x4*)&s_o[i][hh][d0 + t];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t + e] += f * y[e];
          }
        }
        const int head = kvh * a.g + hbase + hh;
        if (whole_pair) {
          float inv = ll == 0.0f ? 0.0f : 1.0f / ll;     // no visible key: 0
          if (F8 && ll != 0.0f) inv *= a.c.vs[kvh];
          char* dst = a.out + seq * a.o_row + head * a.o_head + 2 * d0;
#pragma unroll
          for (int t = 0; t < VE; t += 4) {
            u32x2 y = {pack16<BF>(acc[t] * inv, acc[t + 1] * inv),
                       pack16<BF>(acc[t + 2] * inv, acc[t + 3] * inv)};
            *(u32x2*)(dst + 2 * t) = y;
          }
          if (a.lse && (tid & 15) == 0)
            a.lse[(long)seq * a.hq + head] = (mm + __builtin_amdgcn_logf(ll)) * kLn2;
        } else {
          float* slot_p = a.part + (2 * (long)blockIdx.x + (b0 == 0)) * dec_slot_floats(D);
          if ((tid & 15) == 0) {
            slot_p[hh] = mm;
            slot_p[16 + hh] = ll;
          }
#pragma unroll
          for (int t = 0; t < VE; t += 4)
            *(f32x4*)(slot_p + kDecPartRow + hh * D + d0 + t) =
                f32x4{acc[t], acc[t + 1], acc[t + 2], acc[t + 3]};
        }
      }
      if (b0 == 0 && tid == 0) {
        // the workgroup of the pair's last unit: the largest w with w U / W <= unit
        const long last = (long)pre * HT + (long)(hti + 1) * ns - 1;
        const long wl = ((last + 1) * W - 1) / U;
        int* me = a.meta + 2 * ((long)seq * HT + hti);
        me[0] = blockIdx.x;
        me[1] = (int)(wl - blockIdx.x) + 1;
      }
    }
    __syncthreads();
    u += b1 - b0;
    if (hti == HT - 1 && b1 == ns) ++seq;
  }
}

// Joins the parts of the pairs that more than one workgroup had, in their
// order, eight parts' loads in flight: up to eight parts by one wave a head (a
// lane has D / 64 values), more by four waves, each every fourth part.
template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256) void decode_join_kernel(AttnArgs a) {
  constexpr int E = D / 64;
  __shared__ float s_ml[4][2];
  __shared__ float s_o[4][D];
  const int ht = (a.g + 15) >> 4, HT = a.c.hkv * ht;
  const int wg0 = a.meta[2 * (long)blockIdx.x], cnt = a.meta[2 * (long)blockIdx.x + 1];
  if (cnt <= 1) return;
  const int seq = blockIdx.x / HT, hti = blockIdx.x - seq * HT;
  const int kvh = hti / ht, hbase = (hti - kvh * ht) * 16;
  const int heads = min(16, a.g - hbase);
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const size_t sf = dec_slot_floats(D);

  struct State {
    float m, l, o[E];
  };
  // adds parts first, first + stride, ... (at most eight) of head hh
  auto add = [&](State& s, int hh, int first, int stride) {
    float pm[8], pl[8], po[8][E];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = first + stride * k, ii = i < cnt ? i : first;
      const float* p = a.part + (2 * (size_t)(wg0 + ii) + (ii == 0)) * sf;
      pm[k] = i < cnt ? p[hh] : kNegInf;
      pl[k] = p[16 + hh];
#pragma unroll
      for (int e = 0; e < E; ++e) po[k][e] = p[kDecPartRow + hh * D + lane * E + e];
    }
    float mn = s.m;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, pm[k]);
    const float mu = mn == kNegInf ? 0.0f : mn;
    const float f0 = exp2_fast(s.m - mu);
    s.l *= f0;
#pragma unroll
    for (int e = 0; e < E; ++e) s.o[e] *= f0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (first + stride * k < cnt) {
        const float f = exp2_fast(pm[k] - mu);
        s.l += f * pl[k];
#pragma unroll
        for (int e = 0; e < E; ++e) s.o[e] += f * po[k][e];
      }
    }
    s.m = mn;
  };
  auto write = [&](const State& s, int hh) {
    float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
    if (F8 && s.l != 0.0f) inv *= a.c.vs[kvh];
    const int head = kvh * a.g + hbase + hh;
    char* dst = a.out + seq * a.o_row + head * a.o_head;
    if constexpr (E == 1) {
      *(uint16_t*)(dst + 2 * lane) = (uint16_t)pack16<BF>(s.o[0] * inv, 0.0f);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *(uint32_t*)(dst + 2 * (lane * E + e)) = pack16<BF>(s.o[e] * inv, s.o[e + 1] * inv);
    }
    if (a.lse && lane == 0)
      a.lse[(long)seq * a.hq + head] = (s.m + __builtin_amdgcn_logf(s.l)) * kLn2;
  };
  const State none{kNegInf, 0.0f, {}};

  if (cnt <= 8) {
    for (int hh = 4 * blockIdx.y + w; hh < heads; hh += 4 * gridDim.y) {
      State s = none;
      add(s, hh, 0, 1);
      write(s, hh);
    }
    return;
  }
  for (int hh = blockIdx.y; hh < heads; hh += gridDim.y) {
    State s = none;
    for (int first = w; first < cnt; first += 32) add(s, hh, first, 4);
    if (lane == 0) {
      s_ml[w][0] = s.m;
      s_ml[w][1] = s.l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[w][lane * E + e] = s.o[e];
    __syncthreads();
    if (w == 0) {
      State t = none;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.m = fmaxf(t.m, s_ml[i][0]);
      const float mu = t.m == kNegInf ? 0.0f : t.m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = exp2_fast(s_ml[i][0] - mu);
        t.l += f * s_ml[i][1];
#pragma unroll
        for (int e = 0; e < E; ++e) t.o[e] += f * s_o[i][lane * E + e];
      }
      write(t, hh);
    }
    __syncthreads();
  }
}

template <bool BF, bool F8, int D>
hipError_t run_decode(const AttnArgs& a, hipStream_t s) {
  const int ht = (a.g + 15) / 16, HT = a.c.hkv * ht;
  const long cap = (long)a.t.max_pages * a.t.ps;
  const long seen = a.window ? (long)a.window + a.first + 2 * kDecKeys : cap;
  const long units = ((seen < cap ? seen : cap) + kDecUnit - 1) / kDecUnit + 1;
  const long bound = (long)a.n * HT * units;
  const int wgs = dec_wgs(D, F8), grid = (int)(bound < wgs ? bound : wgs);
  attn_decode_kernel<BF, F8, D><<<grid, 256, 0, s>>>(a);
  const long pairs = (long)a.n * HT;
  const dim3 jg((unsigned)pairs, pairs >= 256 ? 1 : (a.g < 16 ? a.g : 16));
  decode_join_kernel<BF, F8, D><<<jg, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t run_decode_d(const AttnArgs& a, int fmt, hipStream_t s) {
  const bool f8 = a.c.fmt == KV_E4M3;
  if (fmt == KV_BF16)
    return f8 ? run_decode<true, true, D>(a, s) : run_decode<true, false, D>(a, s);
  return f8 ? run_decode<false, true, D>(a, s) : run_decode<false, false, D>(a, s);
}

}  // namespace
}  // namespace moe
