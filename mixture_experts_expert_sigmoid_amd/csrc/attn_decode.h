// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics. Per sequence and key-value head, with the g query heads that
// share it as the columns of Q^T: S^T = K Q^T, p = 2^(S - m) with the running
// maximum m and sum l of a softmax, O^T = V^T P^T, rescaled when m grows.
// One pass over the keys and values, everything else in registers. p is rounded
// to the 16 bits of q for the second product, since the matrix instructions take
// no wider operand at their rate; the sum counts it before. That rounding is of
// the size of the result's own (2^-8 in bf16, 2^-11 in f16): results stand 6-14 %
// further from the 64-bit values than with probabilities of 32 bits.
//
// Layout. A wave takes 32 keys at a time with v_mfma_*_16x16x32. Its K and V
// go straight into its own part of LDS, in loads of whole cache lines (loads
// into the operand registers would take 64 bytes of 16 keys each, half a line,
// and the second half stalled on the first), and no wave waits for another
// while it streams. S^T = K Q^T has a query head in each lane's column (l %
// 16) and 4 keys in its rows, so a lane holds P of 8 keys of one head -- the B
// operand of the second product as it stands, if its 8-key slice of lane group
// l / 16 is taken as keys 4 (l / 16) + 0..3 of both 16-key tiles. V is read
// transposed (ds_read_b64_tr_b16) in that key order; e4m3 values are expanded
// and turned round in the lane.
//
// Split. The keys that each sequence sees are cut into units; the units of all
// (sequence, key-value head) pairs, laid end to end, are dealt out evenly to
// teams whatever the lengths. A team finishes every pair that lies wholly in
// its run; of the first and the last it leaves fp32 partial results that the
// join kernel adds in order. A team is a workgroup (units of four blocks, a
// wave each, joined through LDS), or a single wave where there are many pairs:
// short contexts then run side by side instead of four waves waiting for the
// same few loads. Few pairs that are short by their table or window are not
// split: a workgroup each, and no join kernel (a third of such a call).
//
// Bound: HBM reads of K and V; short contexts by latency (length -> table ->
// keys -> join). Measured: 64 sequences of 201..4001 keys, 8 heads of 128
// (bf16, 567 MB) 111 us, 5.1 TB/s; two of 130 k keys (e4m3, 509 MB) 97 us, 5.2
// TB/s; windows of f16 heads of 64 (402 MB) 90 us, 4.5 TB/s; one sequence of
// 777 keys 10.2 us; 64 of 16 k keys (4.2 GB) 741 us, 5.7 TB/s; head_dim 256, 64 of
// 1500 keys (789 MB, e4m3 395 MB) 151 us and 79 us, 5.2 and 5.0 TB/s. A bare read of pages in scattered order takes 5.5 TB/s.
#pragma once
#include <type_traits>

#include "attn_dev.h"

namespace moe {
namespace {

constexpr int kDecPartRow = 32;       // maxima and sums of 16 heads, before their D floats each

// Probabilities are taken 2^lift times as large, at most 2^15 in f16, whose
// numbers end at 2^-24: keys down to 2^-40 of the largest enter the product,
// where many of them beside one strong key would otherwise count in the sum but
// not in the product (130 k keys at 2^-26: 0.2 %). bf16 has the exponents of
// fp32. Sums and O are as much larger; a quotient of them is not.
template <bool BF> constexpr float kDecLift = BF ? 0.0f : 15.0f;

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
template <int TS>
__device__ __forceinline__ int dec_units(const DecSpan& s) {
  const int u = (s.nb + TS - 1) / TS;
  return u > 0 ? u : 1;               // a sequence without keys still gets its row written
}

// Waits until at most N of the wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Reads of LDS by byte address with their wait in the same statement, ordered
// among the loads into LDS as written (volatile, memory).
template <int T>
__device__ __forceinline__ void lds_read_b128x2(u32x4& a, u32x4& b, uint32_t at) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b)
               : "v"(at), "n"(T)
               : "memory");
}
template <int T>
__device__ __forceinline__ void lds_read_tr16x4(u32x2& a0, u32x2& a1, u32x2& b0, u32x2& b1,
                                                uint32_t a, uint32_t b) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
      "ds_read_b64_tr_b16 %2, %5\n\tds_read_b64_tr_b16 %3, %5 offset:%6\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a0), "=&v"(a1), "=&v"(b0), "=&v"(b1)
      : "v"(a), "v"(b), "n"(T)
      : "memory");
}
template <int VW> struct Dwords { typedef uint32_t type __attribute__((ext_vector_type(VW))); };
template <> struct Dwords<1> { typedef uint32_t type; };
// VW dwords from each of at, at + S, at + 2 S, at + 3 S
template <int VW, int S, typename Words>
__device__ __forceinline__ void lds_read_x4(Words& a, Words& b, Words& c, Words& d, uint32_t at) {
#define MOE_READ4(OP)                                                                       \
  asm volatile(OP " %0, %4\n\t" OP " %1, %4 offset:%5\n\t" OP " %2, %4 offset:%6\n\t" OP  \
                  " %3, %4 offset:%7\n\ts_waitcnt lgkmcnt(0)"                               \
               : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)                                     \
               : "v"(at), "n"(S), "n"(2 * S), "n"(3 * S)                                    \
               : "memory")
  if constexpr (VW == 1) MOE_READ4("ds_read_b32");
  else if constexpr (VW == 2) MOE_READ4("ds_read_b64");
  else MOE_READ4("ds_read_b128");
#undef MOE_READ4
}

template <bool BF, bool F8, int D, int TS>
__global__ __launch_bounds__(256, dec_waves(D, F8)) void attn_decode_kernel(AttnArgs a) {
  constexpr int NC = D / 32;             // 32-deep steps of the first product
  constexpr int ND = D / 16;             // 16-row tiles of O^T
  constexpr int ROW = F8 ? D : 2 * D;    // bytes of a key
  constexpr int UPR = ROW / 16;          // 16-byte units of a key
  constexpr int KI = 16 * UPR / 64;      // loads of a 16-key tile
  constexpr int KB = kDecKeys * ROW;     // bytes of a wave's block of K, and of V
  // a wave's LDS: its blocks of K and V, afterwards its result for the join
  constexpr int OB = 16 * (D + 4) * 4, RB = 2 * KB > OB ? 2 * KB : OB;

  __shared__ int s_pref[kDecMaxSeqs + 1];
  __shared__ int s_len[kDecMaxSeqs];
  __shared__ int s_scan[4];
  __shared__ float s_ml[4][2][16];
  __shared__ __align__(16) char s_wave[4][RB];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
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
      un[k] = dec_units<TS>(dec_span(L, a.window, a.first));
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
  const long teams = (long)gridDim.x * (4 / TS), team = TS == 4 ? blockIdx.x : 4 * blockIdx.x + w;
  const long W = U < teams ? U : teams;
  if (team >= W) return;
  long u = team * U / W, u_end = (team + 1) * U / W;
  int seq = 0;
  if (TS == 4 && a.whole) {
    // a pair for each workgroup
    seq = blockIdx.x / HT;
    const int pre = s_pref[seq], ns = s_pref[seq + 1] - pre;
    u = (long)pre * HT + (blockIdx.x - seq * HT) * ns;
    u_end = u + ns;
  } else {
    // the sequence of unit u: the last i with pref[i] * HT <= u
    int hi = n - 1;
    while (seq < hi) {
      const int mid = (seq + hi + 1) >> 1;
      if ((long)s_pref[mid] * HT <= u) seq = mid; else hi = mid - 1;
    }
  }
  seq = __builtin_amdgcn_readfirstlane(seq);

  // K and V go to LDS 64 units a load, whole cache lines at a time. Unit u of
  // row r lies at u ^ swz(r): a read of the first product takes one unit of 16
  // rows, a transposed one of the second 32 bytes of 16 rows.
  auto k_swz = [](int r) { return r & (UPR < 16 ? UPR - 1 : 15); };
  auto v_swz = [](int r) { return F8 ? 0 : UPR == 8 ? ((r >> 1) & 3) << 1 : (r & 7) << 1; };
  uint32_t k_from[KI], v_from[KI];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = i * (64 / UPR) + lane / UPR;
    k_from[i] = (uint32_t)r * (uint32_t)a.c.st + 16 * (lane % UPR ^ k_swz(r));
    v_from[i] = (uint32_t)r * (uint32_t)a.c.st + 16 * (lane % UPR ^ v_swz(r));
  }
  const uint32_t k_at = lc * ROW + 16 * (lg ^ k_swz(lc));      // turned by 64 bytes a step
  // V: key row v_row of a tile. 16 bits: lane i of 16 reads row i / 4, 4
  // values from 4 (i % 4), and gets column i; e4m3: D / 16 values of row 4 lg
  const int v_row = 4 * lg + (F8 ? 0 : lc >> 2);
  const uint32_t v_at =
      v_row * ROW + (F8 ? lc * (D / 16) : 16 * ((lc & 3) >> 1 ^ v_swz(v_row)) + 8 * (lc & 1));
  char* const my = s_wave[w];
  const uint32_t my_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)my;

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

    // blocks TS x + (w of a team of four) of units x = b0 .. b1 - 1 are this wave's
    const int wt = TS == 4 ? w : 0;
    const int x_end = __builtin_amdgcn_readfirstlane(min(b1, (sp.nb - wt + TS - 1) / TS));
    auto key_of = [&](int x) {
      const int bi = TS * x + wt;
      return kDecKeys * (bi < sp.nb1 ? bi : sp.b2 + bi - sp.nb1);
    };
    // Byte offset in the cache of the two 16-key tiles of the next 64 blocks,
    // a block a lane; negative where a tile has no page or no visible key
    int at0 = b0;
    auto lookup = [&](int x, int t) {
      const int kt = key_of(x) + 16 * t;
      if (x >= x_end || kt >= sp.L || !(kt + 16 > sp.lo || kt < sp.nf)) return -1L;
      const int i = kv_entry(a.t, kt), p = row[i];
      if (p >= 0 && p < a.t.n_pages) return p * a.c.sp + (kt - i * a.t.ps) * a.c.st;
      atomicOr(a.err, kErrPage);
      return -1L;
    };
    long offs[2] = {lookup(b0 + lane, 0), lookup(b0 + lane, 1)};
    struct Place {
      long off[2];                       // 0 without one
      bool there[2];
    };
    auto place_of = [&](int x) {         // x one after another
      if (x - at0 == 64) {
        at0 = x;
        offs[0] = lookup(x + lane, 0);
        offs[1] = lookup(x + lane, 1);
      }
      Place p;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t lo = __builtin_amdgcn_readlane((int)offs[t], x - at0);
        const int hi = __builtin_amdgcn_readlane((int)(offs[t] >> 32), x - at0);
        p.there[t] = hi >= 0;
        p.off[t] = hi >= 0 ? (long)(((uint64_t)(uint32_t)hi << 32) | lo) : 0L;
      }
      return p;
    };

    // head lc of the tile, D values in the order of the K reads
    u32x4 q[NC];
    {
      const char* src = a.q + seq * a.q_row + (long)(kvh * a.g + hbase + lc) * a.q_head;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = F8 ? 64 * (c >> 1) + 16 * lg + 8 * (c & 1) : 32 * c + 8 * lg;
        q[c] = lc < heads ? *(const u32x4*)(src + 2 * d) : u32x4{0, 0, 0, 0};
      }
    }
    const float sc = F8 ? a.scale * a.c.ks[kvh] : a.scale;

    f32x4 o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = f32x4{0, 0, 0, 0};
    float m = kNegInf, l = 0.0f;

    const char* kb = a.c.k + kvh * a.c.sh;
    const char* vb = a.c.v + kvh * a.c.sh;
    auto load = [&](const char* base, const Place& p, const uint32_t (&from)[KI], char* to) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          uint32_t f = from[i];
          asm volatile("" : "+v"(f));    // added by the load, not ahead of it
          __builtin_amdgcn_global_load_lds(
              (const __attribute__((address_space(1))) void*)(base + p.off[t] + f),
              (__attribute__((address_space(3))) void*)(to + (t * KI + i) * 1024), 16, 0, 0);
        }
    };

    // One block: the loads of K and V of block x (place p) have been started,
    // in this order; NEXT: those of block x + 1 (place pn) follow into the same
    // room as soon as each has been read, so that they fly while the block is
    // worked on. Loads complete in their order: all but the newest N are done
    // once vmcnt <= N. The reads are written with their waits (lds_read); left
    // to the compiler, each would wait for every load in flight.
    constexpr int LOADS = 2 * KI;        // of K, and of V
    auto block = [&](auto next, int x, const Place& p, const Place& pn) {
      constexpr bool NEXT = decltype(next)::value;
      const int key = key_of(x);
      // every key of the block visible and there
      const bool whole = p.there[0] && p.there[1] && key + kDecKeys <= sp.L &&
                         (key >= sp.lo || key + kDecKeys <= sp.nf);
      f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
      wait_loads<LOADS>();               // all but V's
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        // 16 bits: steps c and c + 1; e4m3: both in one unit
        u32x4 r[4];                      // [step][tile]
        if constexpr (F8) {
          lds_read_b128x2<16 * ROW>(r[0], r[1], my_at + (k_at ^ (32 * c)));
        } else {
          lds_read_b128x2<16 * ROW>(r[0], r[1], my_at + (k_at ^ (64 * c)));
          lds_read_b128x2<16 * ROW>(r[2], r[3], my_at + (k_at ^ (64 * c + 64)));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            u32x4 ka;
            if constexpr (F8) {
              const uint32_t y0 = r[t][2 * e], y1 = r[t][2 * e + 1];
              ka = u32x4{from_e4m3<BF, false>(y0), from_e4m3<BF, true>(y0),
                         from_e4m3<BF, false>(y1), from_e4m3<BF, true>(y1)};
            } else {
              ka = r[2 * e + t];
            }
            s[t] = mfma16<BF>(ka, q[c + e], s[t]);
          }
      }
      if (NEXT) load(kb, pn, k_from, my);          // K has been read

      float sv[8];
      uint32_t seen = 0xFF;
#pragma unroll
      for (int j = 0; j < 8; ++j) sv[j] = s[j >> 2][j & 3] * sc;
      if (!whole) {
        seen = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int kj = key + 16 * (j >> 2) + 4 * lg + (j & 3);
          const bool ok = p.there[j >> 2] & (kj < sp.L) & ((kj >= sp.lo) | (kj < sp.nf));
          seen |= ok ? 1u << j : 0u;
          sv[j] = ok ? sv[j] : kNegInf;
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
        sv[j] = exp2_fast(BF ? sv[j] - mu : sv[j] - mu + kDecLift<BF>);
        ps += sv[j];
      }
      l = l * alpha + ps;
#pragma unroll
      for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] *= alpha;
      u32x4 pb;
#pragma unroll
      for (int j = 0; j < 4; ++j) pb[j] = pack16<BF>(sv[2 * j], sv[2 * j + 1]);
      // what lies in masked places is not to enter, NaN included: keys of
      // pairs (2 j, 2 j + 1) of the lane
      uint32_t keep[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        keep[j] = ((seen >> (2 * j)) & 1 ? 0xFFFFu : 0u) |
                  ((seen >> (2 * j + 1)) & 1 ? 0xFFFF0000u : 0u);

      wait_loads<NEXT ? LOADS : 0>();    // all but the next K's
      const uint32_t va0 = my_at + KB + v_at;
      if constexpr (F8) {
        constexpr int VW = D / 64;       // dwords of D / 16 values
        uint32_t v[8][VW];
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          typename Dwords<VW>::type y[4];
          lds_read_x4<VW, ROW>(y[0], y[1], y[2], y[3], va0 + 16 * (j >> 2) * ROW);
#pragma unroll
          for (int i = 0; i < 4; ++i) __builtin_memcpy(v[j + i], &y[i], 4 * VW);
        }
#pragma unroll
        for (int e = 0; e < ND / 2; ++e) {
          // values d, d + 1 of the lane's 8 keys, turned to pairs of keys
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            y[j] = e & 1 ? from_e4m3<BF, true>(v[j][e >> 1]) : from_e4m3<BF, false>(v[j][e >> 1]);
          u32x4 lo, hi;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo[j] = pair_lo(y[2 * j], y[2 * j + 1]) & keep[j];
            hi[j] = pair_hi(y[2 * j], y[2 * j + 1]) & keep[j];
          }
          o[2 * e] = mfma16<BF>(lo, pb, o[2 * e]);
          o[2 * e + 1] = mfma16<BF>(hi, pb, o[2 * e + 1]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < ND; t += 2) {
          u32x2 z[4];                    // [tile of O][16-key tile]
          lds_read_tr16x4<16 * ROW>(z[0], z[1], z[2], z[3],
                                    my_at + KB + (v_at ^ (32 * t)),
                                    my_at + KB + (v_at ^ (32 * t + 32)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            u32x4 va = {z[2 * e][0], z[2 * e][1], z[2 * e + 1][0], z[2 * e + 1][1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) va[j] &= keep[j];
            o[t + e] = mfma16<BF>(va, pb, o[t + e]);
          }
        }
      }
      if (NEXT) load(vb, pn, v_from, my + KB);     // V has been read
    };

    if (b0 < x_end) {
      Place p = place_of(b0);
      load(kb, p, k_from, my);
      load(vb, p, v_from, my + KB);
      int x = b0;
      for (; x + 1 < x_end; ++x) {
        const Place pn = place_of(x + 1);
        block(std::true_type{}, x, p, pn);
        p = pn;
      }
      block(std::false_type{}, x, p, p);
    }

    l = xor32_reduce(xor16_reduce(l, OpSum{}), OpSum{});
    const bool whole_pair = b0 == 0 && b1 == ns;
    const int hs = min(16, a.g);         // rows of a slot
    float* const slot_p = a.part + (2 * team + (b0 == 0)) * (kDecPartRow + (long)hs * D);
    if (b0 == 0 && (TS == 4 ? tid : lane) == 0) {
      // the team of the pair's last unit: the largest w with w U / W <= unit
      const long last = (long)pre * HT + (long)(hti + 1) * ns - 1;
      const long wl = ((last + 1) * W - 1) / U;
      int* me = a.meta + 2 * ((long)seq * HT + hti);
      me[0] = (int)team;
      me[1] = (int)(wl - team) + 1;
    }
    const float vs = F8 ? a.c.vs[kvh] : 1.0f;
    if constexpr (TS == 1) {
      if (lc < heads) {
        const int head = kvh * a.g + hbase + lc;
        const float inv = vs / l;
        char* dst = a.out + seq * a.o_row + head * a.o_head;
        float* part = slot_p + kDecPartRow + lc * D;
        // four values of the head from d on; e4m3: row 4 lg + i of tile t is
        // value (D / 16) row + t
        auto put = [&](int d, f32x4 y) {
          if (whole_pair)
            *(u32x2*)(dst + 2 * d) =
                u32x2{pack16<BF>(of_sum(y[0], inv, l), of_sum(y[1], inv, l)),
                      pack16<BF>(of_sum(y[2], inv, l), of_sum(y[3], inv, l))};
          else
            *(f32x4*)(part + d) = y;
        };
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < ND; t += 4)
              put(ND * (4 * lg + i) + t, f32x4{o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]});
        } else {
#pragma unroll
          for (int t = 0; t < ND; ++t) put(16 * t + 4 * lg, o[t]);
        }
        if (lg == 0) {
          if (!whole_pair) {
            slot_p[lc] = m;
            slot_p[16 + lc] = l;
          } else if (a.lse) {
            a.lse[(long)seq * a.hq + head] = (m + (__builtin_amdgcn_logf(l) - kDecLift<BF>)) * kLn2;
          }
        }
      }
    } else {
      // join the four waves
      if (lg == 0) {
        s_ml[w][0][lc] = m;
        s_ml[w][1][lc] = l;
      }
      if (lc < heads) {
        float* dst = (float*)my + lc * (D + 4);
        if constexpr (F8) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < ND; t += 4)
              *(f32x4*)(dst + ND * (4 * lg + i) + t) =
                  f32x4{o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]};
        } else {
#pragma unroll
          for (int t = 0; t < ND; ++t) *(f32x4*)(dst + 16 * t + 4 * lg) = o[t];
        }
      }
      __syncthreads();
      // thread: head hh, values d0 .. d0 + D / 16 - 1
      constexpr int VE = D / 16;
      const int hh = tid >> 4, d0 = (tid & 15) * VE;
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
            const f32x4 y = *(const f32x4*)((const float*)s_wave[i] + hh * (D + 4) + d0 + t);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t + e] += f * y[e];
          }
        }
        const int head = kvh * a.g + hbase + hh;
        if (whole_pair) {
          const float inv = vs / ll;
          char* dst = a.out + seq * a.o_row + head * a.o_head + 2 * d0;
#pragma unroll
          for (int t = 0; t < VE; t += 4) {
            u32x2 y = {pack16<BF>(of_sum(acc[t], inv, ll), of_sum(acc[t + 1], inv, ll)),
                       pack16<BF>(of_sum(acc[t + 2], inv, ll), of_sum(acc[t + 3], inv, ll))};
            *(u32x2*)(dst + 2 * t) = y;
          }
          if (a.lse && (tid & 15) == 0)
            a.lse[(long)seq * a.hq + head] =
                (mm + (__builtin_amdgcn_logf(ll) - kDecLift<BF>)) * kLn2;
        } else {
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
      __syncthreads();
    }
    u += b1 - b0;
    if (hti == HT - 1 && b1 == ns) ++seq;
  }
}

// Joins the parts of the pairs that more than one team had, in their
// order, eight parts' loads in flight: up to eight parts by one wave a head (a
// lane has D / 64 values), more by four waves, each every fourth part.
template <bool BF, bool F8, int D>
__global__ __launch_bounds__(256) void decode_join_kernel(AttnArgs a) {
  constexpr int E = D / 64;
  __shared__ float s_ml[4][2];
  __shared__ float s_o[4][D];
  const int ht = (a.g + 15) >> 4, HT = a.c.hkv * ht;
  const int team0 = a.meta[2 * (long)blockIdx.x], cnt = a.meta[2 * (long)blockIdx.x + 1];
  if (cnt <= 1) return;
  const int seq = blockIdx.x / HT, hti = blockIdx.x - seq * HT;
  const int kvh = hti / ht, hbase = (hti - kvh * ht) * 16;
  const int heads = min(16, a.g - hbase);
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const size_t sf = kDecPartRow + (size_t)min(16, a.g) * D;

  struct State {
    float m, l, o[E];
  };
  // adds parts first, first + stride, ... (at most eight) of head hh
  auto add = [&](State& s, int hh, int first, int stride) {
    float pm[8], pl[8], po[8][E];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = first + stride * k, ii = i < cnt ? i : first;
      const float* p = a.part + (2 * (size_t)(team0 + ii) + (ii == 0)) * sf;
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
    const float inv = (F8 ? a.c.vs[kvh] : 1.0f) / s.l;
    const int head = kvh * a.g + hbase + hh;
    char* dst = a.out + seq * a.o_row + head * a.o_head;
    if constexpr (E == 1) {
      *(uint16_t*)(dst + 2 * lane) = (uint16_t)pack16<BF>(of_sum(s.o[0], inv, s.l), 0.0f);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *(uint32_t*)(dst + 2 * (lane * E + e)) =
            pack16<BF>(of_sum(s.o[e], inv, s.l), of_sum(s.o[e + 1], inv, s.l));
    }
    if (a.lse && lane == 0)
      a.lse[(long)seq * a.hq + head] = (s.m + (__builtin_amdgcn_logf(s.l) - kDecLift<BF>)) * kLn2;
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
hipError_t run_decode(const AttnArgs& all, hipStream_t s) {
  AttnArgs a = all;
  const int ht = (a.g + 15) / 16, HT = a.c.hkv * ht;
  const long pairs = (long)a.n * HT;
  const int ts = dec_team(pairs, D, F8);
  const long cap = (long)a.t.max_pages * a.t.ps;
  const long seen = a.window ? (long)a.window + a.first + 2 * kDecKeys : cap;
  const long units = ((seen < cap ? seen : cap) + ts * kDecKeys - 1) / (ts * kDecKeys) + 1;
  const long bound = (pairs * units * ts + 3) / 4;         // workgroups with anything to do
  const int wgs = dec_wgs(D, F8), grid = (int)(bound < wgs ? bound : wgs);
  a.whole = ts == 4 && pairs <= wgs && dec_whole(pairs, units - 1, D, F8);
  if (a.whole)
    attn_decode_kernel<BF, F8, D, 4><<<(unsigned)pairs, 256, 0, s>>>(a);
  else if (ts == 1)
    attn_decode_kernel<BF, F8, D, 1><<<grid, 256, 0, s>>>(a);
  else
    attn_decode_kernel<BF, F8, D, 4><<<grid, 256, 0, s>>>(a);
  if (a.whole) return hipGetLastError();
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
