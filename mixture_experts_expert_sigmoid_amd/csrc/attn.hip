// Launchers of the attention kernels: workspace layout, the split of large
// batches into launches, the choice of the head_dim instantiation.
#include "kv.h"

namespace moe {

hipError_t launch_decode_64(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_decode_128(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_decode_256(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_prefill_64(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_prefill_128(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_prefill_256(const AttnArgs& a, int fmt, hipStream_t s);

namespace {
inline size_t al16(size_t b) { return (b + 15) & ~(size_t)15; }
size_t dec_part_bytes(long pairs, int g, int D, bool f8) {
  const size_t teams = (size_t)dec_wgs(D, f8) * 4 / dec_team(pairs, D, f8);
  return teams * 2 * (32 + (g < 16 ? g : 16) * D) * 4;
}
}  // namespace

size_t decode_ws_bytes(long n, int hq, int hkv, int D, bool f8) {
  // the first launch of a large batch has the most pairs
  const long m = n < kDecMaxSeqs ? n : kDecMaxSeqs;
  const int g = hq / hkv;
  const long pairs = m * hkv * ((g + 15) / 16);
  return dec_part_bytes(pairs, g, D, f8) + al16((size_t)pairs * 8);
}

hipError_t launch_attn_decode(const AttnArgs& all, int fmt, hipStream_t s) {
  // a workgroup keeps the lengths of its launch's sequences in LDS
  for (long b = 0; b < all.n; b += kDecMaxSeqs) {
    AttnArgs a = all;
    a.n = (int)(all.n - b < kDecMaxSeqs ? all.n - b : kDecMaxSeqs);
    if (a.slots) {
      a.slots += b;
    } else {
      a.t.table += b * a.t.ld;
      a.t.len += b;
      a.t.n_slots -= (int)b;
    }
    a.q += b * a.q_row;
    a.out += b * a.o_row;
    if (a.lse) a.lse += b * a.hq;
    const long pairs = (long)a.n * a.c.hkv * ((a.g + 15) / 16);
    a.meta = (int*)((char*)a.part + dec_part_bytes(pairs, a.g, a.c.D, a.c.fmt == KV_E4M3));
    hipError_t e = a.c.D == 64    ? launch_decode_64(a, fmt, s)
                   : a.c.D == 128 ? launch_decode_128(a, fmt, s)
                                  : launch_decode_256(a, fmt, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// See pre_parts. Measured at 600 / 2400 / 5000 / 10000 / no bound, us: 13
// prompts of 660 tokens, 4 heads of head_dim 256: 61 / 60 / 61 / 64 / 72; 200
// tokens, 32 heads, over 8000 keys 65 / 54 / 48 / 63 / 63; 900 tokens, 16 heads
// of 256: 48 / 44 / 38 / 47 / 47; 16 tokens over 20000 keys 36 / 37 / 38 / 41 / 41.
constexpr float kSplitGain = 5000;

// parts per tile so that about 512 workgroups run
int prefill_splits(long n, long T, int hq, int hkv) {
  const long tiles = prefill_tiles(n, T, hq / hkv) * hkv;
  if (tiles >= 384) return 1;
  const long s = (512 + tiles - 1) / tiles;
  return (int)(s < kPreMaxParts ? s : kPreMaxParts);
}

size_t prefill_ws_bytes(long n, long T, int hq, int hkv, int D) {
  const int s = prefill_splits(n, T, hq, hkv);
  return s > 1 ? (size_t)s * T * hq * (D + 2) * 4 : 0;
}

hipError_t launch_attn_prefill(const AttnArgs& all, int fmt, hipStream_t s) {
  AttnArgs a = all;
  // no more parts than the most keys that a tile can see pay for, so that calls
  // over short tables, or of many rows, need no join
  const long cap = (long)a.t.max_pages * a.t.ps;
  const long span = a.window ? (long)a.window + a.first + kPreRows / a.g + 64 : cap;
  const long nb = (span < cap ? span : cap) / (a.c.D == 256 ? 32 : 64);
  a.split_gain = kSplitGain / ((float)(a.T ? a.T : 1) * a.hq);
  const double pay = __builtin_sqrt((double)nb * a.split_gain);
  long most = prefill_splits(a.n, a.T, a.hq, a.hq / a.g);
  if (most > nb / 4) most = nb / 4;
  if (most > pay) most = (long)pay;
  a.n_split = most < 1 ? 1 : (int)most;
  return a.c.D == 64    ? launch_prefill_64(a, fmt, s)
         : a.c.D == 128 ? launch_prefill_128(a, fmt, s)
                        : launch_prefill_256(a, fmt, s);
}

}  // namespace moe
