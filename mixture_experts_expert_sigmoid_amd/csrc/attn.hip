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
hipError_t launch_latent_256(const AttnArgs& a, int fmt, int grid, hipStream_t s);
hipError_t launch_latent_512(const AttnArgs& a, int fmt, int grid, hipStream_t s);
hipError_t launch_dense_128(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_tree_64(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_tree_128(const AttnArgs& a, int fmt, hipStream_t s);
hipError_t launch_tree_256(const AttnArgs& a, int fmt, hipStream_t s);

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
  if (tiles < 1 || tiles >= 384) return 1;        // (0: a batch without a sequence)
  const long s = (512 + tiles - 1) / tiles;
  return (int)(s < kPreMaxParts ? s : kPreMaxParts);
}

size_t prefill_ws_bytes(long n, long T, int hq, int hkv, int D) {
  const int s = prefill_splits(n, T, hq, hkv);
  return s > 1 ? (size_t)s * T * hq * (D + 2) * 4 : 0;
}

// Trees: parts for as many workgroups as run at a time, whatever the tiles. With
// 384 / 512 / 768 / 1536 of them, us: two trees of 41 and 61 tokens, 64 heads, over
// 50..60 k e4m3 keys 304 / 260 / 298 / 292; 48 of 9..33 over 201..4001 keys 115 /
// 117 / 120 / 120. With head_dim 256, whose workgroups have a CU each, no more than
// fit: a few beyond 256 are a second round (8 trees of 2..23 tokens, 64 heads over 4,
// 1400 keys: 47 us, with 320 workgroups 60). A part of a tree has two tiles of keys at
// least, of a prompt four: one tree over 777 keys 14.9 us against 16.6, three of 1..8
// tokens within a window of 907 31.8 against 29.9.
int tree_splits(long n, long T, int hq, int hkv, int D) {
  const long tiles = prefill_tiles(n, T, hq / hkv) * hkv;
  if (tiles < 1) return 1;
  const long s = D == 256 ? kTreeParts / 2 / tiles : (kTreeParts + tiles - 1) / tiles;
  return (int)(s < 1 ? 1 : s < kPreMaxParts ? s : kPreMaxParts);
}

size_t tree_ws_bytes(long n, long T, int hq, int hkv, int D) {
  const int s = tree_splits(n, T, hq, hkv, D);
  return s > 1 ? (size_t)s * T * hq * (D + 2) * 4 : 0;
}

namespace {
AttnArgs split_prefill(const AttnArgs& all, long most, int part_min) {
  AttnArgs a = all;
  // no more parts than the most keys that a tile can see pay for, so that calls
  // over short tables, or of many rows, need no join
  const long cap = (long)a.t.max_pages * a.t.ps;
  const long span = a.window ? (long)a.window + a.first + kPreRows / a.g + 64 : cap;
  const long nb = (span < cap ? span : cap) / (a.c.D == 256 ? 32 : 64);
  a.split_gain = kSplitGain / ((float)(a.T ? a.T : 1) * a.hq);
  const double pay = __builtin_sqrt((double)nb * a.split_gain);
  if (most > nb / part_min) most = nb / part_min;
  if (most > pay) most = (long)pay;
  a.n_split = most < 1 ? 1 : (int)most;
  return a;
}
}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& all, int fmt, hipStream_t s) {
  const AttnArgs a = split_prefill(all, prefill_splits(all.n, all.T, all.hq, all.hq / all.g), kPartMin);
  return a.c.D == 64    ? launch_prefill_64(a, fmt, s)
         : a.c.D == 128 ? launch_prefill_128(a, fmt, s)
                        : launch_prefill_256(a, fmt, s);
}

hipError_t launch_attn_tree(const AttnArgs& all, int fmt, hipStream_t s) {
  const AttnArgs a = split_prefill(all, tree_splits(all.n, all.T, all.hq, all.hq / all.g, all.c.D),
                                   kTreePartMin);
  return a.c.D == 64    ? launch_tree_64(a, fmt, s)
         : a.c.D == 128 ? launch_tree_128(a, fmt, s)
                        : launch_tree_256(a, fmt, s);
}

hipError_t launch_attn_dense(const AttnArgs& all, int fmt, hipStream_t s) {
  return launch_dense_128(split_prefill(all, prefill_splits(all.n, all.T, all.hq, all.hq), kPartMin),
                          fmt, s);
}

size_t latent_ws_bytes(int D) {
  return (size_t)kLatGrid * (2 * lat_part_floats(D) * 4 + 16);
}

hipError_t launch_attn_latent(const AttnArgs& all, int fmt, hipStream_t s) {
  const int D = all.c.D;
  // a workgroup keeps the prefix sums of its launch's sequences in LDS
  for (long b = 0; b < all.n; b += kLatSeqs) {
    AttnArgs a = all;
    a.n = (int)(all.n - b < kLatSeqs ? all.n - b : kLatSeqs);
    if (a.slots) {
      a.slots += b;
    } else {
      a.t.table += b * a.t.ld;
      a.t.len += b;
      a.t.n_slots -= (int)b;
    }
    if (a.cu) {
      a.cu += b;
    } else {
      a.q += b * a.q_row;
      a.out += b * a.o_row;
      if (a.lse) a.lse += b * a.hq;
      if (a.parent) a.parent += b;
    }
    a.meta = (int*)(a.part + kLatGrid * 2 * lat_part_floats(D));
    // no more workgroups than the table's longest contexts can keep busy
    const long tiles = a.cu ? a.T * a.hq / kLatRows + a.n
                            : a.n * (((long)a.hq + kLatRows - 1) / kLatRows);
    const long units = tiles * ((long)a.t.max_pages * a.t.ps / 32 + 1 + kLatStart);
    const long want = (units + kLatMinUnits - 1) / kLatMinUnits;
    const int grid = (int)(want < kLatGrid ? want : kLatGrid);
    // few tiles, many parts of each: a workgroup a run joins them, else a wave. So / by
    // waves, us: 30 sequences of 16 heads over 1500 keys (8 parts) 39 / 30; 4 of 8 heads
    // over 7..30 k keys (64 parts) 30 / 87.
    a.spread = tiles * kLatFew < grid ? (int)tiles : 0;
    a.teams = grid;
    a.h_inv = ((1u << 22) + a.hq - 1) / a.hq;
    const hipError_t e = D == 256 ? launch_latent_256(a, fmt, grid, s)
                                  : launch_latent_512(a, fmt, grid, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
