// Paged key-value cache: kernel arguments, internal launchers and the device
// helpers that its kernels share. The public entry points in kv_api.hip
// validate the descriptors and fill these.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// err_word bits, equal to the public header's MOE_DEVERR_CACHE_*
constexpr int kErrPage = 0x8, kErrFull = 0x10, kErrBusy = 0x20, kErrTree = 0x40;

enum { KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2 };
inline int kv_esize(int fmt) { return fmt == KV_E4M3 ? 1 : 2; }

struct KvCache {
  char* k;
  char* v;
  long sp, sh, st;       // page, head, token strides in BYTES
  const float* ks;       // E4M3: [hkv] scales
  const float* vs;
  int fmt, n_pages, ps, hkv, D;
};

struct KvTable {
  int* table;
  int* len;
  int* refs;
  long ld;
  int n_slots, max_pages, n_pages, ps;
  uint64_t ps_inv;       // ceil(2^32 / (ps / 16)), see kv_entry
};

struct AttnArgs {
  KvCache c;
  KvTable t;
  const int* slots;      // nullable
  int n;                 // sequences of this launch
  const char* q;
  char* out;
  long q_row, q_head, o_row, o_head;    // strides in BYTES
  float* lse;            // nullable, [rows][hq]
  int hq, g;             // query heads; query heads per key-value head
  float scale;           // softmax scale * log2(e)
  int window, first;
  int* err;
  // prefill
  const int* cu;
  long T;
  int n_split;
  float split_gain;      // see pre_parts
  int n_tiles;           // of a key-value head
  int block0;            // first of all workgroups that this launch runs
  const int* parent;     // of each row, trees only
  uint32_t h_inv;        // latent: see lat_token
  int spread;            // latent: tiles, if they are few, with many parts to be joined
  int teams;             // latent: workgroups of the first launch
  // dense keys (c.k, c.st, c.sh) and values (c.v): rows cu_k[i].. of S, and the
  // values that a key's heads share; strides in bytes
  const int* cu_k;
  long S;
  long v_row, v_head;
  const char* kr;
  long kr_row;
  // decode: every pair is one team's
  int whole;
  // partial results of split rows
  float* part;
  int* meta;
};

// Decode: dec_wgs workgroups, all resident at once on 256 CUs, so that an even
// share of the keys for each is one even pass. More than two of them a CU read
// slower: scattered 16 KB pieces at 5.5 TB/s by 512 workgroups and at 4.9 by
// 1024 (three a CU for head_dim 64, whose pieces are half as long).
constexpr int dec_waves(int D, bool f8) {        // per SIMD, as LDS allows
  return D == 64 ? 4 : D == 128 ? (f8 ? 4 : 2) : (f8 ? 2 : 1);
}
constexpr int dec_wgs(int D, bool f8) {
  return D == 64 ? 768 : dec_waves(D, f8) < 2 ? 256 : 512;
}
// waves of a team: one where there are enough (sequence, key-value head, 16
// query heads) pairs for half of the single waves, else a workgroup. With one
// wave: 512 x 64 keys x 8 heads 46 -> 35.5 us, 256 x 100 keys 33 -> 30.6, 64
// query heads a key-value head 123 -> 80; with a quarter as many pairs as
// waves it lost (64 x 2000 keys of 8 heads 75 -> 80 us).
constexpr int dec_team(long pairs, int D, bool f8) {
  return pairs * 2 >= 4L * dec_wgs(D, f8) ? 1 : 4;
}
// Pairs not split, a workgroup each and no join, if the table or the window
// leaves each of them few units (keys in 128s). Split / not, us: one sequence
// of 500 keys of 8 heads 10.6 / 8.8, of 1000 10.5 / 12.1, e4m3 10.6 / 13.0; 4 x
// 400 keys of head_dim 256 13.5 / 15.3, of 250 12.6 / 11.1. With half as many
// pairs as workgroups and more, 32 x 50..1000 keys 23.5 / 17.4, 56 x 50..1000
// 35 / 31.7.
constexpr bool dec_whole(long pairs, long units, int D, bool f8) {
  const int many = pairs * 2 >= dec_wgs(D, f8) ? 2 : 1;
  return units <= 4 * many && units * (f8 ? D : 2 * D) <= 1024 * many;
}
// Workspace: partial-result slots, two a team (the pair it continues, the one
// it leaves open), of min(16, g) rows of D floats + 16 maxima + 16 sums; and
// one (first team, count) per pair.
constexpr int kDecMaxSeqs = 512;        // sequences per launch
constexpr int kDecKeys = 32;            // keys of one wave's step
size_t decode_ws_bytes(long n, int hq, int hkv, int D, bool f8);
hipError_t launch_attn_decode(const AttnArgs& a, int fmt, hipStream_t s);

// Prefill: tiles of kPreRows rows, a row being a (token, query head) pair of
// one key-value head; when the tiles cannot fill the GPU the keys of each are
// split over up to prefill_splits workgroups, whose partial results (fp32
// rows, maxima, sums) the join kernel adds in order.
constexpr int kPreRows = 128;
// tiles that n sequences of T tokens can have, per key-value head
inline long prefill_tiles(long n, long T, int g) { return T * g / kPreRows + n; }
constexpr int kPreMaxParts = 64;
constexpr int kPartMin = 4, kTreePartMin = 2;   // tiles of keys that a part has at least
int prefill_splits(long n, long T, int hq, int hkv);
size_t prefill_ws_bytes(long n, long T, int hq, int hkv, int D);
hipError_t launch_attn_prefill(const AttnArgs& a, int fmt, hipStream_t s);

// Drafted tokens that form a tree behind the context run through the prompt
// kernels, with ancestors in place of the tokens before.
constexpr int kTreeMax = 256;           // tokens of one tree
constexpr int kTreeParts = 512;         // workgroups that a call's parts are for
size_t tree_ws_bytes(long n, long T, int hq, int hkv, int D);
hipError_t launch_attn_tree(const AttnArgs& a, int fmt, hipStream_t s);
// So do prompts whose keys and values are dense rows.
constexpr int kDenseDim = 128;          // values of a head, and of a key's own
hipError_t launch_attn_dense(const AttnArgs& a, int fmt, hipStream_t s);

// Latent cache: c.D the latent vector's length, one head. A workgroup takes tiles
// of kLatRows rows, a row being a (token, query head) pair; the keys of all tiles,
// laid end to end, are dealt out evenly to at most kLatGrid workgroups.
constexpr int kLatRows = 64;
constexpr int kLatWaves = 8;            // of a workgroup
constexpr int kLatGrid = 256;           // workgroups, one a CU
constexpr int kLatSeqs = 128;           // sequences per launch
constexpr int kLatStart = 7;            // units of 32 keys that a tile's start counts for
// Parts of a tile that a wave by itself joins; measured on either side of it, with 8
// and 64 of them (launch_attn_latent), not near it.
constexpr int kLatFew = 16;
// Units that a workgroup is there for; with 1 / 2 / 3 / 4 / 6, us: one token of 16
// heads over 777 keys 16.5 / 18.0 / 18.6 / 19.1 / 21.3, of 4 sequences over 2400 e4m3
// keys 26.0 / 23.0 / 22.4 / 22.8 / 24.4. The best for neither, and within a tenth of it
// for both.
constexpr int kLatMinUnits = 2;
constexpr long lat_part_floats(int D) { return (long)kLatRows * (D + 2); }
size_t latent_ws_bytes(int D);
hipError_t launch_attn_latent(const AttnArgs& a, int fmt, hipStream_t s);

// Workgroups of 256 threads in one launch: a grid has fewer than 2^32 threads.
// Calls that need more (a list of a million sequences and many heads, rows by
// the hundred million) take several launches.
constexpr long kMaxGrid = 1L << 23;

struct AppendArgs {
  KvCache c;
  KvTable t;
  const int* slots;      // nullable
  const int* start;
  const int* cu;         // nullable
  int n;
  long T;
  const char* k;
  const char* v;
  long k_row, k_head, v_row, v_head;    // bytes
  int* err;
  long row0;             // first row that this launch takes
};
hipError_t launch_append(const AppendArgs& a, int fmt, hipStream_t s);
constexpr int kLatRope = 64;            // rotary values behind a latent vector
hipError_t launch_latent_append(const AppendArgs& a, int fmt, hipStream_t s);

// K and V of up to kCopyLayers layers by pointer; more take more launches
constexpr int kCopyLayers = 32;
struct CopyLayers {
  char* p[2 * kCopyLayers];   // k0, v0, k1, v1, ...
  int n;                      // arrays in p
  long sp, sh, st;            // bytes
  int hkv, ps, row_bytes;     // row_bytes = D * element size
  int linear;                 // a page is one contiguous block
};

hipError_t launch_cache_grow(const KvTable& t, const int* slots, const int* n_new,
                             long n, int* start, int* err, void* ws, hipStream_t s);
hipError_t launch_cache_free(const KvTable& t, const int* slots, long n, int* err,
                             hipStream_t s);
hipError_t launch_cache_trim(const KvTable& t, const int* slots, long n, int window,
                             int first, int* err, hipStream_t s);
hipError_t launch_cache_fork(const CopyLayers* cl, int n_cl, const KvTable& t,
                             const int* src, const int* dst, long n, int* err, void* ws,
                             hipStream_t s);
hipError_t launch_cache_compact(const CopyLayers* cl, int n_cl, const KvTable& t,
                                int* n_used, void* ws, hipStream_t s);
hipError_t launch_cache_copy(const CopyLayers* cl, int n_cl, const int* src,
                             const int* dst, long n, int n_pages, int* err,
                             hipStream_t s);
struct KeepArgs {
  KvTable t;
  const int* slots;      // nullable
  const int* n_draft;
  const int* cu;
  const int* path;
  long n_path;
  long i0;               // first list entry of this launch
  int* err;
};
hipError_t launch_cache_keep(const CopyLayers* cl, int n_cl, const KeepArgs& a, long n,
                             hipStream_t s);
size_t cache_ws_bytes(int n_pages, long n);

// the slot of list entry i, or -1 for none (error bit for one too large)
__device__ __forceinline__ int kv_slot(const int* slots, int i, int n_slots, int* err) {
  const int s = slots ? slots[i] : i;
  if (s >= n_slots) {
    atomicOr(err, kErrPage);
    return -1;
  }
  return s < 0 ? -1 : s;
}

// tokens of a slot, within what its table row can hold
__device__ __forceinline__ int kv_len(const KvTable& t, int slot) {
  if (slot < 0) return 0;
  const int L = t.len[slot];
  const int cap = t.max_pages * t.ps;
  return L < 0 ? 0 : (L > cap ? cap : L);
}

// table entry of token j: j / ps by the reciprocal of ps / 16.
// Exact: j / 16 < 2^24 and the reciprocal's excess is below ps / 16 <= 256
// in units of 2^-32, so the excess of the product stays below one.
__device__ __forceinline__ int kv_entry(const KvTable& t, int j) {
  return (int)(((uint64_t)(uint32_t)(j >> 4) * t.ps_inv) >> 32);
}

}  // namespace moe
