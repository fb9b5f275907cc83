// Upkeep of the pages of a key-value cache: taking free pages (grow, fork),
// giving them back (free, trim, keep), and moving or copying their contents
// (fork, compact, copy_pages, keep).
//
// A page is free when no table entry names it (refs 0), so there is no free
// list: the lowest free pages are found by ranking the zeros of refs. One
// workgroup does that for a call's list of slots, 8192 counts at a time (a
// ballot per 64 of them gives each free page its rank), and stops at the last
// page it needs; a rank's slot is found in the prefix sums of the slots'
// needs. The order is that of the pages and of the list, so the result is the
// same every time.
//
// Measured: free, trim, grow and fork for 96 slots of a pool of 4096 pages 24
// us for the four calls, launches and their latencies (2.7, 3.5, 7.3 and 9.5 us
// on the GPU; that grow looks at the last page's count shows in no figure); compaction of 1.07 GB of pages, read and written, 216 us, and
// copy_pages of 2.15 GB 429 us, 5.0 TB/s, the rate of a large copy.
#include "kv.h"

namespace moe {
namespace {

constexpr int kThreads = 1024;          // of the allocating workgroup
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 8;                 // counts per thread and step
constexpr int kSeg = kThreads * kPer;   // pages per step

// Pools larger than this get their free pages counted per kSeg pages by a
// launch of its own first, and the allocating workgroup passes over segments
// without any.
constexpr int kCountedPool = 65536;

__host__ __device__ __forceinline__ long div_up(long a, long b) { return (a + b - 1) / b; }

// inclusive prefix sum over the workgroup; s_w holds one long per wave
__device__ __forceinline__ long block_scan(long v, long* s_w, long* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int d = 1; d < 64; d <<= 1) {
    const long o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  if (lane == 63) s_w[w] = v;
  __syncthreads();
  long before = 0, all = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) before += s_w[i];
    all += s_w[i];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

struct Scan {
  long pos;      // next page to look at, a multiple of kSeg
};

// Finds the next `total` free pages from sc.pos on and calls put(rank, page)
// for each by some thread; returns how many there were (less than total only
// at the pool's end). s_cnt: one int per wave. seg_free: free pages per kSeg
// pages, or NULL.
template <typename Put>
__device__ long take_free(const int* refs, int P, long total, Scan* sc, int* s_cnt,
                          const int* seg_free, Put put) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  long found = 0;
  long pos = sc->pos;
  while (found < total && pos < P) {
    if (seg_free && seg_free[pos / kSeg] == 0) {
      pos += kSeg;
      continue;
    }
    const long end = min((long)P, pos + kSeg);
    const long first = pos + (long)w * (64 * kPer) + lane;
    uint64_t m[kPer];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long p = first + 64 * k;
      const int r = p < end ? refs[p] : 1;
      m[k] = __ballot(r == 0);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) mine += __popcll(m[k]);
    if (lane == 0) s_cnt[w] = mine;
    __syncthreads();
    long rank = found;
    int all = 0;
    for (int i = 0; i < kWaves; ++i) {
      if (i < w) rank += s_cnt[i];
      all += s_cnt[i];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long r = rank + __popcll(m[k] & ((1ull << lane) - 1));
      if (((m[k] >> lane) & 1) && r < total) put(r, (int)(first + 64 * k));
      rank += __popcll(m[k]);
    }
    found += all;
    // a step with free pages left over is looked at again by the next call
    if (found <= total) pos = end;
  }
  if (found > total) found = total;
  sc->pos = pos;
  return found;
}

// free pages per segment, for large pools
__global__ __launch_bounds__(256) void count_free_kernel(const int* refs, int P, int* seg_free) {
  __shared__ int s[4];
  const long base = (long)blockIdx.x * kSeg;
  int c = 0;
  for (int i = threadIdx.x; i < kSeg; i += 256)
    if (base + i < P) c += refs[base + i] == 0;
  for (int d = 32; d > 0; d >>= 1) c += __shfl_down(c, d);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) seg_free[blockIdx.x] = s[0] + s[1] + s[2] + s[3];
}

// the index of the list entry that rank r falls to: the first with
// incl[i] > r
__device__ __forceinline__ int owner_of(const long* incl, int n, long r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > r) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// One workgroup; bound by latency (a scan of the list, then a step per 8192
// pages looked at). A slot that ends inside a page of another slot too is not let
// on: its next tokens would be written over the other's (keep leaves such slots,
// where it cuts back tokens that a fork shares).
__global__ __launch_bounds__(kThreads) void grow_kernel(KvTable t, const int* slots,
                                                        const int* n_new, int n, int* start,
                                                        const int* seg_free, int* err) {
  __shared__ long s_incl[kThreads];
  __shared__ int s_slot[kThreads], s_have[kThreads], s_need[kThreads];
  __shared__ long s_w[kWaves];
  __shared__ int s_cnt[kWaves];
  Scan sc{0};
  bool spent = false;      // the list has asked for more pages than were free
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x, m = min(n - base, kThreads);
    int slot = -1, L = 0, add = 0;
    long have = 0, need = 0;
    bool full = false, shared = false;
    if (i < n) {
      slot = kv_slot(slots, i, t.n_slots, err);
      L = kv_len(t, slot);
      add = max(0, n_new[i]);
      if (slot >= 0) {
        have = div_up(L, t.ps);
        const long want = div_up((long)L + add, t.ps);
        if (add > 0 && L % t.ps) {
          const int e = t.table[slot * t.ld + kv_entry(t, L)];
          shared = e >= 0 && e < t.n_pages && t.refs[e] > 1;
        }
        full = want > t.max_pages || (!shared && spent && want > have);
        need = full || shared ? 0 : want - have;
      }
    }
    s_slot[threadIdx.x] = slot;
    s_have[threadIdx.x] = (int)have;
    s_need[threadIdx.x] = (int)need;
    long total;
    const long incl = block_scan(need, s_w, &total);
    s_incl[threadIdx.x] = incl;
    __syncthreads();
    const long found =
        take_free(t.refs, t.n_pages, total, &sc, s_cnt, seg_free, [&](long r, int page) {
          const int o = owner_of(s_incl, m, r);
          const long j = r - (s_incl[o] - s_need[o]);
          t.table[s_slot[o] * t.ld + s_have[o] + j] = page;
          t.refs[page] = 1;
        });
    __syncthreads();
    if (i < n) {
      if (need > 0 && incl > found) {
        // the pool ended inside or before this slot's share: what it was
        // given goes back
        full = true;
        for (long j = 0; j < found - (incl - need); ++j) {
          int* e = t.table + slot * t.ld + have + j;
          t.refs[*e] = 0;
          *e = -1;
        }
      }
      const bool ok = slot >= 0 && !full && !shared;
      start[i] = ok ? L : -1;
      if (ok && add > 0) t.len[slot] = L + add;
      if (slot >= 0 && !ok) atomicOr(err, full ? kErrFull : kErrBusy);
    }
    spent |= found < total;
    __syncthreads();
  }
}

// the whole row, kFreePer entries a thread: a caller may have put pages there
// ahead of the slot's tokens
constexpr int kFreePer = 4;

__global__ __launch_bounds__(256) void free_kernel(KvTable t, const int* slots, int* err) {
  const int slot = kv_slot(slots, blockIdx.x, t.n_slots, err);
  if (slot < 0) return;
  int* row = t.table + slot * t.ld;
  int e[kFreePer];
#pragma unroll
  for (int k = 0; k < kFreePer; ++k) {
    const int j = ((int)blockIdx.y * kFreePer + k) * 256 + threadIdx.x;
    e[k] = j < t.max_pages ? row[j] : -1;
  }
#pragma unroll
  for (int k = 0; k < kFreePer; ++k) {
    if (e[k] == -1) continue;
    row[((int)blockIdx.y * kFreePer + k) * 256 + threadIdx.x] = -1;
    if (e[k] >= 0 && e[k] < t.n_pages) atomicSub(&t.refs[e[k]], 1);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) t.len[slot] = 0;
}

__global__ __launch_bounds__(256) void trim_kernel(KvTable t, const int* slots, int window,
                                                   int first, int* err) {
  const int slot = kv_slot(slots, blockIdx.x, t.n_slots, err);
  if (slot < 0) return;
  const long lo = (long)kv_len(t, slot) - window;      // first token that stays
  if (lo <= 0) return;
  int* row = t.table + slot * t.ld;
  const long to = lo / t.ps;                           // pages wholly below lo
  for (long j = div_up(first, t.ps) + threadIdx.x; j < to; j += 256) {
    const int e = row[j];
    if (e < 0) continue;
    row[j] = -1;
    if (e < t.n_pages) atomicSub(&t.refs[e], 1);
  }
}

// fork, first launch: which destinations get a page for their last tokens.
// ws: length of the copy (-1: refused), source and destination page of the
// partly filled last page (-1: none), one of each per pair.
struct ForkPlan {
  int* len;
  int* from;
  int* to;
};

__global__ __launch_bounds__(kThreads) void fork_plan_kernel(KvTable t, const int* src,
                                                             const int* dst, int n, ForkPlan p,
                                                             const int* seg_free, int* err) {
  __shared__ long s_incl[kThreads];
  __shared__ long s_w[kWaves];
  __shared__ int s_cnt[kWaves];
  Scan sc{0};
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x, m = min(n - base, kThreads);
    int L = -1, from = -1;
    if (i < n) {
      const int a = kv_slot(src, i, t.n_slots, err), b = kv_slot(dst, i, t.n_slots, err);
      if (a >= 0 && b >= 0) {
        if (t.len[b] != 0) {
          atomicOr(err, kErrBusy);
        } else {
          L = kv_len(t, a);
          if (L % t.ps) {
            from = t.table[a * t.ld + L / t.ps];
            if (from < 0 || from >= t.n_pages) {
              from = -1;
              atomicOr(err, kErrPage);
            }
          }
        }
      }
    }
    const long need = from >= 0;
    long total;
    const long incl = block_scan(need, s_w, &total);
    s_incl[threadIdx.x] = incl;
    if (i < n) {
      p.from[i] = from;
      p.to[i] = -1;
    }
    __syncthreads();
    const long found =
        take_free(t.refs, t.n_pages, total, &sc, s_cnt, seg_free, [&](long r, int page) {
          p.to[base + owner_of(s_incl, m, r)] = page;
          t.refs[page] = 1;
        });
    if (i < n) {
      if (need && incl > found) {
        L = -1;
        p.from[i] = -1;
        atomicOr(err, kErrFull);
      }
      p.len[i] = L;
    }
    __syncthreads();
  }
}

// second launch, beside the copies: the table rows, lengths and counts of the
// shared pages; one workgroup per pair
__device__ void fork_rows(const KvTable& t, const int* src, const int* dst, const ForkPlan& p,
                          int i) {
  const int L = p.len[i];
  if (L < 0) return;
  const int* from = t.table + src[i] * t.ld;
  int* to = t.table + dst[i] * t.ld;
  const int whole = L / t.ps;
  for (int j = threadIdx.x; j < whole; j += 256) {
    const int e = from[j];
    to[j] = e;
    if (e >= 0 && e < t.n_pages) atomicAdd(&t.refs[e], 1);
  }
  if (threadIdx.x == 0) {
    if (L % t.ps) to[whole] = p.to[i];
    t.len[dst[i]] = L;
  }
}

// ----------------------------------------------------------- page contents
// Copies page from[i] to page to[i] in every array of cl. A workgroup moves
// 256 x NU units of 16 bytes at a time, NU loads of each thread in flight.
// n_dev: the number of pairs in device memory, or NULL (then n). Bound by HBM:
// every byte moved is read once and written once.
template <int NU>
__device__ void copy_pages(const CopyLayers& cl, const int* from, const int* to, long n,
                           const int* n_dev, int n_pages, int* err, int wg, int wgs) {
  if (n_dev) n = *n_dev;
  const int rows = cl.hkv * cl.ps, upr = cl.row_bytes >> 4;
  const int units = rows * upr, parts = (units + 256 * NU - 1) / (256 * NU);
  const int lg = __builtin_ctz(upr);    // 4..32 units in a row
  const int per = parts * cl.n;         // items of a pair
  const long items = n * per;
  for (long it = wg; it < items; it += wgs) {
    const long pair = it / per;
    const int rest = (int)(it - pair * per), part = rest / cl.n, arr = rest - part * cl.n;
    const int a = from[pair], b = to[pair];
    if (a < 0 || b < 0) continue;
    if (a >= n_pages || b >= n_pages) {
      if (err && threadIdx.x == 0) atomicOr(err, kErrPage);
      continue;
    }
    const char* s = cl.p[arr] + a * cl.sp;
    char* d = cl.p[arr] + b * cl.sp;
    uint4 v[NU];
    long off[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = (part * NU + k) * 256 + threadIdx.x;
      if (cl.linear) {
        off[k] = (long)u << 4;
      } else {
        const int row = u >> lg, h = row / cl.ps;
        off[k] = h * cl.sh + (row - h * cl.ps) * cl.st + ((u & (upr - 1)) << 4);
      }
      if (u < units) v[k] = *(const uint4*)(s + off[k]);
    }
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = (part * NU + k) * 256 + threadIdx.x;
      if (u < units) *(uint4*)(d + off[k]) = v[k];
    }
  }
}

// 16 KB a step for many pages, 4 KB for few, which then spread over more CUs
constexpr int kMany = 4, kFew = 1;
// enough workgroups for the copies' loads to cover the memory latency; a
// call with fewer parts launches one each
constexpr long kCopyGrid = 4096;

long copy_items(const CopyLayers& cl, long n, int nu) {
  const long units = (long)cl.hkv * cl.ps * (cl.row_bytes >> 4);
  return n * ((units + 256 * nu - 1) / (256 * nu)) * cl.n;
}
int copy_nu(const CopyLayers& cl, long n) {
  return copy_items(cl, n, kMany) >= 1024 ? kMany : kFew;
}
int copy_grid(const CopyLayers& cl, long n, int nu) {
  const long items = copy_items(cl, n, nu);
  return (int)(items < kCopyGrid ? items : kCopyGrid);
}

template <int NU>
__global__ __launch_bounds__(256) void copy_pages_kernel(CopyLayers cl, const int* from,
                                                         const int* to, long n,
                                                         const int* n_dev, int n_pages,
                                                         int* err) {
  copy_pages<NU>(cl, from, to, n, n_dev, n_pages, err, blockIdx.x, gridDim.x);
}

// the pairs' rows by the first n workgroups, copies by the others
template <int NU>
__global__ __launch_bounds__(256) void fork_kernel(CopyLayers cl, KvTable t, const int* src,
                                                   const int* dst, int n, ForkPlan p) {
  if ((int)blockIdx.x < n)
    fork_rows(t, src, dst, p, blockIdx.x);
  else
    copy_pages<NU>(cl, p.from, p.to, n, nullptr, t.n_pages, nullptr, blockIdx.x - n,
                   gridDim.x - n);
}

hipError_t copy_all(const CopyLayers* cl, int n_cl, const int* from, const int* to, long n,
                    const int* n_dev, int n_pages, int* err, hipStream_t s) {
  for (int i = 0; i < n_cl; ++i) {
    const int nu = copy_nu(cl[i], n), grid = copy_grid(cl[i], n, nu);
    if (grid == 0) continue;
    if (nu == kMany)
      copy_pages_kernel<kMany><<<grid, 256, 0, s>>>(cl[i], from, to, n, n_dev, n_pages, err);
    else
      copy_pages_kernel<kFew><<<grid, 256, 0, s>>>(cl[i], from, to, n, n_dev, n_pages, err);
  }
  return hipGetLastError();
}

// -------------------------------------------------------------------- keep
// The accepted path of a tree of drafted tokens: its j-th token, the a_j-th
// drafted one, goes to place j behind the C tokens of context. a is ascending,
// so a_j >= j, and a token's place lies behind those already written: moved one
// by one in the path's order, each is read before it is overwritten. A thread keeps
// to its 16 bytes of every token, so nothing is to be ordered between threads.
//
// A slot that is to be kept gets its new length with the sign bit set from the
// copy's first workgroup for it, and without from the launch after the copies:
// that one gives pages back, after which refs no longer tell who was to be left.
// Measured: 256 paths of up to 12 tokens in 8 layers of 8 heads of 128 (93 MB) 21 us
// and 4 for the second launch, 4.4 TB/s; 16 paths of up to 5 in 4 layers 6 and 3 us.
struct Path {
  int slot, L, C, m, k;  // tokens now, those before the tree, drafted, accepted
  const int* at;
  bool marked;           // found right by another workgroup
};
constexpr uint32_t kKeptBit = 0x80000000u;

// entry i's path, read and checked by the whole workgroup alike; false: none,
// or one that the slot is to be left for
__device__ bool path_of(const KeepArgs& a, long i, bool tell, Path& p) {
  p.slot = kv_slot(a.slots, (int)i, a.t.n_slots, a.err);
  if (p.slot < 0) return false;
  const int m = a.n_draft[i], c0 = a.cu[i], c1 = a.cu[i + 1];
  // one read for all: the length may be marked meanwhile
  __shared__ int s_len;
  if (threadIdx.x == 0) s_len = a.t.len[p.slot];
  __syncthreads();
  const int len = s_len, cap = a.t.max_pages * a.t.ps;
  const int now = (int)((uint32_t)len & ~kKeptBit);
  p.m = m;
  p.k = c1 - c0;
  p.at = a.path + c0;
  p.marked = len < 0 && now <= cap;
  if (p.marked) {
    p.C = now - p.k;
    p.L = p.C + m;
    // right as checked before it was marked, unless another entry names the slot
    return c0 >= 0 && p.k >= 0 && c1 <= a.n_path && p.C >= 0 && p.k <= m && m <= cap - p.C;
  }
  p.L = max(0, min(len, cap));
  p.C = p.L - m;
  int bad = 0;
  if (c0 < 0 || c1 < c0 || c1 > a.n_path || m < 0 || m > p.L || p.k > m) {
    bad = kErrTree;
  } else {
    const int* row = a.t.table + p.slot * a.t.ld;
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
      const int x = p.at[j];
      if (x <= (j ? p.at[j - 1] : -1) || x >= m) {
        bad |= kErrTree;
      } else if (x != j) {
        const int e = row[kv_entry(a.t, p.C + j)];
        if (e >= 0 && e < a.t.n_pages && a.t.refs[e] > 1) bad |= kErrBusy;
      }
    }
  }
  const int tree = __syncthreads_or(bad & kErrTree), busy = __syncthreads_or(bad & kErrBusy);
  if (!(tree | busy)) return true;
  if (tell && threadIdx.x == 0) atomicOr(a.err, tree ? kErrTree : kErrBusy);
  return false;
}

constexpr int kKeepTokens = 64;         // of a path, found at a time

// Workgroup (i, y): 256 of the 16-byte columns that all arrays' tokens have, of
// entry i. One token after the other: the workgroups of a large batch cover each
// other's latency, and 2, 4, 8 or 16 loads of a thread in flight (each batch read
// before it is written) took longer, with 256 paths of
// up to 12 tokens in 8 layers (93 MB) 39, 38, 48 and 51 us against 29 (copies
// that put the lengths back included), and no less with 1 to 64 paths of up to
// 60. For a step's few tokens the time is that of finding the places (slot ->
// length, path -> entries).
__global__ __launch_bounds__(256) void keep_copy_kernel(CopyLayers cl, KeepArgs a) {
  __shared__ long s_from[kKeepTokens], s_to[kKeepTokens];
  Path p;
  if (!path_of(a, a.i0 + blockIdx.x, blockIdx.y == 0, p)) return;
  if (blockIdx.y == 0 && !p.marked && threadIdx.x == 0)
    a.t.len[p.slot] = (int)((uint32_t)(p.C + p.k) | kKeptBit);
  const int upr = cl.row_bytes >> 4, lg = __builtin_ctz(upr);
  const int per = cl.hkv * upr, col = (int)blockIdx.y * 256 + threadIdx.x;
  const int arr = col / per, u = col - arr * per;
  const bool mine = arr < cl.n;
  char* const base = cl.p[mine ? arr : 0] + (u >> lg) * cl.sh + ((u & (upr - 1)) << 4);
  const int* row = a.t.table + p.slot * a.t.ld;
  auto place = [&](int pos) {
    const int i = kv_entry(a.t, pos), e = row[i];
    return e >= 0 && e < a.t.n_pages ? e * cl.sp + (pos - i * a.t.ps) * cl.st : -1L;
  };
  for (int j0 = 0; j0 < p.k; j0 += kKeepTokens) {
    const int cnt = min(kKeepTokens, p.k - j0);
    if (j0) __syncthreads();
    if ((int)threadIdx.x < cnt) {
      const int j = j0 + threadIdx.x, x = p.at[j];
      long from = -1, to = -1;
      if (x > j && x < p.m) {
        from = place(p.C + x);
        to = place(p.C + j);
        if ((from | to) < 0) {
          atomicOr(a.err, kErrPage);
          from = -1;
        }
      }
      s_from[threadIdx.x] = from;
      s_to[threadIdx.x] = to;
    }
    __syncthreads();
    if (!mine) continue;
    for (int t = 0; t < cnt; ++t)
      if (s_from[t] >= 0) *(uint4*)(base + s_to[t]) = *(const uint4*)(base + s_from[t]);
  }
}

// the lengths, and the pages of rejected tokens given back, once every layer
// has been moved
__global__ __launch_bounds__(256) void keep_kernel(KeepArgs a) {
  Path p;
  if (!path_of(a, blockIdx.x, false, p) || !p.marked) return;
  int* row = a.t.table + p.slot * a.t.ld;
  const int end = (int)div_up(p.L, a.t.ps);
  for (int j = (int)div_up(p.C + p.k, a.t.ps) + threadIdx.x; j < end; j += 256) {
    const int e = atomicExch(&row[j], -1);
    if (e >= 0 && e < a.t.n_pages) atomicSub(&a.t.refs[e], 1);
  }
  if (threadIdx.x == 0) a.t.len[p.slot] = p.C + p.k;
}

// ----------------------------------------------------------------- compact
// ws: hdr {U, pairs}, used pages per segment, holes, movers, rank of each
// page among the movers
struct CompactPlan {
  int* hdr;
  int* seg_used;
  int* holes;
  int* movers;
  int* rank;
};

__global__ __launch_bounds__(kThreads) void count_used_kernel(const int* refs, int P,
                                                              int* seg_used) {
  __shared__ int s[kWaves];
  const long base = (long)blockIdx.x * kSeg;
  int c = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const long p = base + k * kThreads + threadIdx.x;
    c += p < P ? refs[p] > 0 : 0;
  }
  for (int d = 32; d > 0; d >>= 1) c += __shfl_down(c, d);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int all = 0;
    for (int i = 0; i < kWaves; ++i) all += s[i];
    seg_used[blockIdx.x] = all;
  }
}

// one workgroup per segment: free page p < U has rank p - used(p) among the
// holes, used page p >= U rank used(p) - used(U) among the movers, with
// used(p) the number of used pages before p
__global__ __launch_bounds__(kThreads) void rank_kernel(const int* refs, int P, int segs,
                                                        CompactPlan pl, int* n_used) {
  __shared__ long s_w[kWaves];
  __shared__ int s_cnt[kWaves], s_low[kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long wave0 = (long)blockIdx.x * kSeg + (long)w * (64 * kPer), first = wave0 + lane;
  uint64_t m[kPer];
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const long p = first + 64 * k;
    m[k] = __ballot(p < P && refs[p] > 0);
    mine += __popcll(m[k]);
  }
  if (lane == 0) s_cnt[w] = mine;
  long U = 0, base = 0, used_u = 0;
  if (segs == 1) {                       // all from the ballots, no launch before this one
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) U += s_cnt[i];
    int low = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long below = U - (wave0 + 64 * k);
      low += __popcll(below >= 64 ? m[k] : below > 0 ? m[k] & ((1ull << below) - 1) : 0);
    }
    if (lane == 0) s_low[w] = low;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) used_u += s_low[i];
  } else {
    long all = 0, before = 0;
    for (int i = threadIdx.x; i < segs; i += kThreads) {
      const int c = pl.seg_used[i];
      all += c;
      if (i < (int)blockIdx.x) before += c;
    }
    block_scan(all, s_w, &U);
    block_scan(before, s_w, &base);
    // used(U): the segments before U's, and the used pages of its own below U
    const int useg = (int)(U / kSeg);
    long part = 0;
    for (int i = threadIdx.x; i < segs && i < useg; i += kThreads) part += pl.seg_used[i];
    for (long p = (long)useg * kSeg + threadIdx.x; p < U; p += kThreads) part += refs[p] > 0;
    block_scan(part, s_w, &used_u);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    pl.hdr[0] = (int)U;
    pl.hdr[1] = (int)(U - used_u);
    if (n_used) *n_used = (int)U;
  }
  long u = base;
  for (int i = 0; i < w; ++i) u += s_cnt[i];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const long p = first + 64 * k;
    const long up = u + __popcll(m[k] & ((1ull << lane) - 1));
    if (p < P) {
      const bool used = (m[k] >> lane) & 1;
      if (!used && p < U) pl.holes[p - up] = (int)p;
      if (used && p >= U) {
        pl.movers[up - used_u] = (int)p;
        pl.rank[p] = (int)(up - used_u);
      }
    }
    u += __popcll(m[k]);
  }
}

// table entries and counts follow the pages
__device__ void remap(const KvTable& t, const CompactPlan& pl, int wg, int wgs) {
  const int U = pl.hdr[0], K = pl.hdr[1];
  const long stride = (long)wgs * 256, tid = (long)wg * 256 + threadIdx.x;
  for (long i = tid; i < K; i += stride) {
    const int h = pl.holes[i], m = pl.movers[i];
    t.refs[h] = t.refs[m];
    t.refs[m] = 0;
  }
  const long entries = (long)t.n_slots * t.max_pages;
  for (long i = tid; i < entries; i += stride) {
    const long slot = i / t.max_pages;
    int* e = t.table + slot * t.ld + (i - slot * t.max_pages);
    const int p = *e;
    // an entry that names a page without references is not a page in use
    if (p >= U && p < t.n_pages) {
      const int r = pl.rank[p];
      if (r >= 0 && r < K && pl.movers[r] == p) *e = pl.holes[r];
    }
  }
}

// the tables by the first `remaps` workgroups, copies by the others
template <int NU>
__global__ __launch_bounds__(256) void compact_kernel(CopyLayers cl, KvTable t, CompactPlan pl,
                                                      int remaps) {
  if ((int)blockIdx.x < remaps)
    remap(t, pl, blockIdx.x, remaps);
  else
    copy_pages<NU>(cl, pl.movers, pl.holes, 0, pl.hdr + 1, t.n_pages, nullptr,
                   blockIdx.x - remaps, gridDim.x - remaps);
}

inline size_t al16(size_t b) { return (b + 15) & ~(size_t)15; }
inline int segs_of(int P) { return (int)(((long)P + kSeg - 1) / kSeg); }

// free pages per segment of a large pool, or NULL
const int* count_free(const KvTable& t, void* ws, hipStream_t s) {
  if (t.n_pages <= kCountedPool) return nullptr;
  count_free_kernel<<<segs_of(t.n_pages), 256, 0, s>>>(t.refs, t.n_pages, (int*)ws);
  return (const int*)ws;
}

}  // namespace

size_t cache_ws_bytes(int P, long n) {
  const size_t seg = al16((size_t)segs_of(P) * 4);
  const size_t fork = seg + 3 * al16((size_t)n * 4);
  const size_t compact = 16 + seg + 3 * al16((size_t)P * 4);
  return fork > compact ? fork : compact;
}

hipError_t launch_cache_grow(const KvTable& t, const int* slots, const int* n_new, long n,
                             int* start, int* err, void* ws, hipStream_t s) {
  const int* seg = count_free(t, ws, s);
  grow_kernel<<<1, kThreads, 0, s>>>(t, slots, n_new, (int)n, start, seg, err);
  return hipGetLastError();
}

hipError_t launch_cache_free(const KvTable& t, const int* slots, long n, int* err,
                             hipStream_t s) {
  const unsigned parts = (unsigned)((t.max_pages + 256 * kFreePer - 1) / (256 * kFreePer));
  free_kernel<<<dim3((unsigned)n, parts), 256, 0, s>>>(t, slots, err);
  return hipGetLastError();
}

hipError_t launch_cache_trim(const KvTable& t, const int* slots, long n, int window, int first,
                             int* err, hipStream_t s) {
  trim_kernel<<<(int)n, 256, 0, s>>>(t, slots, window, first, err);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const CopyLayers* cl, int n_cl, const KvTable& t, const int* src,
                             const int* dst, long n, int* err, void* ws, hipStream_t s) {
  const int* seg = count_free(t, ws, s);
  char* w = (char*)ws + al16((size_t)segs_of(t.n_pages) * 4);
  const size_t a = al16((size_t)n * 4);
  ForkPlan p{(int*)w, (int*)(w + a), (int*)(w + 2 * a)};
  fork_plan_kernel<<<1, kThreads, 0, s>>>(t, src, dst, (int)n, p, seg, err);
  const int nu = copy_nu(cl[0], n), grid = (int)n + copy_grid(cl[0], n, nu);
  if (nu == kMany)
    fork_kernel<kMany><<<grid, 256, 0, s>>>(cl[0], t, src, dst, (int)n, p);
  else
    fork_kernel<kFew><<<grid, 256, 0, s>>>(cl[0], t, src, dst, (int)n, p);
  return copy_all(cl + 1, n_cl - 1, p.from, p.to, n, nullptr, t.n_pages, nullptr, s);
}

hipError_t launch_cache_keep(const CopyLayers* cl, int n_cl, const KeepArgs& all, long n,
                             hipStream_t s) {
  KeepArgs a = all;
  for (int i = 0; i < n_cl; ++i) {
    const long cols = (long)cl[i].n * cl[i].hkv * (cl[i].row_bytes >> 4);
    const unsigned wgs = (unsigned)div_up(cols, 256);
    const long most = kMaxGrid / wgs;             // entries of one launch
    for (a.i0 = 0; a.i0 < n; a.i0 += most) {
      const unsigned m = (unsigned)(n - a.i0 < most ? n - a.i0 : most);
      keep_copy_kernel<<<dim3(m, wgs), 256, 0, s>>>(cl[i], a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  keep_kernel<<<(unsigned)n, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CopyLayers* cl, int n_cl, const KvTable& t, int* n_used,
                                void* ws, hipStream_t s) {
  const int segs = segs_of(t.n_pages);
  char* w = (char*)ws;
  const size_t a = al16((size_t)t.n_pages * 4);
  CompactPlan pl;
  pl.hdr = (int*)w;
  pl.seg_used = (int*)(w + 16);
  w += 16 + al16((size_t)segs * 4);
  pl.holes = (int*)w;
  pl.movers = (int*)(w + a);
  pl.rank = (int*)(w + 2 * a);
  if (segs > 1) count_used_kernel<<<segs, kThreads, 0, s>>>(t.refs, t.n_pages, pl.seg_used);
  rank_kernel<<<segs, kThreads, 0, s>>>(t.refs, t.n_pages, segs, pl, n_used);
  const long entries = (long)t.n_slots * t.max_pages;
  const long blocks = (entries + 1023) / 1024;
  const int remaps = (int)(blocks < 1024 ? blocks : 1024);
  // at most half of the pool moves
  const long most = t.n_pages / 2;
  const int nu = copy_nu(cl[0], most), grid = remaps + copy_grid(cl[0], most, nu);
  if (nu == kMany)
    compact_kernel<kMany><<<grid, 256, 0, s>>>(cl[0], t, pl, remaps);
  else
    compact_kernel<kFew><<<grid, 256, 0, s>>>(cl[0], t, pl, remaps);
  return copy_all(cl + 1, n_cl - 1, pl.movers, pl.holes, most, pl.hdr + 1, t.n_pages, nullptr,
                  s);
}

hipError_t launch_cache_copy(const CopyLayers* cl, int n_cl, const int* src, const int* dst,
                             long n, int n_pages, int* err, hipStream_t s) {
  return copy_all(cl, n_cl, src, dst, n, nullptr, n_pages, err, s);
}

}  // namespace moe
