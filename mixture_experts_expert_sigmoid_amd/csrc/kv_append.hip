// New keys and values into the pages of a cache. A workgroup takes a few rows
// (tokens): one thread a row finds its page -- sequence, slot, start, table
// entry: four or more dependent loads -- while the others' loads of the rows
// are on their way, then all quantise (e4m3 caches) and store. Bound by HBM
// for prompts (input read once, codes written once), by latency and launch for
// single tokens. Measured: 8 prompts of 500..8001 tokens, 8 heads of 128, into
// e4m3 (223 MB) 62 us, 3.6 TB/s (a large copy: 4.8), into bf16 (297 MB) 65 us,
// 4.6 TB/s; a token of each of 64 sequences 6.8 us a call, 4.2 us of it the
// kernel. 8 rows a workgroup and 4
// loads in flight: 16 rows, 4 rows, 8 or 2 loads were all slower (8: 67 us).
// Rows of a latent cache (a vector and its rotary key, one head, one scale) go the
// same way: 36,000 of them into an e4m3 cache (63 MB) 17.5-18.4 us, 3.4-3.6 TB/s, a
// token of each of 64 sequences 6.5-7.2 us a call, 3.6 us of it the kernel.
#include "common.h"
#include "kv.h"

namespace moe {
namespace {

template <int IN>
__device__ __forceinline__ float in_f32(uint32_t b) {
  if (IN == KV_BF16) return bf16_bits_to_f32(b);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

// four quotients -> four e4m3 codes: saturated to +-448 first (the conversion
// alone gives NaN beyond), NaN -> 0x7F
// (finite: there is none)
__device__ __forceinline__ uint32_t pack4(const float (&q)[4], bool finite) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  uint32_t o = (uint32_t)w;
  if (finite) return o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (q[i] != q[i]) o = (o & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
  return o;
}

constexpr int kMaxRows = 8;      // rows of a workgroup
constexpr int kBatch = 4;        // 16-byte loads of a thread in flight
// The same of a latent cache, whose rows are shorter: 14 rows of 512 + 64 values
// are four units a thread less a part of one. 36,000 rows into an e4m3 cache
// (63 MB) took 17.8 us with 14 rows and 1 load, 18.6 with 2, 20.6 with 4, 18.8
// with 7 rows and 1 load, 19.0 with 28; as above, 21.2.
constexpr int kLatMaxRows = 14;
constexpr int kLatBatch = 1;

// IN: type of the rows; Q: into an e4m3 cache; LAT: a latent cache, whose
// tokens are D values of k and then kLatRope of v, in one array with one scale
template <int IN, bool Q, bool LAT>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int rows) {
  constexpr int B = LAT ? kLatBatch : kBatch;
  __shared__ long s_off[LAT ? kLatMaxRows : kMaxRows];  // place of the row's token; -1: none
  const int upr = a.c.D >> 3;                     // 16-byte units per head, a power of two
  const int lg = __builtin_ctz(upr);
  const int per = LAT ? upr + kLatRope / 8 : 2 * a.c.hkv * upr;      // units per token
  const int tid = threadIdx.x;
  const long r0 = a.row0 + (long)blockIdx.x * rows;
  const int nr = (int)min((long)rows, a.T - r0);

  // unit x of row `row`, 256 units on a time
  int row = tid / per, x = tid - row * per;
  const int step_row = 256 / per, step_x = 256 - step_row * per;
  bool first = true;
  while (true) {
    int br[B], bx[B];
    uint4 in[B];
    bool any = false;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      br[k] = row;
      bx[k] = x;
      in[k] = make_uint4(0, 0, 0, 0);
      if (row < nr) {
        const int kvh = x >> lg, val = LAT ? kvh > 0 : kvh >= a.c.hkv;
        const int h = LAT ? 0 : kvh - val * a.c.hkv;
        const long r = r0 + row;
        in[k] = *(const uint4*)((val ? a.v + r * a.v_row + h * a.v_head
                                     : a.k + r * a.k_row + h * a.k_head) +
                                (x & (upr - 1)) * 16);
        any = true;
      }
      row += step_row;
      x += step_x;
      if (x >= per) {
        x -= per;
        ++row;
      }
    }
    if (first) {
      first = false;
      if (tid < nr) {
        // the sequence of row r: the last i with cu[i] <= r
        const long r = r0 + tid;
        int i = (int)r, at0 = (int)r;
        bool have = true;
        if (a.cu) {
          int lo = 0, hi = a.n - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= r) lo = mid; else hi = mid - 1;
          }
          i = lo;
          at0 = a.cu[i];
          have = r >= at0 && r < a.cu[i + 1];
        }
        long off = -1;
        if (have) {
          const int start = a.start[i], slot = kv_slot(a.slots, i, a.t.n_slots, a.err);
          if (slot >= 0 && start >= 0) {
            const long pos = (long)start + (r - at0);
            int page = -1, e = 0;
            if (pos < (long)a.t.max_pages * a.t.ps) {
              e = kv_entry(a.t, (int)pos);
              page = a.t.table[slot * a.t.ld + e];
            }
            if (page >= 0 && page < a.t.n_pages)
              off = page * a.c.sp + (pos - (long)e * a.t.ps) * a.c.st;
            else
              atomicOr(a.err, kErrPage);
          }
        }
        s_off[tid] = off;
      }
      __syncthreads();
    }
    if (!any) return;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (br[k] >= nr) continue;
      const long off = s_off[br[k]];
      if (off < 0) continue;
      const int kvh = bx[k] >> lg, val = LAT ? 0 : kvh >= a.c.hkv;
      const int h = LAT ? 0 : kvh - val * a.c.hkv;
      const int c8 = LAT ? bx[k] : bx[k] & (upr - 1);
      char* dst = (val ? a.c.v : a.c.k) + off + h * a.c.sh;
      if (Q) {
        // x / s: with y = RN(1 / s), q0 = RN(x y) and the residual r = q0 s - x,
        // exact by FMA, q = RN(q0 - r y). q0 is within 1.5 units of its last
        // place u of x / s, so q0 - r y within 2^-23 u, and q is RN(x / s) but
        // where x / s lies that close to a point halfway between two floats;
        // there it may be the other of the two. The code is the quotient's all
        // the same: it could differ only beside a tie T of the codes (5 bits,
        // 16 <= T < 32), where x 2^a = (T 2^20 +- 1) S + d, |d| <= 8, S the 24
        // bits of s. x has at most 11 bits, so a > 30, which asks for S = j 2^20
        // -+ d and j = T d: but 8 <= j < 16. A zero keeps its sign: r is +0 for
        // zeros of both signs, so q0 - r y is q0. All this in the normal range
        // and for s > 0; other lanes divide. Three operations a value instead of
        // the division's ten.
        const float s = (val ? a.c.vs : a.c.ks)[h];
        const uint32_t w[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
        float f[8];
        bool fast = s >= 0x1p-60f && s <= 0x1p60f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = in_f32<IN>(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFF);
          fast &= f[j] == 0.0f || (fabsf(f[j]) >= 0x1p-60f && fabsf(f[j]) <= 0x1p60f);
        }
        if (fast) {
          const float y = 1.0f / s;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float q0 = __fmul_rn(f[j], y);
            f[j] = __builtin_fmaf(-__builtin_fmaf(q0, s, -f[j]), y, q0);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = f[j] / s;
        }
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float q[4] = {f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]};
          o[j] = pack4(q, fast);
        }
        *(uint2*)(dst + c8 * 8) = make_uint2(o[0], o[1]);
      } else {
        *(uint4*)(dst + c8 * 16) = in[k];
      }
    }
  }
}

template <bool LAT>
hipError_t run_append(const AppendArgs& a, int fmt, hipStream_t s) {
  // a row a workgroup as long as there are few, so that single tokens spread
  // over the CUs; more of them share one lookup's latency for prompts
  constexpr int kMost = LAT ? kLatMaxRows : kMaxRows;
  const int rows = (int)(a.T >= 1024 * kMost ? kMost : a.T < 2048 ? 1 : a.T / 1024);
  const bool q = a.c.fmt == KV_E4M3;
  AppendArgs p = a;
  for (p.row0 = 0; p.row0 < a.T; p.row0 += kMaxGrid * rows) {
    const long left = (a.T - p.row0 + rows - 1) / rows;
    const unsigned grid = (unsigned)(left < kMaxGrid ? left : kMaxGrid);
    if (!q)
      append_kernel<KV_BF16, false, LAT><<<grid, 256, 0, s>>>(p, rows);   // bits only, any type
    else if (fmt == KV_BF16)
      append_kernel<KV_BF16, true, LAT><<<grid, 256, 0, s>>>(p, rows);
    else
      append_kernel<KV_F16, true, LAT><<<grid, 256, 0, s>>>(p, rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int fmt, hipStream_t s) {
  return run_append<false>(a, fmt, s);
}

hipError_t launch_latent_append(const AppendArgs& a, int fmt, hipStream_t s) {
  return run_append<true>(a, fmt, s);
}

}  // namespace moe
