// New keys and values into the pages of a cache. One thread per 8 values:
// a 16-byte load, the quantisation for e4m3 caches, an 8- or 16-byte store.
// Bound by HBM for prompts (input read once, codes written once) and by the
// launch for single tokens.
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
__device__ __forceinline__ uint32_t pack4(const float (&q)[4]) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  uint32_t o = (uint32_t)w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (q[i] != q[i]) o = (o & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
  return o;
}

// IN: type of the rows; Q: into an e4m3 cache
template <int IN, bool Q>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  const int upr = a.c.D >> 3;                     // 16-byte units per row, a power of two
  const int lg = __builtin_ctz(upr);
  const int per = 2 * a.c.hkv * upr;              // units per token
  const long total = a.T * per, step = (long)gridDim.x * 256;
  for (long u = (long)blockIdx.x * 256 + threadIdx.x; u < total; u += step) {
    const long r = u / per;
    const int x = (int)(u - r * per), c8 = x & (upr - 1);
    const int kvh = x >> lg, val = kvh >= a.c.hkv, h = kvh - val * a.c.hkv;
    // the sequence of row r: the last i with cu[i] <= r
    int i = (int)r;
    int first = (int)r;
    if (a.cu) {
      int lo = 0, hi = a.n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= r) lo = mid; else hi = mid - 1;
      }
      i = lo;
      first = a.cu[i];
      if (r < first || r >= a.cu[i + 1]) continue;
    }
    const char* src = (val ? a.v + r * a.v_row + h * a.v_head : a.k + r * a.k_row + h * a.k_head) +
                      c8 * 16;
    const uint4 in = *(const uint4*)src;
    const int slot = kv_slot(a.slots, i, a.t.n_slots, a.err);
    const int at = a.start[i];
    if (slot < 0 || at < 0) continue;
    const long pos = (long)at + (r - first);
    int page = -1;
    if (pos < (long)a.t.max_pages * a.t.ps) page = a.t.table[slot * a.t.ld + pos / a.t.ps];
    if (page < 0 || page >= a.t.n_pages) {
      atomicOr(a.err, kErrPage);
      continue;
    }
    char* dst = (val ? a.c.v : a.c.k) + page * a.c.sp + h * a.c.sh + (pos % a.t.ps) * a.c.st;
    if (Q) {
      const float s = (val ? a.c.vs : a.c.ks)[h];
      const uint32_t w[4] = {in.x, in.y, in.z, in.w};
      uint32_t o[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f[4] = {in_f32<IN>(w[2 * j] & 0xFFFF) / s, in_f32<IN>(w[2 * j] >> 16) / s,
                            in_f32<IN>(w[2 * j + 1] & 0xFFFF) / s,
                            in_f32<IN>(w[2 * j + 1] >> 16) / s};
        o[j] = pack4(f);
      }
      *(uint2*)(dst + c8 * 8) = make_uint2(o[0], o[1]);
    } else {
      *(uint4*)(dst + c8 * 16) = in;
    }
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, int fmt, hipStream_t s) {
  const long total = a.T * 2 * a.c.hkv * (a.c.D >> 3);
  const long blocks = (total + 255) / 256;
  const int grid = (int)(blocks < 16384 ? blocks : 16384);
  const bool q = a.c.fmt == KV_E4M3;
  if (!q)
    append_kernel<KV_BF16, false><<<grid, 256, 0, s>>>(a);   // bits only, either type
  else if (fmt == KV_BF16)
    append_kernel<KV_BF16, true><<<grid, 256, 0, s>>>(a);
  else
    append_kernel<KV_F16, true><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
