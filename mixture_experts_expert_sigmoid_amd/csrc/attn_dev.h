// Device helpers of the attention kernels: 16-bit operand types, matrix
// instructions, e4m3 expansion.
#pragma once
#include "common.h"
#include "kv.h"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// BF: operands are bf16, else f16. Operands are passed as four dwords of
// pairs.
template <bool BF>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <bool BF>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// two fp32 -> a pair of 16-bit values, round to nearest even
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF) {
    bf16x2 r = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, r);
  } else {
    f16x2 r = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, r);
  }
}

// a pair of e4m3 codes (half HI of w) -> a pair of 16-bit values, exact
template <bool BF, bool HI>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
  if constexpr (BF)
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// low / high halves of two dwords: {lo(b), lo(a)} and {hi(b), hi(a)}, a low
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Loads of 16 bytes a lane from base + at straight into LDS, lane l's to LDS address
// `to` + 16 l (base alike in the wave; at below 2^31); those at offsets from `bytes` on
// read nothing and write zeros. The whole offset is the lane's: it alone is what the
// bound is compared with, whatever a scalar offset would do beside it. In assembly,
// since the compiler takes loads into one array of LDS for loads into any, and would
// wait for those in flight wherever LDS is read; they are to be waited for by count
// (wait_counts), before a barrier if other waves read them.
__device__ __forceinline__ uint32_t lds_of(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"      // (m0 has no value to be preserved)
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t bytes, int at,
                                            uint32_t to) {
  auto alike = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); };
  const uint64_t b = (uint64_t)base;
  const u32x4 rsrc = {alike((uint32_t)b), alike((uint32_t)(b >> 32) & 0xFFFFu), alike(bytes),
                      0x00020000u};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(alike(to)), "v"(at), "s"(rsrc)
               : "memory", "m0");
}

// The same from an address of each lane's own, without a bound.
__device__ __forceinline__ void load_lanes_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from)
               : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A value of the result, of the sum l of its row's probabilities: 0 without one,
// whatever infinities the values of keys that score -infinity left in y.
__device__ __forceinline__ float of_sum(float y, float inv, float l) {
  return l == 0.0f ? 0.0f : y * inv;
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;

// A maximum is followed when it has grown by more than 2^kDefer. In f16, whose
// numbers end at 2^-24 and have all their bits from 2^-14 on, probabilities are
// taken 2^kLift times as large, so that many weak keys beside a strong one are
// not lost from the product while they count in the sum; both together stay
// below 2^16. bf16 has the exponents of fp32. Following so much sooner costs
// f16 prompts of 6000 tokens 1 % at head_dim 64 and 128, 5 % at 256 (8 % over
// e4m3), whose O takes three instructions a register to rescale. No lift for a
// maximum (of scores in base 2) whose own rounding could take them past 2^16.
template <bool BF> constexpr float kDefer = BF ? 8.0f : 3.9f;
constexpr float kLift = 12.0f;
template <bool BF>
__device__ __forceinline__ float pre_lift(float m) {
  return !BF && fabsf(m) < 0x1p18f ? kLift : 0.0f;
}

}  // namespace moe
