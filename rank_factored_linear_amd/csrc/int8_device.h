// 8-bit integers with one scale per row: the number format of the integer
// product, shared by the kernels that make it and those that multiply it.
//
// A row (an activation token, or an output channel of a weight) is held as
// whole numbers -127 .. 127 and one fp32 scale.  With a = max |value| of the row
// and a' = max(a, 2^-100):
//   scale = a' * (1 / 127),  q = round(value * (127 * (1 / a'))),
// each fp32 operation rounded once, ties to even.  The floor keeps 127 / a'
// finite; a row below it is scaled as if its largest value were 2^-100.  q is
// off by at most half of the scale.  A row that holds an infinity or NaN gets a
// NaN scale and zeros: such a row has no finite scale, and a product with it
// must not look valid.
#pragma once

#include "fp8_device.h"

namespace tb {
namespace int8 {

constexpr float kMax = 127.f;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Of a row's largest magnitude (its fp32 bits, sign cleared; as integers
// infinities and NaN are the largest): the stored scale, and the factor that
// values are multiplied by (0 marks a row that has no finite scale).
__device__ __forceinline__ void row_scale(uint32_t amax, float& stored, float& by) {
  const bool finite = amax < 0x7f800000u;
  const float a = fmaxf(__uint_as_float(amax), fp8::kLeast);
  stored = finite ? a * (1.f / kMax) : __builtin_nanf("");
  by = finite ? kMax * (1.f / a) : 0.f;
}

// Four values times by as whole numbers, one to a byte (the first in the
// lowest).  The product is rounded to fp32 before it is rounded to a whole
// number, so it is kept from being fused with the sum.  1.5 * 2^23 + v holds
// round(v) in its low bits, as a signed byte in the lowest.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float by) {
#pragma clang fp contract(off)
  constexpr float kShift = 12582912.f;
  const uint32_t ia = __float_as_uint(a * by + kShift), ib = __float_as_uint(b * by + kShift);
  const uint32_t ic = __float_as_uint(c * by + kShift), id = __float_as_uint(d * by + kShift);
  const uint32_t lo = __builtin_amdgcn_perm(ib, ia, 0x0c0c0400u), hi = __builtin_amdgcn_perm(id, ic, 0x0c0c0400u);
  return by == 0.f ? 0u : lo | hi << 16;
}

// c += A . B of 16 x 64 by 64 x 16 whole numbers.  Lane l gives 16 bytes of A's
// row l % 16 and of B's column l % 16 (which 16 of the 64 k is free as long as A
// and B agree) and receives rows 4 (l / 16) + 0..3 of column l % 16.  Sums are
// 32-bit and exact: 2^16 products of 127 x 127 stay below 2^31.
__device__ __forceinline__ i32x4 mma(fp8::u32x4 a, fp8::u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Behind a group of products.  Each adds to an accumulator that an earlier one
// has added to, and takes operands from registers that vector code may be given
// next: the form that mfma_operand_guard is for.  The integer products have never
// been wrong (every test of them is bit for bit), but the cause in the others is
// not known, so they keep the same distance: products_issued waits behind the
// group's last product, which the sums passed through it keep in front of it.
// Operands that are kept behind it have registers of their own until then.
__device__ __forceinline__ void keep(const fp8::u32x4& operand) { asm volatile("" ::"v"(operand)); }
template <int R, int N>
__device__ __forceinline__ void products_issued(i32x4 (&acc)[R][N]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < N; ++n) asm volatile("" : "+v"(acc[r][n]));
  __builtin_amdgcn_sched_barrier(0);
  mfma_operand_guard();
  __builtin_amdgcn_sched_barrier(0);
}

// Four sums of one token, whose scale is xs, and their outputs' scales ws.
__device__ __forceinline__ f32x4 scaled(i32x4 sum, float xs, const f32x4& ws) {
  f32x4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = float(sum[e]) * (xs * ws[e]);
  return y;
}

}  // namespace int8

// A wave's sum and maximum, in every lane: across the lanes of each sixteen by
// cross-lane adds (neighbours, pairs, then halves of eight and sixteen mirrored,
// which by then hold the same in every lane), across the four sixteens through
// LDS permutes.  The order is fixed.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, false));
}
constexpr int kDppSwap1 = 0xb1, kDppSwap2 = 0x4e, kDppHalfMirror = 0x141, kDppMirror = 0x140;
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp<kDppSwap1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppSwap2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppMirror>(__float_as_uint(v)));
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {   // over sixteen lanes
  v = max(v, dpp<kDppSwap1>(v));
  v = max(v, dpp<kDppSwap2>(v));
  v = max(v, dpp<kDppHalfMirror>(v));
  return max(v, dpp<kDppMirror>(v));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max16(v);
  v = max(v, uint32_t(__shfl_xor(int(v), 16)));
  return max(v, uint32_t(__shfl_xor(int(v), 32)));
}

// Sums and maxima over the threads that hold a row: one wave, or the whole
// workgroup.  Every call uses the other half of `lds`, so one barrier is enough:
// a wave writes a half again only behind the barrier of the call in between,
// which every wave reaches after it has read that half.
constexpr int kRowMaxParts = 64;
struct RowThreads {
  float (*lds)[kRowMaxParts];   // [2][kRowMaxParts]
  int waves;                    // of a row
  int half;

  // Of CH parts, where part c of wave w is number c * waves + w of the row: each
  // is summed over its wave, then they are added in the order of their numbers.
  // So the sum depends on what each part is, not on how the parts are spread over
  // threads.  CH * waves <= kRowMaxParts.
  template <int CH>
  __device__ __forceinline__ float sum(const float (&v)[CH]) {
    float s[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) s[c] = wave_sum(v[c]);
    float t = 0.f;
    if (waves == 1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) t += s[c];
      return t;
    }
    if (threadIdx.x % kWave == 0)
#pragma unroll
      for (int c = 0; c < CH; ++c) lds[half][c * waves + int(threadIdx.x) / kWave] = s[c];
    __syncthreads();
    for (int p = 0; p < CH * waves; ++p) t += lds[half][p];
    half ^= 1;
    return t;
  }
  // Of fp32 bits with the sign cleared.
  __device__ __forceinline__ uint32_t max_bits(uint32_t v) {
    v = wave_max(v);
    if (waves == 1) return v;
    lds[half][threadIdx.x / kWave] = __uint_as_float(v);
    __syncthreads();
    uint32_t m = 0;
    for (int w = 0; w < waves; ++w) m = max(m, __float_as_uint(lds[half][w]));
    half ^= 1;
    return m;
  }
};

}  // namespace tb
