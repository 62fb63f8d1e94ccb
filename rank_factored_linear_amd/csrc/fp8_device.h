// 8-bit blocks: the number formats of the block-scaled product, shared by the
// kernels that make them and those that multiply them.
//
// A block (128 columns of one activation row, or a 128 x 128 block of a
// weight) is held as e4m3 numbers q (4 exponent bits, 3 mantissa bits, largest
// value 448, no infinities) and one scale.  With a = max |value| of the block:
//   power-of-two scale (one byte, exponent + 127):
//       scale = 2^max(ceil(log2(a / 448)), -127),  q = e4m3(value / scale).
//     Nothing is rounded but q itself.
//   fp32 scale, with a' = max(a, 2^-100):
//       scale = a' * (1 / 448),  q = e4m3(value * (448 * (1 / a'))),
//     each fp32 operation rounded once.  The floor keeps 448 / a' finite; a
//     block below it is scaled as if its largest value were 2^-100.
// q rounds to nearest, ties to even: off by at most 2^-4 of the value (2^-10
// of the scale below 2^-6 scales).  A block that holds an infinity or NaN gets
// a NaN scale and NaN in every q: such a value has no finite scale, and a
// product with it must not look valid.
#pragma once

#include "tb_device.h"
#include "tb_host.h"

namespace tb {
namespace fp8 {

constexpr int kBlock = kFp8Block;
constexpr float kMax = 448.f;
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Loads through buffer descriptors.  The range check covers the sum of the lane
// offset and the scalar offset, for loads to registers and for loads to LDS
// (probed on gfx950, inside one allocation, up to scalar offsets far past the
// descriptor): what lies past num_records reads as zeros.  So rows past a tile's
// end may be named by either offset, and kPast names nothing at all.
constexpr unsigned kRsrcFlags = 0x00020000u;  // descriptor word 3: 32-bit data format
constexpr int kPast = int(0x80000000u);       // lane offset past every buffer

typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// One direct-to-LDS load of a wave: 16 bytes per lane, 1 KB at dst.  M0 takes one
// wait state before a load reads it.  Written as assembly so that the compiler
// does not drain it before each LDS read; wait_loads is the wait.
__device__ __forceinline__ void dma(unsigned dst, __amdgpu_buffer_rsrc_t r, int v, int soff) {
  asm volatile("s_mov_b32 m0, %[d]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v], %[r], %[s] offen lds" ::[d] "s"(dst),
               [v] "v"(v), [r] "s"(r), [s] "s"(soff)
               : "memory", "m0");
}
// One scale per lane, four bytes apart in LDS (a byte is widened).
template <int SC>
__device__ __forceinline__ void dma_scale(unsigned dst, __amdgpu_buffer_rsrc_t r, int v, int soff) {
  if constexpr (SC == TB_SCALE_E8M0)
    asm volatile("s_mov_b32 m0, %[d]\n\ts_nop 0\n\tbuffer_load_ubyte %[v], %[r], %[s] offen lds" ::[d] "s"(dst),
                 [v] "v"(v), [r] "s"(r), [s] "s"(soff)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %[d]\n\ts_nop 0\n\tbuffer_load_dword %[v], %[r], %[s] offen lds" ::[d] "s"(dst),
                 [v] "v"(v), [r] "s"(r), [s] "s"(soff)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// At most N of this wave's loads are still out, and its LDS reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Scale storage by scale type.
template <int SC> struct ScaleOf;
template <> struct ScaleOf<TB_SCALE_F32> { typedef float type; };
template <> struct ScaleOf<TB_SCALE_E8M0> { typedef uint8_t type; };
template <int SC> using scale_t = typename ScaleOf<SC>::type;

// A stored scale as fp32 (a power of two down to 2^-127, the latter subnormal).
__device__ __forceinline__ float scale_value(float s) { return s; }
__device__ __forceinline__ float scale_value(uint8_t s) {
  const uint32_t bits = s == 0 ? 0x00400000u : uint32_t(s) << 23;
  return s == 255 ? __builtin_nanf("") : __uint_as_float(bits);
}

// Of a block's largest magnitude (its fp32 bits, sign cleared; as integers
// infinities and NaN are the largest): the stored scale, and the factor that
// values are multiplied by before they are rounded to e4m3.
template <int SC>
__device__ __forceinline__ void block_scale(uint32_t amax, scale_t<SC>& stored, float& by) {
  const bool finite = amax < 0x7f800000u;
  if constexpr (SC == TB_SCALE_E8M0) {
    // 448 = 1.75 * 2^8: a mantissa above 1.75 needs one power more.
    const int e = max(int(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
    stored = finite ? uint8_t(e) : uint8_t(255);
    by = finite ? __uint_as_float(uint32_t(254 - e) << 23) : __builtin_nanf("");
  } else {
    const float a = fmaxf(__uint_as_float(amax), kLeast);
    stored = finite ? a * (1.f / kMax) : __builtin_nanf("");
    by = finite ? kMax * (1.f / a) : __builtin_nanf("");
  }
}

// Four values as e4m3 bytes (the first in the lowest byte).
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// Eight consecutive elements as fp32.
__device__ __forceinline__ void unpack8(const Frag8<bf16_t>& f, float (&t)[8]) {
  const uint32_t w[4] = {f.v.x, f.v.y, f.v.z, f.v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t[2 * e] = __uint_as_float(w[e] << 16);
    t[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Frag8<float>& f, float (&t)[8]) {
  t[0] = f.lo.x; t[1] = f.lo.y; t[2] = f.lo.z; t[3] = f.lo.w;
  t[4] = f.hi.x; t[5] = f.hi.y; t[6] = f.hi.z; t[7] = f.hi.w;
}

// One product of 16 x 128 by 128 x 16 e4m3 numbers, unscaled.  Lane l gives 32
// bytes of A's row l % 16 and of B's column l % 16 (which 32 of the 128 k is
// free as long as A and B agree) and receives rows 4 (l / 16) + 0..3 of column
// l % 16.
//
// EXACT false: the 8-bit matrix instruction.  It adds the eight products of
// each eight consecutive bytes of a lane in fixed point: measured on gfx950,
// every product is cut (towards zero) at 2^-13 of the largest 2^(a + b) in the
// group, a and b the exponents of a product's factors; from there on sums are
// fp32.  A sum is off by at most 7 * 2^-13 of its terms' magnitudes.  For
// normally distributed values that is about 2^-16 of a block's sum, far below
// half a step of bf16 (2^-8 of a value), so a bf16 result does not see it; where
// large terms cancel it does (seven products of 30 beside one of +-448^2, signs
// alternating from group to group: 24192 for 30240), and fp32 results are the way
// to avoid it.
// EXACT true, for fp32 results, which would: the same bytes widened to bf16
// (exact) for four bf16 products, whose sums are fp32 throughout, at half the
// rate.
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// An operand as the instruction takes it.
template <bool EXACT> struct Operand;
template <> struct Operand<false> { i32x8 v; };
template <> struct Operand<true> { bf16x8 v[4]; };

template <bool EXACT>
__device__ __forceinline__ Operand<EXACT> operand(const i32x8& b) {
  Operand<EXACT> r;
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = widen(b[2 * j], b[2 * j + 1]);
  } else {
    r.v = b;
  }
  return r;
}

__device__ __forceinline__ f32x4 mma(const Operand<false>& a, const Operand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Operand<true>& a, const Operand<true>& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

// Behind a group of products.  The exact form is a chain of 16x16x32 ops into
// one accumulator whose operands vector code has just written and will rewrite:
// the case that mfma_operand_guard is for.  So products_issued waits behind the
// group's last op, and the operands are kept past that: until then they have
// registers of their own, which nothing rewrites (the compiler stays free to
// widen one operand while others multiply).  Call products_issued, then keep
// each operand.
__device__ __forceinline__ void keep(const Operand<false>&) {}
__device__ __forceinline__ void keep(const Operand<true>& o) {
#pragma unroll
  for (int j = 0; j < 4; ++j) asm volatile("" ::"v"(o.v[j]));
}
template <bool EXACT> __device__ __forceinline__ void products_issued() {
  if constexpr (EXACT) {
    __builtin_amdgcn_sched_barrier(0);
    mfma_operand_guard();
    __builtin_amdgcn_sched_barrier(0);
  }
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
}

}  // namespace fp8
}  // namespace tb
