// 8-bit blocks of activations and of weights (the formats are in
// fp8_device.h).
#include "fp8_device.h"
#include "tb_rebuild.h"

namespace tb {

namespace {

using namespace fp8;

constexpr int kThreads = 256;

// ---- activations: one scale per row and 128 columns -------------------------
//
// Sixteen lanes hold a block, eight elements each, so a block is one 16-byte
// (bf16) load, four cross-lane maxima and one 8-byte store per lane: one pass
// over the data, bound by HBM for long inputs and by launch latency for a few
// rows.  A wave takes kSeg blocks of one row (four at a time); the row's
// segments go over blockIdx.y so that a few long rows still fill the chip.
constexpr int kSeg = 8;

template <typename E, int SC>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const E* __restrict__ x, uint8_t* __restrict__ q,
                                                                 scale_t<SC>* __restrict__ scale, ScaleStrides ss,
                                                                 int64_t M, int I, int KB) {
  const int l = int(threadIdx.x) & 63;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / kWave) + (threadIdx.x >> 6);
  if (row >= M) return;
  const E* xr = x + row * I;
  uint8_t* qr = q + row * I;
  Frag8<E> f[kSeg / 4];
#pragma unroll
  for (int p = 0; p < kSeg / 4; ++p) {
    const int c = (int(blockIdx.y) * kSeg + p * 4) * kBlock + l * 8;   // I % 8 == 0: all eight or none
    f[p] = load_frag_if<E>(xr + c, c < I);
  }
#pragma unroll
  for (int p = 0; p < kSeg / 4; ++p) {
    const int kb = int(blockIdx.y) * kSeg + p * 4 + (l >> 4), c = kb * kBlock + (l & 15) * 8;
    float t[8];
    unpack8(f[p], t);
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = max(a, abs_bits(t[e]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2) a = max(a, uint32_t(__shfl_xor(int(a), d)));
    scale_t<SC> st;
    float by;
    block_scale<SC>(a, st, by);
    if (c < I)
      *reinterpret_cast<u32x2*>(qr + c) = u32x2{pack4(t[0] * by, t[1] * by, t[2] * by, t[3] * by),
                                                pack4(t[4] * by, t[5] * by, t[6] * by, t[7] * by)};
    if ((l & 15) == 0 && kb < KB) scale[row * ss.token + kb * ss.block] = st;
  }
}

// ---- weights: W = diag(s) W0 + U V^T, one scale per 128 x 128 block ---------
//
// One workgroup makes one block: the product U V^T on the matrix cores, then
// through LDS (fp32) so that sixteen lanes cover a row of 128: W0 is read in
// 16- or 32-byte pieces per lane and the e4m3 bytes leave 128 to a row.  The
// W0 loads are issued ahead of the product's; loads retire in order, so its first
// step waits for them as well.  Each thread
// keeps its 64 rebuilt values in registers between the block's maximum and
// their rounding, so W is formed once, in fp32, and never written wide: bf16
// bundles move 3 bytes per weight through HBM.  This kernel serves fp32 bundles,
// ranks that the ring kernel below does not take, and dense weights, where there
// is no product (8192 x 5376: 29 us in bf16, 37 us in fp32).
constexpr int kPitch = 132;  // floats per row of the tile in LDS: 16-byte aligned, rows 4 banks apart

// The fp32 product of a block with rank % 4 == 0: four waves of 64 x 64 in
// v_mfma_f32_32x32x2_f32, k-tiles of 32 in two LDS buffers, the next one in
// registers meanwhile.  A lane reads four consecutive k of a row for four
// products, lanes 0..31 the first four of eight and lanes 32..63 the others:
// U and V are paired alike, so only the order of the sum is another.  Rows are
// 36 floats apart, so sixteen rows' pieces of four meet all 64 banks.
//
// Calls, beside four 64 x 64 products without prefetch (kAny, which other ranks
// still take): 21504 x 5376 rank 256: 546 us (1166), 108 TFLOP/s against 138 of
// a library product; 4096 x 5376 rank 64: 52 (79), 21469 x 432 rank 128: 44
// (88). At rank 64 neither the matrix rate (20 us) nor HBM (22) is reached;
// what holds it there was not measured.
namespace f128 {

constexpr int kStep = 32, kRow = 36, kOpFloats = kBlock * kRow;
constexpr int kLdsBytes = 2 * 2 * kOpFloats * 4;   // [buffer][U, V]
using f32x16 = rebuild::t128::f32x16;

__device__ __forceinline__ void product(const float* u, const float* v, int O, int I, int R, int o0, int i0,
                                        float* lds, f32x16 (&acc)[2][2]) {
  const int tid = int(threadIdx.x), w = tid >> 6, l = tid & 63, h = l >> 5, lr = l & 31;
  const int wi = w & 1, wo = w >> 1, row0 = tid >> 3, piece = (tid & 7) * 4;
  f32x4 next[2][4];
  auto load = [&](int k0) {
    const int k = k0 + piece;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + 32 * j;
      const f32x4 none = {0.f, 0.f, 0.f, 0.f};
      next[0][j] = o0 + row < O && k < R ? *reinterpret_cast<const f32x4*>(u + size_t(o0 + row) * R + k) : none;
      next[1][j] = i0 + row < I && k < R ? *reinterpret_cast<const f32x4*>(v + size_t(i0 + row) * R + k) : none;
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int op = 0; op < 2; ++op)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(lds + (2 * buf + op) * kOpFloats + (row0 + 32 * j) * kRow + piece) = next[op][j];
  };
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.f;
  load(0);
  store(0);
  __syncthreads();
  int buf = 0;
  for (int k0 = 0; k0 < R; k0 += kStep, buf ^= 1) {
    const bool more = k0 + kStep < R;
    if (more) load(k0 + kStep);
    const float* lu = lds + 2 * buf * kOpFloats + (wo * 64 + lr) * kRow + 4 * h;
    const float* lv = lds + (2 * buf + 1) * kOpFloats + (wi * 64 + lr) * kRow + 4 * h;
#pragma unroll
    for (int kk = 0; kk < kStep; kk += 8) {
      f32x4 fu[2], fv[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        fu[b] = *reinterpret_cast<const f32x4*>(lu + b * 32 * kRow + kk);
        fv[b] = *reinterpret_cast<const f32x4*>(lv + b * 32 * kRow + kk);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int cb = 0; cb < 2; ++cb)
            acc[rb][cb] = __builtin_amdgcn_mfma_f32_32x32x2f32(fv[rb][e], fu[cb][e], acc[rb][cb], 0, 0, 0);
    }
    // The other buffer's readers passed the barrier that ended the last step.
    if (more) store(buf ^ 1);
    __syncthreads();
  }
}

}  // namespace f128

enum Product { kNone, kMfma, kMfma32, kAny };

template <typename EI, int SC, int PROD>
__global__ __launch_bounds__(kThreads, 2) void rebuild_blocks_kernel(const EI* __restrict__ s,
                                                                     const EI* __restrict__ w0,
                                                                     const EI* __restrict__ u,
                                                                     const EI* __restrict__ v,
                                                                     uint8_t* __restrict__ q,
                                                                     scale_t<SC>* __restrict__ scale, int O, int I,
                                                                     int R, int KB) {
  constexpr int kTile = PROD == kNone ? 16 : PROD == kMfma32 ? f128::kLdsBytes : kBlock * kPitch * 4;
  static_assert(f128::kLdsBytes >= kBlock * kPitch * 4, "the tile fits the fp32 product's staging");
  static_assert(kTile == 16 || kTile >= rebuild::t128::kLdsBytes, "the product's staging fits the tile's room");
  __shared__ __attribute__((aligned(16))) unsigned char lds[kTile];
  __shared__ uint32_t wave_max[kThreads / kWave];
  const int tid = int(threadIdx.x), w = tid >> 6, l = tid & 63;
  const int ob = int(blockIdx.x) / KB, kb = int(blockIdx.x) % KB;
  const int o0 = ob * kBlock, i0 = kb * kBlock;
  const int c = (tid & 15) * 8, r0 = tid >> 4;   // thread: columns c..c+7 of rows r0 + 16 p

  Frag8<EI> f[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int o = o0 + r0 + 16 * p;
    f[p] = load_frag_if<EI>(w0 + size_t(o) * I + i0 + c, o < O && i0 + c < I);   // I % 8 == 0
  }

  float* tile = reinterpret_cast<float*>(lds);
  if constexpr (PROD == kMfma || PROD == kMfma32) {
    namespace t = rebuild::t128;
    t::f32x16 acc[2][2];
    if constexpr (PROD == kMfma32)
      f128::product(u, v, O, I, R, o0, i0, tile, acc);
    else
      t::product(u, v, O, I, R, o0, i0, lds, acc);
    __syncthreads();   // every wave has read the last k-tile
    const int wi = w & 1, wo = w >> 1, h = l >> 5, lr = l & 31;
#pragma unroll
    for (int cb = 0; cb < 2; ++cb)
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const t::f32x16& a = acc[rb][cb];
          *reinterpret_cast<f32x4*>(tile + (wo * 64 + cb * 32 + lr) * kPitch + wi * 64 + rb * 32 + 8 * b + 4 * h) =
              f32x4{a[4 * b], a[4 * b + 1], a[4 * b + 2], a[4 * b + 3]};
        }
    __syncthreads();
  } else if constexpr (PROD == kAny) {
    namespace t = rebuild::t64;
    for (int qd = 0; qd < 4; ++qd) {
      const int to = (qd >> 1) * t::BT, ti = (qd & 1) * t::BT;
      f32x4 acc[4];
      t::product<EI>(u, v, O, I, R, o0 + to, i0 + ti, acc);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tile[(to + w * 16 + (l >> 4) * 4 + e) * kPitch + ti + ct * 16 + (l & 15)] = acc[ct][e];
    }
    __syncthreads();
  }

  float val[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int row = r0 + 16 * p, o = o0 + row;
    unpack8(f[p], val[p]);
    const float so = s != nullptr && o < O ? to_f32<EI>(s[o]) : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = s != nullptr ? so * val[p][e] : val[p][e];
      if constexpr (PROD != kNone) t = tile[row * kPitch + c + e] + t;
      val[p][e] = t;
      // Rows and columns past the matrix hold zeros (W0, U and V read as zero there).
      a = max(a, abs_bits(t));
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) a = max(a, uint32_t(__shfl_xor(int(a), d)));
  if (l == 0) wave_max[w] = a;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kThreads / kWave; ++j) a = max(a, wave_max[j]);
  scale_t<SC> st;
  float by;
  block_scale<SC>(a, st, by);
  if (tid == 0) scale[size_t(ob) * KB + kb] = st;
  if (i0 + c >= I) return;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int o = o0 + r0 + 16 * p;
    if (o >= O) continue;
    const float(&t)[8] = val[p];
    *reinterpret_cast<u32x2*>(q + size_t(o) * I + i0 + c) =
        u32x2{pack4(t[0] * by, t[1] * by, t[2] * by, t[3] * by), pack4(t[4] * by, t[5] * by, t[6] * by, t[7] * by)};
  }
}

// ---- bf16 bundles with rank % 8 == 0, up to 256 ------------------------------
//
// The same block per workgroup, with U and V coming in k-tiles of 32 straight
// into a ring of three LDS slots of 16 KB, two k-tiles ahead, and the product
// passing through LDS in two halves, so that three workgroups fit a compute
// unit and hide each other's waits.
//
// 21504 x 5376 at rank 256: 120 to 135 us by card and clock (2.6 to 2.9 TB/s of
// W0 read and e4m3 written; staged through registers, two workgroups per compute
// unit: 154 us). HBM does not bound it (8192 x 5376 at rank 64: 3.7 TB/s; rank 0:
// 4.5 TB/s). Counters at rank 256: 10300 cycles of a compute unit per block,
// matrix units busy 20 % of them, vector instructions 26 %, LDS reads and writes
// of the waves 19 % with no bank conflict; waves spend 45 % of their cycles in
// waits and 35 % ready but not issued. No unit is full; which wait costs most was
// not measured (direct-to-LDS writes and L1 are not in these counters). One of
// them is for W0: a wave's loads retire in order, so the first k-tile's wait is
// for W0 too. U and V through registers with three workgroups a unit took 125 us,
// two persistent workgroups that keep loading across blocks 153.
namespace ring {

constexpr int BK = 32, kRingSlots = 3;
constexpr int kOpBytes = kBlock * BK * 2;      // one operand's k-tile: 128 rows of 64 bytes
constexpr int kSlotBytes = 2 * kOpBytes;
constexpr int kLds = kRingSlots * kSlotBytes;
static_assert(kLds >= 64 * kPitch * 4, "half a tile of fp32 fits the ring's room");

typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef rebuild::t128::f32x16 f32x16;

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Two direct-to-LDS loads: load j fills 1 KB at dst + j KB, lane l at + 16 l.
__device__ __forceinline__ void dma2(unsigned dst, __amdgpu_buffer_rsrc_t r, int v0, int v1, int soff) {
  asm volatile(
      "s_mov_b32 m0, %[d0]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[v0], %[r], %[so] offen lds\n\t"
      "s_mov_b32 m0, %[d1]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[v1], %[r], %[so] offen lds"
      :
      : [d0] "s"(dst), [d1] "s"(dst + 1024u), [v0] "v"(v0), [v1] "v"(v1), [r] "s"(r), [so] "s"(soff)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// KT: k-tiles of the rank (those past it load zeros).
template <int SC, int KT>
__global__ __launch_bounds__(kThreads, 3) void rebuild_ring_kernel(const bf16_t* __restrict__ s,
                                                                   const bf16_t* __restrict__ w0,
                                                                   const bf16_t* __restrict__ u,
                                                                   const bf16_t* __restrict__ v,
                                                                   uint8_t* __restrict__ q,
                                                                   scale_t<SC>* __restrict__ scale, int O, int I,
                                                                   int R, int KB) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  __shared__ uint32_t wave_max[kThreads / kWave];
  lds_byte* const base = (lds_byte*)lds;
  const int tid = int(threadIdx.x), w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int ob = int(blockIdx.x) / KB, kb = int(blockIdx.x) % KB;
  const int o0 = ob * kBlock, i0 = kb * kBlock;
  const int c = (tid & 15) * 8, r0 = tid >> 4;   // epilogue: columns c..c+7 of rows r0 + 16 p

  // A wave fills rows 32 w + 16 j + l / 4 of a k-tile; chunk c of row r sits at
  // c ^ ((r >> 2) & 3), so that fragment reads of 16 rows meet all banks.
  const unsigned dst = unsigned(uintptr_t(base)) + unsigned(w) * 2048u;
  const int drow = w * 32 + (l >> 2), dc = (l & 3) ^ ((l >> 4) & 3);
  const int orows = min(O - o0, kBlock), irows = min(I - i0, kBlock);
  const __amdgpu_buffer_rsrc_t ru =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t*>(u + size_t(o0) * R), 0, orows * R * 2, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rv =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t*>(v + size_t(i0) * R), 0, irows * R * 2, kRsrcFlags);
  auto issue = [&](int slot, int kt) {
    const bool ok = dc * 8 < R - kt * BK;
    const int a0 = drow * R * 2 + dc * 16, a1 = a0 + 32 * R;
    dma2(dst + slot * kSlotBytes, ru, ok ? a0 : kPast, ok ? a1 : kPast, kt * BK * 2);
    dma2(dst + slot * kSlotBytes + kOpBytes, rv, ok ? a0 : kPast, ok ? a1 : kPast, kt * BK * 2);
  };

  // W0 first.  Loads retire in order, so the first step's wait below is for W0 as
  // well: it hides behind the other workgroups of the compute unit, not behind
  // this one's product.
  Frag8<bf16_t> f[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int o = o0 + r0 + 16 * p;
    f[p] = load_frag_if<bf16_t>(w0 + size_t(o) * I + i0 + c, o < O && i0 + c < I);   // I % 8 == 0
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int e = 0; e < kRingSlots - 1; ++e)
    if (e < KT) issue(e, e);

  const int wi = w & 1, wo = w >> 1, h = l >> 5, lr = l & 31;
  f32x16 acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.f;

#pragma unroll
  for (int st = 0; st < KT; ++st) {
    // Loads land in order: k-tile st has when at most the four of the next one are out.
    if (st + 1 < KT) wait_loads<4>();
    else wait_loads<0>();
    __builtin_amdgcn_s_barrier();   // published; and every wave has left the slot filled next
    if (st + kRingSlots - 1 < KT) issue((st + kRingSlots - 1) % kRingSlots, st + kRingSlots - 1);
    __builtin_amdgcn_sched_barrier(0);
    const int off = (st % kRingSlots) * kSlotBytes;
    u32x4 fv[2][2], fu[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) {
        const int pos = ((ks * 2 + h) ^ ((lr >> 2) & 3)) << 4;
        fv[rb][ks] = *reinterpret_cast<const lds_u32x4*>(base + off + kOpBytes + (wi * 64 + rb * 32 + lr) * 64 + pos);
        fu[rb][ks] = *reinterpret_cast<const lds_u32x4*>(base + off + (wo * 64 + rb * 32 + lr) * 64 + pos);
      }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int cb = 0; cb < 2; ++cb)
          acc[rb][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fv[rb][ks]),
                                                                __builtin_bit_cast(bf16x8, fu[cb][ks]), acc[rb][cb], 0,
                                                                0, 0);
    __builtin_amdgcn_sched_barrier(0);
    mfma_operand_guard();
    __builtin_amdgcn_sched_barrier(0);
  }

  // The product through LDS, 64 rows at a time: waves 2 half, 2 half + 1 hold
  // them (columns in fours per lane), every thread then takes eight columns of
  // its rows.
  float val[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
    if (wo == half) {
#pragma unroll
      for (int cb = 0; cb < 2; ++cb)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const f32x16& m = acc[rb][cb];
            *reinterpret_cast<lds_f32x4*>(base + ((cb * 32 + lr) * kPitch + wi * 64 + rb * 32 + 8 * b + 4 * h) * 4) =
                f32x4{m[4 * b], m[4 * b + 1], m[4 * b + 2], m[4 * b + 3]};
          }
    }
    __syncthreads();
#pragma unroll
    for (int pp = 0; pp < 4; ++pp) {
      const int p = half * 4 + pp, o = o0 + r0 + 16 * p;
      const f32x4 lo = *reinterpret_cast<const lds_f32x4*>(base + ((r0 + 16 * pp) * kPitch + c) * 4);
      const f32x4 hi = *reinterpret_cast<const lds_f32x4*>(base + ((r0 + 16 * pp) * kPitch + c + 4) * 4);
      unpack8(f[p], val[p]);
      const float so = s != nullptr && o < O ? to_f32<bf16_t>(s[o]) : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        val[p][e] = so * val[p][e] + (e < 4 ? lo[e & 3] : hi[e & 3]);
        a = max(a, abs_bits(val[p][e]));
      }
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) a = max(a, uint32_t(__shfl_xor(int(a), d)));
  if (l == 0) wave_max[w] = a;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kThreads / kWave; ++j) a = max(a, wave_max[j]);
  scale_t<SC> st;
  float by;
  block_scale<SC>(a, st, by);
  if (tid == 0) scale[size_t(ob) * KB + kb] = st;
  if (i0 + c >= I) return;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int o = o0 + r0 + 16 * p;
    if (o >= O) continue;
    const float(&t)[8] = val[p];
    *reinterpret_cast<u32x2*>(q + size_t(o) * I + i0 + c) =
        u32x2{pack4(t[0] * by, t[1] * by, t[2] * by, t[3] * by), pack4(t[4] * by, t[5] * by, t[6] * by, t[7] * by)};
  }
}

}  // namespace ring

template <typename E, int SC>
hipError_t rows_typed(const void* x, void* q, void* scale, ScaleStrides ss, int64_t m, int64_t in_dim,
                      hipStream_t stream) {
  const int KB = int(fp8_blocks(in_dim));
  const dim3 grid(unsigned((m + kThreads / kWave - 1) / (kThreads / kWave)), unsigned((KB + kSeg - 1) / kSeg));
  hipLaunchKernelGGL((quantize_rows_kernel<E, SC>), grid, dim3(kThreads), 0, stream, static_cast<const E*>(x),
                     static_cast<uint8_t*>(q), static_cast<scale_t<SC>*>(scale), ss, m, int(in_dim), KB);
  return hipGetLastError();
}

template <typename EI, int SC>
hipError_t blocks_typed(const void* s, const void* w0, const void* u, const void* v, void* q, void* scale,
                        int64_t out_dim, int64_t in_dim, int64_t rank, hipStream_t stream) {
  const int KB = int(fp8_blocks(in_dim));
  const dim3 grid(unsigned(fp8_blocks(out_dim) * KB));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, static_cast<const EI*>(s), static_cast<const EI*>(w0),
                       static_cast<const EI*>(u), static_cast<const EI*>(v), static_cast<uint8_t*>(q),
                       static_cast<scale_t<SC>*>(scale), int(out_dim), int(in_dim), int(rank), KB);
    return hipGetLastError();
  };
  if (rank == 0) return go(rebuild_blocks_kernel<EI, SC, kNone>);
  if constexpr (sizeof(EI) == 2) {
    if (rank % 8 == 0 && rank <= 64) return go(ring::rebuild_ring_kernel<SC, 2>);
    if (rank % 8 == 0 && rank <= 128) return go(ring::rebuild_ring_kernel<SC, 4>);
    if (rank % 8 == 0 && rank <= 256) return go(ring::rebuild_ring_kernel<SC, 8>);
    if (rank % 8 == 0) return go(rebuild_blocks_kernel<EI, SC, kMfma>);
  } else if (rank % 4 == 0) {
    return go(rebuild_blocks_kernel<EI, SC, kMfma32>);
  }
  return go(rebuild_blocks_kernel<EI, SC, kAny>);
}

}  // namespace

hipError_t launch_quantize_rows(tb_dtype dtype, tb_scale scale_type, const void* x, void* q, void* scale,
                                ScaleStrides ss, int64_t m, int64_t in_dim, hipStream_t stream) {
  const bool e8 = scale_type == TB_SCALE_E8M0;
  if (dtype == TB_BF16)
    return e8 ? rows_typed<bf16_t, TB_SCALE_E8M0>(x, q, scale, ss, m, in_dim, stream)
              : rows_typed<bf16_t, TB_SCALE_F32>(x, q, scale, ss, m, in_dim, stream);
  return e8 ? rows_typed<float, TB_SCALE_E8M0>(x, q, scale, ss, m, in_dim, stream)
            : rows_typed<float, TB_SCALE_F32>(x, q, scale, ss, m, in_dim, stream);
}

hipError_t launch_rebuild_blocks(tb_dtype dtype, tb_scale scale_type, const void* s, const void* w0, const void* u,
                                 const void* v, void* q, void* scale, int64_t out_dim, int64_t in_dim, int64_t rank,
                                 hipStream_t stream) {
  const bool e8 = scale_type == TB_SCALE_E8M0;
  if (dtype == TB_BF16)
    return e8 ? blocks_typed<bf16_t, TB_SCALE_E8M0>(s, w0, u, v, q, scale, out_dim, in_dim, rank, stream)
              : blocks_typed<bf16_t, TB_SCALE_F32>(s, w0, u, v, q, scale, out_dim, in_dim, rank, stream);
  return e8 ? blocks_typed<float, TB_SCALE_E8M0>(s, w0, u, v, q, scale, out_dim, in_dim, rank, stream)
            : blocks_typed<float, TB_SCALE_F32>(s, w0, u, v, q, scale, out_dim, in_dim, rank, stream);
}

}  // namespace tb
