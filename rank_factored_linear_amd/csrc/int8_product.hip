// y = xq . wq^T of 8-bit integers with a scale per token and per output channel:
//   y[t, o] = (sum_i xq[t, i] wq[o, i]) * (xs[t] * ws[o])
// The sums are whole numbers held in 32 bits and exact in any order, so however
// the reduction is split the result is the same bit for bit; it is turned to
// fp32 (one rounding), scaled (two) and rounded to y's type.
//
// W's rows are the products' A operand (output rows), x's the B operand
// (output columns): a lane then holds four consecutive outputs of one token.
#include "int8_device.h"

#include <algorithm>

namespace tb {

namespace {

using namespace fp8;
using int8::i32x4;

template <typename YE>
__device__ __forceinline__ void store_out4(YE* y, const f32x4& v, int n, bool wide) {
  if constexpr (sizeof(YE) == 2) {
    if (wide) {
      *reinterpret_cast<u32x2*>(y) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      return;
    }
  } else if (wide) {
    *reinterpret_cast<f32x4*>(y) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) y[e] = from_f32<YE>(v[e]);
}

// The scales of outputs o .. o + 3 (those past the last: any).
__device__ __forceinline__ f32x4 channel_scales(const float* ws, int o, int O) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = ws[min(o + e, O - 1)];
  return v;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), kRsrcFlags);
}

// ---------------------------------------------------------------------------
// 64 tokens x 128 outputs per workgroup, four waves of 64 outputs x 32 tokens,
// 128 columns per step.  Both operands come straight into a ring of three LDS
// slots, two steps ahead.  Rows of 128 bytes keep their 16-byte pieces
// XOR-swizzled by (row >> 1) & 7, so that the fragment reads of 16 rows meet
// all banks.  With few tiles the reduction is cut into S slices; each writes its
// sums and a second launch adds and scales them.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, TM = 64, kSlots = 3;   // outputs and tokens of a tile; LDS slots
constexpr int kThreads = 256;

struct Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* y;
  int* part;   // [S][tiles][8][kThreads] pieces of four, or NULL with one slice
  int M, O, I, KB;
  int tiles_m, tiles_n, S;
  int wide;
};

// Tile u's first token and output: groups of eight token tiles walked column
// by column, so that workgroups that run together share rows in L2.
__device__ __forceinline__ void tile_at(const Args& a, int u, int& m0, int& n0) {
  const int per_group = 8 * a.tiles_n, first = u / per_group * 8, gs = min(a.tiles_m - first, 8), r = u % per_group;
  m0 = (first + r % gs) * TM;
  n0 = r / gs * kTile;
}

template <typename YE>
__global__ __launch_bounds__(kThreads, 2) void int8_ring_kernel(Args a) {
  constexpr int kX = kTile * 128, kSlot = kX + TM * 128, kLoads = 6;   // loads of a wave and step: four of W, two of x
  __shared__ __attribute__((aligned(16))) uint8_t ring[kSlots * kSlot];
  lds_byte* const base = (lds_byte*)ring;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  // Workgroup g runs on XCD g % 8: each XCD takes a run of the tiles of few
  // slices, so that what it reads again fits its own L2.
  const int tiles = a.tiles_m * a.tiles_n, total = tiles * a.S, xcd = int(blockIdx.x) % 8;
  const int at = xcd * (total / 8) + min(xcd, total % 8) + int(blockIdx.x) / 8;
  const int slice = at / tiles, tile = at % tiles;
  int m0, n0;
  tile_at(a, tile, m0, n0);
  const int kb0 = int(int64_t(slice) * a.KB / a.S), kb1 = int(int64_t(slice + 1) * a.KB / a.S);

  const int rows_w = min(a.O - n0, kTile), rows_x = min(a.M - m0, TM);
  const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + size_t(n0) * a.I, int64_t(rows_w) * a.I);
  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x + size_t(m0) * a.I, int64_t(rows_x) * a.I);
  // Load j of an operand: row 8 (w loads + j) + l / 8, the piece that the
  // swizzle keeps at position l % 8; eight rows further on the swizzle differs
  // in its upper bit only.
  const int dr = l >> 3, pe = (l & 7) ^ (dr >> 1), po = pe ^ 4;
  const unsigned b0 = unsigned(uintptr_t(base));
  auto issue = [&](int slot, int kb) {
    const int left = kb < kb1 ? a.I - kb * kBlock : 0, k = min(kb, kb1 - 1) * kBlock;
    const int ve = pe * 16 < left ? dr * a.I + pe * 16 : kPast, vo = po * 16 < left ? dr * a.I + po * 16 : kPast;
    const unsigned d = b0 + unsigned(slot * kSlot);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row8 = w * 4 + j;
      dma(d + row8 * 1024, rw, (row8 & 1) ? vo : ve, k + row8 * 8 * a.I);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) dma(d + kX + (w * 2 + j) * 1024, rx, j ? vo : ve, k + (w * 2 + j) * 8 * a.I);
  };

  i32x4 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  const int sw = (lr >> 1) & 7, p0 = (q ^ sw) << 4, p1 = ((q + 4) ^ sw) << 4;
  auto step = [&](auto which, int kb) {
    constexpr int slot = decltype(which)::value;
    wait_loads<kLoads>();             // block kb has landed; kb + 1 may be out
    __builtin_amdgcn_s_barrier();     // published; and every wave has left the slot filled next
    issue((slot + 2) % kSlots, kb + 2);
    const lds_byte* const s = base + slot * kSlot;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = h ? p1 : p0;
      u32x4 fx[2], fw[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) fx[j] = *reinterpret_cast<const lds_u32x4*>(s + kX + (wt * 32 + j * 16 + lr) * 128 + p);
#pragma unroll
      for (int i = 0; i < 4; ++i) fw[i] = *reinterpret_cast<const lds_u32x4*>(s + (wo * 64 + i * 16 + lr) * 128 + p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = int8::mma(fw[i], fx[j], acc[i][j]);
    }
  };
  issue(0, kb0);
  issue(1, kb0 + 1);
  int kb = kb0;
  for (; kb + 2 < kb1; kb += 3) {
    step(std::integral_constant<int, 0>{}, kb);
    step(std::integral_constant<int, 1>{}, kb + 1);
    step(std::integral_constant<int, 2>{}, kb + 2);
  }
  if (kb < kb1) step(std::integral_constant<int, 0>{}, kb);
  if (kb + 1 < kb1) step(std::integral_constant<int, 1>{}, kb + 1);
  wait_loads<0>();   // nothing lands in LDS after the workgroup has ended

  if (a.S > 1) {
    i32x4* p = reinterpret_cast<i32x4*>(a.part) + (size_t(slice) * tiles + tile) * 8 * kThreads + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) p[(i * 2 + j) * kThreads] = acc[i][j];
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = m0 + wt * 32 + j * 16 + lr;
    if (t >= a.M) continue;
    const float xs = a.xs[t];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = n0 + wo * 64 + i * 16 + q * 4;
      if (o < a.O)
        store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o,
                   int8::scaled(acc[i][j], xs, channel_scales(a.ws, o, a.O)), a.O - o, a.wide && o + 4 <= a.O);
    }
  }
}

// The slices' sums of a split product: one workgroup for the pieces of 16
// outputs of each of a tile's waves.
template <typename YE>
__global__ __launch_bounds__(kThreads) void int8_join_kernel(Args a) {
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  const int tile = int(blockIdx.x) >> 2, tiles = a.tiles_m * a.tiles_n, i = int(blockIdx.x) & 3;
  int m0, n0;
  tile_at(a, tile, m0, n0);
  const i32x4* p = reinterpret_cast<const i32x4*>(a.part) + (size_t(tile) * 4 + i) * 2 * kThreads + threadIdx.x;
  i32x4 sum[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) sum[j] = p[j * kThreads];
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) sum[j] += p[(size_t(s) * tiles * 8 + j) * kThreads];
  const int o = n0 + wo * 64 + i * 16 + q * 4;
  if (o >= a.O) return;
  const f32x4 ws = channel_scales(a.ws, o, a.O);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = m0 + wt * 32 + j * 16 + lr;
    if (t < a.M)
      store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, int8::scaled(sum[j], a.xs[t], ws), a.O - o,
                 a.wide && o + 4 <= a.O);
  }
}

template <typename YE>
hipError_t ring_go(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((int8_ring_kernel<YE>), dim3(unsigned(a.tiles_m * a.tiles_n * a.S)), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 1) return e;
  hipLaunchKernelGGL((int8_join_kernel<YE>), dim3(unsigned(a.tiles_m * a.tiles_n * 4)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

Int8Plan plan_int8(int64_t m, int64_t out_dim, int64_t in_dim, bool quantised, tb_dtype y_dtype, int cus) {
  Int8Plan p{};
  const int64_t KB = fp8_blocks(in_dim);
  p.S = 1;
  size_t at = 0;
  if (!quantised) {
    p.off_xq = at;
    at = align_up(at + size_t(m) * in_dim, 256);
    p.off_xs = at;
    at = align_up(at + size_t(m) * 4, 256);
  }
  p.tiles_n = int((out_dim + kTile - 1) / kTile);
  p.tiles_m = int((m + TM - 1) / TM);
  // Slices for the two workgroups that a compute unit holds, of at least four
  // blocks, where that saves more than the second launch costs (as much as
  // about 12 blocks).
  const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
  const int64_t s = std::min<int64_t>(2 * cus / tiles, KB / 4);
  if (s > 1 && KB - KB / s >= 12) p.S = int(s);
  if (p.S > 1) {
    p.off_part = at;
    at += size_t(p.S) * tiles * kTile * TM * 4;
  }
  p.bytes = at;
  return p;
}

hipError_t launch_int8_product(const Int8Plan& p, tb_dtype x_dtype, tb_dtype y_dtype, const void* x, const float* xs,
                               const void* w, const float* ws, void* y, int64_t m, int64_t out_dim, int64_t in_dim,
                               char* data, hipStream_t stream) {
  if (x_dtype != TB_INT8) {
    void* xq = data + p.off_xq;
    float* sq = reinterpret_cast<float*>(data + p.off_xs);
    hipError_t e = launch_int8_rows(x_dtype, x, xq, sq, m, in_dim, stream);
    if (e != hipSuccess) return e;
    x = xq;
    xs = sq;
  }
  const size_t ys = y_dtype == TB_BF16 ? 2 : 4;
  const int wide = out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * ys - 1)) == 0;
  const Args a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, y,
               reinterpret_cast<int*>(data + p.off_part), int(m), int(out_dim), int(in_dim), int(fp8_blocks(in_dim)),
               p.tiles_m, p.tiles_n, p.S, wide};
  return y_dtype == TB_BF16 ? ring_go<bf16_t>(a, stream) : ring_go<float>(a, stream);
}

}  // namespace tb
