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
// Few tokens (m <= 64): the weight streams once, at HBM rate.
//
// Each workgroup owns an equal share of the output rows, in tiles of 16 that
// need not be full: rows past its share are not loaded.  Its eight waves take
// blocks of 128 columns in turn, so that together they read runs of a kilobyte
// of each row; their sums meet in LDS.  Weights go from global memory straight
// into registers, kDepth blocks ahead: each byte is used once.  A lane's 32
// bytes of a block are two 16-byte pieces 64 apart, so that one load of a wave
// covers 64 contiguous bytes of each of 16 rows.
//
// Bound by HBM for large weights and few tokens (1 x 5376 x 21504, x given: 22.0 us,
// 5.3 TB/s; quantised in the kernel 24.9), by latency for small ones (1 x 1536 x 1152:
// 4.6 us, quantised), and with more tokens by the reads of x, which every workgroup
// repeats (plan_int8).
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8, kDecodeThreads = kDecodeWaves * kWave;
static_assert(kDecodeThreads == kFp8DecodeThreads, "what the launch's size is checked against");
constexpr int kDepth = 2;   // blocks of each wave in flight

struct DecodeArgs {
  const void* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* y;
  int M, O, I, KB;
  int wide;   // y rows can be written four outputs at a time
  int rows;   // output rows of a workgroup
};

// Q(x) of a workgroup's own in LDS: rows 16 bytes apart beyond whole blocks, so
// that the pieces of 16 tokens spread over the banks.
constexpr int x_pitch(int KB) { return KB * kBlock + 16; }

// All tokens (at most 16) into LDS by the whole workgroup: a power of two of them
// side by side, each by an equal share of the threads, which keep their first
// kHeld pieces in registers between the maximum and the rounding and read any
// others again.  red: kDecodeWaves words.
constexpr int kHeld = 6;
template <typename XE>
__device__ __forceinline__ void quantise_tokens(const DecodeArgs& a, uint8_t* xq, float* xs, uint32_t* red) {
  int p2 = 1;
  while (p2 < a.M) p2 *= 2;
  const int G = kDecodeThreads / p2, t = int(threadIdx.x) / G, li = int(threadIdx.x) % G;
  const XE* x = static_cast<const XE*>(a.x) + size_t(min(t, a.M - 1)) * a.I;
  Frag8<XE> held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int c = (j * G + li) * 8;
    held[j] = load_frag_if<XE>(x + c, c < a.I);
  }
  uint32_t top = 0;
  auto raise = [&](const Frag8<XE>& p) {
    float f[8];
    unpack8(p, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(f[e]));
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j) raise(held[j]);
  for (int c = (kHeld * G + li) * 8; c < a.I; c += G * 8) raise(load_frag<XE>(x + c));
  for (int d = 1; d < min(G, kWave); d *= 2) top = max(top, uint32_t(__shfl_xor(int(top), d)));
  if (G > kWave) {
    const int w = int(threadIdx.x) / kWave, per = G / kWave;
    red[w] = top;
    __syncthreads();
    for (int j = w / per * per; j < w / per * per + per; ++j) top = max(top, red[j]);
  }
  float stored, by;
  int8::row_scale(top, stored, by);
  if (t >= a.M) return;
  if (li == 0) xs[t] = stored;
  uint8_t* q = xq + t * x_pitch(a.KB);
  auto put = [&](const Frag8<XE>& p, int c) {
    float f[8];
    unpack8(p, f);
    *reinterpret_cast<u32x2*>(q + c) = u32x2{int8::pack4(f[0], f[1], f[2], f[3], by), int8::pack4(f[4], f[5], f[6], f[7], by)};
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if ((j * G + li) * 8 < a.I) put(held[j], (j * G + li) * 8);
  for (int c = (kHeld * G + li) * 8; c < a.I; c += G * 8) put(load_frag<XE>(x + c), c);
  // Columns past the last up to a whole block meet weights that were read as zeros.
}

constexpr int kLdsX = 65536;   // bytes of Q(x) a workgroup keeps

// XE: uint8_t where x comes in 8 bits, else the type it is quantised from.
template <int NT, int RT, typename XE, typename YE>
__global__ __launch_bounds__(kDecodeThreads) void int8_decode_kernel(DecodeArgs a) {
  constexpr bool kFused = sizeof(XE) > 1;
  __shared__ i32x4 red[kDecodeWaves / 2][RT * NT][kWave];
  __shared__ __attribute__((aligned(16))) uint8_t xlds[kFused ? kLdsX : 16];
  __shared__ float xslds[16];
  __shared__ uint32_t tops[kDecodeWaves];
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, kq = (l >> 4) * 16;
  const int o0 = int(blockIdx.x) * a.rows, rows = min(a.rows, a.O - o0);   // rows <= 16 RT
  const int nkb = (a.KB - w + kDecodeWaves - 1) / kDecodeWaves;            // this wave's blocks w, w + 8, ..

  const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + size_t(o0) * a.I, int64_t(rows) * a.I);
  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, kFused ? 0 : int64_t(a.M) * a.I);
  const int row = lr * a.I + kq;
  // Tokens past the last repeat it; their results are not stored.
  const uint8_t* xl[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xl[n] = xlds + (kFused ? min(n * 16 + lr, a.M - 1) * x_pitch(a.KB) + kq : 0);

  i32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = i32x4{0, 0, 0, 0};

  struct Stage {
    u32x4 w[2][RT], x[2][kFused ? 1 : NT];
  } st[kDepth];

  // Lane offsets of the two pieces of this wave's block i.
  struct Where { int at[2]; };
  auto where = [&](int i) {
    const int left = a.I - (w + i * kDecodeWaves) * kBlock;   // I % 16 == 0: a piece is all in or all out
    return Where{{kq < left ? row : kPast, kq + 64 < left ? row + 64 : kPast}};
  };
  auto fetch = [&](Stage& s, const Where& p, int i) {
    const int k = (w + i * kDecodeWaves) * kBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < RT; ++r) s.w[h][r] = __builtin_amdgcn_raw_buffer_load_b128(rw, p.at[h], k + r * 16 * a.I, 0);
      if constexpr (!kFused) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s.x[h][n] = __builtin_amdgcn_raw_buffer_load_b128(rx, p.at[h], k + n * 16 * a.I, 0);
      }
    }
  };
  struct Tokens { u32x4 v[2][NT]; };
  auto multiply = [&](const Stage& s, int i) {
    const int k = (w + i * kDecodeWaves) * kBlock;
    Tokens x;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (kFused) x.v[h][n] = *reinterpret_cast<const u32x4*>(xl[n] + k + 64 * h);
        else x.v[h][n] = s.x[h][n];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][n] = int8::mma(s.w[h][r], x.v[h][n], acc[r][n]);
      }
    return x;
  };
  auto keep_tokens = [&](const Tokens& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) int8::keep(x.v[h][n]);
  };

#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (d < nkb) fetch(st[d], where(d), d);
  // The first weight blocks are on their way while x is quantised.
  if constexpr (kFused) {
    quantise_tokens<XE>(a, xlds, xslds, tops);
    __syncthreads();
  }
  // Rounds without a branch: a branch around a refill would make the compiler
  // wait for the refill itself before it uses the next stage.  A refill's offsets are
  // made before the products, so that it leaves right behind them, and the guard's wait
  // is spent while it is on its way.
  int i = 0;
  for (; i + 2 * kDepth <= nkb; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const Where next = where(i + d + kDepth);
      __builtin_amdgcn_sched_barrier(0);
      const Tokens x = multiply(st[d], i + d);
      __builtin_amdgcn_sched_barrier(0);
      fetch(st[d], next, i + d + kDepth);
      int8::products_issued(acc);
      if constexpr (kFused) keep_tokens(x);
    }
  }
  for (; i < nkb; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (i + d < nkb) {
        const Tokens x = multiply(st[d], i + d);
        int8::products_issued(acc);
        keep_tokens(x);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r) int8::keep(st[d].w[h][r]);
        if (i + d + kDepth < nkb) fetch(st[d], where(i + d + kDepth), i + d + kDepth);
      }
    }
  }

  // The eight waves' sums: wave w + 4's into wave w's, then those four.
  if (w >= kDecodeWaves / 2) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) red[w - kDecodeWaves / 2][r * NT + n][l] = acc[r][n];
  }
  __syncthreads();
  if (w < kDecodeWaves / 2) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) red[w][r * NT + n][l] += acc[r][n];
  }
  __syncthreads();
  for (int j = int(threadIdx.x); j < RT * NT * kWave; j += kDecodeThreads) {
    const int tile = j / kWave, ln = j % kWave;
    const int t = (tile % NT) * 16 + (ln & 15), o = (tile / NT) * 16 + (ln >> 4) * 4;
    if (t >= a.M || o >= rows) continue;
    i32x4 v = red[0][tile][ln];
#pragma unroll
    for (int q = 1; q < kDecodeWaves / 2; ++q) v += red[q][tile][ln];
    store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o0 + o,
               int8::scaled(v, kFused ? xslds[t] : a.xs[t], channel_scales(a.ws, o0 + o, a.O)), rows - o,
               a.wide && o + 4 <= rows);
  }
}

// ---------------------------------------------------------------------------
// Tiles of TM tokens x TN outputs (64 or 128 each): TM / 16 waves, each 32 tokens
// by half of the outputs, 128 columns per step.  Both operands come straight into a
// ring of LDS slots, and a step's fragments are read while the step before
// multiplies.  Rows of 128 bytes keep their 16-byte pieces XOR-swizzled by (row >>
// 1) & 7, so that the fragment reads of 16 rows meet all banks.  With few tiles the
// reduction is cut into S slices; each writes its sums and a second launch adds
// and scales them.
//
// A step of 64 x 64 tiles (16 KB) takes 0.2 us, one of 128 x 128 tiles (32 KB) 0.55.  No
// unit that was counted is full: with 64 x 64 tiles the matrix cores are busy for 20 %
// of the time that a unit works (128 x 128: 39 %), its L1 returns data for half of it
// and waits for L2 in 45 %, which answers in 370 cycles, and waves wait in 40 % of their
// cycles.  Rings of three to six slots, fragments read a step ahead or not, and waves of
// 64 x 64 that share the columns and read up to half as much from LDS all took the same
// within 3 %, hot or cold.  777 x 1152 x 6912 15 to 16 us (16.8 in a trace), 512 x 8192 x
// 5376 28.8 (1.57 Pop/s).
// Which tiles a call takes: plan_int8.
// ---------------------------------------------------------------------------
struct Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* y;
  int* part;   // [S][tiles][TN / 16][4 TM] pieces of four, or NULL with one slice
  int M, O, I, KB;
  int tiles_m, tiles_n, S;
  int wide;
};

// Tile u's first token and output: groups of eight token tiles walked column
// by column, so that workgroups that run together share rows in L2.
template <int TM, int TN>
__device__ __forceinline__ void tile_at(const Args& a, int u, int& m0, int& n0) {
  const int per_group = 8 * a.tiles_n, first = u / per_group * 8, gs = min(a.tiles_m - first, 8), r = u % per_group;
  m0 = (first + r % gs) * TM;
  n0 = r / gs * TN;
}

template <typename YE, int TM, int TN, int kSlots>
__global__ __launch_bounds__(4 * TM) void int8_ring_kernel(Args a) {
  constexpr int kThreads = 4 * TM, kWaves = TM / 16, kW = TN / 8 / kWaves;   // kW, 2: loads of W and x per wave and step
  constexpr int kI = TN / 32;   // W fragments of a wave
  constexpr int kX = TN * 128, kSlot = kX + TM * 128, kLoads = kW + 2;
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
  tile_at<TM, TN>(a, tile, m0, n0);
  const int kb0 = int(int64_t(slice) * a.KB / a.S), kb1 = int(int64_t(slice + 1) * a.KB / a.S);

  const int rows_w = min(a.O - n0, TN), rows_x = min(a.M - m0, TM);
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
    for (int j = 0; j < kW; ++j) {
      const int row8 = w * kW + j;
      dma(d + row8 * 1024, rw, (row8 & 1) ? vo : ve, k + row8 * 8 * a.I);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) dma(d + kX + (w * 2 + j) * 1024, rx, j ? vo : ve, k + (w * 2 + j) * 8 * a.I);
  };

  i32x4 acc[kI][2];
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // A step's fragments are read while the step before multiplies.
  struct Fragments {
    u32x4 w[2][kI], x[2][2];
  } f[2];
  const int sw = (lr >> 1) & 7, p0 = (q ^ sw) << 4, p1 = ((q + 4) ^ sw) << 4;
  auto read = [&](int slot, Fragments& g) {
    const lds_byte* const s = base + slot * kSlot;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = h ? p1 : p0;
#pragma unroll
      for (int j = 0; j < 2; ++j) g.x[h][j] = *reinterpret_cast<const lds_u32x4*>(s + kX + (wt * 32 + j * 16 + lr) * 128 + p);
#pragma unroll
      for (int i = 0; i < kI; ++i)
        g.w[h][i] = *reinterpret_cast<const lds_u32x4*>(s + (wo * (TN / 2) + i * 16 + lr) * 128 + p);
    }
  };
  auto step = [&](auto which, int kb) {
    constexpr int U = decltype(which)::value;
    if (kb >= kb1) return;
    wait_loads<kLoads*(kSlots - 2)>();   // block kb + 1 has landed, those behind it may be out; this wave holds block kb
    __builtin_amdgcn_s_barrier();        // and so does every other
    issue(U % kSlots, kb + kSlots);
    read((U + 1) % kSlots, f[(U + 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = int8::mma(f[U & 1].w[h][i], f[U & 1].x[h][j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    // With the wait and the barrier, mfma_operand_guard's distance to the vector code of the next step; in 64 x 64 tiles
    // they alone are enough (eight states more take 3 % there: 777 x 1152 x 6912).
    if constexpr (TN == 128) asm volatile("s_nop 3");
  };
#pragma unroll
  for (int d = 0; d < kSlots; ++d) issue(d, kb0 + d);
  wait_loads<kLoads*(kSlots - 1)>();
  __builtin_amdgcn_s_barrier();
  read(0, f[0]);
  constexpr int kUnroll = kSlots % 2 ? 2 * kSlots : kSlots;
  for (int kb = kb0; kb < kb1; kb += kUnroll) {
    step(std::integral_constant<int, 0>{}, kb);
    step(std::integral_constant<int, 1>{}, kb + 1);
    step(std::integral_constant<int, 2>{}, kb + 2);
    step(std::integral_constant<int, 3>{}, kb + 3);
    if constexpr (kUnroll > 4) {
      step(std::integral_constant<int, 4>{}, kb + 4);
      step(std::integral_constant<int, 5>{}, kb + 5);
    }
  }
  int8::products_issued(acc);
  wait_loads<0>();   // nothing lands in LDS after the workgroup has ended

  if (a.S > 1) {
    i32x4* p = reinterpret_cast<i32x4*>(a.part) + (size_t(slice) * tiles + tile) * 2 * kI * kThreads + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kI; ++i)
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
    for (int i = 0; i < kI; ++i) {
      const int o = n0 + wo * (TN / 2) + i * 16 + q * 4;
      if (o < a.O)
        store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o,
                   int8::scaled(acc[i][j], xs, channel_scales(a.ws, o, a.O)), a.O - o, a.wide && o + 4 <= a.O);
    }
  }
}

// The slices' sums of a split product: one workgroup for the pieces of 16
// outputs of each of a tile's waves.
template <typename YE, int TM, int TN>
__global__ __launch_bounds__(4 * TM) void int8_join_kernel(Args a) {
  constexpr int kThreads = 4 * TM, kI = TN / 32;
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  const int tile = int(blockIdx.x) / kI, tiles = a.tiles_m * a.tiles_n, i = int(blockIdx.x) % kI;
  int m0, n0;
  tile_at<TM, TN>(a, tile, m0, n0);
  const i32x4* p = reinterpret_cast<const i32x4*>(a.part) + (size_t(tile) * kI + i) * 2 * kThreads + threadIdx.x;
  i32x4 sum[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) sum[j] = p[j * kThreads];
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) sum[j] += p[(size_t(s) * tiles * 2 * kI + j) * kThreads];
  const int o = n0 + wo * (TN / 2) + i * 16 + q * 4;
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

template <typename YE, int TM, int TN, int SLOTS>
hipError_t ring_go(const Args& a, hipStream_t stream) {
  const unsigned tiles = unsigned(a.tiles_m * a.tiles_n);
  hipLaunchKernelGGL((int8_ring_kernel<YE, TM, TN, SLOTS>), dim3(tiles * unsigned(a.S)), dim3(4 * TM), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 1) return e;
  hipLaunchKernelGGL((int8_join_kernel<YE, TM, TN>), dim3(tiles * (TN / 32)), dim3(4 * TM), 0, stream, a);
  return hipGetLastError();
}

template <int NT, int RT, typename XE, typename YE>
hipError_t decode_go(const DecodeArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned((a.O + a.rows - 1) / a.rows));
  hipLaunchKernelGGL((int8_decode_kernel<NT, RT, XE, YE>), grid, dim3(kDecodeThreads), 0, stream, a);
  return hipGetLastError();
}

template <int NT, typename XE, typename YE>
hipError_t decode_rt(const DecodeArgs& a, hipStream_t stream) {
  const int rt = (a.rows + 15) / 16;
  if (rt == 1) return decode_go<NT, 1, XE, YE>(a, stream);
  if (rt == 2) return decode_go<NT, 2, XE, YE>(a, stream);
  if (rt == 3) return decode_go<NT, 3, XE, YE>(a, stream);
  if constexpr (NT <= 2)
    if (rt == 4) return decode_go<NT, 4, XE, YE>(a, stream);
  if constexpr (NT == 1)
    if (rt <= 6) return decode_go<NT, 6, XE, YE>(a, stream);
  return hipErrorInvalidValue;
}

template <typename YE>
hipError_t decode_x(tb_dtype x_dtype, const DecodeArgs& a, hipStream_t stream) {
  if (x_dtype == TB_BF16) return decode_rt<1, bf16_t, YE>(a, stream);
  if (x_dtype == TB_F32) return decode_rt<1, float, YE>(a, stream);
  if (a.M <= 16) return decode_rt<1, uint8_t, YE>(a, stream);
  return a.M <= 32 ? decode_rt<2, uint8_t, YE>(a, stream) : decode_rt<4, uint8_t, YE>(a, stream);
}

// Output rows of a workgroup: equal shares of the weight for every compute
// unit (one with twice the rows of another would finish last), in as few
// workgroups per unit as the widest kernel for these tokens allows; from 17
// tokens on in multiples of four, so that results leave four at a time.
int decode_rows(int64_t m, int64_t out_dim, int cus) {
  const int most = fp8_decode_most_rows(m);
  const int64_t k = (out_dim + int64_t(cus) * most - 1) / (int64_t(cus) * most);
  const int64_t rows = (out_dim + cus * k - 1) / (cus * k);
  return int(m <= 16 ? rows : (rows + 3) / 4 * 4);
}

// The kernel, its tiles and its slices are those that a simple estimate finds
// fastest (us, at 256 compute units).  It was set by the sizes below and 30 like them, from
// 1 to 4000 tokens, x given; what it picks was the fastest of everything measured
// there, or within 10 % of it.
//   Few-token kernel: a start, and the rates at which a unit reads its rows (from
//   HBM) and x (from its XCD's L2): 16 x 5376 x 5376 8.8 us (64 x 64 tiles 12.0),
//   but 16 x 5376 x 21504 27.4 (25.3), 33 x 5376 x 21504 46 (26.1) and 64 x 21504 x 5376
//   47 (29.8 with 64 x 128).
//   Tiles: a start, and a step for every 128 columns; a unit's workgroups share it;
//   no less than the weights take from HBM.  Slices are written, read and joined by
//   another launch.  300 x 1536 x 1152 6.0 with 64 x 64, 8.3 with 64 x 128, 9.9 with 128 x
//   128; 777 x 1152 x 6912 15.5, 18.5 in two slices, 20.2 in three; 512 x 8192 x 5376
//   39.3, 32.4, 28.9, and 42.4 with 256 x 256 in four; 128 x 5376 x 21504 43.1 in three,
//   39.2 in three, 33.3 in six; 2000 x 8192 x 5376 143, 114, 108 and 71 with 256 x 256.
struct Shape { int tm, tn; double start, step; };
constexpr Shape kShapes[] = {{64, 64, 4.2, 0.22}, {64, 128, 5.2, 0.37}, {128, 128, 5.5, 0.57}};

double joined(int64_t slices, double sums) { return slices > 1 ? 3.5 + double(slices) * sums * 8 / 6e6 : 0.; }

double streamed(int64_t m, int64_t out_dim, int64_t in_dim, int rows, int cus) {
  const int64_t rounds = ((out_dim + rows - 1) / rows + cus - 1) / cus;
  return 1. + double(rounds) * (2.5 + double(rows) * double(in_dim) / 25e3 + double(m) * double(in_dim) / 45e3);
}

}  // namespace

Int8Plan plan_int8(int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype, int cus) {
  Int8Plan p{};
  const int64_t KB = fp8_blocks(in_dim);
  const double weights = 2. + double(out_dim) * double(in_dim) / 6e6;
  p.tile = plan_int8_tiles(m, out_dim, in_dim, cus);
  const int64_t big_tiles = int64_t(p.tile.tiles_m) * p.tile.tiles_n, cut = p.tile.S > 1 ? p.tile.split_tiles : 0;
  p.big = 1;
  p.S = 1;
  double best = std::max(weights, 4. + 1.6 * (double((big_tiles - cut + cus - 1) / cus) * double(KB) +
                                              (cut > 0 ? double((KB + p.tile.S - 1) / p.tile.S) : 0.))) +
                joined(p.tile.S, double(cut) * 65536);
  for (const Shape& t : kShapes) {
    const int64_t tm = (m + t.tm - 1) / t.tm, tn = (out_dim + t.tn - 1) / t.tn;
    for (int64_t s = 1; s <= 8 && (s == 1 || s * 4 <= KB); ++s) {
      if (tm * tn * s * (4 * t.tm) >= int64_t(1) << 32) continue;   // (a launch holds fewer threads)
      const double cost =
          std::max(weights, t.start + t.step * double((tm * tn * s + cus - 1) / cus) * double((KB + s - 1) / s)) +
          joined(s, double(m) * double(out_dim));
      if (cost >= best) continue;
      best = cost;
      p.big = 0;
      p.tm = t.tm;
      p.tn = t.tn;
      p.tiles_m = int(tm);
      p.tiles_n = int(tn);
      p.S = int(s);
    }
  }
  if (m <= kDecodeMaxTokens) {
    // Up to 16 tokens the few-token kernel can quantise x itself, which costs each workgroup a pass over x and a wait
    // (about 1.5 us) instead of a launch (about 3.5).
    p.rows = decode_rows(m, out_dim, cus);
    const bool quantises = x_dtype != TB_INT8 && m <= 16 && m * x_pitch(int(KB)) <= kLdsX;
    const double passes = 1.5 + double(m * in_dim) * (x_dtype == TB_BF16 ? 2 : 4) / 60e3, launch = x_dtype != TB_INT8 ? 3.5 : 0.;
    p.fused = quantises && passes < launch;
    p.decode = streamed(m, out_dim, in_dim, p.rows, cus) + (p.fused ? passes : launch) <= best + launch;
    p.fused = p.fused && p.decode;
  }
  size_t at = 0;
  if (x_dtype != TB_INT8 && !p.fused) {
    p.off_xq = at;
    at = align_up(at + size_t(m) * in_dim, 256);
    p.off_xs = at;
    at = align_up(at + size_t(m) * 4, 256);
  }
  p.off_part = at;
  if (!p.decode && p.big) at += p.tile.part_bytes;
  else if (!p.decode && p.S > 1)
    at += size_t(p.S) * size_t(p.tiles_m) * size_t(p.tiles_n) * size_t(p.tm) * size_t(p.tn) * 4;
  p.bytes = at;
  return p;
}

hipError_t launch_int8_product(const Int8Plan& p, tb_dtype x_dtype, tb_dtype y_dtype, const void* x, const float* xs,
                               const void* w, const float* ws, void* y, int64_t m, int64_t out_dim, int64_t in_dim,
                               char* data, hipStream_t stream) {
  if (x_dtype != TB_INT8 && !p.fused) {
    void* xq = data + p.off_xq;
    float* sq = reinterpret_cast<float*>(data + p.off_xs);
    hipError_t e = launch_int8_rows(x_dtype, x, xq, sq, m, in_dim, stream);
    if (e != hipSuccess) return e;
    x = xq;
    xs = sq;
    x_dtype = TB_INT8;
  }
  const size_t ys = y_dtype == TB_BF16 ? 2 : 4;
  const int wide = out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * ys - 1)) == 0;
  if (p.decode) {
    const DecodeArgs a{x, xs, static_cast<const uint8_t*>(w), ws, y, int(m), int(out_dim), int(in_dim),
                       int(fp8_blocks(in_dim)), wide && p.rows % 4 == 0, p.rows};
    return y_dtype == TB_BF16 ? decode_x<bf16_t>(x_dtype, a, stream) : decode_x<float>(x_dtype, a, stream);
  }
  if (p.big)
    return launch_int8_tiles(p.tile, y_dtype, x, xs, w, ws, y, reinterpret_cast<int*>(data + p.off_part), m, out_dim,
                             in_dim, stream);
  const Args a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, y,
               reinterpret_cast<int*>(data + p.off_part), int(m), int(out_dim), int(in_dim), int(fp8_blocks(in_dim)),
               p.tiles_m, p.tiles_n, p.S, wide};
  auto go = [&](auto tm, auto tn, auto slots) {
    constexpr int TM = decltype(tm)::value, TN = decltype(tn)::value, SLOTS = decltype(slots)::value;
    return y_dtype == TB_BF16 ? ring_go<bf16_t, TM, TN, SLOTS>(a, stream) : ring_go<float, TM, TN, SLOTS>(a, stream);
  };
  using std::integral_constant;
  if (p.tm == 128) return go(integral_constant<int, 128>{}, integral_constant<int, 128>{}, integral_constant<int, 3>{});
  if (p.tn == 128) return go(integral_constant<int, 64>{}, integral_constant<int, 128>{}, integral_constant<int, 3>{});
  return go(integral_constant<int, 64>{}, integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

}  // namespace tb
