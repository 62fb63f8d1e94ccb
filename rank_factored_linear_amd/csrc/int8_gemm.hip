// The 8-bit integer product for many tokens: output tiles of 256 outputs x 256
// tokens (the formula and the other kernels are in int8_product.hip).
//
// Eight waves, each 128 outputs x 64 tokens in products of 16 x 16 x 64 that
// add to 32 accumulators of four whole numbers.  The reduction runs by 128
// columns (128 bytes of each of 512 rows, 64 KB) through a two-buffer LDS ring
// filled by direct-to-LDS loads; rows keep their 16-byte pieces XOR-swizzled by
// (row >> 1) & 7, so the fragment reads of 16 consecutive rows meet all 64 banks.
//
// Workgroups are persistent, one per compute unit, and take whole tiles in
// rounds.  What is left over for a last, partly filled round is cut into
// slices of in_dim, whose sums a second launch adds.  A tile's scales come to
// LDS with its first loads, so that its end waits for nothing.
//
// 8192 x 8192 x 8192: 400 us (2.75 Pop/s; a library product 446 to 507); 4096 x
// 21504 x 5376: 365 to 386 from card to card and 15 to join (2.36 to 2.49 with the join;
// a library product 438 to 473).  The products alone,
// in registers, run at 4.1 (power; 32 x 32 x 32 ones at 3.5).  With zeros, which draw
// less power, it takes 10 % less, so most of the rest is waiting: the matrix cores are
// busy for 65 % of the time, waves wait in a third of their cycles, L1 for L2 in 56 %.
// Tried at 4096 x 4096 x 32768 (412 us): four waves of 128 x 128, which read a
// third less from LDS but leave nothing to run at a barrier, 427; stages of 64
// columns, four in the ring, whose loads fetch half lines, 503.
#include "int8_device.h"

#include <algorithm>

namespace tb {

namespace {

using namespace fp8;
using int8::i32x4;

constexpr int BT = 256;                       // outputs and tokens of a tile
constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kOpBytes = BT * kBlock;         // one operand's block in LDS
constexpr int kBOffset = 2 * kOpBytes;        // ring [W0][W1][x0][x1]
constexpr int kRingBytes = 4 * kOpBytes;
constexpr int kScales = 2 * BT;               // floats: a tile's channels, then its tokens; two tiles' in turn
// Finished tiles leave through LDS, 16 tokens x 128 bytes at a time per wave,
// rows 144 bytes apart, beside the ring.
constexpr int kStagePitch = 144, kStageBytes = 16 * kStagePitch;
static_assert(kRingBytes + 2 * kScales * 4 + kWaves * kStageBytes <= 160 * 1024, "ring, scales and staging fit the LDS");
static_assert(int64_t(BT) * TB_INT8_MAX_IN_DIM < (int64_t(1) << 31), "a tile's rows are addressed with 31-bit offsets");
constexpr int kPieces = 32;                   // pieces of four sums per lane and tile

struct Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* y;
  int* part;         // [S][split_tiles][kPieces][kThreads] pieces of four
  int M, O, I, KB;
  int tiles_m, tiles_n;
  int split_tiles, S;   // the first split_tiles tiles are cut into S slices
  int xcd_major;        // workgroup g takes position (g % 8) * (grid / 8) + g / 8
  int wide;             // y 16-byte aligned and O a multiple of 8
};

// Tile u of the processing order: groups of eight token tiles walked column by
// column, so that workgroups that run together share rows of both operands.
__device__ __forceinline__ void tile_at(const Args& a, int u, int& m0, int& n0) {
  const int per_group = 8 * a.tiles_n, first = u / per_group * 8, gs = min(a.tiles_m - first, 8), r = u % per_group;
  m0 = (first + r % gs) * BT;
  n0 = r / gs * BT;
}

struct Item {
  int u, slice, m0, n0, kb0, kb1;
};

__device__ __forceinline__ Item item_at(const Args& a, int v) {
  Item it;
  const int cut = a.split_tiles * a.S;
  it.slice = v < cut ? v / a.split_tiles : -1;
  it.u = v < cut ? v % a.split_tiles : v - cut + a.split_tiles;
  it.kb0 = v < cut ? int(int64_t(it.slice) * a.KB / a.S) : 0;
  it.kb1 = v < cut ? int(int64_t(it.slice + 1) * a.KB / a.S) : a.KB;
  tile_at(a, it.u, it.m0, it.n0);
  return it;
}

// An LDS address kept as one register, so that the displacements of buffers
// and fragments fold into the instructions' offsets.
__device__ __forceinline__ lds_byte* opaque(lds_byte* p) {
  asm volatile("" : "+v"(p));
  return p;
}

struct Lanes {
  unsigned dma_w, dma_x, dma_s;  // where this wave's loads land in buffer 0
  int w, row;                    // the wave; first row of its loads in the tile
  int ce, co;                    // lane offsets' pieces (bytes) in loads of even and of odd groups of eight rows
  int dr;                        // row of the lane in a load
  lds_byte* w_rd[2];             // the fragment's pieces q and q + 4 of W row wo * 128 + lane % 16
  lds_byte* x_rd[2];             // and of x row wt * 64 + lane % 16
};

__device__ __forceinline__ Lanes make_lanes(uint8_t* ring, float* scales) {
  lds_byte* base = (lds_byte*)ring;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  Lanes ln;
  ln.w = w;
  ln.row = w * 32;
  const unsigned b0 = unsigned(uintptr_t(base));
  ln.dma_w = __builtin_amdgcn_readfirstlane(b0 + unsigned(ln.row) * kBlock);
  ln.dma_x = __builtin_amdgcn_readfirstlane(b0 + unsigned(kBOffset) + unsigned(ln.row) * kBlock);
  ln.dma_s = __builtin_amdgcn_readfirstlane(unsigned(uintptr_t((lds_byte*)scales)) + unsigned(w) * 256u);
  // Groups of eight rows start at multiples of eight: their swizzle is the
  // row's half, with the upper bit flipped in every second group.
  ln.dr = l >> 3;
  ln.ce = ((l & 7) ^ (ln.dr >> 1)) << 4;
  ln.co = ln.ce ^ 64;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = ((q + 4 * h) ^ ((lr >> 1) & 7)) << 4;
    ln.w_rd[h] = opaque(base + (wo * 128 + lr) * kBlock + piece);
    ln.x_rd[h] = opaque(base + kBOffset + (wt * 64 + lr) * kBlock + piece);
  }
  return ln;
}

__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const void*>((uint64_t(hi) << 32) | lo);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(uniform_ptr(p)), 0, __builtin_amdgcn_readfirstlane(bytes),
                                           kRsrcFlags);
}

// One item's operands (all uniform; lanes address them by offset).
struct Source {
  const uint8_t* w;
  const uint8_t* x;
  int wbytes, xbytes;
};

__device__ __forceinline__ Source source_of(const Args& a, const Item& it) {
  Source s;
  s.w = a.w + size_t(it.n0) * a.I;
  s.x = a.x + size_t(it.m0) * a.I;
  s.wbytes = min(a.O - it.n0, BT) * a.I;
  s.xbytes = min(a.M - it.m0, BT) * a.I;
  return s;
}

// The loads of a block: 0..3 its x rows, 4..7 its W rows.  Pieces past the
// reduction, rows past the matrix and every piece of a block at or past kb1 are
// fetched from past the buffers and so land as zeros without memory traffic.
// There is no branch: one here would let the compiler move products of a step
// into the block behind it, and the waits count loads.
constexpr int kBlockLoads = 8;

struct Issue {
  __amdgpu_buffer_rsrc_t rw, rx;
  int ve, vo;          // lane offsets of even and of odd groups of eight rows
  int at, step;        // offset of the wave's first row; bytes of eight rows
};

__device__ __forceinline__ Issue issue_of(const Args& a, const Source& s, const Lanes& ln, int kb, int kb1) {
  Issue i;
  const int left = kb < kb1 ? a.I - kb * kBlock : 0, k = min(kb, kb1 - 1) * kBlock;
  i.ve = ln.ce < left ? ln.dr * a.I + ln.ce : kPast;
  i.vo = ln.co < left ? ln.dr * a.I + ln.co : kPast;
  i.rw = uniform_rsrc(s.w, s.wbytes);
  i.rx = uniform_rsrc(s.x, s.xbytes);
  i.at = __builtin_amdgcn_readfirstlane(ln.row * a.I + k);
  i.step = 8 * a.I;
  return i;
}

template <int BUF, int J>
__device__ __forceinline__ void load(const Lanes& ln, const Issue& i) {
  if constexpr (J < 4)
    dma(ln.dma_x + unsigned(BUF * kOpBytes + J * 1024), i.rx, J & 1 ? i.vo : i.ve, i.at + J * i.step);
  else
    dma(ln.dma_w + unsigned(BUF * kOpBytes + (J - 4) * 1024), i.rw, J & 1 ? i.vo : i.ve, i.at + (J - 4) * i.step);
}

// Both halves of a fragment: 16 rows x 128 columns.
struct Frag { u32x4 h[2]; };

template <int BUF>
__device__ __forceinline__ Frag read_w(const Lanes& ln, int i) {
  return Frag{{*reinterpret_cast<const lds_u32x4*>(ln.w_rd[0] + BUF * kOpBytes + i * 16 * kBlock),
               *reinterpret_cast<const lds_u32x4*>(ln.w_rd[1] + BUF * kOpBytes + i * 16 * kBlock)}};
}
template <int BUF>
__device__ __forceinline__ Frag read_x(const Lanes& ln, int j) {
  return Frag{{*reinterpret_cast<const lds_u32x4*>(ln.x_rd[0] + BUF * kOpBytes + j * 16 * kBlock),
               *reinterpret_cast<const lds_u32x4*>(ln.x_rd[1] + BUF * kOpBytes + j * 16 * kBlock)}};
}

// One block in software-pipelined form.  On entry block kb sits in buffer BUF,
// its x fragments in fb and its W fragments 0..3 in fa; the loads of block kb + 1
// into the other buffer are out.
//   - The first half of the products (W fragments 0..3) frees fa for fragments
//     4..7, the last that are read from BUF.
//   - A few products into the second half, one barrier: every wave holds all of
//     block kb, and block kb + 1 has landed.  From there on block kb + 2 is
//     asked for into BUF, and each x fragment's registers take the next block's
//     as soon as their last products are under way, then fa.
// The loads go out one by one between products: issued together behind a
// barrier they keep every wave from its products until the address units have
// taken them.  Products come in pairs, so that none follows one that adds to the
// same accumulator.
#define TB_FENCE __builtin_amdgcn_sched_barrier(0)
#define TB_MUL(I, F, J, H) acc[I][J] = int8::mma(fa[F].h[H], fb[J].h[H], acc[I][J])
// W fragments I0 and I1 (in fa[F0], fa[F1]) with x fragments J0 and J1; MID between the halves.
#define TB_PAIR(I0, F0, J0, I1, F1, J1, MID) \
  TB_MUL(I0, F0, J0, 0);                     \
  TB_MUL(I1, F1, J1, 0);                     \
  MID;                                       \
  TB_MUL(I0, F0, J0, 1);                     \
  TB_MUL(I1, F1, J1, 1)
#define TB_LOAD(J)      \
  TB_FENCE;             \
  load<BUF, J>(ln, next); \
  TB_FENCE
template <int BUF>
__device__ __forceinline__ void k_step(const Args& a, const Source& s, const Lanes& ln, int kb, int kb1, Frag (&fa)[4],
                                       Frag (&fb)[4], i32x4 (&acc)[8][4]) {
  const Issue next = issue_of(a, s, ln, kb + 2, kb1);
  TB_PAIR(0, 0, 0, 0, 0, 1, );
  TB_PAIR(0, 0, 2, 0, 0, 3, );
  TB_PAIR(1, 1, 0, 1, 1, 1, );
  TB_PAIR(1, 1, 2, 1, 1, 3, );
  TB_FENCE;
  fa[0] = read_w<BUF>(ln, 4);
  fa[1] = read_w<BUF>(ln, 5);
  TB_FENCE;
  TB_PAIR(2, 2, 0, 2, 2, 1, );
  TB_PAIR(2, 2, 2, 2, 2, 3, );
  TB_FENCE;
  fa[2] = read_w<BUF>(ln, 6);
  TB_FENCE;
  TB_PAIR(3, 3, 0, 3, 3, 1, );
  TB_PAIR(3, 3, 2, 3, 3, 3, );
  TB_FENCE;
  fa[3] = read_w<BUF>(ln, 7);
  TB_FENCE;
  TB_PAIR(4, 0, 0, 5, 1, 0, );
  TB_PAIR(4, 0, 1, 5, 1, 1, );
  TB_FENCE;
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  TB_FENCE;
  TB_PAIR(6, 2, 0, 7, 3, 0, TB_LOAD(0));
  TB_FENCE;
  fb[0] = read_x<1 - BUF>(ln, 0);
  TB_LOAD(1);
  TB_PAIR(6, 2, 1, 7, 3, 1, TB_LOAD(2));
  TB_FENCE;
  fb[1] = read_x<1 - BUF>(ln, 1);
  TB_LOAD(3);
  TB_PAIR(4, 0, 2, 5, 1, 2, TB_LOAD(4));
  TB_LOAD(5);
  TB_PAIR(6, 2, 2, 7, 3, 2, TB_LOAD(6));
  TB_FENCE;
  fb[2] = read_x<1 - BUF>(ln, 2);
  TB_LOAD(7);
  TB_PAIR(4, 0, 3, 5, 1, 3, );
  TB_FENCE;
  fa[0] = read_w<1 - BUF>(ln, 0);
  fa[1] = read_w<1 - BUF>(ln, 1);
  TB_FENCE;
  TB_PAIR(6, 2, 3, 7, 3, 3, );
  TB_FENCE;
  fb[3] = read_x<1 - BUF>(ln, 3);
  fa[2] = read_w<1 - BUF>(ln, 2);
  fa[3] = read_w<1 - BUF>(ln, 3);
  TB_FENCE;
}
#undef TB_LOAD
#undef TB_PAIR
#undef TB_MUL
#undef TB_FENCE

__device__ __forceinline__ void k_run(const Args& a, const Source& s, const Lanes& ln, int kb0, int kb1,
                                      i32x4 (&acc)[8][4]) {
  Frag fa[4], fb[4];
  // Block kb0 has landed (the loads of the next one may be out).
  wait_loads<kBlockLoads>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) fb[j] = read_x<0>(ln, j);
#pragma unroll
  for (int i = 0; i < 4; ++i) fa[i] = read_w<0>(ln, i);
  int kb = kb0;
  for (; kb + 1 < kb1; kb += 2) {
    k_step<0>(a, s, ln, kb, kb1, fa, fb, acc);
    k_step<1>(a, s, ln, kb + 1, kb1, fa, fb, acc);
  }
  if (kb < kb1) k_step<0>(a, s, ln, kb, kb1, fa, fb, acc);
  int8::products_issued(acc);
  wait_loads<0>();
  __syncthreads();   // the ring is free
}

template <int BUF>
__device__ __forceinline__ void load_block(const Args& a, const Source& s, const Lanes& ln, int kb, int kb1) {
  const Issue i = issue_of(a, s, ln, kb, kb1);
  load<BUF, 0>(ln, i);
  load<BUF, 1>(ln, i);
  load<BUF, 2>(ln, i);
  load<BUF, 3>(ln, i);
  load<BUF, 4>(ln, i);
  load<BUF, 5>(ln, i);
  load<BUF, 6>(ln, i);
  load<BUF, 7>(ln, i);
}

// The scales of an item's tile (into half `half` of their buffer) and its first
// two blocks (the ring must be free).  Waves 0..3 bring the channels', the others
// the tokens'; scales past the last land as zeros.
__device__ __forceinline__ void prefetch(const Args& a, const Source& s, const Lanes& ln, const Item& it, int half) {
  const bool tokens = ln.w >= 4;
  const int first = (ln.w & 3) * 64, left = max((tokens ? a.M - it.m0 : a.O - it.n0) - first, 0);
  dma_scale<TB_SCALE_F32>(ln.dma_s + unsigned(half * kScales * 4),
                          uniform_rsrc((tokens ? a.xs + it.m0 : a.ws + it.n0) + (left > 0 ? first : 0), min(left, 64) * 4),
                          (int(threadIdx.x) % kWave) * 4, 0);
  load_block<0>(a, s, ln, it.kb0, it.kb1);
  load_block<1>(a, s, ln, it.kb0 + 1, it.kb1);
}

// The wave's 128 outputs x 64 tokens: 16 tokens x 128 bytes at a time through
// its staging area, so that eight lanes write 128 bytes of a token.
template <typename YE>
__device__ __forceinline__ void store_tile(const Args& a, int m0, int n0, const i32x4 (&acc)[8][4], lds_byte* stage,
                                           const float* scales) {
  constexpr int kPer = 8 / int(sizeof(YE));   // W fragments whose 16 outputs make 128 bytes
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4;
  lds_byte* const base = stage + w * kStageBytes;
  lds_byte* const wr = base + lr * kStagePitch + q * 4 * int(sizeof(YE));   // token lr, outputs 4 q (+ 16 i)
  lds_byte* const rd = base + (l >> 3) * kStagePitch + (l & 7) * 16;        // token l / 8 (+ 8 r)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float xs = scales[BT + (w >> 1) * 64 + j * 16 + lr];
#pragma unroll
    for (int h = 0; h < 8 / kPer; ++h) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const f32x4 ws = *reinterpret_cast<const f32x4*>(scales + (w & 1) * 128 + (h * kPer + i) * 16 + q * 4);
        const f32x4 v = int8::scaled(acc[h * kPer + i][j], xs, ws);
        if constexpr (sizeof(YE) == 2)
          *reinterpret_cast<lds_u32x2*>(wr + i * 32) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        else
          *reinterpret_cast<lds_u32x4*>(wr + i * 64) = __builtin_bit_cast(u32x4, v);
      }
      // A wave reads back what it wrote itself, and its LDS operations complete in order.
      asm volatile("" ::: "memory");
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        constexpr int kN = 16 / int(sizeof(YE));   // outputs of 16 bytes
        const u32x4 v = *reinterpret_cast<const lds_u32x4*>(rd + r * 8 * kStagePitch);
        const int t = m0 + (w >> 1) * 64 + j * 16 + r * 8 + (l >> 3);
        const int o = n0 + (w & 1) * 128 + h * kPer * 16 + (l & 7) * kN;
        if (t >= a.M || o >= a.O) continue;
        YE* dst = static_cast<YE*>(a.y) + size_t(t) * a.O + o;
        if (a.wide) {
          *reinterpret_cast<u32x4*>(dst) = v;
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (o + e < a.O) {
              if constexpr (sizeof(YE) == 2) dst[e] = bf16_t{uint16_t(v[e / 2] >> (16 * (e % 2)))};
              else dst[e] = __uint_as_float(v[e]);
            }
        }
      }
      asm volatile("" ::: "memory");
    }
  }
}

template <typename YE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void int8_tiles_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes];
  __shared__ __attribute__((aligned(16))) float scales[2 * kScales];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves * kStageBytes];
  const int g = int(blockIdx.x), G = int(gridDim.x);
  const int pos = a.xcd_major ? (g % 8) * (G / 8) + g / 8 : g;
  const int total = a.split_tiles * a.S + (a.tiles_m * a.tiles_n - a.split_tiles);
  if (pos >= total) return;
  const Lanes ln = make_lanes(ring, scales);
  Item it = item_at(a, pos);
  Source src = source_of(a, it);
  int half = 0;
  prefetch(a, src, ln, it, half);
  for (int v = pos; v < total; v += G) {
    i32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    k_run(a, src, ln, it.kb0, it.kb1, acc);
    const Item cur = it;
    if (v + G < total) {   // the next item's first blocks load while this one is stored
      it = item_at(a, v + G);
      src = source_of(a, it);
      prefetch(a, src, ln, it, 1 - half);
    }
    if (cur.slice < 0) {
      store_tile<YE>(a, cur.m0, cur.n0, acc, (lds_byte*)stage, scales + half * kScales);
    } else {
      i32x4* p = reinterpret_cast<i32x4*>(a.part) +
                 (size_t(cur.slice) * a.split_tiles + cur.u) * kPieces * kThreads + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[(i * 4 + j) * kThreads] = acc[i][j];
    }
    half = 1 - half;
  }
}

// The slices of the cut tiles: one workgroup for 16 of each wave's tokens (x
// fragment j) and 64 of its outputs (W fragments 4 h .. + 3), so that a token's
// outputs leave as a whole line.
template <typename YE>
__global__ __launch_bounds__(kThreads) void int8_tiles_join_kernel(Args a) {
  const int u = int(blockIdx.x) >> 3, j = int(blockIdx.x) & 3, h = (int(blockIdx.x) >> 2) & 1;
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4;
  int m0, n0;
  tile_at(a, u, m0, n0);
  const i32x4* p = reinterpret_cast<const i32x4*>(a.part) + (size_t(u) * kPieces + h * 16 + j) * kThreads + threadIdx.x;
  const size_t next = size_t(a.split_tiles) * kPieces * kThreads;
  i32x4 sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = __builtin_nontemporal_load(p + i * 4 * kThreads);
#pragma unroll 4
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += __builtin_nontemporal_load(p + s * next + i * 4 * kThreads);
  const int t = m0 + (w >> 1) * 64 + j * 16 + lr;
  if (t >= a.M) return;
  const float xs = a.xs[t];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = n0 + (w & 1) * 128 + h * 64 + i * 16 + q * 4;
    if (o >= a.O) continue;
    f32x4 ws;
#pragma unroll
    for (int e = 0; e < 4; ++e) ws[e] = a.ws[min(o + e, a.O - 1)];
    const f32x4 v = int8::scaled(sum[i], xs, ws);
    YE* dst = static_cast<YE*>(a.y) + size_t(t) * a.O + o;
    if (a.wide) {
      if constexpr (sizeof(YE) == 2) *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      else *reinterpret_cast<f32x4*>(dst) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (o + e < a.O) dst[e] = from_f32<YE>(v[e]);
    }
  }
}

template <typename YE>
hipError_t tiles_go(const Int8TilePlan& p, const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((int8_tiles_kernel<YE>), dim3(unsigned(p.grid)), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.S == 1) return e;
  hipLaunchKernelGGL((int8_tiles_join_kernel<YE>), dim3(unsigned(p.split_tiles * 8)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

Int8TilePlan plan_int8_tiles(int64_t m, int64_t out_dim, int64_t in_dim, int cus) {
  Int8TilePlan p{};
  p.tiles_m = int((m + BT - 1) / BT);
  p.tiles_n = int((out_dim + BT - 1) / BT);
  const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n, KB = fp8_blocks(in_dim);
  p.S = 1;
  // What does not fill a round is cut so that its slices do, where that saves
  // more blocks of work than writing, launching and joining the slices cost
  // (about as much as 12 blocks).
  const int64_t rest = tiles % cus;
  if (rest > 0) {
    const int64_t s = std::min<int64_t>({cus / rest, KB / 4, 8});
    if (s > 1 && KB - KB / s > 12) {
      p.S = int(s);
      p.split_tiles = int(rest);
    }
  }
  const int64_t items = tiles - p.split_tiles + int64_t(p.split_tiles) * p.S;
  p.grid = int(std::min<int64_t>(items, cus));
  p.xcd_major = p.grid % 8 == 0;
  p.part_bytes = p.S > 1 ? size_t(p.split_tiles) * p.S * BT * BT * 4 : 0;
  return p;
}

hipError_t launch_int8_tiles(const Int8TilePlan& p, tb_dtype y_dtype, const void* x, const float* xs, const void* w,
                             const float* ws, void* y, int* part, int64_t m, int64_t out_dim, int64_t in_dim,
                             hipStream_t stream) {
  const int wide = out_dim % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  const Args a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, y, part, int(m), int(out_dim),
               int(in_dim), int(fp8_blocks(in_dim)), p.tiles_m, p.tiles_n, p.split_tiles, p.S, p.xcd_major, wide};
  return y_dtype == TB_BF16 ? tiles_go<bf16_t>(p, a, stream) : tiles_go<float>(p, a, stream);
}

}  // namespace tb
