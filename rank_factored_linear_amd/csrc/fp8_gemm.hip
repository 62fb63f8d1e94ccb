// The 8-bit block-scaled product for many tokens and bf16 results: output
// tiles of 256 outputs x 256 tokens (the formula and the other kernels are in
// fp8_product.hip).
//
// Eight waves, each 128 outputs x 64 tokens in products of 16 x 16 x 128, so
// that a wave's outputs share one weight scale and a lane's four outputs one
// activation scale.  The reduction runs block by block (128 bytes of each of
// 512 rows, 64 KB) through a two-buffer LDS ring filled by direct-to-LDS
// loads; rows keep their 16-byte pieces XOR-swizzled by (row >> 1) & 7, so the
// fragment reads of 16 consecutive rows meet all 64 banks.
//
// Scales of both types, turned into floats, cost one multiply-add per result
// and block (four for each product of 32 cycles); each product's results are
// added while the next one runs.
//
// 4096 x 5376 x 8192, powers of two: 161 us of a call of 194; 4096 x 21504 x
// 5376, fp32 scales: 420 us (2.26 PFLOP/s) of a call of 444 (2.13), calls 438 to
// 472 from one card to another.  Both under the power limit: in a burst after
// idling the second takes 430 us at first, 470 from the fourth call to about the
// fifteenth, and settles at 420.
//
// Workgroups are persistent, one per compute unit, and take whole tiles in
// rounds.  What is left over for a last, partly filled round is cut into
// slices of in_dim, whose fp32 sums a second launch adds in slice order.
#include "fp8_device.h"

#include <algorithm>

namespace tb {

namespace {

using namespace fp8;

constexpr int BT = 256;                       // outputs and tokens of a tile
constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kOpBytes = BT * kBlock;         // one operand's block in LDS
constexpr int kBOffset = 2 * kOpBytes;        // ring [W0][W1][x0][x1]
constexpr int kRingBytes = 4 * kOpBytes;
constexpr int kScaleBytes = 2 * kWaves * 256; // each wave's 64 activation scales of two blocks
// Finished tiles leave through LDS, 16 tokens x 64 outputs of bf16 at a time
// per wave, rows 144 bytes apart, beside the ring.
constexpr int kStagePitch = 144, kStageBytes = 16 * kStagePitch;
static_assert(kRingBytes + kScaleBytes + kWaves * kStageBytes <= 160 * 1024, "ring, scales and staging fit the LDS");
static_assert(int64_t(BT) * TB_FP8_MAX_IN_DIM < (int64_t(1) << 31), "a tile's rows are addressed with 31-bit offsets");
constexpr int kPieces = 32;                   // pieces of four results per lane and tile

struct Args {
  const uint8_t* x;
  const void* xs;
  const uint8_t* w;
  const void* ws;
  bf16_t* y;
  float* part;       // [S][split_tiles][kPieces][kThreads] pieces of four
  int M, O, I, KB;
  int tiles_m, tiles_n;
  int split_tiles, S;   // the first split_tiles tiles are cut into S slices
  int xcd_major;        // workgroup g takes position (g % 8) * (grid / 8) + g / 8
  int wide;             // y 16-byte aligned and O a multiple of 8
  int64_t xs_t, xs_k;   // strides of xs (ScaleStrides)
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
  int row, tok;         // first row of its loads in the tile; its first token
  int ce, co;                    // lane offsets' pieces (bytes) in loads of even and of odd groups of eight rows
  int dr;                        // row of the lane in a load
  lds_byte* w_rd[2];             // the fragment's pieces q and q + 4 of W row wo * 128 + lane % 16
  lds_byte* x_rd[2];             // and of x row wt * 64 + lane % 16
  lds_byte* s_rd;                // the scale of that x row
};

__device__ __forceinline__ Lanes make_lanes(uint8_t* ring, uint8_t* scales) {
  lds_byte* base = (lds_byte*)ring;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  Lanes ln;
  ln.row = w * 32;
  ln.tok = wt * 64;
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
  ln.s_rd = opaque((lds_byte*)scales + w * 256 + lr * 4);
  return ln;
}

__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t(hi) << 32) | lo);
}

// One item's operands and scales (all uniform; lanes address them by offset).
template <int SC>
struct Source {
  const uint8_t* w;
  const uint8_t* x;
  const scale_t<SC>* xs;
  int wbytes, xbytes, xsbytes;
  const scale_t<SC>* ws;
};

template <int SC>
__device__ __forceinline__ Source<SC> source_of(const Args& a, const Item& it) {
  Source<SC> s;
  const int rows_w = min(a.O - it.n0, BT), rows_x = min(a.M - it.m0, BT);
  s.w = a.w + size_t(it.n0) * a.I;
  s.x = a.x + size_t(it.m0) * a.I;
  s.wbytes = rows_w * a.I;
  s.xbytes = rows_x * a.I;
  s.xs = static_cast<const scale_t<SC>*>(a.xs) + it.m0 * a.xs_t;
  s.xsbytes = int(((rows_x - 1) * a.xs_t + 1) * int64_t(sizeof(scale_t<SC>)));
  // The wave's 128 outputs are one weight block (a block past the last: any will do).
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), blocks = (a.O + kBlock - 1) / kBlock;
  s.ws = static_cast<const scale_t<SC>*>(a.ws) + size_t(min(it.n0 / kBlock + (w & 1), blocks - 1)) * a.KB;
  return s;
}

// The loads of a block: 0..3 its x rows, 4..7 its W rows, 8 its activation
// scales.  Pieces past the
// reduction, rows past the matrix and every piece of a block at or past kb1 are
// fetched from past the buffers and so land as zeros without memory traffic.
// There is no branch: one here would let the compiler move products of a step
// into the block behind it, and the waits count loads.
constexpr int kBlockLoads = 9;

template <int SC>
struct Issue {
  __amdgpu_buffer_rsrc_t rw, rx, rs;
  int ve, vo, vs;      // lane offsets of even and of odd groups of eight rows; of the scales
  int x, w;            // offsets of the wave's first rows
  int step;            // bytes of eight rows
};

template <int SC>
__device__ __forceinline__ Issue<SC> issue_of(const Args& a, const Source<SC>& s, const Lanes& ln, int kb, int kb1) {
  Issue<SC> i;
  const int left = kb < kb1 ? a.I - kb * kBlock : 0, k = min(kb, kb1 - 1) * kBlock, n = int(sizeof(scale_t<SC>));
  i.ve = ln.ce < left ? ln.dr * a.I + ln.ce : kPast;
  i.vo = ln.co < left ? ln.dr * a.I + ln.co : kPast;
  i.vs = (ln.tok + int(threadIdx.x) % kWave) * int(a.xs_t) * n;
  i.rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(uniform_ptr(s.w)), 0,
                                           __builtin_amdgcn_readfirstlane(s.wbytes), kRsrcFlags);
  i.rx = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(uniform_ptr(s.x)), 0,
                                           __builtin_amdgcn_readfirstlane(s.xbytes), kRsrcFlags);
  i.rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(uniform_ptr(reinterpret_cast<const uint8_t*>(s.xs + min(kb, kb1 - 1) * a.xs_k))), 0,
                                           __builtin_amdgcn_readfirstlane(s.xsbytes), kRsrcFlags);
  i.x = __builtin_amdgcn_readfirstlane(ln.row * a.I + k);
  i.w = __builtin_amdgcn_readfirstlane(ln.row * a.I + k);
  i.step = 8 * a.I;
  return i;
}

template <int BUF, int J, int SC>
__device__ __forceinline__ void load(const Lanes& ln, const Issue<SC>& i) {
  if constexpr (J < 4)
    dma(ln.dma_x + unsigned(BUF * kOpBytes + J * 1024), i.rx, J & 1 ? i.vo : i.ve, i.x + J * i.step);
  else if constexpr (J < 8) {
    dma(ln.dma_w + unsigned(BUF * kOpBytes + (J - 4) * 1024), i.rw, J & 1 ? i.vo : i.ve, i.w + (J - 4) * i.step);
  } else
    dma_scale<SC>(ln.dma_s + unsigned(BUF * kWaves * 256), i.rs, i.vs, 0);
}

template <int BUF>
__device__ __forceinline__ i32x8 read_w(const Lanes& ln, int i) {
  return join(*reinterpret_cast<const lds_u32x4*>(ln.w_rd[0] + BUF * kOpBytes + i * 16 * kBlock),
              *reinterpret_cast<const lds_u32x4*>(ln.w_rd[1] + BUF * kOpBytes + i * 16 * kBlock));
}
template <int BUF>
__device__ __forceinline__ i32x8 read_x(const Lanes& ln, int j) {
  return join(*reinterpret_cast<const lds_u32x4*>(ln.x_rd[0] + BUF * kOpBytes + j * 16 * kBlock),
              *reinterpret_cast<const lds_u32x4*>(ln.x_rd[1] + BUF * kOpBytes + j * 16 * kBlock));
}

// xs * ws of the lane's token in each x fragment.
struct Scales { float x[4]; };

template <int BUF, int SC>
__device__ __forceinline__ Scales read_scales(const Source<SC>& s, const Lanes& ln, int kb) {
  Scales r;
  const float w = scale_value(s.ws[kb]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t raw = *reinterpret_cast<const lds_u32*>(ln.s_rd + BUF * (kWaves * 256) + j * 64);
    r.x[j] = (SC == TB_SCALE_E8M0 ? scale_value(uint8_t(raw)) : __uint_as_float(raw)) * w;
  }
  return r;
}

// The product of W fragment I (f) and x fragment J for acc[I][J].  Its results
// stay in `pend` and are scaled and added, to where PI, PJ say, under the
// product that follows (PI < 0: nothing is pending).
template <int I, int J, int PI, int PJ>
__device__ __forceinline__ void product(const i32x8& f, const i32x8& fx, const Scales& sc, f32x4 (&acc)[8][4],
                                        f32x4& pend) {
  const f32x4 p =
      __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f, fx, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
  if constexpr (PI >= 0) acc[PI][PJ] += pend * sc.x[PJ];
  pend = p;
}

// One block in software-pipelined form.  On entry block kb sits in buffer BUF,
// its x fragments in fb, its W fragments 0..3 in fa0 and fa1 and its scales in
// sc; the loads of block kb + 1 into the other buffer are out.
//   - The first half of the products (W fragments 0..3) frees fa0 and fa1 for
//     fragments 4..7, the last that are read from BUF.
//   - A few products into the second half, one barrier: every wave holds all of
//     block kb, and block kb + 1 has landed.  From there on block kb + 2 is
//     asked for into BUF, and each x fragment's registers take the next block's
//     as soon as their last products are under way, then fa0 and fa1.  So the
//     reads of a block are spread over half a step (packed into its last
//     quarter they outlast the products there).
// The loads go out one by one between products: issued together behind a
// barrier they keep every wave from its products until the address units have
// taken them.
#define TB_FENCE __builtin_amdgcn_sched_barrier(0)
#define TB_LOAD(J)              \
  TB_FENCE;                     \
  load<BUF, J, SC>(ln, next);   \
  TB_FENCE
template <int BUF, int SC>
__device__ __forceinline__ void k_step(const Args& a, const Source<SC>& s, const Lanes& ln, int kb, int kb1,
                                       i32x8 (&fa0)[2], i32x8 (&fa1)[2], i32x8 (&fb)[4], Scales& sc,
                                       f32x4 (&acc)[8][4]) {
  f32x4 pend;
  const Issue<SC> next = issue_of<SC>(a, s, ln, kb + 2, kb1);
  product<0, 0, -1, 3>(fa0[0], fb[0], sc, acc, pend);
  product<0, 1, 0, 0>(fa0[0], fb[1], sc, acc, pend);
  product<0, 2, 0, 1>(fa0[0], fb[2], sc, acc, pend);
  product<0, 3, 0, 2>(fa0[0], fb[3], sc, acc, pend);
  product<1, 0, 0, 3>(fa0[1], fb[0], sc, acc, pend);
  product<1, 1, 1, 0>(fa0[1], fb[1], sc, acc, pend);
  product<1, 2, 1, 1>(fa0[1], fb[2], sc, acc, pend);
  product<1, 3, 1, 2>(fa0[1], fb[3], sc, acc, pend);
  TB_FENCE;
  fa0[0] = read_w<BUF>(ln, 4);
  fa0[1] = read_w<BUF>(ln, 5);
  TB_FENCE;
  product<2, 0, 1, 3>(fa1[0], fb[0], sc, acc, pend);
  product<2, 1, 2, 0>(fa1[0], fb[1], sc, acc, pend);
  product<2, 2, 2, 1>(fa1[0], fb[2], sc, acc, pend);
  product<2, 3, 2, 2>(fa1[0], fb[3], sc, acc, pend);
  TB_FENCE;
  fa1[0] = read_w<BUF>(ln, 6);
  TB_FENCE;
  product<3, 0, 2, 3>(fa1[1], fb[0], sc, acc, pend);
  product<3, 1, 3, 0>(fa1[1], fb[1], sc, acc, pend);
  product<3, 2, 3, 1>(fa1[1], fb[2], sc, acc, pend);
  product<3, 3, 3, 2>(fa1[1], fb[3], sc, acc, pend);
  TB_FENCE;
  fa1[1] = read_w<BUF>(ln, 7);
  TB_FENCE;
  product<4, 0, 3, 3>(fa0[0], fb[0], sc, acc, pend);
  product<5, 0, 4, 0>(fa0[1], fb[0], sc, acc, pend);
  product<4, 1, 5, 0>(fa0[0], fb[1], sc, acc, pend);
  product<5, 1, 4, 1>(fa0[1], fb[1], sc, acc, pend);
  TB_FENCE;
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  const Scales now = sc;
  sc = read_scales<1 - BUF, SC>(s, ln, min(kb + 1, kb1 - 1));
  TB_FENCE;
  product<6, 0, 5, 1>(fa1[0], fb[0], now, acc, pend);
  TB_LOAD(0);
  product<7, 0, 6, 0>(fa1[1], fb[0], now, acc, pend);
  TB_FENCE;
  fb[0] = read_x<1 - BUF>(ln, 0);
  TB_LOAD(1);
  product<6, 1, 7, 0>(fa1[0], fb[1], now, acc, pend);
  TB_LOAD(2);
  product<7, 1, 6, 1>(fa1[1], fb[1], now, acc, pend);
  TB_FENCE;
  fb[1] = read_x<1 - BUF>(ln, 1);
  TB_LOAD(3);
  product<4, 2, 7, 1>(fa0[0], fb[2], now, acc, pend);
  TB_LOAD(4);
  product<5, 2, 4, 2>(fa0[1], fb[2], now, acc, pend);
  TB_LOAD(5);
  product<6, 2, 5, 2>(fa1[0], fb[2], now, acc, pend);
  TB_LOAD(6);
  product<7, 2, 6, 2>(fa1[1], fb[2], now, acc, pend);
  TB_FENCE;
  fb[2] = read_x<1 - BUF>(ln, 2);
  TB_LOAD(7);
  product<4, 3, 7, 2>(fa0[0], fb[3], now, acc, pend);
  product<5, 3, 4, 3>(fa0[1], fb[3], now, acc, pend);
  TB_FENCE;
  fa0[0] = read_w<1 - BUF>(ln, 0);
  fa0[1] = read_w<1 - BUF>(ln, 1);
  TB_LOAD(8);
  product<6, 3, 5, 3>(fa1[0], fb[3], now, acc, pend);
  product<7, 3, 6, 3>(fa1[1], fb[3], now, acc, pend);
  TB_FENCE;
  fb[3] = read_x<1 - BUF>(ln, 3);
  fa1[0] = read_w<1 - BUF>(ln, 2);
  fa1[1] = read_w<1 - BUF>(ln, 3);
  acc[7][3] += pend * now.x[3];
  TB_FENCE;
}
#undef TB_LOAD
#undef TB_FENCE

template <int SC>
__device__ __forceinline__ void k_run(const Args& a, const Source<SC>& s, const Lanes& ln, int kb0, int kb1,
                                      f32x4 (&acc)[8][4]) {
  i32x8 fa0[2], fa1[2], fb[4];
  // Block kb0 has landed (the nine loads of the next one may be out).
  wait_loads<kBlockLoads>();
  __syncthreads();
  Scales sc = read_scales<0, SC>(s, ln, kb0);
#pragma unroll
  for (int j = 0; j < 4; ++j) fb[j] = read_x<0>(ln, j);
  fa0[0] = read_w<0>(ln, 0);
  fa0[1] = read_w<0>(ln, 1);
  fa1[0] = read_w<0>(ln, 2);
  fa1[1] = read_w<0>(ln, 3);
  int kb = kb0;
  for (; kb + 1 < kb1; kb += 2) {
    k_step<0, SC>(a, s, ln, kb, kb1, fa0, fa1, fb, sc, acc);
    k_step<1, SC>(a, s, ln, kb + 1, kb1, fa0, fa1, fb, sc, acc);
  }
  if (kb < kb1) k_step<0, SC>(a, s, ln, kb, kb1, fa0, fa1, fb, sc, acc);
  wait_loads<0>();
  __syncthreads();   // the ring is free
}

template <int BUF, int SC>
__device__ __forceinline__ void load_block(const Args& a, const Source<SC>& s, const Lanes& ln, int kb, int kb1) {
  const Issue<SC> i = issue_of<SC>(a, s, ln, kb, kb1);
  load<BUF, 0, SC>(ln, i);
  load<BUF, 1, SC>(ln, i);
  load<BUF, 2, SC>(ln, i);
  load<BUF, 3, SC>(ln, i);
  load<BUF, 4, SC>(ln, i);
  load<BUF, 5, SC>(ln, i);
  load<BUF, 6, SC>(ln, i);
  load<BUF, 7, SC>(ln, i);
  load<BUF, 8, SC>(ln, i);
}

// The first two blocks of an item (the ring must be free).
template <int SC>
__device__ __forceinline__ void prefetch(const Args& a, const Source<SC>& s, const Lanes& ln, const Item& it) {
  load_block<0, SC>(a, s, ln, it.kb0, it.kb1);
  load_block<1, SC>(a, s, ln, it.kb0 + 1, it.kb1);
}

// The wave's 128 outputs x 64 tokens as bf16: 16 tokens x 64 outputs at a time
// through its staging area, so that eight lanes write 128 bytes of a token.
__device__ __forceinline__ void store_tile(const Args& a, int m0, int n0, const f32x4 (&acc)[8][4], lds_byte* stage) {
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4;
  lds_byte* const base = stage + w * kStageBytes;
  lds_byte* const wr = base + lr * kStagePitch + q * 8;                  // token lr, outputs 4 q (+ 16 i)
  lds_byte* const rd = base + (l >> 3) * kStagePitch + (l & 7) * 16;     // token l / 8 (+ 8 r), outputs 8 (l % 8)
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4& v = acc[4 * h + i][j];
        *reinterpret_cast<lds_u32x2*>(wr + i * 32) =
            u32x2{pack_bf16(v[0], v[1]),
                  pack_bf16(v[2], v[3])};
      }
      // A wave reads back what it wrote itself, and its LDS operations complete in order.
      asm volatile("" ::: "memory");
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const u32x4 v = *reinterpret_cast<const lds_u32x4*>(rd + r * 8 * kStagePitch);
        const int t = m0 + (w >> 1) * 64 + j * 16 + r * 8 + (l >> 3), o = n0 + (w & 1) * 128 + h * 64 + (l & 7) * 8;
        if (t >= a.M || o >= a.O) continue;
        bf16_t* dst = a.y + size_t(t) * a.O + o;
        if (a.wide) {
          *reinterpret_cast<u32x4*>(dst) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (o + e < a.O) dst[e] = bf16_t{uint16_t(v[e / 2] >> (16 * (e % 2)))};
        }
      }
      asm volatile("" ::: "memory");
    }
}

template <int SC>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void fp8_tiles_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRingBytes];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kScaleBytes];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves * kStageBytes];
  const int g = int(blockIdx.x), G = int(gridDim.x);
  const int pos = a.xcd_major ? (g % 8) * (G / 8) + g / 8 : g;
  const int total = a.split_tiles * a.S + (a.tiles_m * a.tiles_n - a.split_tiles);
  if (pos >= total) return;
  const Lanes ln = make_lanes(ring, scales);
  Item it = item_at(a, pos);
  Source<SC> src = source_of<SC>(a, it);
  prefetch<SC>(a, src, ln, it);
  for (int v = pos; v < total; v += G) {
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    k_run<SC>(a, src, ln, it.kb0, it.kb1, acc);
    const Item cur = it;
    if (v + G < total) {   // the next item's first blocks load while this one is stored
      it = item_at(a, v + G);
      src = source_of<SC>(a, it);
      prefetch<SC>(a, src, ln, it);
    }
    if (cur.slice < 0) {
      store_tile(a, cur.m0, cur.n0, acc, (lds_byte*)stage);
    } else {
      f32x4* p = reinterpret_cast<f32x4*>(a.part) +
                 (size_t(cur.slice) * a.split_tiles + cur.u) * kPieces * kThreads + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[(i * 4 + j) * kThreads] = acc[i][j];
    }
  }
}

// The slices of the cut tiles, added in slice order: one workgroup for 16 of
// each wave's tokens (x fragment j) and 64 of its outputs (W fragments 4 h ..
// + 3), so that a token's outputs leave as a whole line.
__global__ __launch_bounds__(kThreads) void fp8_tiles_join_kernel(Args a) {
  const int u = int(blockIdx.x) >> 3, j = int(blockIdx.x) & 3, h = (int(blockIdx.x) >> 2) & 1;
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4;
  int m0, n0;
  tile_at(a, u, m0, n0);
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (size_t(u) * kPieces + h * 16 + j) * kThreads + threadIdx.x;
  const size_t next = size_t(a.split_tiles) * kPieces * kThreads;
  f32x4 sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = __builtin_nontemporal_load(p + i * 4 * kThreads);
#pragma unroll 4
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += __builtin_nontemporal_load(p + s * next + i * 4 * kThreads);
  const int t = m0 + (w >> 1) * 64 + j * 16 + lr;
  if (t >= a.M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = n0 + (w & 1) * 128 + h * 64 + i * 16 + q * 4;
    if (o >= a.O) continue;
    bf16_t* dst = a.y + size_t(t) * a.O + o;
    if (a.wide) {
      *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16(sum[i][0], sum[i][1]), pack_bf16(sum[i][2], sum[i][3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (o + e < a.O) dst[e] = bf16_t{f32_to_bf16(sum[i][e])};
    }
  }
}

}  // namespace

Fp8TilePlan plan_fp8_tiles(int64_t m, int64_t out_dim, int64_t in_dim, int cus) {
  Fp8TilePlan p{};
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

hipError_t launch_fp8_tiles(const Fp8TilePlan& p, tb_scale scale_type, const void* x, const void* xs, ScaleStrides ss,
                            const void* w, const void* ws, void* y, float* part, int64_t m, int64_t out_dim, int64_t in_dim,
                            hipStream_t stream) {
  const int wide = out_dim % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  const Args a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, static_cast<bf16_t*>(y), part,
               int(m), int(out_dim), int(in_dim), int(fp8_blocks(in_dim)), p.tiles_m, p.tiles_n, p.split_tiles, p.S,
               p.xcd_major, wide, ss.token, ss.block};
  const dim3 grid(unsigned(p.grid)), block(kThreads);
  if (scale_type == TB_SCALE_E8M0)
    hipLaunchKernelGGL(fp8_tiles_kernel<TB_SCALE_E8M0>, grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL(fp8_tiles_kernel<TB_SCALE_F32>, grid, block, 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.S == 1) return e;
  hipLaunchKernelGGL(fp8_tiles_join_kernel, dim3(unsigned(p.split_tiles * 8)), block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace tb
