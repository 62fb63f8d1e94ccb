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
// Powers of two as scales go into the matrix instruction itself, which scales
// its operands' exponents: nothing is left for the vector unit.  fp32 scales
// need one multiply-add per result and block (four for each product of 32
// cycles); each product's results are added while the next one runs.
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
constexpr unsigned kRsrcFlags = 0x00020000u;  // buffer descriptor word 3: 32-bit data format
constexpr int kPast = int(0x80000000u);       // lane offset past every buffer: the load returns zeros
// Finished tiles leave through LDS, 16 tokens x 64 outputs of bf16 at a time
// per wave, rows 144 bytes apart, beside the ring.
constexpr int kStagePitch = 144, kStageBytes = 16 * kStagePitch;
static_assert(kRingBytes + kWaves * kStageBytes <= 160 * 1024, "ring and staging fit the LDS");
constexpr int kPieces = 32;                   // pieces of four results per lane and tile

typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

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
  unsigned dma_w, dma_x;   // this wave's 4 KB of each operand in buffer 0
  int row, ce, co;         // load j: row + 8 j, piece ce (even j) or co (odd j)
  lds_byte* w_rd[2];       // the fragment's pieces q and q + 4 of W row wo * 128 + lane % 16
  lds_byte* x_rd[2];       // and of x row wt * 64 + lane % 16
  int xs_off;              // bytes from the tile's first activation scale to those of that row
};

__device__ __forceinline__ Lanes make_lanes(uint8_t* ring, int scale_row_bytes) {
  lds_byte* base = (lds_byte*)ring;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  Lanes ln;
  const unsigned b0 = unsigned(uintptr_t(base));
  ln.dma_w = __builtin_amdgcn_readfirstlane(b0 + unsigned(w) * 4096u);
  ln.dma_x = __builtin_amdgcn_readfirstlane(b0 + unsigned(kBOffset) + unsigned(w) * 4096u);
  ln.xs_off = (wt * 64 + lr) * scale_row_bytes;
  ln.row = w * 32 + (l >> 3);
  ln.ce = (l & 7) ^ ((ln.row >> 1) & 7);
  ln.co = (l & 7) ^ (((ln.row + 8) >> 1) & 7);
  // Fragment rows are 16 apart: the swizzle of row r + 16 i is that of r.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = ((q + 4 * h) ^ ((lr >> 1) & 7)) << 4;
    ln.w_rd[h] = opaque(base + (wo * 128 + lr) * kBlock + piece);
    ln.x_rd[h] = opaque(base + kBOffset + (wt * 64 + lr) * kBlock + piece);
  }
  return ln;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Four direct-to-LDS loads of a wave: load j fills 1 KB at dst + j KB from the
// rows at soff + j * step.  M0 takes one wait state before a load reads it.
// Written as assembly so that the compiler does not drain them before each LDS
// read; wait_dma is the wait.
__device__ __forceinline__ void dma4(unsigned dst, __amdgpu_buffer_rsrc_t r, int ve, int vo, int soff, int step) {
  asm volatile(
      "s_mov_b32 m0, %[d0]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[ve], %[r], %[s0] offen lds\n\t"
      "s_mov_b32 m0, %[d1]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[vo], %[r], %[s1] offen lds\n\t"
      "s_mov_b32 m0, %[d2]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[ve], %[r], %[s2] offen lds\n\t"
      "s_mov_b32 m0, %[d3]\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %[vo], %[r], %[s3] offen lds"
      :
      : [d0] "s"(dst), [d1] "s"(dst + 1024u), [d2] "s"(dst + 2048u), [d3] "s"(dst + 3072u), [ve] "v"(ve), [vo] "v"(vo),
        [r] "s"(r), [s0] "s"(soff), [s1] "s"(soff + step), [s2] "s"(soff + 2 * step), [s3] "s"(soff + 3 * step)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// Every load of this wave has landed.
__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

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
  const uint8_t* xs;
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
  s.xs = static_cast<const uint8_t*>(a.xs) + size_t(it.m0) * a.KB * sizeof(scale_t<SC>);
  s.xsbytes = rows_x * a.KB * int(sizeof(scale_t<SC>));
  // The wave's 128 outputs are one weight block (a block past the last: any will do).
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), blocks = (a.O + kBlock - 1) / kBlock;
  s.ws = static_cast<const scale_t<SC>*>(a.ws) + size_t(min(it.n0 / kBlock + (w & 1), blocks - 1)) * a.KB;
  return s;
}

// Block kb of both operands into LDS buffer BUF; pieces past the reduction, and
// every piece of a block at or past kb1, are fetched from past the buffers and
// so land as zeros without memory traffic.  There is no branch: one here would
// let the compiler move products of a step into the block behind it.
template <int BUF, int SC>
__device__ __forceinline__ void issue(const Args& a, const Source<SC>& s, const Lanes& ln, int kb, int kb1) {
  const int left = kb < kb1 ? a.I - kb * kBlock : 0;
  const int ve = ln.ce * 16 < left ? ln.row * a.I + (ln.ce << 4) : kPast;
  const int vo = ln.co * 16 < left ? ln.row * a.I + (ln.co << 4) : kPast;
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(uniform_ptr(s.w)), 0, __builtin_amdgcn_readfirstlane(s.wbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(uniform_ptr(s.x)), 0, __builtin_amdgcn_readfirstlane(s.xbytes), kRsrcFlags);
  const int soff = __builtin_amdgcn_readfirstlane(min(kb, kb1 - 1) * kBlock), step = 8 * a.I;
  dma4(ln.dma_w + BUF * kOpBytes, rw, ve, vo, soff, step);
  dma4(ln.dma_x + BUF * kOpBytes, rx, ve, vo, soff, step);
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

// The scales of a block as the products take them: bytes for the matrix
// instruction, or xs * ws.
template <int SC> struct Scales;
template <> struct Scales<TB_SCALE_E8M0> { int w, x[4]; };
template <> struct Scales<TB_SCALE_F32> { float x[4]; };

template <int SC>
struct RawScales {
  scale_t<SC> w, x[4];
};

// xs_off: this lane's token of x fragment 0 in the tile, times KB scales.
// Tokens past the last read a zero scale.
template <int SC>
__device__ __forceinline__ RawScales<SC> load_scales(const Args& a, const Source<SC>& s, int xs_off, int kb) {
  RawScales<SC> r;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(uniform_ptr(s.xs)), 0, __builtin_amdgcn_readfirstlane(s.xsbytes), kRsrcFlags);
  r.w = s.ws[kb];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int soff = __builtin_amdgcn_readfirstlane((j * 16 * a.KB + kb) * int(sizeof(scale_t<SC>)));
    if constexpr (SC == TB_SCALE_E8M0)
      r.x[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, xs_off, soff, 0);
    else
      r.x[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, xs_off, soff, 0));
  }
  return r;
}

__device__ __forceinline__ Scales<TB_SCALE_E8M0> use_scales(const RawScales<TB_SCALE_E8M0>& r) {
  return {int(r.w), {int(r.x[0]), int(r.x[1]), int(r.x[2]), int(r.x[3])}};
}
__device__ __forceinline__ Scales<TB_SCALE_F32> use_scales(const RawScales<TB_SCALE_F32>& r) {
  return {{r.x[0] * r.w, r.x[1] * r.w, r.x[2] * r.w, r.x[3] * r.w}};
}

// The product of W fragment i (f) and x fragment j into acc[i][j].  With fp32
// scales its results stay in `pend` and are added, to where PI, PJ say, under
// the product that follows (PI < 0: nothing is pending).
template <int I, int J, int PI, int PJ>
__device__ __forceinline__ void product(const i32x8& f, const i32x8& fx, const Scales<TB_SCALE_E8M0>& sc,
                                        f32x4 (&acc)[8][4], f32x4&) {
  acc[I][J] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f, fx, acc[I][J], 0, 0, 0, sc.w, 0, sc.x[J]);
}
template <int I, int J, int PI, int PJ>
__device__ __forceinline__ void product(const i32x8& f, const i32x8& fx, const Scales<TB_SCALE_F32>& sc,
                                        f32x4 (&acc)[8][4], f32x4& pend) {
  const f32x4 p =
      __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f, fx, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
  if constexpr (PI >= 0) acc[PI][PJ] += pend * sc.x[PJ];
  pend = p;
}
__device__ __forceinline__ void finish_block(const Scales<TB_SCALE_E8M0>&, f32x4 (&)[8][4], f32x4&) {}
__device__ __forceinline__ void finish_block(const Scales<TB_SCALE_F32>& sc, f32x4 (&acc)[8][4], f32x4& pend) {
  acc[7][3] += pend * sc.x[3];
}

// W fragments 2 S and 2 S + 1 with the four x fragments.
template <int S, int SC>
__device__ __forceinline__ void mma_pair(const i32x8 (&fa)[2], const i32x8 (&fb)[4], const Scales<SC>& sc,
                                         f32x4 (&acc)[8][4], f32x4& pend) {
  product<2 * S, 0, 2 * S - 1, 3>(fa[0], fb[0], sc, acc, pend);
  product<2 * S, 1, 2 * S, 0>(fa[0], fb[1], sc, acc, pend);
  product<2 * S, 2, 2 * S, 1>(fa[0], fb[2], sc, acc, pend);
  product<2 * S, 3, 2 * S, 2>(fa[0], fb[3], sc, acc, pend);
  product<2 * S + 1, 0, 2 * S, 3>(fa[1], fb[0], sc, acc, pend);
  product<2 * S + 1, 1, 2 * S + 1, 0>(fa[1], fb[1], sc, acc, pend);
  product<2 * S + 1, 2, 2 * S + 1, 1>(fa[1], fb[2], sc, acc, pend);
  product<2 * S + 1, 3, 2 * S + 1, 2>(fa[1], fb[3], sc, acc, pend);
}

// One block in software-pipelined form.  On entry block kb sits in buffer BUF,
// its x fragments in fb and W fragments 0, 1 in fa0, its scales in sc; the
// loads of block kb + 1 into the other buffer and of its scales (raw) are in
// flight.  The barrier falls before the last quarter of the products, once
// block kb + 1 has landed and every wave holds its last fragments of BUF;
// block kb + 2 is then issued into BUF.  The last quarter goes x fragment by x
// fragment, so that each one's registers take the next block's as soon as its
// two products are under way.
template <int BUF, int SC>
__device__ __forceinline__ void k_step(const Args& a, const Source<SC>& s, const Lanes& ln, int kb, int kb1,
                                       i32x8 (&fa0)[2], i32x8 (&fa1)[2], i32x8 (&fb)[4], Scales<SC>& sc,
                                       RawScales<SC>& raw, f32x4 (&acc)[8][4]) {
  f32x4 pend;
#define TB_FENCE __builtin_amdgcn_sched_barrier(0)
  fa1[0] = read_w<BUF>(ln, 2);
  fa1[1] = read_w<BUF>(ln, 3);
  TB_FENCE;
  mma_pair<0>(fa0, fb, sc, acc, pend);
  TB_FENCE;
  fa0[0] = read_w<BUF>(ln, 4);
  fa0[1] = read_w<BUF>(ln, 5);
  TB_FENCE;
  mma_pair<1>(fa1, fb, sc, acc, pend);
  TB_FENCE;
  fa1[0] = read_w<BUF>(ln, 6);
  fa1[1] = read_w<BUF>(ln, 7);
  TB_FENCE;
  mma_pair<2>(fa0, fb, sc, acc, pend);
  TB_FENCE;
  wait_dma();
  __syncthreads();
  const Scales<SC> now = sc;
  sc = use_scales(raw);
  fa0[0] = read_w<1 - BUF>(ln, 0);
  fa0[1] = read_w<1 - BUF>(ln, 1);
  TB_FENCE;
  raw = load_scales<SC>(a, s, ln.xs_off, min(kb + 2, kb1 - 1));
  issue<BUF, SC>(a, s, ln, kb + 2, kb1);
  TB_FENCE;
  product<6, 0, 5, 3>(fa1[0], fb[0], now, acc, pend);
  product<7, 0, 6, 0>(fa1[1], fb[0], now, acc, pend);
  TB_FENCE;
  fb[0] = read_x<1 - BUF>(ln, 0);
  TB_FENCE;
  product<6, 1, 7, 0>(fa1[0], fb[1], now, acc, pend);
  product<7, 1, 6, 1>(fa1[1], fb[1], now, acc, pend);
  TB_FENCE;
  fb[1] = read_x<1 - BUF>(ln, 1);
  TB_FENCE;
  product<6, 2, 7, 1>(fa1[0], fb[2], now, acc, pend);
  product<7, 2, 6, 2>(fa1[1], fb[2], now, acc, pend);
  TB_FENCE;
  fb[2] = read_x<1 - BUF>(ln, 2);
  TB_FENCE;
  product<6, 3, 7, 2>(fa1[0], fb[3], now, acc, pend);
  product<7, 3, 6, 3>(fa1[1], fb[3], now, acc, pend);
  TB_FENCE;
  fb[3] = read_x<1 - BUF>(ln, 3);
  finish_block(now, acc, pend);
  TB_FENCE;
#undef TB_FENCE
}

template <int SC>
__device__ __forceinline__ void k_run(const Args& a, const Source<SC>& s, const Lanes& ln, int kb0, int kb1,
                                      RawScales<SC> first, RawScales<SC> raw, f32x4 (&acc)[8][4]) {
  i32x8 fa0[2], fa1[2], fb[4];
  wait_dma();
  __syncthreads();
  Scales<SC> sc = use_scales(first);
#pragma unroll
  for (int j = 0; j < 4; ++j) fb[j] = read_x<0>(ln, j);
  fa0[0] = read_w<0>(ln, 0);
  fa0[1] = read_w<0>(ln, 1);
  int kb = kb0;
  for (; kb + 1 < kb1; kb += 2) {
    k_step<0, SC>(a, s, ln, kb, kb1, fa0, fa1, fb, sc, raw, acc);
    k_step<1, SC>(a, s, ln, kb + 1, kb1, fa0, fa1, fb, sc, raw, acc);
  }
  if (kb < kb1) k_step<0, SC>(a, s, ln, kb, kb1, fa0, fa1, fb, sc, raw, acc);
  wait_dma();
  __syncthreads();   // the ring is free
}

template <int SC>
__device__ __forceinline__ void prefetch(const Args& a, const Source<SC>& s, const Lanes& ln, const Item& it,
                                         RawScales<SC>& first, RawScales<SC>& raw) {
  first = load_scales<SC>(a, s, ln.xs_off, it.kb0);
  raw = load_scales<SC>(a, s, ln.xs_off, min(it.kb0 + 1, a.KB - 1));
  issue<0, SC>(a, s, ln, it.kb0, it.kb1);
  issue<1, SC>(a, s, ln, it.kb0 + 1, it.kb1);
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
  __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves * kStageBytes];
  const int g = int(blockIdx.x), G = int(gridDim.x);
  const int pos = a.xcd_major ? (g % 8) * (G / 8) + g / 8 : g;
  const int total = a.split_tiles * a.S + (a.tiles_m * a.tiles_n - a.split_tiles);
  if (pos >= total) return;
  const Lanes ln = make_lanes(ring, a.KB * int(sizeof(scale_t<SC>)));
  Item it = item_at(a, pos);
  Source<SC> src = source_of<SC>(a, it);
  RawScales<SC> first, raw;
  prefetch<SC>(a, src, ln, it, first, raw);
  for (int v = pos; v < total; v += G) {
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    k_run<SC>(a, src, ln, it.kb0, it.kb1, first, raw, acc);
    const Item cur = it;
    if (v + G < total) {   // the next item's first blocks load while this one is stored
      it = item_at(a, v + G);
      src = source_of<SC>(a, it);
      prefetch<SC>(a, src, ln, it, first, raw);
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

// The slices of the cut tiles, added in slice order: one workgroup for four
// outputs' pieces (i) of a tile, all its tokens.
__global__ __launch_bounds__(kThreads) void fp8_tiles_join_kernel(Args a) {
  const int u = int(blockIdx.x) >> 3, i = int(blockIdx.x) & 7;
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4;
  int m0, n0;
  tile_at(a, u, m0, n0);
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (size_t(u) * kPieces + i * 4) * kThreads + threadIdx.x;
  f32x4 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = p[j * kThreads];
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += p[(size_t(s) * a.split_tiles * kPieces + j) * kThreads];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = m0 + (w >> 1) * 64 + j * 16 + lr, o = n0 + (w & 1) * 128 + i * 16 + q * 4;
    if (t >= a.M || o >= a.O) continue;
    bf16_t* dst = a.y + size_t(t) * a.O + o;
    if (a.wide) {
      *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16(sum[j][0], sum[j][1]),
                                             pack_bf16(sum[j][2], sum[j][3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (o + e < a.O) dst[e] = bf16_t{f32_to_bf16(sum[j][e])};
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

hipError_t launch_fp8_tiles(const Fp8TilePlan& p, tb_scale scale_type, const void* x, const void* xs, const void* w,
                            const void* ws, void* y, float* part, int64_t m, int64_t out_dim, int64_t in_dim,
                            hipStream_t stream) {
  const int wide = out_dim % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  const Args a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, static_cast<bf16_t*>(y), part,
               int(m), int(out_dim), int(in_dim), int(fp8_blocks(in_dim)), p.tiles_m, p.tiles_n, p.split_tiles, p.S,
               p.xcd_major, wide};
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
