// y = Q(x) . Wq^T in 8-bit blocks:
//   y[t, o] = sum_b xs[t, b] ws[o / 128, b] sum_{i in block b} xq[t, i] wq[o, i]
// over blocks b of 128 columns.  A block's inner sum is one matrix-core product
// of depth 128; its fp32 result is scaled by xs * ws (one fp32
// product) and added in fp32 in block order.  y is rounded once.
//
// W's rows are the products' A operand (output rows), x's the B operand
// (output columns): a lane then holds four consecutive outputs of one token,
// whose activation scale is one register, while the weight scale is uniform.
#include "fp8_device.h"

#include <algorithm>

namespace tb {

namespace {

using namespace fp8;

template <typename YE>
__device__ __forceinline__ void store_out4(YE* y, const f32x4& v, int n, bool wide) {
  if constexpr (sizeof(YE) == 2) {
    if (wide) {
      *reinterpret_cast<u32x2*>(y) = u32x2{pack_bf16(v[0], v[1]),
                                           pack_bf16(v[2], v[3])};
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

// ---------------------------------------------------------------------------
// Few tokens (m <= 64): the weight streams once, at HBM rate.
//
// Each workgroup owns an equal share of the output rows (decode_rows), in tiles
// of 16 that need not be full: rows past its share are not loaded.  Its eight
// waves take blocks of 128 columns in turn, so that together they read runs of
// a kilobyte of each row (against a contiguous range for each wave: 53 -> 45 us
// at 64 x 21504 x 5376); the eight fp32 partials meet in LDS and are added in
// a fixed order (no atomics, no workspace).  Weights go from global memory
// straight into registers, kDepth blocks ahead: each byte is used once.  A
// lane's 32 bytes of a block are two 16-byte pieces 64 apart, so that one load
// of a wave covers 64 contiguous bytes of each of 16 rows.
//
// Bound by HBM for large weights (4 x 21504 x 5376: 24.2 us, 4.8 TB/s, 94% of
// a large copy's rate; 1 x 5376 x 21504: 27 to 28 us, 4.1 to 4.3 TB/s) and by
// latency for small ones (1 x 1536 x 1152: 4.0 us).  From 33 tokens on it is
// neither (64 x 21504 x 5376: 43.7 us); which of the reads of x, which every
// workgroup repeats, the second round of workgroups and their start and end
// bounds it was not measured.
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;
static_assert(kDecodeWaves * kWave == kFp8DecodeThreads, "what the launch's size is checked against");
constexpr int kDecodeLdsX = 32768;   // bytes of Q(x) a workgroup keeps in LDS
constexpr int kDepth = 2;            // blocks of each wave in flight (3 and 4 gained nothing and cost occupancy)

struct DecodeArgs {
  const void* x;
  const void* xs;
  const uint8_t* w;
  const void* ws;
  void* y;
  int M, O, I, KB;
  int wide;  // y rows can be written four outputs at a time
  int rows;  // output rows of a workgroup
  int xs_t, xs_k;   // strides of xs (ScaleStrides)
};

// Loads go through buffer descriptors: rows, pieces and blocks past the end are
// given an offset past the buffer and read as zeros, without a branch that
// would keep the compiler from having many loads in flight.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), kRsrcFlags);
}

template <typename XE> struct XFrag;
template <> struct XFrag<uint8_t> { u32x4 v[2]; };
template <> struct XFrag<bf16_t> { u32x4 v[4]; };
template <> struct XFrag<float> { u32x4 v[8]; };

// The lane's two 16-element pieces of a row's block, 64 elements apart: at lo
// and hi (bytes from the descriptor's base, plus soff).
template <typename XE>
__device__ __forceinline__ XFrag<XE> load_x(__amdgpu_buffer_rsrc_t r, int lo, int hi, int soff) {
  constexpr int kN = int(sizeof(XE));   // 16-byte loads per piece
  XFrag<XE> f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    f.v[j] = __builtin_amdgcn_raw_buffer_load_b128(r, lo + 16 * j, soff, 0);
    f.v[kN + j] = __builtin_amdgcn_raw_buffer_load_b128(r, hi + 16 * j, soff, 0);
  }
  return f;
}

__device__ __forceinline__ void unpack_x(const XFrag<bf16_t>& f, float (&t)[4][8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[j][2 * e] = __uint_as_float(f.v[j][e] << 16);
      t[j][2 * e + 1] = __uint_as_float(f.v[j][e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack_x(const XFrag<float>& f, float (&t)[4][8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[j / 2][(j % 2) * 4 + e] = __uint_as_float(f.v[j][e]);
}

template <int SC>
__device__ __forceinline__ scale_t<SC> load_scale(__amdgpu_buffer_rsrc_t r, int off, int soff) {
  if constexpr (SC == TB_SCALE_E8M0)
    return __builtin_amdgcn_raw_buffer_load_b8(r, off, soff, 0);
  else
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off * 4, soff * 4, 0));
}

template <typename XE, int SC>
__device__ __forceinline__ i32x8 operand_x(const XFrag<XE>& r, float& scale) {
  if constexpr (sizeof(XE) == 1) {
    return join(r.v[0], r.v[1]);
  } else {
    float t[4][8];
    uint32_t a = 0;
    unpack_x(r, t);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) a = max(a, abs_bits(t[j][e]));
    a = max(a, uint32_t(__shfl_xor(int(a), 16)));
    a = max(a, uint32_t(__shfl_xor(int(a), 32)));
    scale_t<SC> st;
    float by;
    block_scale<SC>(a, st, by);
    scale = scale_value(st);
    i32x8 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = int(pack4(t[j][0] * by, t[j][1] * by, t[j][2] * by, t[j][3] * by));
      v[2 * j + 1] = int(pack4(t[j][4] * by, t[j][5] * by, t[j][6] * by, t[j][7] * by));
    }
    return v;
  }
}

// Where the products' x comes from.
enum XMode {
  kXGiven,      // e4m3 in memory
  kXInRegs,     // quantised by every wave, in the registers that hold a block
  kXInLds,      // quantised by every wave into LDS, token by token
};

// kXInLds: a wave's blocks w, w + 8, .. of every token, 16 lanes to a block as
// in quantize_rows_kernel, into LDS ([token][block][128] and [token][block]
// scales).  Nobody else reads them.
template <int SC, typename XE>
__device__ __forceinline__ void quantise_run(const DecodeArgs& a, int w, int nkb, uint8_t* xq, float* xs) {
  const int l = int(threadIdx.x) % kWave;
  const int passes = (nkb + 3) / 4;
  for (int j = 0; j < a.M * passes; ++j) {
    const int t = j / passes, b = (j % passes) * 4 + (l >> 4), c = (w + b * kDecodeWaves) * kBlock + (l & 15) * 8;
    float f[8];
    unpack8(load_frag_if<XE>(static_cast<const XE*>(a.x) + size_t(t) * a.I + c, b < nkb && c < a.I), f);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(f[e]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2) m = max(m, uint32_t(__shfl_xor(int(m), d)));
    scale_t<SC> st;
    float by;
    block_scale<SC>(m, st, by);
    if (b < nkb) {
      *reinterpret_cast<u32x2*>(xq + (t * nkb + b) * kBlock + (l & 15) * 8) =
          u32x2{pack4(f[0] * by, f[1] * by, f[2] * by, f[3] * by), pack4(f[4] * by, f[5] * by, f[6] * by, f[7] * by)};
      if ((l & 15) == 0) xs[t * nkb + b] = scale_value(st);
    }
  }
}

template <int SC, int NT, int RT, int XM, typename XE, typename YE>
__global__ __launch_bounds__(kDecodeWaves* kWave) void fp8_decode_kernel(DecodeArgs a) {
  constexpr bool kExact = sizeof(YE) == 4;
  __shared__ f32x4 red[kDecodeWaves / 2][RT * NT][kWave];
  __shared__ __attribute__((aligned(16))) uint8_t xlds[XM == kXInLds ? kDecodeLdsX : 16];
  __shared__ float xslds[XM == kXInLds ? kDecodeLdsX / kBlock : 1];
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, kq = (l >> 4) * 16;
  const int o0 = int(blockIdx.x) * a.rows, rows = min(a.rows, a.O - o0);   // rows <= 16 RT
  // The waves take blocks in turn, so that together they read runs of a
  // kilobyte of each row.
  const int nkb = (a.KB - w + kDecodeWaves - 1) / kDecodeWaves;   // this wave's blocks w, w + 8, ..

  const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + size_t(o0) * a.I, int64_t(rows) * a.I);
  const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, int64_t(a.M) * a.I * int(sizeof(XE)));
  const __amdgpu_buffer_rsrc_t rxs = rows_rsrc(a.xs, (int64_t(a.M - 1) * a.xs_t + int64_t(a.KB - 1) * a.xs_k + 1) * int(sizeof(scale_t<SC>)));
  // The rows lie in one weight block or, from row `edge` on, in the next one too.
  const int edge = kBlock - o0 % kBlock;
  const bool two = edge < rows;
  const __amdgpu_buffer_rsrc_t rws = rows_rsrc(static_cast<const scale_t<SC>*>(a.ws) + size_t(o0 / kBlock) * a.KB,
                                               int64_t(two ? 2 : 1) * a.KB * int(sizeof(scale_t<SC>)));
  const int wrow = lr * a.I + kq;
  const int lds0 = a.M * (w * (a.KB / kDecodeWaves) + min(w, a.KB % kDecodeWaves));   // blocks of the waves before
  const int xrow = (lr * a.I + kq) * int(sizeof(XE));

  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    u32x4 lo[RT], hi[RT];
    XFrag<XE> x[XM == kXInLds ? 1 : NT];
    scale_t<SC> xs[NT], ws[2];
  } st[kDepth];

  auto fetch = [&](Stage& s, int i) {
    const int kb = w + i * kDecodeWaves, k = kb * kBlock, left = a.I - k;   // I % 16 == 0: a piece is all in or all out
    const bool lo = kq < left, hi = kq + 64 < left;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      s.lo[r] = __builtin_amdgcn_raw_buffer_load_b128(rw, lo ? wrow : kPast, k + r * 16 * a.I, 0);
      s.hi[r] = __builtin_amdgcn_raw_buffer_load_b128(rw, hi ? wrow + 64 : kPast, k + r * 16 * a.I, 0);
    }
    if constexpr (XM != kXInLds) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        s.x[n] = load_x<XE>(rx, lo ? xrow : kPast, hi ? xrow + 64 * int(sizeof(XE)) : kPast,
                            (k + n * 16 * a.I) * int(sizeof(XE)));
    }
    if constexpr (XM == kXGiven) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s.xs[n] = load_scale<SC>(rxs, (lr + n * 16) * a.xs_t, kb * a.xs_k);
    }
    s.ws[0] = load_scale<SC>(rws, 0, kb);
    s.ws[1] = load_scale<SC>(rws, 0, kb + a.KB);   // (past the descriptor where there is one block: zero)
  };
  auto multiply = [&](const Stage& s, int i) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float xsc;
      i32x8 xb;
      if constexpr (XM == kXInLds) {
        // Tokens past the last repeat it; their results are not stored.
        const int t = min(n * 16 + lr, a.M - 1), at = lds0 + t * nkb + i;
        const uint8_t* p = xlds + at * kBlock + kq;
        xb = join(*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + 64));
        xsc = xslds[at];
      } else {
        xb = operand_x<XE, SC>(s.x[n], xsc);
        if constexpr (XM == kXGiven) xsc = scale_value(s.xs[n]);
      }
      const Operand<kExact> xv = operand<kExact>(xb);
      if constexpr (kExact) {
        const float s0 = xsc * scale_value(s.ws[0]), s1 = xsc * scale_value(s.ws[1]);
        // Two row tiles' products at a time where there are no more.
        constexpr int kGroup = RT <= 2 ? RT : 1;
#pragma unroll
        for (int r = 0; r < RT; r += kGroup) {
          Operand<kExact> wv[kGroup];
          f32x4 p[kGroup];
#pragma unroll
          for (int h = 0; h < kGroup; ++h) {
            i32x8 wb = join(s.lo[r + h], s.hi[r + h]);
            // Widened anew for every 16 tokens: kept, they would not fit the registers.
            if constexpr (NT > 1 && RT > 2) asm volatile("" : "+v"(wb));
            wv[h] = operand<kExact>(wb);
          }
#pragma unroll
          for (int h = 0; h < kGroup; ++h) p[h] = mma(wv[h], xv);
          products_issued<kExact>();
#pragma unroll
          for (int h = 0; h < kGroup; ++h) keep(wv[h]);
          keep(xv);
#pragma unroll
          for (int h = 0; h < kGroup; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[r + h][n][e] += p[h][e] * ((r + h) * 16 + (l >> 4) * 4 + e < edge ? s0 : s1);
        }
      } else if constexpr (NT == 1) {
        const float s0 = xsc * scale_value(s.ws[0]);
        if (!two) {
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][n] += mma(operand<kExact>(join(s.lo[r], s.hi[r])), xv) * s0;
        } else {
          const float s1 = xsc * scale_value(s.ws[1]);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const f32x4 p = mma(operand<kExact>(join(s.lo[r], s.hi[r])), xv);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][n][e] += p[e] * (r * 16 + (l >> 4) * 4 + e < edge ? s0 : s1);
          }
        }
      } else {
        // Workgroups start at multiples of four rows here: a lane's four share a scale.
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r][n] += mma(operand<kExact>(join(s.lo[r], s.hi[r])), xv) *
                       (xsc * scale_value(r * 16 + (l >> 4) * 4 < edge ? s.ws[0] : s.ws[1]));
      }
    }
  };

#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (d < nkb) fetch(st[d], d);
  // The first weight blocks are on their way while x is quantised.
  if constexpr (XM == kXInLds) {
    quantise_run<SC, XE>(a, w, nkb, xlds + lds0 * kBlock, xslds + lds0);
    // Lanes read what others of their wave wrote: its LDS operations complete in order, once the compiler keeps it.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  // Rounds without a branch: a branch around a refill would make the compiler
  // wait for the refill itself before it uses the next stage.
  int i = 0;
  for (; i + 2 * kDepth <= nkb; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      multiply(st[d], i + d);
      __builtin_amdgcn_sched_barrier(0);
      fetch(st[d], i + d + kDepth);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  for (; i < nkb; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (i + d < nkb) {
        multiply(st[d], i + d);
        if (i + d + kDepth < nkb) fetch(st[d], i + d + kDepth);
      }
    }
  }

  // The eight waves' sums, added in a fixed order: wave w + 4's to wave w's,
  // then those four.
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
  for (int j = int(threadIdx.x); j < RT * NT * kWave; j += kDecodeWaves * kWave) {
    const int tile = j / kWave, ln = j % kWave;
    f32x4 v = red[0][tile][ln];
#pragma unroll
    for (int q = 1; q < kDecodeWaves / 2; ++q) v += red[q][tile][ln];
    const int t = (tile % NT) * 16 + (ln & 15), o = (tile / NT) * 16 + (ln >> 4) * 4;
    if (t < a.M && o < rows)
      store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o0 + o, v, rows - o, a.wide && o + 4 <= rows);
  }
}

// ---------------------------------------------------------------------------
// More tokens (the 256 x 256 tiles of fp8_gemm.hip aside): 64 tokens x 128
// outputs per workgroup, four waves of 64 outputs x 32 tokens, one block of
// 128 columns per step.  Both operands' blocks and the tokens' scales come
// straight into a ring of three LDS slots, two blocks ahead, so that a step
// waits for a block asked for two steps before (staged through registers, one
// block ahead took 27 us at 777 x 1152 x 6912 in fp32, and two blocks ahead
// did not fit the registers).  Rows of 128 bytes keep their 16-byte pieces
// XOR-swizzled by (row >> 1) & 7, so that the fragment reads of 16 rows meet
// all banks.
// With few tiles the reduction is cut into S slices; each slice writes its
// fp32 sums and a second launch adds them in slice order, so the result does
// not depend on timing.
//
// Bound by the rate at which blocks reach LDS from the memory-side cache (24 KB
// per block and tile) and, for fp32 results, by the bf16 matrix rate and the
// widening beside it: 777 x 1152 x 6912 takes 23.3 us in fp32 (four slices, and
// 4.4 us to join them) and 15.6 us in bf16; 2000 x 8192 x 5376 in fp32 220 us in
// a long burst and up to 250 in a short one (0.80 PFLOP/s).  fp32 results keep a
// step's operands to its end (fp8_device.h, keep), which costs 8 to 15 %.  128
// tokens per workgroup (eight waves) were no faster when that was not so: 22.3,
// 16.4 and 232 us against 21.3, 16.7 and 216.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, TM = 64, kSlots = 3;   // outputs and tokens of a tile; LDS slots
constexpr int kGemmThreads = 4 * TM;

struct GemmArgs {
  const uint8_t* x;
  const void* xs;
  const uint8_t* w;
  const void* ws;
  void* y;
  float* part;   // [S][tiles][8][4 TM] pieces of four, or NULL with one slice
  int M, O, I, KB;
  int tiles_m, tiles_n, S;
  int wide;
  int64_t xs_t, xs_k;   // strides of xs (ScaleStrides)
};

// Tile u's first token and output: groups of eight token tiles walked column
// by column, so that workgroups that run together share rows in L2.
__device__ __forceinline__ void tile_at(const GemmArgs& a, int u, int& m0, int& n0) {
  const int per_group = 8 * a.tiles_n, first = u / per_group * 8, gs = min(a.tiles_m - first, 8), r = u % per_group;
  m0 = (first + r % gs) * TM;
  n0 = r / gs * kTile;
}

template <int SC, typename YE>
__global__ __launch_bounds__(kGemmThreads, 2) void fp8_gemm_kernel(GemmArgs a) {
  constexpr bool kExact = sizeof(YE) == 4;
  constexpr int kWaves = TM / 16, kW = 16 / kWaves;   // kW, 2: loads of W and x per wave and block
  constexpr int kX = kTile * 128, kScales = kX + TM * 128, kSlot = kScales + kWaves * 256;
  constexpr int kLoads = kW + 2 + 1;
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
  const scale_t<SC>* ws = static_cast<const scale_t<SC>*>(a.ws) + size_t(n0 / kBlock) * a.KB;
  // Load j of an operand: row 8 (w loads + j) + l / 8, the piece that the
  // swizzle keeps at position l % 8; eight rows further on the swizzle differs
  // in its upper bit only.
  const int dr = l >> 3, pe = (l & 7) ^ (dr >> 1), po = pe ^ 4;
  const unsigned b0 = unsigned(uintptr_t(base));
  const scale_t<SC>* xs = static_cast<const scale_t<SC>*>(a.xs) + int64_t(m0) * a.xs_t;
  const int64_t xs_bytes = (int64_t(rows_x - 1) * a.xs_t + 1) * int(sizeof(scale_t<SC>));
  const int xs_off = (wt * 32 + (l & 31)) * int(a.xs_t) * int(sizeof(scale_t<SC>));
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
    dma_scale<SC>(d + kScales + w * 256, rows_rsrc(xs + min(kb, kb1 - 1) * a.xs_k, xs_bytes), xs_off, 0);
  };

  f32x4 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int sw = (lr >> 1) & 7, p0 = (q ^ sw) << 4, p1 = ((q + 4) ^ sw) << 4;
  auto step = [&](auto which, int kb) {
    constexpr int slot = decltype(which)::value;
    wait_loads<kLoads>();             // block kb has landed; kb + 1 may be out
    __builtin_amdgcn_s_barrier();     // published; and every wave has left the slot filled next
    issue((slot + 2) % kSlots, kb + 2);
    const lds_byte* const s = base + slot * kSlot;
    const float wsc = scale_value(ws[kb]);
    Operand<kExact> fx[2];
    float sc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const lds_byte* r = s + kX + (wt * 32 + j * 16 + lr) * 128;
      fx[j] = operand<kExact>(join(*reinterpret_cast<const lds_u32x4*>(r + p0), *reinterpret_cast<const lds_u32x4*>(r + p1)));
      const uint32_t raw = *reinterpret_cast<const lds_u32*>(s + kScales + w * 256 + (j * 16 + lr) * 4);
      if constexpr (SC == TB_SCALE_E8M0) sc[j] = scale_value(uint8_t(raw)) * wsc;
      else sc[j] = __uint_as_float(raw) * wsc;
    }
    Operand<kExact> fw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const lds_byte* r = s + (wo * 64 + i * 16 + lr) * 128;
      fw[i] = operand<kExact>(join(*reinterpret_cast<const lds_u32x4*>(r + p0), *reinterpret_cast<const lds_u32x4*>(r + p1)));
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] += mma(fw[i], fx[j]) * sc[j];
    }
    products_issued<kExact>();
#pragma unroll
    for (int i = 0; i < 4; ++i) keep(fw[i]);
#pragma unroll
    for (int j = 0; j < 2; ++j) keep(fx[j]);
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
    f32x4* p = reinterpret_cast<f32x4*>(a.part) +
               (size_t(slice) * tiles + tile) * 8 * kGemmThreads + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) p[(i * 2 + j) * kGemmThreads] = acc[i][j];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = m0 + wt * 32 + j * 16 + lr, o = n0 + wo * 64 + i * 16 + q * 4;
      if (t < a.M && o < a.O)
        store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, acc[i][j], a.O - o, a.wide && o + 4 <= a.O);
    }
}

// The slices' sums of a split product, added in slice order: one workgroup for
// the pieces of 16 outputs of each of a tile's waves.
template <typename YE>
__global__ __launch_bounds__(kGemmThreads) void fp8_join_kernel(GemmArgs a) {
  const int w = int(threadIdx.x) / kWave, l = int(threadIdx.x) % kWave, lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  const int tile = int(blockIdx.x) >> 2, tiles = a.tiles_m * a.tiles_n, i = int(blockIdx.x) & 3;
  int m0, n0;
  tile_at(a, tile, m0, n0);
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (size_t(tile) * 4 + i) * 2 * kGemmThreads + threadIdx.x;
  f32x4 sum[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) sum[j] = p[j * kGemmThreads];
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) sum[j] += p[(size_t(s) * tiles * 8 + j) * kGemmThreads];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = m0 + wt * 32 + j * 16 + lr, o = n0 + wo * 64 + i * 16 + q * 4;
    if (t < a.M && o < a.O)
      store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, sum[j], a.O - o, a.wide && o + 4 <= a.O);
  }
}

template <int SC, int NT, int RT, int XM, typename XE, typename YE>
hipError_t decode_go(const DecodeArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned((a.O + a.rows - 1) / a.rows));
  hipLaunchKernelGGL((fp8_decode_kernel<SC, NT, RT, XM, XE, YE>), grid, dim3(kDecodeWaves * kWave), 0, stream, a);
  return hipGetLastError();
}

template <int SC, int NT, typename YE>
hipError_t decode_given(const DecodeArgs& a, hipStream_t stream) {
  const int rt = (a.rows + 15) / 16;
  if (rt == 1) return decode_go<SC, NT, 1, kXGiven, uint8_t, YE>(a, stream);
  if (rt == 2) return decode_go<SC, NT, 2, kXGiven, uint8_t, YE>(a, stream);
  if (rt == 3) return decode_go<SC, NT, 3, kXGiven, uint8_t, YE>(a, stream);
  if constexpr (NT <= 2)
    if (rt == 4) return decode_go<SC, NT, 4, kXGiven, uint8_t, YE>(a, stream);
  if constexpr (NT == 1)
    if (rt <= 6) return decode_go<SC, NT, 6, kXGiven, uint8_t, YE>(a, stream);
  return hipErrorInvalidValue;
}

// Up to 16 tokens, quantised in the kernel (decode_fused).
template <int SC, typename XE, typename YE>
hipError_t decode_quantising(const DecodeArgs& a, hipStream_t stream) {
  const int rt = (a.rows + 15) / 16;
  if (rt == 1) return decode_go<SC, 1, 1, kXInLds, XE, YE>(a, stream);
  if (rt == 2) return decode_go<SC, 1, 2, kXInLds, XE, YE>(a, stream);
  if (rt == 3) return decode_go<SC, 1, 3, kXInRegs, XE, YE>(a, stream);
  if (rt == 4) return decode_go<SC, 1, 4, kXInRegs, XE, YE>(a, stream);
  if (rt <= 6) return decode_go<SC, 1, 6, kXInRegs, XE, YE>(a, stream);
  return hipErrorInvalidValue;
}

// Output rows of a workgroup: equal shares of the weight for every compute
// unit (a unit with twice the rows of another would finish last: a compute
// unit takes at most ~22 GB/s from HBM here), in as few workgroups per unit as
// the widest kernel for these tokens allows.
int decode_rows(int64_t m, int64_t out_dim, int cus) {
  const int most = fp8_decode_most_rows(m);
  const int64_t k = (out_dim + int64_t(cus) * most - 1) / (int64_t(cus) * most);
  const int64_t rows = (out_dim + cus * k - 1) / (cus * k);
  return int(m <= 16 ? rows : (rows + 3) / 4 * 4);
}

// Whether the kernel quantises x itself: always where it can do so while the
// weights stream (more than 32 rows a workgroup; 16 x 21504 x 5376: 26.9 us
// against 25.0 and a launch of about 3), and else where Q(x) fits its LDS
// (1 x 5376 x 21504: 28.3 us against 28.0 and a launch).  Where neither holds
// the work per workgroup is mostly that quantisation (8 x 1152 x 6912 in fp32:
// 13.1 us against 7.3 and a launch of 3.1).
bool decode_fused(int64_t m, int64_t out_dim, int64_t in_dim, int cus) {
  return m <= kFp8FusedTokens &&
         (decode_rows(m, out_dim, cus) > 32 || m * fp8_blocks(in_dim) * kBlock <= kDecodeLdsX);
}

template <int SC, typename YE>
hipError_t decode_x(tb_dtype x_dtype, const DecodeArgs& a, hipStream_t stream) {
  if (x_dtype == TB_BF16) return decode_quantising<SC, bf16_t, YE>(a, stream);
  if (x_dtype == TB_F32) return decode_quantising<SC, float, YE>(a, stream);
  if (a.M <= 16) return decode_given<SC, 1, YE>(a, stream);
  return a.M <= 32 ? decode_given<SC, 2, YE>(a, stream) : decode_given<SC, 4, YE>(a, stream);
}

template <int SC, typename YE>
hipError_t gemm_go(const GemmArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((fp8_gemm_kernel<SC, YE>), dim3(unsigned(a.tiles_m * a.tiles_n * a.S)), dim3(kGemmThreads), 0,
                     stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 1) return e;
  hipLaunchKernelGGL((fp8_join_kernel<YE>), dim3(unsigned(a.tiles_m * a.tiles_n * 4)), dim3(kGemmThreads), 0, stream,
                     a);
  return hipGetLastError();
}

}  // namespace

Fp8Plan plan_fp8(int64_t m, int64_t out_dim, int64_t in_dim, bool quantised, tb_dtype y_dtype, tb_scale scale_type,
                 int cus) {
  Fp8Plan p{};
  const int64_t KB = fp8_blocks(in_dim);
  p.decode = m <= kDecodeMaxTokens;
  p.rows = p.decode ? decode_rows(m, out_dim, cus) : 0;
  p.fused = p.decode && !quantised && decode_fused(m, out_dim, in_dim, cus);
  p.S = 1;
  size_t at = 0;
  if (!quantised && !p.fused) {
    p.off_xq = at;
    at = align_up(at + size_t(m) * in_dim, 256);
    p.off_xs = at;
    at = align_up(at + size_t(m) * KB * (scale_type == TB_SCALE_E8M0 ? 1 : 4), 256);
  }
  // The 256 x 256 kernel makes bf16 results and needs tiles for half the compute
  // units.
  p.big = !p.decode && y_dtype == TB_BF16 && ((m + 255) / 256) * ((out_dim + 255) / 256) * 2 >= cus;
  if (p.big) {
    p.tile = plan_fp8_tiles(m, out_dim, in_dim, cus);
    p.off_part = at;
    at += p.tile.part_bytes;
  } else if (!p.decode) {
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
  }
  p.bytes = at;
  return p;
}

hipError_t launch_fp8_product(const Fp8Plan& p, tb_dtype x_dtype, tb_dtype y_dtype, tb_scale scale_type, const void* x,
                              const void* xs, const void* w, const void* ws, void* y, int64_t m, int64_t out_dim,
                              int64_t in_dim, char* data, hipStream_t stream) {
  const bool e8 = scale_type == TB_SCALE_E8M0;
  ScaleStrides ss{fp8_blocks(in_dim), 1};
  if (x_dtype != TB_E4M3 && !p.fused) {
    void* xq = data + p.off_xq;
    void* sq = data + p.off_xs;
    ss = ScaleStrides{1, m};
    hipError_t e = launch_quantize_rows(x_dtype, scale_type, x, xq, sq, ss, m, in_dim, stream);
    if (e != hipSuccess) return e;
    x = xq;
    xs = sq;
    x_dtype = TB_E4M3;
  }
  const size_t ys = y_dtype == TB_BF16 ? 2 : 4;
  const int wide = out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * ys - 1)) == 0;
  const int KB = int(fp8_blocks(in_dim));
  if (p.decode) {
    const DecodeArgs a{x, xs, static_cast<const uint8_t*>(w), ws, y, int(m), int(out_dim), int(in_dim), KB,
                       wide && p.rows % 4 == 0, p.rows, int(ss.token), int(ss.block)};
    if (y_dtype == TB_BF16)
      return e8 ? decode_x<TB_SCALE_E8M0, bf16_t>(x_dtype, a, stream) : decode_x<TB_SCALE_F32, bf16_t>(x_dtype, a, stream);
    return e8 ? decode_x<TB_SCALE_E8M0, float>(x_dtype, a, stream) : decode_x<TB_SCALE_F32, float>(x_dtype, a, stream);
  }
  if (p.big)
    return launch_fp8_tiles(p.tile, scale_type, x, xs, ss, w, ws, y, reinterpret_cast<float*>(data + p.off_part), m,
                            out_dim, in_dim, stream);
  const GemmArgs a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, y,
                   reinterpret_cast<float*>(data + p.off_part), int(m), int(out_dim), int(in_dim), KB, p.tiles_m,
                   p.tiles_n, p.S, wide, ss.token, ss.block};
  if (y_dtype == TB_BF16) return e8 ? gemm_go<TB_SCALE_E8M0, bf16_t>(a, stream) : gemm_go<TB_SCALE_F32, bf16_t>(a, stream);
  return e8 ? gemm_go<TB_SCALE_E8M0, float>(a, stream) : gemm_go<TB_SCALE_F32, float>(a, stream);
}

}  // namespace tb
