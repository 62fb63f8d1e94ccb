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
      *reinterpret_cast<u32x2*>(y) = u32x2{f32_to_bf16(v[0]) | (uint32_t(f32_to_bf16(v[1])) << 16),
                                           f32_to_bf16(v[2]) | (uint32_t(f32_to_bf16(v[3])) << 16)};
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
// A workgroup owns 16 RT output rows and its eight waves split in_dim into
// contiguous runs of blocks, so that even a small weight keeps every compute
// unit loading; the eight fp32 partials meet in LDS and are added in wave
// order (no atomics, no workspace).  Fragments go from global memory straight
// into registers, kDepth blocks ahead: each weight byte is used once.  A lane's
// 32 bytes of a block are two 16-byte pieces 64 apart, so that one load of a
// wave covers 64 contiguous bytes of each of 16 rows.
// XE uint8_t: x comes in e4m3 with its scales.  XE bf16_t or float: each wave
// quantises the blocks it multiplies, in registers: a block of 16 tokens sits
// in its 64 lanes exactly as the product wants it, so the block's maximum is
// two cross-lane steps and no launch or memory is spent on Q(x).
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;

struct DecodeArgs {
  const void* x;
  const void* xs;
  const uint8_t* w;
  const void* ws;
  void* y;
  int M, O, I, KB;
  int wide;  // y rows can be written four outputs at a time
};

template <typename XE> struct XFrag;
template <> struct XFrag<uint8_t> { u32x4 lo, hi; };
template <> struct XFrag<bf16_t> { Frag8<bf16_t> f[4]; };
template <> struct XFrag<float> { Frag8<float> f[4]; };

// The lane's two 16-element pieces of a row's block at p (element pointer),
// 64 elements apart; a piece past the row's end reads as zeros.
template <typename XE>
__device__ __forceinline__ XFrag<XE> load_x(const XE* p, bool lo, bool hi) {
  XFrag<XE> r;
  if constexpr (sizeof(XE) == 1) {
    r.lo = lo ? *reinterpret_cast<const u32x4*>(p) : u32x4{0, 0, 0, 0};
    r.hi = hi ? *reinterpret_cast<const u32x4*>(p + 64) : u32x4{0, 0, 0, 0};
  } else {
    r.f[0] = load_frag_if<XE>(p, lo);
    r.f[1] = load_frag_if<XE>(p + 8, lo);
    r.f[2] = load_frag_if<XE>(p + 64, hi);
    r.f[3] = load_frag_if<XE>(p + 72, hi);
  }
  return r;
}

template <typename XE, int SC>
__device__ __forceinline__ i32x8 operand_x(const XFrag<XE>& r, float& scale) {
  if constexpr (sizeof(XE) == 1) {
    return join(r.lo, r.hi);
  } else {
    float t[4][8];
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack8(r.f[j], t[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = max(a, abs_bits(t[j][e]));
    }
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

template <int SC, int NT, int RT, typename XE, typename YE>
__global__ __launch_bounds__(kDecodeWaves* kWave) void fp8_decode_kernel(DecodeArgs a) {
  constexpr bool kFused = sizeof(XE) != 1, kExact = sizeof(YE) == 4;
  constexpr int kDepth = NT * sizeof(XE) >= 4 ? 2 : 4;
  __shared__ f32x4 red[kDecodeWaves][RT * NT][kWave];
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), l = int(threadIdx.x) % kWave;
  const int lr = l & 15, kq = (l >> 4) * 16;
  const int o0 = int(blockIdx.x) * 16 * RT;
  const int kb0 = int(int64_t(w) * a.KB / kDecodeWaves), kb1 = int(int64_t(w + 1) * a.KB / kDecodeWaves);
  const scale_t<SC>* ws = static_cast<const scale_t<SC>*>(a.ws) + size_t(o0 / kBlock) * a.KB;

  // Rows and tokens past the end repeat the last one; their results are not stored.
  const uint8_t* wp[RT];
  const XE* xp[NT];
  const scale_t<SC>* xsp[NT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wp[r] = a.w + size_t(min(o0 + r * 16 + lr, a.O - 1)) * a.I + kq;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = min(n * 16 + lr, a.M - 1);
    xp[n] = static_cast<const XE*>(a.x) + size_t(t) * a.I + kq;
    if constexpr (!kFused) xsp[n] = static_cast<const scale_t<SC>*>(a.xs) + size_t(t) * a.KB;
  }

  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    u32x4 lo[RT], hi[RT];
    XFrag<XE> x[NT];
    scale_t<SC> xs[NT];
    scale_t<SC> ws;
  } st[kDepth];

  auto fetch = [&](Stage& s, int kb) {
    const int k = kb * kBlock;
    const bool lo = k + kq < a.I, hi = k + kq + 64 < a.I;   // I % 16 == 0: a piece is all in or all out
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      s.lo[r] = lo ? *reinterpret_cast<const u32x4*>(wp[r] + k) : u32x4{0, 0, 0, 0};
      s.hi[r] = hi ? *reinterpret_cast<const u32x4*>(wp[r] + k + 64) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s.x[n] = load_x<XE>(xp[n] + k, lo, hi);
      if constexpr (!kFused) s.xs[n] = xsp[n][kb];
    }
    s.ws = ws[kb];
  };
  auto multiply = [&](const Stage& s) {
    const float wsc = scale_value(s.ws);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float xsc = 0.f;
      const Operand<kExact> xv = operand<kExact>(operand_x<XE, SC>(s.x[n], xsc));
      if constexpr (!kFused) xsc = scale_value(s.xs[n]);
      const float sc = xsc * wsc;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        acc[r][n] += mma(operand<kExact>(join(s.lo[r], s.hi[r])), xv) * sc;
      }
    }
  };

#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (kb0 + d < kb1) fetch(st[d], kb0 + d);
  for (int kb = kb0; kb < kb1; kb += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (kb + d < kb1) {
        multiply(st[d]);
        if (kb + d + kDepth < kb1) fetch(st[d], kb + d + kDepth);
      }
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[w][r * NT + n][l] = acc[r][n];
  __syncthreads();
  for (int j = int(threadIdx.x); j < RT * NT * kWave; j += kDecodeWaves * kWave) {
    const int tile = j / kWave, ln = j % kWave;
    f32x4 v = red[0][tile][ln];
#pragma unroll
    for (int q = 1; q < kDecodeWaves; ++q) v += red[q][tile][ln];
    const int t = (tile % NT) * 16 + (ln & 15), o = o0 + (tile / NT) * 16 + (ln >> 4) * 4;
    if (t < a.M && o < a.O)
      store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, v, a.O - o, a.wide && o + 4 <= a.O);
  }
}

// ---------------------------------------------------------------------------
// Many tokens: 128 outputs x 128 tokens per workgroup, four waves of 64 x 64,
// one block of 128 columns per step.  Both operands' blocks are staged in LDS
// (two buffers; rows of 128 bytes with their 16-byte pieces XOR-swizzled by
// row, so that the fragment reads of 16 rows meet all banks) through
// registers, so the next block's loads fly while this one multiplies.
// With few tiles the reduction is cut into S slices over blockIdx.y; each
// slice writes its fp32 sums and a second launch adds them in slice order, so
// the result does not depend on timing.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, kGemmThreads = 256;

struct GemmArgs {
  const uint8_t* x;
  const void* xs;
  const uint8_t* w;
  const void* ws;
  void* y;
  float* part;   // [S][tiles][64][256] pieces of four, or NULL with one slice
  int M, O, I, KB;
  int tiles_m, tiles_n, S;
  int wide;
};

__device__ __forceinline__ int swz(int row, int piece) { return row * 128 + ((piece ^ ((row >> 1) & 7)) << 4); }

template <int SC, typename YE>
__global__ __launch_bounds__(kGemmThreads, 2) void fp8_gemm_kernel(GemmArgs a) {
  constexpr bool kExact = sizeof(YE) == 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][kTile * 128];  // [buffer][W or x]
  const int tid = int(threadIdx.x), w = tid / kWave, l = tid % kWave;
  const int lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  // Tiles in groups of eight token tiles, so that workgroups that run together
  // share rows of both operands in L2.
  const int per_group = 8 * a.tiles_n, first = int(blockIdx.x) / per_group * 8, gs = min(a.tiles_m - first, 8);
  const int tm = first + (int(blockIdx.x) % per_group) % gs, tn = (int(blockIdx.x) % per_group) / gs;
  const int m0 = tm * kTile, n0 = tn * kTile;
  const int slice = int(blockIdx.y);
  const int kb0 = int(int64_t(slice) * a.KB / a.S), kb1 = int(int64_t(slice + 1) * a.KB / a.S);

  const int sr = tid >> 3, sp = tid & 7;   // staging: piece sp of rows sr + 32 j
  const scale_t<SC>* ws = static_cast<const scale_t<SC>*>(a.ws) + size_t(tn) * a.KB;
  const scale_t<SC>* xs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    xs[j] = static_cast<const scale_t<SC>*>(a.xs) + size_t(min(m0 + wt * 64 + j * 16 + lr, a.M - 1)) * a.KB;

  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 rw[4], rx[4];
  scale_t<SC> nws{}, nxs[4]{};
  auto fetch = [&](int kb) {
    const int k = kb * kBlock + sp * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = n0 + sr + 32 * j, t = m0 + sr + 32 * j;
      rw[j] = o < a.O && k < a.I ? *reinterpret_cast<const u32x4*>(a.w + size_t(o) * a.I + k) : u32x4{0, 0, 0, 0};
      rx[j] = t < a.M && k < a.I ? *reinterpret_cast<const u32x4*>(a.x + size_t(t) * a.I + k) : u32x4{0, 0, 0, 0};
      nxs[j] = xs[j][kb];
    }
    nws = ws[kb];
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<u32x4*>(&lds[buf][0][swz(sr + 32 * j, sp)]) = rw[j];
      *reinterpret_cast<u32x4*>(&lds[buf][1][swz(sr + 32 * j, sp)]) = rx[j];
    }
  };
  if (kb0 < kb1) {
    fetch(kb0);
    stage(0);
  }
  for (int kb = kb0; kb < kb1; ++kb) {
    const int buf = (kb - kb0) & 1;
    float sc[4];
    const float wsc = scale_value(nws);
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[j] = scale_value(nxs[j]) * wsc;
    __syncthreads();   // this block is staged, and every wave has left the other buffer
    if (kb + 1 < kb1) fetch(kb + 1);
    Operand<kExact> fx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = wt * 64 + j * 16 + lr;
      fx[j] = operand<kExact>(join(*reinterpret_cast<const u32x4*>(&lds[buf][1][swz(row, q)]),
                                   *reinterpret_cast<const u32x4*>(&lds[buf][1][swz(row, q + 4)])));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wo * 64 + i * 16 + lr;
      const Operand<kExact> fw = operand<kExact>(join(*reinterpret_cast<const u32x4*>(&lds[buf][0][swz(row, q)]),
                                                      *reinterpret_cast<const u32x4*>(&lds[buf][0][swz(row, q + 4)])));
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += mma(fw, fx[j]) * sc[j];
    }
    if (kb + 1 < kb1) stage(buf ^ 1);
  }

  if (a.S > 1) {
    f32x4* p = reinterpret_cast<f32x4*>(a.part) +
               (size_t(slice) * a.tiles_m * a.tiles_n + blockIdx.x) * 16 * kGemmThreads + tid;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[(i * 4 + j) * kGemmThreads] = acc[i][j];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = m0 + wt * 64 + j * 16 + lr, o = n0 + wo * 64 + i * 16 + q * 4;
      if (t < a.M && o < a.O)
        store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, acc[i][j], a.O - o, a.wide && o + 4 <= a.O);
    }
}

// The slices' sums of a split product, added in slice order: one workgroup for
// four of a tile's sixteen pieces.
template <typename YE>
__global__ __launch_bounds__(kGemmThreads) void fp8_join_kernel(GemmArgs a) {
  const int tid = int(threadIdx.x), w = tid / kWave, l = tid % kWave, lr = l & 15, q = l >> 4, wo = w & 1, wt = w >> 1;
  const int tile = int(blockIdx.x) >> 2, tiles = a.tiles_m * a.tiles_n, i = int(blockIdx.x) & 3;
  const int per_group = 8 * a.tiles_n, first = tile / per_group * 8, gs = min(a.tiles_m - first, 8);
  const int m0 = (first + (tile % per_group) % gs) * kTile, n0 = (tile % per_group) / gs * kTile;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (size_t(tile) * 16 + i * 4) * kGemmThreads + tid;
  f32x4 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = p[j * kGemmThreads];
  for (int s = 1; s < a.S; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += p[(size_t(s) * tiles * 16 + j) * kGemmThreads];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = m0 + wt * 64 + j * 16 + lr, o = n0 + wo * 64 + i * 16 + q * 4;
    if (t < a.M && o < a.O)
      store_out4(static_cast<YE*>(a.y) + size_t(t) * a.O + o, sum[j], a.O - o, a.wide && o + 4 <= a.O);
  }
}

template <int SC, int NT, int RT, typename XE, typename YE>
hipError_t decode_go(const DecodeArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned((a.O + 16 * RT - 1) / (16 * RT)));
  hipLaunchKernelGGL((fp8_decode_kernel<SC, NT, RT, XE, YE>), grid, dim3(kDecodeWaves * kWave), 0, stream, a);
  return hipGetLastError();
}

template <int SC, typename XE, typename YE>
hipError_t decode_typed(const DecodeArgs& a, hipStream_t stream) {
  if (a.M <= 16) return decode_go<SC, 1, 1, XE, YE>(a, stream);
  if constexpr (sizeof(XE) == 1) {
    if (a.M <= 32) return decode_go<SC, 2, 1, XE, YE>(a, stream);
    return decode_go<SC, 4, 1, XE, YE>(a, stream);
  }
  return hipErrorInvalidValue;
}

template <int SC, typename YE>
hipError_t decode_x(tb_dtype x_dtype, const DecodeArgs& a, hipStream_t stream) {
  if (x_dtype == TB_E4M3) return decode_typed<SC, uint8_t, YE>(a, stream);
  // Quantised in the kernel: y has x's type or either.
  if (x_dtype == TB_BF16) return decode_typed<SC, bf16_t, YE>(a, stream);
  return decode_typed<SC, float, YE>(a, stream);
}

template <int SC, typename YE>
hipError_t gemm_go(const GemmArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((fp8_gemm_kernel<SC, YE>), dim3(unsigned(a.tiles_m * a.tiles_n), unsigned(a.S)),
                     dim3(kGemmThreads), 0, stream, a);
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
  p.fused = !quantised && m <= kFp8FusedTokens;
  p.S = 1;
  size_t at = 0;
  if (!quantised && !p.fused) {
    p.off_xq = at;
    at = align_up(at + size_t(m) * in_dim, 256);
    p.off_xs = at;
    at = align_up(at + size_t(m) * KB * (scale_type == TB_SCALE_E8M0 ? 1 : 4), 256);
  }
  // The 256 x 256 kernel makes bf16 results, needs tiles for half the compute
  // units and addresses a tile's rows with 31-bit offsets.
  p.big = !p.decode && y_dtype == TB_BF16 && in_dim <= (int64_t(1) << 31) / 256 - 128 &&
          ((m + 255) / 256) * ((out_dim + 255) / 256) * 2 >= cus;
  if (p.big) {
    p.tile = plan_fp8_tiles(m, out_dim, in_dim, cus);
    p.off_part = at;
    at += p.tile.part_bytes;
  } else if (!p.decode) {
    p.tiles_m = int((m + kTile - 1) / kTile);
    p.tiles_n = int((out_dim + kTile - 1) / kTile);
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    // Two workgroups fit a compute unit; a slice keeps at least four blocks.
    if (tiles < cus) p.S = int(std::max<int64_t>(1, std::min<int64_t>(2 * cus / tiles, KB / 4)));
    if (p.S > 1) {
      p.off_part = at;
      at += size_t(p.S) * tiles * kTile * kTile * 4;
    }
  }
  p.bytes = at;
  return p;
}

hipError_t launch_fp8_product(const Fp8Plan& p, tb_dtype x_dtype, tb_dtype y_dtype, tb_scale scale_type, const void* x,
                              const void* xs, const void* w, const void* ws, void* y, int64_t m, int64_t out_dim,
                              int64_t in_dim, char* data, hipStream_t stream) {
  const bool e8 = scale_type == TB_SCALE_E8M0;
  if (x_dtype != TB_E4M3 && !p.fused) {
    void* xq = data + p.off_xq;
    void* sq = data + p.off_xs;
    hipError_t e = launch_quantize_rows(x_dtype, scale_type, x, xq, sq, m, in_dim, stream);
    if (e != hipSuccess) return e;
    x = xq;
    xs = sq;
    x_dtype = TB_E4M3;
  }
  const size_t ys = y_dtype == TB_BF16 ? 2 : 4;
  const int wide = out_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * ys - 1)) == 0;
  const int KB = int(fp8_blocks(in_dim));
  if (p.decode) {
    const DecodeArgs a{x, xs, static_cast<const uint8_t*>(w), ws, y, int(m), int(out_dim), int(in_dim), KB, wide};
    if (y_dtype == TB_BF16)
      return e8 ? decode_x<TB_SCALE_E8M0, bf16_t>(x_dtype, a, stream) : decode_x<TB_SCALE_F32, bf16_t>(x_dtype, a, stream);
    return e8 ? decode_x<TB_SCALE_E8M0, float>(x_dtype, a, stream) : decode_x<TB_SCALE_F32, float>(x_dtype, a, stream);
  }
  if (p.big)
    return launch_fp8_tiles(p.tile, scale_type, x, xs, w, ws, y, reinterpret_cast<float*>(data + p.off_part), m,
                            out_dim, in_dim, stream);
  const GemmArgs a{static_cast<const uint8_t*>(x), xs, static_cast<const uint8_t*>(w), ws, y,
                   reinterpret_cast<float*>(data + p.off_part), int(m), int(out_dim), int(in_dim), KB, p.tiles_m,
                   p.tiles_n, p.S, wide};
  if (y_dtype == TB_BF16) return e8 ? gemm_go<TB_SCALE_E8M0, bf16_t>(a, stream) : gemm_go<TB_SCALE_F32, bf16_t>(a, stream);
  return e8 ? gemm_go<TB_SCALE_E8M0, float>(a, stream) : gemm_go<TB_SCALE_F32, float>(a, stream);
}

}  // namespace tb
