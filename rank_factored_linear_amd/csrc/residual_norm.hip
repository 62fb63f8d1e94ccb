// The norms before and after a block in one pass over the residual stream: for
// each row
//   a = y, or y / sqrt(mean(y^2) + eps) * (post_weight + offset)
//   h' = residual_scale * h + gate * a
//   z = h' / sqrt(mean(h'^2) + eps) * (weight + offset)
// with z in the type that the next projection takes: wide, 8-bit integers with a
// scale per row, or e4m3 with a scale per 128 columns.
//
// A row's threads hold it from its load to its last store, in fp32 and in registers
// (but for what spills, see Reach): z is made from h' as it is before it is rounded
// to be stored.  Each element is read and written once, so the call is bound by HBM
// for many rows and by latency (two sums over the row, one behind the other) for a
// few.
//
// h' goes past the caches: the block that reads it next has a layer's weights
// before it, while z is read at once.  With y the z of the call before and h
// cold, bf16: 4096 x 5376 33.4 us against 34.2 with both kept and 35.4 with both past
// them, 1024 x 5376 10.9 (12.0, 10.3), 4096 x 1152 9.3 (10.7, 8.9).  All loads of a row,
// y's behind h's, before the first use: 37.4 -> 34.2 (5.15 TB/s).  Loading the next row
// ahead of the present one gained nothing.
#include "int8_device.h"

#include <algorithm>

namespace tb {

namespace {

struct NormArgs {
  tb_residual r;
  int64_t M;
  int n, T;            // elements of a row, threads that hold it
  float scale, eps, offset, inv_n;
  int post;
};

// How a row's pieces of eight elements are read and written: at multiples of 16
// bytes; where its length, strides or addresses are not, at those of an element
// (n >= 8: the last piece is then read as the row's last eight elements, so that no
// load needs a branch around it, and shifted; what it holds of its neighbour's, which
// may be written already, is dropped); or, in rows shorter than a piece, element by
// element.  1022 rows, bf16, per call: of 5376 10.3 us, 5377 11.7 (by single elements
// 30), 8193 20 (235), 16384 26.6, 16385 42.5 (393), 24583 94, 32768 48.  Part of what kAny
// takes longer are spills: a launch may have 1024 threads, which leaves a thread 128
// registers, and three pieces of a row spill 6 to 22 of them, four (rows of more than
// 24576) 43 to 64.  With kPieces it is 4 to 25 with four pieces, none with fewer.
enum Reach { kPieces, kAny, kShort };

// Sixteen bytes as they are reached (an alignment does not pass through a template's type argument).
template <typename E, int R> struct Sixteen { typedef fp8::u32x4 type; };
template <> struct Sixteen<bf16_t, kAny> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct Sixteen<float, kAny> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };

template <typename E, int R>
__device__ __forceinline__ Frag8<E> fetch(const E* p, int at, int n) {
  if constexpr (R == kPieces) {
    return load_frag_if<E>(p + at, at < n);
  } else {
    typedef typename Sixteen<E, R>::type T;
    T v[sizeof(E) / 2];
    if constexpr (R == kAny) {
      const T* from = reinterpret_cast<const T*>(p + min(at, n - 8));
#pragma unroll
      for (int i = 0; i < int(sizeof(E)) / 2; ++i) v[i] = from[i];
    } else {
      E e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = at + i < n ? p[at + i] : from_f32<E>(0.f);
      __builtin_memcpy(v, e, sizeof(v));
    }
    Frag8<E> f;
    static_assert(sizeof(f) == sizeof(v), "eight elements");
    __builtin_memcpy(&f, v, sizeof(f));
    return f;
  }
}
// A fetched piece as fp32, zeros behind the row's end.
template <typename E, int R>
__device__ __forceinline__ void widen(const Frag8<E>& p, int at, int n, float (&f)[8]) {
  fp8::unpack8(p, f);
  if constexpr (R == kAny) {
    const int past = at + 8 - n;
    if (past > 0) {
#pragma unroll
      for (int by = 4; by > 0; by /= 2)
        if (past & by) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = e + by < 8 ? f[(e + by) & 7] : 0.f;
        }
      if (past >= 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
      }
    }
  }
}

// PASS: written past the caches.
template <typename E, int R, bool PASS>
__device__ __forceinline__ void store_piece(E* p, int at, int n, const float (&f)[8]) {
  typedef typename Sixteen<E, R>::type T;
  if (at >= n) return;
  p += at;
  if (R != kPieces && at + 8 > n) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < n) p[e] = from_f32<E>(f[e]);
    return;
  }
  T v[sizeof(E) / 2];
  if constexpr (sizeof(E) == 2) {
    v[0] = T{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = T{__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
               __float_as_uint(f[4 * h + 3])};
  }
#pragma unroll
  for (int i = 0; i < int(sizeof(E)) / 2; ++i) {
    if constexpr (PASS) __builtin_nontemporal_store(v[i], reinterpret_cast<T*>(p) + i);
    else reinterpret_cast<T*>(p)[i] = v[i];
  }
}

// The sum of a row's squares by groups of 64 consecutive pieces (a wave's), so that
// it does not depend on the threads that hold the row, which depend on how many rows
// there are: a row's results are the same in any batch.
template <int CH>
__device__ __forceinline__ float square_sum(const float (&f)[CH][8], RowThreads& row_threads) {
  float s[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    s[c] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[c] = __builtin_fmaf(f[c][e], f[c][e], s[c]);
  }
  return row_threads.sum<CH>(s);
}

// What z is held in.
enum Held { kWide, kInt8, kE4m3F32, kE4m3E8m0 };

// E: type of y, the gate, the weights and a wide z; H: of the residual.  A row
// is held in CH pieces of eight elements by each of T threads: one wave, with four
// rows to a workgroup, or a whole workgroup.
template <typename E, typename H, int Z, int R, int CH>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a) {
  // Fused where it is written so: what the compiler would choose may differ from one CH to another.
#pragma clang fp contract(off)
  __shared__ float lds[2][kRowMaxParts];
  RowThreads row_threads{lds, a.T / kWave, 0};
  const int li = a.T == kWave ? int(threadIdx.x) % kWave : int(threadIdx.x), rows = a.T == kWave ? int(blockDim.x) / kWave : 1;
  for (int64_t row = int64_t(blockIdx.x) * rows + (rows > 1 ? int(threadIdx.x) / kWave : 0); row < a.M;
       row += int64_t(gridDim.x) * rows) {
    // (Pieces of R == kAny are widened only when all of a row's loads are out: that takes a branch.)
    float f[CH][8];
    {
      const H* h = static_cast<const H*>(a.r.h) + row * a.r.h_stride;
      Frag8<H> raw[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) raw[c] = fetch<H, R>(h, (c * a.T + li) * 8, a.n);
      if (!a.r.y) {
#pragma unroll
        for (int c = 0; c < CH; ++c) widen<H, R>(raw[c], (c * a.T + li) * 8, a.n, f[c]);
      } else {
        float y[CH][8];
        const E* yr = static_cast<const E*>(a.r.y) + row * a.r.y_stride;
        Frag8<E> t[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) t[c] = fetch<E, R>(yr, (c * a.T + li) * 8, a.n);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          widen<H, R>(raw[c], (c * a.T + li) * 8, a.n, f[c]);
          widen<E, R>(t[c], (c * a.T + li) * 8, a.n, y[c]);
        }
        if (a.post) {
          const float r = 1.f / sqrtf(square_sum<CH>(y, row_threads) * a.inv_n + a.eps);
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[c][e] *= r;
          if (a.r.post_weight) {
            const E* pw = static_cast<const E*>(a.r.post_weight);
#pragma unroll
            for (int c = 0; c < CH; ++c) t[c] = fetch<E, R>(pw, (c * a.T + li) * 8, a.n);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              float w[8];
              widen<E, R>(t[c], (c * a.T + li) * 8, a.n, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[c][e] *= w[e] + a.offset;
            }
          }
        }
        if (a.r.gate) {
          const E* gate = static_cast<const E*>(a.r.gate) + (unsigned(row) / unsigned(a.r.gate_rows)) * a.r.gate_stride;
          if (a.r.gate_channels) {
#pragma unroll
            for (int c = 0; c < CH; ++c) t[c] = fetch<E, R>(gate, (c * a.T + li) * 8, a.n);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              float g[8];
              widen<E, R>(t[c], (c * a.T + li) * 8, a.n, g);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[c][e] *= g[e];
            }
          } else {
            const float g = to_f32<E>(*gate);   // one for the row
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) y[c][e] *= g;
          }
        }
        H* out = static_cast<H*>(a.r.h_out) + row * a.r.h_out_stride;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[c][e] = __builtin_fmaf(f[c][e], a.scale, y[c][e]);
          store_piece<H, R, true>(out, (c * a.T + li) * 8, a.n, f[c]);
        }
      }
    }
    if (!a.r.z) continue;
    const float r = 1.f / sqrtf(square_sum<CH>(f, row_threads) * a.inv_n + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[c][e] *= r;
    if (a.r.weight) {
      const E* weight = static_cast<const E*>(a.r.weight);
      Frag8<E> t[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) t[c] = fetch<E, R>(weight, (c * a.T + li) * 8, a.n);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float w[8];
        widen<E, R>(t[c], (c * a.T + li) * 8, a.n, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[c][e] *= w[e] + a.offset;
      }
    }
    if constexpr (Z == kWide) {
      E* z = static_cast<E*>(a.r.z) + row * a.r.z_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) store_piece<E, R, false>(z, (c * a.T + li) * 8, a.n, f[c]);
    } else {
      static_assert(R == kPieces, "8-bit results are written eight at a time");
      uint8_t* z = static_cast<uint8_t*>(a.r.z) + row * a.n;
      if constexpr (Z == kInt8) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((c * a.T + li) * 8 < a.n) top = max(top, fp8::abs_bits(f[c][e]));
        float stored, by;
        int8::row_scale(row_threads.max_bits(top), stored, by);
        if (li == 0) static_cast<float*>(a.r.z_scale)[row] = stored;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int at = (c * a.T + li) * 8;
          if (at < a.n)
            *reinterpret_cast<fp8::u32x2*>(z + at) =
                fp8::u32x2{int8::pack4(f[c][0], f[c][1], f[c][2], f[c][3], by),
                           int8::pack4(f[c][4], f[c][5], f[c][6], f[c][7], by)};
        }
      } else {
        // Sixteen lanes hold a block of 128 columns.
        constexpr int SC = Z == kE4m3F32 ? TB_SCALE_F32 : TB_SCALE_E8M0;
        const int blocks = (a.n + fp8::kBlock - 1) / fp8::kBlock;
        fp8::scale_t<SC>* zs = static_cast<fp8::scale_t<SC>*>(a.r.z_scale) + row * blocks;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int at = (c * a.T + li) * 8;
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (at < a.n) top = max(top, fp8::abs_bits(f[c][e]));
          top = max16(top);
          fp8::scale_t<SC> stored;
          float by;
          fp8::block_scale<SC>(top, stored, by);
          if (at < a.n) {
            *reinterpret_cast<fp8::u32x2*>(z + at) =
                fp8::u32x2{fp8::pack4(f[c][0] * by, f[c][1] * by, f[c][2] * by, f[c][3] * by),
                           fp8::pack4(f[c][4] * by, f[c][5] * by, f[c][6] * by, f[c][7] * by)};
            if (at % fp8::kBlock == 0) zs[at / fp8::kBlock] = stored;
          }
        }
      }
    }
  }
}

template <typename E, typename H, int Z, int R>
hipError_t norm_sized(NormArgs& a, hipStream_t stream) {
  // For many rows the fewest threads that hold a row in three pieces each (4096 x
  // 5376: 33.0 us with 256 threads, 37.9 with 512, 43.6 with 1024), for fewer up to
  // one piece each, as long as there are no more than 1024 threads for every
  // compute unit (1 x 5376: 3.6 us with 1024 threads, 3.8 with 512, 4.4 with 256;
  // 512 x 5376: 7.1 with 512, 7.2 with 1024).
  a.T = kWave;
  while (a.T < 1024 && (a.T * 24 < a.n || (a.T * 8 < a.n && a.M * a.T * 2 <= 1 << 18))) a.T *= 2;
  const int ch = (a.n + 8 * a.T - 1) / (8 * a.T), threads = a.T == kWave ? 256 : a.T, rows = threads / a.T;
  const dim3 grid(unsigned(std::min<int64_t>((a.M + rows - 1) / rows, 1 << 20)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a);
    return hipGetLastError();
  };
  if (ch == 1) return go(residual_norm_kernel<E, H, Z, R, 1>);
  if constexpr (R != kShort) {
    if (ch == 2) return go(residual_norm_kernel<E, H, Z, R, 2>);
    if (ch == 3) return go(residual_norm_kernel<E, H, Z, R, 3>);
    if (ch == 4) return go(residual_norm_kernel<E, H, Z, R, 4>);
  }
  return hipErrorInvalidValue;
}

// Whether every row can be taken in 16-byte pieces.
bool pieces_fit(const NormArgs& a) {
  const tb_residual& r = a.r;
  const int64_t strides = r.h_stride | r.y_stride | r.h_out_stride | r.z_stride | (r.gate_channels ? r.gate_stride : 0);
  uintptr_t at = 0;
  for (const void* p : {r.h, r.y, r.post_weight, r.weight, (const void*)r.h_out, (const void*)r.z,
                        r.gate_channels ? r.gate : nullptr})
    at |= reinterpret_cast<uintptr_t>(p);
  return a.n % 8 == 0 && strides % 8 == 0 && at % 16 == 0;
}

template <typename E, typename H>
hipError_t norm_typed(NormArgs& a, tb_dtype z_dtype, tb_scale scale_type, hipStream_t stream) {
  if (z_dtype == TB_INT8) return norm_sized<E, H, kInt8, kPieces>(a, stream);
  if (z_dtype == TB_E4M3)
    return scale_type == TB_SCALE_F32 ? norm_sized<E, H, kE4m3F32, kPieces>(a, stream)
                                      : norm_sized<E, H, kE4m3E8m0, kPieces>(a, stream);
  if (pieces_fit(a)) return norm_sized<E, H, kWide, kPieces>(a, stream);
  return a.n < 8 ? norm_sized<E, H, kWide, kShort>(a, stream) : norm_sized<E, H, kWide, kAny>(a, stream);
}

}  // namespace

hipError_t launch_residual_norm(const tb_residual& r, int64_t m, int64_t n, float residual_scale, float eps,
                                float weight_offset, bool post_norm, tb_dtype dtype, tb_dtype h_dtype, tb_dtype z_dtype,
                                tb_scale scale_type, hipStream_t stream) {
  NormArgs a{};
  a.r = r;
  a.r.gate_rows = std::max<int64_t>(1, std::min(r.gate_rows, m));   // (m fits 32 bits)
  a.M = m;
  a.n = int(n);
  a.scale = residual_scale;
  a.eps = eps;
  a.offset = weight_offset;
  a.inv_n = 1.f / float(n);
  a.post = post_norm;
  if (dtype == TB_BF16)
    return h_dtype == TB_BF16 ? norm_typed<bf16_t, bf16_t>(a, z_dtype, scale_type, stream)
                              : norm_typed<bf16_t, float>(a, z_dtype, scale_type, stream);
  return h_dtype == TB_BF16 ? norm_typed<float, bf16_t>(a, z_dtype, scale_type, stream)
                            : norm_typed<float, float>(a, z_dtype, scale_type, stream);
}

}  // namespace tb
