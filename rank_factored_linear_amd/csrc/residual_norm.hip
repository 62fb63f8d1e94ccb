// The norms before and after a block in one pass over the residual stream: for
// each row
//   a = y, or y / sqrt(mean(y^2) + eps) * (post_weight + offset)
//   h' = residual_scale * h + gate * a
//   z = h' / sqrt(mean(h'^2) + eps) * (weight + offset)
// with z in the type that the next projection takes: wide, 8-bit integers with a
// scale per row, or e4m3 with a scale per 128 columns.
//
// A row's threads hold it in registers from its load to its last store, in
// fp32: z is made from h' as it is before it is rounded to be stored.  Each
// element is read and written once, so the call is bound by HBM for many rows
// and by latency (two sums over the row, one behind the other) for a few.
//
// h' goes past the caches: the block that reads it next has a layer's weights
// before it, while z is read at once.  With y the z of the call before and h
// cold, bf16: 4096 x 5376 36.3 us (4.9 TB/s) against 37.5 with both kept and 38.1
// with both past them, 1024 x 5376 10.4 (11.5, 10.0), 4096 x 1152 9.2 (10.6, 8.9).
// Loading the next row ahead of the present one gained nothing (40.9 -> 41.9 us).
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

// V elements as fp32.
template <typename E, int V>
__device__ __forceinline__ void load_v(const E* p, bool ok, float (&f)[V]) {
  if constexpr (V == 8) {
    fp8::unpack8(load_frag_if<E>(p, ok), f);
  } else {
    static_assert(V == 1, "pieces of eight or one");
    f[0] = ok ? to_f32<E>(*p) : 0.f;
  }
}

// PASS: written past the caches where the piece allows it.
template <typename T, bool PASS>
__device__ __forceinline__ void put(T* p, const T& v) {
  if constexpr (PASS) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <typename E, int V, bool PASS>
__device__ __forceinline__ void store_v(E* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<E>(f[0]);
  } else if constexpr (sizeof(E) == 2) {
    put<fp8::u32x4, PASS>(reinterpret_cast<fp8::u32x4*>(p), fp8::u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])});
  } else {
    put<f32x4, PASS>(reinterpret_cast<f32x4*>(p), f32x4{f[0], f[1], f[2], f[3]});
    put<f32x4, PASS>(reinterpret_cast<f32x4*>(p) + 1, f32x4{f[4], f[5], f[6], f[7]});
  }
}

// The sum of a row's squares.  Pieces of eight: by groups of 64 consecutive pieces
// (a wave's), so that it does not depend on the threads that hold the row, which
// depend on how many rows there are: a row's results are the same in any batch.
// (The threads for single elements depend on n alone.)
template <int V, int CH>
__device__ __forceinline__ float square_sum(const float (&f)[CH][V], RowThreads& row_threads) {
  constexpr int kParts = V == 8 ? CH : 1;
  float s[kParts];
#pragma unroll
  for (int c = 0; c < kParts; ++c) s[c] = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < V; ++e) s[kParts == 1 ? 0 : c] = __builtin_fmaf(f[c][e], f[c][e], s[kParts == 1 ? 0 : c]);
  return row_threads.sum<kParts>(s);
}

// What z is held in.
enum Held { kWide, kInt8, kE4m3F32, kE4m3E8m0 };

// E: type of y, the gate, the weights and a wide z; H: of the residual.  A row
// is held in CH pieces of V elements by each of T threads: one wave, with four
// rows to a workgroup, or a whole workgroup.
template <typename E, typename H, int Z, int V, int CH>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a) {
  // Fused where it is written so: what the compiler would choose may differ from one CH to another.
#pragma clang fp contract(off)
  __shared__ float lds[2][kRowMaxParts];
  RowThreads row_threads{lds, a.T / kWave, 0};
  const int li = a.T == kWave ? int(threadIdx.x) % kWave : int(threadIdx.x), rows = a.T == kWave ? int(blockDim.x) / kWave : 1;
  for (int64_t row = int64_t(blockIdx.x) * rows + (rows > 1 ? int(threadIdx.x) / kWave : 0); row < a.M;
       row += int64_t(gridDim.x) * rows) {
    float f[CH][V];
    {
      const H* h = static_cast<const H*>(a.r.h) + row * a.r.h_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * a.T + li) * V;
        load_v<H, V>(h + at, at < a.n, f[c]);
      }
    }
    if (a.r.y) {
      float y[CH][V];
      const E* yr = static_cast<const E*>(a.r.y) + row * a.r.y_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * a.T + li) * V;
        load_v<E, V>(yr + at, at < a.n, y[c]);
      }
      float r = 1.f;
      if (a.post) r = 1.f / sqrtf(square_sum<V, CH>(y, row_threads) * a.inv_n + a.eps);
      const E* pw = static_cast<const E*>(a.r.post_weight);
      const E* gate = static_cast<const E*>(a.r.gate);
      float whole = 1.f;   // one gate for the row
      if (gate) {
        gate += (unsigned(row) / unsigned(a.r.gate_rows)) * a.r.gate_stride;
        if (!a.r.gate_channels) whole = to_f32<E>(*gate);
      }
      H* out = static_cast<H*>(a.r.h_out) + row * a.r.h_out_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * a.T + li) * V;
        float t[V];
        if (a.post) {
#pragma unroll
          for (int e = 0; e < V; ++e) y[c][e] *= r;
          if (pw) {
            load_v<E, V>(pw + at, at < a.n, t);
#pragma unroll
            for (int e = 0; e < V; ++e) y[c][e] *= t[e] + a.offset;
          }
        }
        if (gate) {
          if (a.r.gate_channels) {
            load_v<E, V>(gate + at, at < a.n, t);
#pragma unroll
            for (int e = 0; e < V; ++e) y[c][e] *= t[e];
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) y[c][e] *= whole;
          }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) f[c][e] = __builtin_fmaf(f[c][e], a.scale, y[c][e]);
        if (at < a.n) store_v<H, V, true>(out + at, f[c]);
      }
    }
    if (!a.r.z) continue;
    const float r = 1.f / sqrtf(square_sum<V, CH>(f, row_threads) * a.inv_n + a.eps);
    const E* wt = static_cast<const E*>(a.r.weight);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * a.T + li) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) f[c][e] *= r;
      if (wt) {
        float t[V];
        load_v<E, V>(wt + at, at < a.n, t);
#pragma unroll
        for (int e = 0; e < V; ++e) f[c][e] *= t[e] + a.offset;
      }
    }
    if constexpr (Z == kWide) {
      E* z = static_cast<E*>(a.r.z) + row * a.r.z_stride;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * a.T + li) * V;
        if (at < a.n) store_v<E, V, false>(z + at, f[c]);
      }
    } else {
      static_assert(Z == kWide || V == 8, "8-bit results are written eight at a time");
      uint8_t* z = static_cast<uint8_t*>(a.r.z) + row * a.n;
      if constexpr (Z == kInt8) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < V; ++e)
            if ((c * a.T + li) * V < a.n) top = max(top, fp8::abs_bits(f[c][e]));
        float stored, by;
        int8::row_scale(row_threads.max_bits(top), stored, by);
        if (li == 0) static_cast<float*>(a.r.z_scale)[row] = stored;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int at = (c * a.T + li) * V;
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
          const int at = (c * a.T + li) * V;
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < V; ++e)
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

template <typename E, typename H, int Z, int V>
hipError_t norm_sized(NormArgs& a, hipStream_t stream) {
  // For many rows the fewest threads that hold a row in three pieces each (4096 x
  // 5376: 40.9 us with 256 threads, 43.2 with 512, 51 with 1024), for fewer up to
  // one piece each, as long as there are no more than 1024 threads for every
  // compute unit (1 x 5376: 4.1 us with 1024 threads, 4.5 with 512, 5.5 with 256;
  // 512 x 5376: 7.5 with 512, 7.7 with 1024).
  constexpr int kMost = V == 8 ? 3 : 8;
  a.T = kWave;
  while (a.T < 1024 && (int64_t(a.T) * V * kMost < a.n || (V == 8 && a.T * V < a.n && a.M * a.T * 2 <= 1 << 18))) a.T *= 2;
  const int ch = (a.n + V * a.T - 1) / (V * a.T), threads = a.T == kWave ? 256 : a.T, rows = threads / a.T;
  const dim3 grid(unsigned(std::min<int64_t>((a.M + rows - 1) / rows, 1 << 20)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a);
    return hipGetLastError();
  };
  if constexpr (V == 8) {
    if (ch == 1) return go(residual_norm_kernel<E, H, Z, V, 1>);
    if (ch == 2) return go(residual_norm_kernel<E, H, Z, V, 2>);
    if (ch == 3) return go(residual_norm_kernel<E, H, Z, V, 3>);
    if (ch == 4) return go(residual_norm_kernel<E, H, Z, V, 4>);
  } else {
    if (ch <= 8) return go(residual_norm_kernel<E, H, Z, V, 8>);
    if (ch <= 32) return go(residual_norm_kernel<E, H, Z, V, 32>);
  }
  return hipErrorInvalidValue;
}

// Whether every row can be taken in 16-byte pieces.
template <typename E, typename H>
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
  if (z_dtype == TB_INT8) return norm_sized<E, H, kInt8, 8>(a, stream);
  if (z_dtype == TB_E4M3)
    return scale_type == TB_SCALE_F32 ? norm_sized<E, H, kE4m3F32, 8>(a, stream)
                                      : norm_sized<E, H, kE4m3E8m0, 8>(a, stream);
  return pieces_fit<E, H>(a) ? norm_sized<E, H, kWide, 8>(a, stream) : norm_sized<E, H, kWide, 1>(a, stream);
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
