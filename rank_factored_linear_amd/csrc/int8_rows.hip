// Rows as 8-bit integers with a scale each (the format is in int8_device.h).
//
// One pass: a row's threads hold it in registers between its maximum and its
// rounding.  Bound by HBM for many rows (5376 x 21504 bf16 61 us, 5.7 TB/s, most of it
// read) and by launch latency for a few (61 x 1152 fp32 3.0).
#include "int8_device.h"

#include <algorithm>

namespace tb {

namespace {

// A row is held by T threads, CH pieces of eight elements each: one wave, with
// four rows to a workgroup, or a whole workgroup.
template <typename E, int CH>
__global__ __launch_bounds__(1024) void int8_rows_kernel(const E* __restrict__ x, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale, int64_t M, int I, int T) {
  __shared__ float lds[2][kRowMaxParts];
  RowThreads row_threads{lds, T / kWave, 0};
  const int li = int(threadIdx.x) % T, rows = int(blockDim.x) / T;
  for (int64_t row = int64_t(blockIdx.x) * rows + int(threadIdx.x) / T; row < M; row += int64_t(gridDim.x) * rows) {
    const E* xr = x + row * I;
    Frag8<E> f[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * T + li) * 8;   // I % 8 == 0: all eight or none
      f[c] = load_frag_if<E>(xr + at, at < I);
    }
    uint32_t a = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float t[8];
      fp8::unpack8(f[c], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = max(a, fp8::abs_bits(t[e]));
    }
    a = row_threads.max_bits(a);
    float stored, by;
    int8::row_scale(a, stored, by);
    if (li == 0) scale[row] = stored;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * T + li) * 8;
      float t[8];
      fp8::unpack8(f[c], t);
      if (at < I)
        *reinterpret_cast<fp8::u32x2*>(q + row * I + at) =
            fp8::u32x2{int8::pack4(t[0], t[1], t[2], t[3], by), int8::pack4(t[4], t[5], t[6], t[7], by)};
    }
  }
}

template <typename E>
hipError_t rows_typed(const void* x, void* q, float* scale, int64_t m, int64_t in_dim, hipStream_t stream) {
  // The fewest threads that hold the row in four pieces each.
  int T = kWave;
  while (T < 1024 && T * 32 < in_dim) T *= 2;
  const int ch = int((in_dim + 8 * T - 1) / (8 * T)), threads = T == kWave ? 256 : T, rows = threads / T;
  const dim3 grid(unsigned(std::min<int64_t>((m + rows - 1) / rows, 1 << 20)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, static_cast<const E*>(x), static_cast<uint8_t*>(q), scale,
                       m, int(in_dim), T);
    return hipGetLastError();
  };
  if (ch == 1) return go(int8_rows_kernel<E, 1>);
  if (ch == 2) return go(int8_rows_kernel<E, 2>);
  if (ch <= 4) return go(int8_rows_kernel<E, 4>);
  return ch <= 8 ? go(int8_rows_kernel<E, 8>) : hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_int8_rows(tb_dtype dtype, const void* x, void* q, float* scale, int64_t m, int64_t in_dim,
                            hipStream_t stream) {
  return dtype == TB_BF16 ? rows_typed<bf16_t>(x, q, scale, m, in_dim, stream)
                          : rows_typed<float>(x, q, scale, m, in_dim, stream);
}

}  // namespace tb
