// Per-head norms with the position rotation in the same pass: for each token
// and head of D elements
//   z = x / sqrt(mean(x^2) + eps) * (weight + offset),
// then the first R elements of z are turned by the token's position: pair p of
// (z_i, z_j) becomes (z_i cos - z_j sin, z_j cos + z_i sin) with the angle
// position * freq[p] (pairs (p, p + R/2), or (2p, 2p + 1) when interleaved).
//
// Each element is read and written once: the call is bound by HBM for a
// prefill and by launch latency for a few tokens.  A group of lanes holds a
// head, a lane two chunks of V elements chosen so that both members of every
// pair meet in one lane; the square sum is a few cross-lane steps.  A wave
// works on one token and keeps its cosines and sines in registers while it
// walks heads, so they are computed once per token, chunk and wave.  Angles
// are fp64 products reduced to a fraction of a turn in fp64 (a position of a
// million leaves fp32 no correct digits of the fraction), then fp32.
#include "tb_device.h"
#include "tb_host.h"

#include <algorithm>

namespace tb {

namespace {

constexpr int kThreads = 256;

struct HeadArgs {
  int n;
  tb_head_part part[kMaxProjections];
  int first[kMaxProjections + 1];   // part j owns heads first[j] .. first[j+1] - 1 of a token
  int64_t T;
  int D, half;      // head size, rotated pairs
  int G;            // lanes per head (a power of two)
  int iters;        // head groups a wave walks
  const int64_t* pos;
  const double* freq;
  float eps, offset, inv_d;
};

template <typename E, int V>
__device__ __forceinline__ void load_chunk(const E* p, float (&f)[V]) {
  if constexpr (V * sizeof(E) == 16) {
    if constexpr (sizeof(E) == 2) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
      const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = to_f32<E>(p[e]);
  }
}

template <typename E, int V>
__device__ __forceinline__ void store_chunk(E* p, const float (&f)[V]) {
  if constexpr (V * sizeof(E) == 16) {
    if constexpr (sizeof(E) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32_to_bf16(f[2 * e]) | (uint32_t(f32_to_bf16(f[2 * e + 1])) << 16);
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = from_f32<E>(f[e]);
  }
}

// V: elements of a chunk (16 bytes, or 1 for any size and alignment); UPL:
// units (pairs of chunks) per lane; INTER: interleaved pairs.
template <typename E, int V, int UPL, bool INTER>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadArgs a) {
  const int l = int(threadIdx.x) & 63;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / kWave) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int lane = l & (a.G - 1), slot = l / a.G, slots = kWave / a.G;
  const int heads = a.first[a.n];
  const int h0 = int(blockIdx.y) * a.iters * slots;

  // Unit u's chunks: interleaved, 2V consecutive elements from 2V u.  Else the
  // rotated units take V elements from V u and their partners R/2 further on,
  // and the units after them 2V consecutive elements of the rest.
  int ea[UPL], eb[UPL];
  float cs[UPL][V], sn[UPL][V];
  const double where = a.half > 0 ? double(a.pos[t]) : 0.;
#pragma unroll
  for (int k = 0; k < UPL; ++k) {
    const int u = lane + k * a.G;
    if (INTER) {
      ea[k] = 2 * V * u;
      eb[k] = ea[k] + V;
    } else if (u * V < a.half) {
      ea[k] = u * V;
      eb[k] = a.half + u * V;
    } else {
      ea[k] = 2 * a.half + 2 * (u * V - a.half);
      eb[k] = ea[k] + V;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int p = u * V + e;   // the pair's frequency
      cs[k][e] = 1.f;
      sn[k][e] = 0.f;
      if (p < a.half) {
        const double turns = where * a.freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
        sincospif(2.f * float(turns - rint(turns)), &sn[k][e], &cs[k][e]);
      }
    }
  }

  for (int it = 0; it < a.iters; ++it) {
    const int h = h0 + it * slots + slot;
    const bool live = h < heads;
    int j = 0;
    while (live && j + 1 < a.n && h >= a.first[j + 1]) ++j;
    const tb_head_part& pt = a.part[j];
    const int hh = live ? h - a.first[j] : 0;
    const E* x = static_cast<const E*>(pt.x) + t * pt.x_token_stride + hh * pt.x_head_stride;
    float fa[UPL][V], fb[UPL][V];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) fa[k][e] = fb[k][e] = 0.f;
      if (live && ea[k] < a.D) load_chunk<E, V>(x + ea[k], fa[k]);
      if (live && eb[k] < a.D) load_chunk<E, V>(x + eb[k], fb[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum += fa[k][e] * fa[k][e] + fb[k][e] * fb[k][e];
    }
    for (int d = 1; d < a.G; d *= 2) sum += __shfl_xor(sum, d);
    const float r = 1.f / sqrtf(sum * a.inv_d + a.eps);
    if (!live) continue;
    const E* wt = static_cast<const E*>(pt.weight);
    E* y = static_cast<E*>(pt.y) + t * pt.y_token_stride + hh * pt.y_head_stride;
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      float wa[V], wb[V];
#pragma unroll
      for (int e = 0; e < V; ++e) wa[e] = wb[e] = 1.f;
      if (wt) {
        if (ea[k] < a.D) load_chunk<E, V>(wt + ea[k], wa);
        if (eb[k] < a.D) load_chunk<E, V>(wt + eb[k], wb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          wa[e] += a.offset;
          wb[e] += a.offset;
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        fa[k][e] *= r * wa[e];
        fb[k][e] *= r * wb[e];
      }
      if constexpr (INTER && V > 1) {
        // The unit's 2V elements are V pairs: the first V/2 in chunk a, the rest in chunk b.
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float x0 = fa[k][e], x1 = fa[k][e + 1], c0 = cs[k][e / 2], s0 = sn[k][e / 2];
          fa[k][e] = x0 * c0 - x1 * s0;
          fa[k][e + 1] = x1 * c0 + x0 * s0;
          const float z0 = fb[k][e], z1 = fb[k][e + 1], c1 = cs[k][V / 2 + e / 2], s1 = sn[k][V / 2 + e / 2];
          fb[k][e] = z0 * c1 - z1 * s1;
          fb[k][e + 1] = z1 * c1 + z0 * s1;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x0 = fa[k][e], x1 = fb[k][e];
          fa[k][e] = x0 * cs[k][e] - x1 * sn[k][e];
          fb[k][e] = x1 * cs[k][e] + x0 * sn[k][e];
        }
      }
      if (ea[k] < a.D) store_chunk<E, V>(y + ea[k], fa[k]);
      if (eb[k] < a.D) store_chunk<E, V>(y + eb[k], fb[k]);
    }
  }
}

template <typename E, int V>
hipError_t heads_typed(HeadArgs& a, bool interleaved, hipStream_t stream) {
  const int units = (a.D + 2 * V - 1) / (2 * V);
  a.G = 1;
  while (a.G < kWave && a.G < units) a.G *= 2;
  const int upl = (units + a.G - 1) / a.G, slots = kWave / a.G;
  const int groups = (a.first[a.n] + slots - 1) / slots;
  // A wave walks all of a token's heads (its angles are then computed once)
  // unless there are too few tokens to fill the chip.
  a.iters = a.T >= 4096 ? groups : std::max(1, int(groups * a.T / 4096));
  const dim3 grid(unsigned((a.T + kThreads / kWave - 1) / (kThreads / kWave)), unsigned((groups + a.iters - 1) / a.iters));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  };
  if (upl == 1) return interleaved ? go(heads_kernel<E, V, 1, true>) : go(heads_kernel<E, V, 1, false>);
  if (upl == 2) return interleaved ? go(heads_kernel<E, V, 2, true>) : go(heads_kernel<E, V, 2, false>);
  if constexpr (V == 1) {
    if (upl <= 4) return interleaved ? go(heads_kernel<E, V, 4, true>) : go(heads_kernel<E, V, 4, false>);
    if (upl <= 8) return interleaved ? go(heads_kernel<E, V, 8, true>) : go(heads_kernel<E, V, 8, false>);
  }
  return hipErrorInvalidValue;
}

template <typename E>
hipError_t heads_vec(HeadArgs& a, bool interleaved, hipStream_t stream) {
  constexpr int V = 16 / sizeof(E);
  // 16-byte chunks need sizes, strides and addresses that are multiples of 16 bytes.
  bool vec = a.D % V == 0 && (interleaved || a.half % V == 0);
  for (int j = 0; j < a.n && vec; ++j) {
    const tb_head_part& p = a.part[j];
    vec = (p.x_token_stride | p.x_head_stride | p.y_token_stride | p.y_head_stride) % V == 0 &&
          ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.weight)) &
           15u) == 0;
  }
  return vec ? heads_typed<E, V>(a, interleaved, stream) : heads_typed<E, 1>(a, interleaved, stream);
}

}  // namespace

hipError_t launch_heads(tb_dtype dtype, int n, const tb_head_part* parts, int64_t tokens, int head_dim, int rot_dim,
                        bool interleaved, const int64_t* positions, const double* freqs, float eps, float offset,
                        hipStream_t stream) {
  HeadArgs a{};
  a.n = n;
  for (int j = 0; j < n; ++j) {
    a.part[j] = parts[j];
    a.first[j + 1] = a.first[j] + int(parts[j].heads);
  }
  a.T = tokens;
  a.D = head_dim;
  a.half = rot_dim / 2;
  a.pos = positions;
  a.freq = freqs;
  a.eps = eps;
  a.offset = offset;
  a.inv_d = 1.f / float(head_dim);
  return dtype == TB_BF16 ? heads_vec<bf16_t>(a, interleaved, stream) : heads_vec<float>(a, interleaved, stream);
}

}  // namespace tb
