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
  int first[kMaxProjections + 1];   // part j owns head groups first[j] .. first[j+1] - 1 of a token
  int64_t T;
  int D, half;      // head size, rotated pairs
  int G;            // lanes per head (a power of two)
  int iters;        // head groups a wave walks
  const int64_t* pos;
  const double* freq;
  float eps, offset, inv_d;
};

// V consecutive elements as they are in memory.
template <typename E, int V> struct Raw { uint4 v; };
template <typename E> struct Raw<E, 1> { E v; };
template <> struct Raw<bf16_t, 2> { uint32_t v; };
template <> struct Raw<float, 2> { float2 v; };

template <typename E, int V>
__device__ __forceinline__ Raw<E, V> load_raw(const E* p) {
  Raw<E, V> r;
  r.v = *reinterpret_cast<const decltype(r.v)*>(p);
  return r;
}
template <typename E, int V> __device__ __forceinline__ Raw<E, V> zero_raw() {
  if constexpr (V == 1) return Raw<E, 1>{from_f32<E>(0.f)};
  else if constexpr (V > 2) return Raw<E, V>{make_uint4(0, 0, 0, 0)};
  else return Raw<E, V>{};
}

template <typename E, int V>
__device__ __forceinline__ void widen(const Raw<E, V>& r, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = to_f32<E>(r.v);
  } else if constexpr (V == 2) {
    if constexpr (sizeof(E) == 2) {
      f[0] = __uint_as_float(r.v << 16);
      f[1] = __uint_as_float(r.v & 0xffff0000u);
    } else {
      f[0] = r.v.x;
      f[1] = r.v.y;
    }
  } else {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (sizeof(E) == 2) f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
      else f[e] = __uint_as_float(w[e]);
    }
  }
}

template <typename E, int V>
__device__ __forceinline__ void store_chunk(E* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<E>(f[0]);
  } else if constexpr (V == 2) {
    if constexpr (sizeof(E) == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16(f[0], f[1]);
    else *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else if constexpr (sizeof(E) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                              pack_bf16(f[6], f[7]));
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  }
}

// V: elements of a chunk (16 bytes, 2, or 1 for any size and alignment); UPL:
// units (pairs of chunks) per lane; INTER: interleaved pairs.
template <typename E, int V, int UPL, bool INTER>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadArgs a) {
  const int l = int(threadIdx.x) & 63;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  if (t >= a.T) return;
  const int lane = l & (a.G - 1), slot = l / a.G, slots = kWave / a.G;
  const int g0 = int(blockIdx.y) * a.iters, g1 = min(g0 + a.iters, a.first[a.n]);

  // Unit u's chunks: interleaved, 2V consecutive elements from 2V u.  Else the
  // rotated units take V elements from V u and their partners R/2 further on,
  // and the units after them 2V consecutive elements of the rest.
  int ea[UPL], eb[UPL];
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
  }

  // The part that owns group g (uniform), and this lane's head of the group.
  int j = 0;
  while (g0 >= a.first[j + 1]) ++j;
  Raw<E, V> ra[UPL], rb[UPL];
  auto fetch = [&](int g, int pj) {
    const tb_head_part& pt = a.part[pj];
    const int h = (g - a.first[pj]) * slots + slot;
    const E* x = static_cast<const E*>(pt.x) + t * pt.x_token_stride + h * pt.x_head_stride;
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      ra[k] = rb[k] = zero_raw<E, V>();
      if (h < int(pt.heads)) {
        if (ea[k] < a.D) ra[k] = load_raw<E, V>(x + ea[k]);
        if (eb[k] < a.D) rb[k] = load_raw<E, V>(x + eb[k]);
      }
    }
  };
  fetch(g0, j);   // under way while the angles are computed

  float cs[UPL][V], sn[UPL][V];
  const double where = a.half > 0 ? double(a.pos[t]) : 0.;
#pragma unroll
  for (int k = 0; k < UPL; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int p = (lane + k * a.G) * V + e;   // the pair's frequency
      cs[k][e] = 1.f;
      sn[k][e] = 0.f;
      if (p < a.half) {
        const double turns = where * a.freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
        sincospif(2.f * float(turns - rint(turns)), &sn[k][e], &cs[k][e]);
      }
    }

  float wa[UPL][V], wb[UPL][V];
  int have = -1;   // the part whose weights are in wa, wb
  for (int g = g0; g < g1; ++g) {
    const tb_head_part& pt = a.part[j];
    const int h = (g - a.first[j]) * slots + slot;
    if (j != have) {
      have = j;
      const E* wt = static_cast<const E*>(pt.weight);
#pragma unroll
      for (int k = 0; k < UPL; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) wa[k][e] = wb[k][e] = 1.f;
        if (wt) {
          if (ea[k] < a.D) widen<E, V>(load_raw<E, V>(wt + ea[k]), wa[k]);
          if (eb[k] < a.D) widen<E, V>(load_raw<E, V>(wt + eb[k]), wb[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            wa[k][e] += a.offset;
            wb[k][e] += a.offset;
          }
        }
      }
    }
    float fa[UPL][V], fb[UPL][V];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      widen<E, V>(ra[k], fa[k]);
      widen<E, V>(rb[k], fb[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum += fa[k][e] * fa[k][e] + fb[k][e] * fb[k][e];
    }
    const int jn = j;
    if (g + 1 < g1) {   // the next group loads while this one is finished
      while (g + 1 >= a.first[j + 1]) ++j;
      fetch(g + 1, j);
    }
    for (int d = 1; d < a.G; d *= 2) sum += __shfl_xor(sum, d);
    const float r = 1.f / sqrtf(sum * a.inv_d + a.eps);
    E* y = static_cast<E*>(a.part[jn].y) + t * a.part[jn].y_token_stride + h * a.part[jn].y_head_stride;
    const bool live = h < int(a.part[jn].heads);
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        fa[k][e] *= r * wa[k][e];
        fb[k][e] *= r * wb[k][e];
      }
      // Elements that are not rotated are left alone: turned by nothing, they
      // would still take on an infinity or NaN of their neighbour.
      const int p0 = (lane + k * a.G) * V;   // the unit's first pair
      if constexpr (INTER && V > 1) {
        // The unit's 2V elements are V pairs: the first V/2 in chunk a, the rest in chunk b.
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float x0 = fa[k][e], x1 = fa[k][e + 1], c0 = cs[k][e / 2], s0 = sn[k][e / 2];
          const bool ta = p0 + e / 2 < a.half, tb = p0 + V / 2 + e / 2 < a.half;
          fa[k][e] = ta ? x0 * c0 - x1 * s0 : x0;
          fa[k][e + 1] = ta ? x1 * c0 + x0 * s0 : x1;
          const float z0 = fb[k][e], z1 = fb[k][e + 1], c1 = cs[k][V / 2 + e / 2], s1 = sn[k][V / 2 + e / 2];
          fb[k][e] = tb ? z0 * c1 - z1 * s1 : z0;
          fb[k][e + 1] = tb ? z1 * c1 + z0 * s1 : z1;
        }
      } else if (p0 < a.half) {   // V divides half: a unit is rotated as a whole
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x0 = fa[k][e], x1 = fb[k][e];
          fa[k][e] = x0 * cs[k][e] - x1 * sn[k][e];
          fb[k][e] = x1 * cs[k][e] + x0 * sn[k][e];
        }
      }
      if (live && ea[k] < a.D) store_chunk<E, V>(y + ea[k], fa[k]);
      if (live && eb[k] < a.D) store_chunk<E, V>(y + eb[k], fb[k]);
    }
  }
}

template <typename E, int V>
hipError_t heads_typed(HeadArgs& a, bool interleaved, hipStream_t stream) {
  const int units = (a.D + 2 * V - 1) / (2 * V);
  a.G = 1;
  while (a.G < kWave && a.G < units) a.G *= 2;
  const int upl = (units + a.G - 1) / a.G, slots = kWave / a.G;
  for (int j = 0; j < a.n; ++j) a.first[j + 1] = a.first[j] + int((a.part[j].heads + slots - 1) / slots);
  const int groups = a.first[a.n];
  // A wave walks all of a token's heads, computing its angles once (4096 tokens
  // of 32 + 8 heads of 256: 34 us, against 40 in two waves and 56 in ten),
  // unless that leaves too few waves for the chip.
  a.iters = std::max(1, int(std::min<int64_t>(groups, groups * a.T / 4096)));
  const dim3 grid(unsigned((a.T + kThreads / kWave - 1) / (kThreads / kWave)), unsigned((groups + a.iters - 1) / a.iters));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  };
  if (upl == 1) return interleaved ? go(heads_kernel<E, V, 1, true>) : go(heads_kernel<E, V, 1, false>);
  if constexpr (V <= 4)
    if (upl == 2) return interleaved ? go(heads_kernel<E, V, 2, true>) : go(heads_kernel<E, V, 2, false>);
  if constexpr (V <= 2)
    if (upl <= 4) return interleaved ? go(heads_kernel<E, V, 4, true>) : go(heads_kernel<E, V, 4, false>);
  if constexpr (V == 1)
    if (upl <= 8) return interleaved ? go(heads_kernel<E, V, 8, true>) : go(heads_kernel<E, V, 8, false>);
  return hipErrorInvalidValue;
}

// Whether every part can be taken in chunks of V elements: sizes, strides and
// addresses are multiples of one.  What is not walks in pairs or single elements,
// whose loads and stores are then what counts: 4096 tokens of 32 + 8 heads of 250,
// 63 pairs rotated, one element at a time: 83 us (2.0 TB/s), against 35 for heads
// of 256 in chunks of 16 bytes.
template <typename E>
bool chunks_fit(const HeadArgs& a, bool interleaved, int V) {
  if (a.D % V != 0 || (!interleaved && a.half % V != 0)) return false;
  for (int j = 0; j < a.n; ++j) {
    const tb_head_part& p = a.part[j];
    if (p.heads > 0 &&
        ((p.x_token_stride | p.x_head_stride | p.y_token_stride | p.y_head_stride) % V != 0 ||
         ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.weight)) &
          (V * sizeof(E) - 1)) != 0))
      return false;
  }
  return true;
}

template <typename E>
hipError_t heads_vec(HeadArgs& a, bool interleaved, hipStream_t stream) {
  constexpr int V = 16 / sizeof(E);
  if (chunks_fit<E>(a, interleaved, V)) return heads_typed<E, V>(a, interleaved, stream);
  return chunks_fit<E>(a, interleaved, 2) ? heads_typed<E, 2>(a, interleaved, stream)
                                          : heads_typed<E, 1>(a, interleaved, stream);
}

}  // namespace

hipError_t launch_heads(tb_dtype dtype, int n, const tb_head_part* parts, int64_t tokens, int head_dim, int rot_dim,
                        bool interleaved, const int64_t* positions, const double* freqs, float eps, float offset,
                        hipStream_t stream) {
  HeadArgs a{};
  a.n = n;
  for (int j = 0; j < n; ++j) {
    a.part[j] = parts[j];
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
