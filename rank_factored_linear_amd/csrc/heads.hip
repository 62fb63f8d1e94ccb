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
// million leaves fp32 no correct digits of the fraction), then fp32, which is what
// sincospif takes: that rounds the fraction by up to 2^-26 of a turn, so a cosine or
// sine is off by up to 1e-7 beside its own rounding.  A bf16 result does not see it; in
// fp32 ones it shows in the last place.
//
// With several axes (time, height, width) a token has a position on each, and a
// pair's angle takes the one of its axis; pairs may then lie within the span of
// their axis, (j, j + count) behind the elements of the axes before, and the
// norm may be left out.  Which axis a pair belongs to travels with the launch
// (two bits each), so it is checked on the host.
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

// What a launch with several axes knows besides.  Where each axis comes in one run
// of pairs that is where the runs begin; else a table, read only then.
struct AxesTable {
  int norm, table;
  int begin[kMaxAxes];                       // runs: their first pairs (behind the last run: none)
  int64_t row[kMaxAxes];                     // where the positions of a run's axis (with a table: of an axis) start
  uint32_t axis[TB_MAX_HEAD_DIM / 2 / 16];   // table: of pair p two bits at 2 (p % 16) of word p / 16
};
// SPAN: pairs lie within the span of their axis (there are runs).  LANES: of the
// narrow layout (spread(1) below) whose units a lane holds, each summed by itself.
template <bool SPAN_, int LANES_> struct AxesArgs : HeadArgs {
  static constexpr bool kAxes = true, kSpan = SPAN_;
  static constexpr int kLanes = LANES_;
  AxesTable m;
};
struct OneAxisArgs : HeadArgs {
  static constexpr bool kAxes = false, kSpan = false;
  static constexpr int kLanes = 1;
};

// What lanes l and l ^ D hold, added: within sixteen lanes by a cross-lane add (the
// mirrors reach a lane that holds the same as l ^ D, as all smaller D are done).
template <int CTRL> __device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, 0xf, 0xf, false)));
}
template <int D> __device__ __forceinline__ float add_lanes(float v) {
  if constexpr (D == 1) return add_dpp<0xb1>(v);         // neighbours
  else if constexpr (D == 2) return add_dpp<0x4e>(v);    // pairs
  else if constexpr (D == 4) return add_dpp<0x141>(v);   // eight mirrored
  else if constexpr (D == 8) return add_dpp<0x140>(v);   // sixteen mirrored
  else return v + __shfl_xor(v, D);
}
// N sums over G lanes each, then with one another, in the order of a tree over N G lanes.
template <int N> __device__ __forceinline__ float sum_lanes(float (&s)[N], int G) {
  auto step = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (D < G) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = add_lanes<D>(s[i]);
    }
  };
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 4>{});
  step(std::integral_constant<int, 8>{});
  step(std::integral_constant<int, 16>{});
  step(std::integral_constant<int, 32>{});
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int i = 0; i < N; i += 2 * w) s[i] += s[i + w];
  return s[0];
}

// With several axes which operations are fused is written out: of a a + b b either
// product may be, and what the compiler takes differs from one number of units to
// another, which is chosen by the number of tokens.  It is what the compiler takes for
// one axis (in all but fp32 heads of 512 and more), where a pair's second element adds
// the other way round if a lane of the narrow layout holds one unit of one pair.
__device__ __forceinline__ float plus_squares(float sum, float a, float b) {
#pragma clang fp contract(off)
  return sum + __builtin_fmaf(a, a, b * b);
}
template <bool ONE_PAIR>
__device__ __forceinline__ void turn(float x0, float x1, float c, float s, float& y0, float& y1) {
#pragma clang fp contract(off)
  y0 = __builtin_fmaf(x0, c, -(x1 * s));
  y1 = ONE_PAIR ? __builtin_fmaf(x0, s, x1 * c) : __builtin_fmaf(x1, c, x0 * s);
}
__device__ __forceinline__ float fraction(double at, double freq) {   // of a turn
#pragma clang fp contract(off)
  const double turns = at * freq * 0.15915494309189533577;   // 1 / (2 pi)
  return float(turns - rint(turns));
}

// The table's words over a wave's lanes, as many as there are pairs for.
__device__ __forceinline__ uint32_t axis_words(const AxesTable& m, int half) {
  const int l = int(threadIdx.x) & 63;
  uint32_t word = 0;
#pragma unroll
  for (int c = 0; c < TB_MAX_HEAD_DIM / 2 / 16; c += 8)
    if (c * 16 < half)
#pragma unroll
      for (int k = c; k < c + 8; ++k) word = l == k ? m.axis[k] : word;
  return word;
}
// One of four values, each a variable of its own: with an array, filled in a loop,
// the compiler chooses among the elements' addresses, and the array goes to memory
// (1009 tokens of 32 heads of 72 in fp32: 21 us against 8.3).
static_assert(kMaxAxes == 4, "two bits name an axis");
template <typename T> struct Four { T a, b, c, d; };
template <typename T> __device__ __forceinline__ T pick(const Four<T>& v, int i) {
  const T lo = i == 0 ? T(v.a) : T(v.b), hi = i == 2 ? T(v.c) : T(v.d);
  return i < 2 ? T(lo) : T(hi);
}

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
// units (pairs of chunks) per lane; INTER: interleaved pairs; A: for one axis or
// for several.
template <typename E, int V, int UPL, bool INTER, typename A>
__global__ __launch_bounds__(kThreads) void heads_kernel(A a) {
  const int l = int(threadIdx.x) & 63;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  if (t >= a.T) return;
  const int lane = l & (a.G - 1), slot = l / a.G, slots = kWave / a.G;
  const int g0 = int(blockIdx.y) * a.iters, g1 = min(g0 + a.iters, a.first[a.n]);

  // Unit u's chunks: interleaved, 2V consecutive elements from 2V u.  Else the
  // rotated units take V elements from V u and their partners R/2 further on,
  // and the units after them 2V consecutive elements of the rest.
  int ea[UPL], eb[UPL];
  uint32_t axes[UPL];   // of the unit's pairs, two bits each: with a table their axes, else their runs
  Four<int> begin{};
  if constexpr (A::kAxes) {
    begin = Four<int>{a.m.begin[0], a.m.begin[1], a.m.begin[2], a.m.begin[3]};
    if (a.m.table) {
      const uint32_t words = axis_words(a.m, a.half);
#pragma unroll
      for (int k = 0; k < UPL; ++k) {
        const int p0 = (lane + k * a.G) * V;   // (V divides 16: a unit's pairs lie in one word)
        axes[k] = uint32_t(__shfl(int(words), p0 >> 4 & 63)) >> (2 * (p0 & 15));
      }
    } else {
#pragma unroll
      for (int k = 0; k < UPL; ++k) {
        axes[k] = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int p = (lane + k * a.G) * V + e;
          axes[k] |= uint32_t((p >= begin.b) + (p >= begin.c) + (p >= begin.d)) << (2 * e);
        }
      }
    }
  }
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
    if constexpr (A::kSpan)
      if (u * V < a.half) {   // (V divides every axis's pairs: a unit belongs to one)
        const int r = int(axes[k] & 3u), first = pick(begin, r);
        const Four<int> end{min(begin.b, a.half), min(begin.c, a.half), min(begin.d, a.half), a.half};
        ea[k] = first + u * V;
        eb[k] = ea[k] + pick(end, r) - first;
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
  double where = 0.;
  Four<double> on{};
  if constexpr (A::kAxes) {   // (unused ones: the first axis's)
    on = Four<double>{double(a.pos[a.m.row[0] + t]), double(a.pos[a.m.row[1] + t]), double(a.pos[a.m.row[2] + t]),
                      double(a.pos[a.m.row[3] + t])};
  } else {
    where = a.half > 0 ? double(a.pos[t]) : 0.;
  }
#pragma unroll
  for (int k = 0; k < UPL; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int p = (lane + k * a.G) * V + e;   // the pair's frequency
      cs[k][e] = 1.f;
      sn[k][e] = 0.f;
      if (p < a.half) {
        double at = where;
        if constexpr (A::kAxes) {
          at = pick(on, int(axes[k] >> (2 * e) & 3u));
          sincospif(2.f * fraction(at, a.freq[p]), &sn[k][e], &cs[k][e]);
        } else {
          const double turns = at * a.freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
          sincospif(2.f * float(turns - rint(turns)), &sn[k][e], &cs[k][e]);
        }
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
    float sum = 0.f, sums[A::kLanes] = {};   // (sums: with several axes, of each lane of the narrow layout)
#pragma unroll
    for (int k = 0; k < UPL; ++k) {
      widen<E, V>(ra[k], fa[k]);
      widen<E, V>(rb[k], fb[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (A::kAxes) sums[k % A::kLanes] = plus_squares(sums[k % A::kLanes], fa[k][e], fb[k][e]);
        else sum += fa[k][e] * fa[k][e] + fb[k][e] * fb[k][e];
      }
    }
    const int jn = j;
    if (g + 1 < g1) {   // the next group loads while this one is finished
      while (g + 1 >= a.first[j + 1]) ++j;
      fetch(g + 1, j);
    }
    float r = 1.f;
    bool normed = true;
    if constexpr (A::kAxes) normed = a.m.norm;
    if (normed) {
      if constexpr (A::kAxes) {
        r = 1.f / sqrtf(__builtin_fmaf(sum_lanes(sums, a.G), a.inv_d, a.eps));
      } else {
        for (int d = 1; d < a.G; d *= 2) sum += __shfl_xor(sum, d);
        r = 1.f / sqrtf(sum * a.inv_d + a.eps);
      }
    }
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
          if constexpr (A::kAxes) {
            float y0, y1;
            turn<false>(x0, x1, c0, s0, y0, y1);
            fa[k][e] = ta ? y0 : x0;
            fa[k][e + 1] = ta ? y1 : x1;
          } else {
            fa[k][e] = ta ? x0 * c0 - x1 * s0 : x0;
            fa[k][e + 1] = ta ? x1 * c0 + x0 * s0 : x1;
          }
          const float z0 = fb[k][e], z1 = fb[k][e + 1], c1 = cs[k][V / 2 + e / 2], s1 = sn[k][V / 2 + e / 2];
          if constexpr (A::kAxes) {
            float y0, y1;
            turn<false>(z0, z1, c1, s1, y0, y1);
            fb[k][e] = tb ? y0 : z0;
            fb[k][e + 1] = tb ? y1 : z1;
          } else {
            fb[k][e] = tb ? z0 * c1 - z1 * s1 : z0;
            fb[k][e + 1] = tb ? z1 * c1 + z0 * s1 : z1;
          }
        }
      } else if (p0 < a.half) {   // V divides half: a unit is rotated as a whole
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x0 = fa[k][e], x1 = fb[k][e];
          if constexpr (A::kAxes) {
            turn<V == 1 && UPL <= A::kLanes>(x0, x1, cs[k][e], sn[k][e], fa[k][e], fb[k][e]);
          } else {
            fa[k][e] = x0 * cs[k][e] - x1 * sn[k][e];
            fb[k][e] = x1 * cs[k][e] + x0 * sn[k][e];
          }
        }
      }
      if (live && ea[k] < a.D) store_chunk<E, V>(y + ea[k], fa[k]);
      if (live && eb[k] < a.D) store_chunk<E, V>(y + eb[k], fb[k]);
    }
  }
}

template <typename E, int V>
hipError_t heads_typed(HeadArgs& a, bool interleaved, bool span, const AxesTable* axes, hipStream_t stream) {
  const int units = (a.D + 2 * V - 1) / (2 * V);
  // Units of a lane: as few as the lanes allow, so that a few tokens have many lanes.  Pieces of two or one element
  // leave a lane little to do for each step of its wave: with several axes and many tokens four units are taken (4096
  // tokens of 32 + 8 heads of 180 in bf16: 27.5 us against 57.4; but 64 of 32 heads of 72, not normed, 5.2 against
  // 3.6).  A head's squares are added in the order that the narrow layout has, so its results do not depend on how many
  // tokens there are.
  auto spread = [&](int per) {
    a.G = 1;
    while (a.G < kWave && a.G * per < units) a.G *= 2;
    const int slots = kWave / a.G;
    for (int j = 0; j < a.n; ++j) a.first[j + 1] = a.first[j] + int((a.part[j].heads + slots - 1) / slots);
    return a.first[a.n];
  };
  int groups = spread(1);
  const int narrow = a.G;
  if (V <= 2 && axes && groups * a.T >= 32768) groups = spread(4);
  const int lanes = narrow / a.G;   // 1, 2 or 4
  const int upl = (units + a.G - 1) / a.G;
  // A wave walks all of a token's heads, computing its angles once (4096 tokens
  // of 32 + 8 heads of 256: 34 us, against 40 in two waves and 56 in ten),
  // unless that leaves too few waves for the chip.
  a.iters = std::max(1, int(std::min<int64_t>(groups, groups * a.T / 4096)));
  const dim3 grid(unsigned((a.T + kThreads / kWave - 1) / (kThreads / kWave)), unsigned((groups + a.iters - 1) / a.iters));
  auto go = [&](auto units) {
    constexpr int UPL = decltype(units)::value;
    auto launch = [&](auto kernel, auto args) {
      static_cast<HeadArgs&>(args) = a;
      if constexpr (decltype(args)::kAxes) args.m = *axes;
      hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, args);
      return hipGetLastError();
    };
    if (!axes)
      return interleaved ? launch(heads_kernel<E, V, UPL, true, OneAxisArgs>, OneAxisArgs{})
                         : launch(heads_kernel<E, V, UPL, false, OneAxisArgs>, OneAxisArgs{});
    auto several = [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      if (interleaved) return launch(heads_kernel<E, V, UPL, true, AxesArgs<false, L>>, AxesArgs<false, L>{});
      return span ? launch(heads_kernel<E, V, UPL, false, AxesArgs<true, L>>, AxesArgs<true, L>{})
                  : launch(heads_kernel<E, V, UPL, false, AxesArgs<false, L>>, AxesArgs<false, L>{});
    };
    if constexpr (V <= 2 && UPL == 4)
      if (lanes == 4) return several(std::integral_constant<int, 4>{});
    if constexpr (V <= 2 && (UPL == 2 || UPL == 4))
      if (lanes == 2) return several(std::integral_constant<int, 2>{});
    return several(std::integral_constant<int, 1>{});
  };
  if (upl == 1) return go(std::integral_constant<int, 1>{});
  if constexpr (V <= 4)
    if (upl == 2) return go(std::integral_constant<int, 2>{});
  if constexpr (V <= 2)
    if (upl <= 4) return go(std::integral_constant<int, 4>{});
  if constexpr (V == 1)
    if (upl <= 8) return go(std::integral_constant<int, 8>{});
  return hipErrorInvalidValue;
}

// Whether every part can be taken in chunks of V elements: sizes, strides and
// addresses are multiples of one.  What is not walks in pairs or single elements,
// whose loads and stores are then what counts: 4096 tokens of 32 + 8 heads of 250,
// 63 pairs rotated, one element at a time: 83 us (2.0 TB/s), against 35 for heads
// of 256 in chunks of 16 bytes.
template <typename E>
bool chunks_fit(const HeadArgs& a, bool interleaved, bool span, const AxesTable* axes, int V) {
  if (a.D % V != 0 || (!interleaved && a.half % V != 0)) return false;
  if (span)
    for (int b : axes->begin)   // (half is a multiple of V, too)
      if (b < a.half && b % V != 0) return false;
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
hipError_t heads_vec(HeadArgs& a, bool interleaved, bool span, const AxesTable* axes, hipStream_t stream) {
  constexpr int V = 16 / sizeof(E);
  if (chunks_fit<E>(a, interleaved, span, axes, V)) return heads_typed<E, V>(a, interleaved, span, axes, stream);
  return chunks_fit<E>(a, interleaved, span, axes, 2) ? heads_typed<E, 2>(a, interleaved, span, axes, stream)
                                                      : heads_typed<E, 1>(a, interleaved, span, axes, stream);
}

HeadArgs head_args(int n, const tb_head_part* parts, int64_t tokens, int head_dim, int rot_dim, const int64_t* positions,
                   const double* freqs, float eps, float offset) {
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
  return a;
}

}  // namespace

hipError_t launch_heads(tb_dtype dtype, int n, const tb_head_part* parts, int64_t tokens, int head_dim, int rot_dim,
                        bool interleaved, const int64_t* positions, const double* freqs, float eps, float offset,
                        hipStream_t stream) {
  HeadArgs a = head_args(n, parts, tokens, head_dim, rot_dim, positions, freqs, eps, offset);
  return dtype == TB_BF16 ? heads_vec<bf16_t>(a, interleaved, false, nullptr, stream)
                          : heads_vec<float>(a, interleaved, false, nullptr, stream);
}

hipError_t launch_heads_axes(tb_dtype dtype, int n, const tb_head_part* parts, int64_t tokens, int head_dim, int rot_dim,
                             const HeadAxes& axes, const int64_t* positions, const double* freqs, float eps, float offset,
                             hipStream_t stream) {
  if (axes.axes == 1 && axes.norm)   // (with one axis its span is all pairs)
    return launch_heads(dtype, n, parts, tokens, head_dim, rot_dim, axes.pairs == TB_PAIRS_INTERLEAVED, positions, freqs,
                        eps, offset, stream);
  HeadArgs a = head_args(n, parts, tokens, head_dim, rot_dim, positions, freqs, eps, offset);
  AxesTable m{};
  m.norm = axes.norm;
  unsigned seen = 0;
  int runs = 0;
  for (int p = 0; p < a.half; ++p) {
    const int ax = axes.pair_axis[p];
    m.axis[p / 16] |= uint32_t(ax) << (2 * (p % 16));
    if (p > 0 && ax == axes.pair_axis[p - 1]) continue;
    if (seen >> ax & 1u) m.table = 1;
    seen |= 1u << ax;
    if (runs < kMaxAxes) {
      m.begin[runs] = p;
      m.row[runs] = ax * tokens;
    }
    ++runs;
  }
  if (m.table)
    for (int i = 0; i < kMaxAxes; ++i) m.row[i] = i < axes.axes ? i * tokens : 0;
  else
    for (int i = runs; i < kMaxAxes; ++i) m.begin[i] = 1 << 30;
  const bool interleaved = axes.pairs == TB_PAIRS_INTERLEAVED, span = axes.pairs == TB_PAIRS_AXIS;
  return dtype == TB_BF16 ? heads_vec<bf16_t>(a, interleaved, span, &m, stream)
                          : heads_vec<float>(a, interleaved, span, &m, stream);
}

}  // namespace tb
