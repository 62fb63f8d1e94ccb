// C ABI of libtb: host-side argument checks and dispatch.  Every check runs
// before anything is enqueued, so a failing call leaves all outputs untouched.
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "tb_host.h"

namespace tb {

namespace {

thread_local char g_last_error[512] = "";

tb_status fail(tb_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return st;
}

tb_status ok() {
  g_last_error[0] = '\0';
  return TB_OK;
}

tb_status hip_fail(hipError_t e, const char* what) {
  return fail(TB_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t esize(tb_dtype d) { return d == TB_BF16 ? 2 : 4; }
bool valid_dtype(tb_dtype d) { return d == TB_F32 || d == TB_BF16; }

constexpr int kMaxDevices = 64;
int g_cus[kMaxDevices];  // 0 = not queried yet (benign race: every writer stores the same value)

// Shapes the kernels index with 32-bit ints.
constexpr int64_t kMaxDim = int64_t(1) << 30;

tb_status check_dims(int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank) {
  if (m < 1 || out_dim < 1 || in_dim < 1 || rank < 0)
    return fail(TB_ERR_INVALID_ARGUMENT, "need m >= 1, out_dim >= 1, in_dim >= 1, rank >= 0 (got %lld, %lld, %lld, %lld)",
                (long long)m, (long long)out_dim, (long long)in_dim, (long long)rank);
  if (m > kMaxDim || out_dim > kMaxDim || in_dim > kMaxDim || rank > kMaxDim)
    return fail(TB_ERR_UNSUPPORTED, "a dimension exceeds 2^30");
  if (in_dim % 8 != 0) return fail(TB_ERR_UNSUPPORTED, "in_dim %lld is not a multiple of 8", (long long)in_dim);
  return TB_OK;
}

}  // namespace

namespace {
std::atomic<int> g_wait_polls{1 << 20};
}  // namespace

int decode_wait_polls() { return g_wait_polls.load(std::memory_order_relaxed); }

int device_cu_count(int* cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return int(e);
  if (dev >= 0 && dev < kMaxDevices && g_cus[dev] > 0) {
    *cus = g_cus[dev];
    return 0;
  }
  int n = 0;
  e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return int(e);
  if (n < 2) n = 2;
  if (dev >= 0 && dev < kMaxDevices) g_cus[dev] = n;
  *cus = n;
  return 0;
}

}  // namespace tb

using namespace tb;

extern "C" {

tb_status tb_band_index(int32_t num_layers, int32_t num_bands, int32_t layer, int32_t* band_out) {
  if (band_out == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "band_out is NULL");
  if (num_layers < 1) return fail(TB_ERR_INVALID_ARGUMENT, "num_layers %d < 1", num_layers);
  if (num_bands < 1 || num_bands > num_layers)
    return fail(TB_ERR_INVALID_ARGUMENT, "num_bands %d outside [1, %d]", num_bands, num_layers);
  if (layer < 0 || layer >= num_layers)
    return fail(TB_ERR_INVALID_ARGUMENT, "layer %d outside [0, %d)", layer, num_layers);
  // q layers per band, the first m bands one more; they end at layer m(q+1).
  const int32_t q = num_layers / num_bands, m = num_layers % num_bands;
  const int32_t big = m * (q + 1);
  *band_out = layer < big ? layer / (q + 1) : m + (layer - big) / q;
  return ok();
}

namespace {

// Data bytes of one projection's buffers: enough for every plan a call of m
// tokens may take (alone or in a group, whatever its streamer budget; the
// last 64-token slice of a longer fp32 call has a plan of its own).
size_t forward_data_bytes(int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype, int cus) {
  if (dtype == TB_BF16 && m > kDecodeMaxTokens) return plan_gemm(1, &out_dim, m, in_dim, rank, cus).bytes;
  size_t bytes = 0;
  const int64_t counts[2] = {m < kDecodeMaxTokens ? m : kDecodeMaxTokens,
                             m > kDecodeMaxTokens ? m % kDecodeMaxTokens : 0};
  for (int64_t mt : counts)
    if (mt > 0) bytes = std::max(bytes, decode_bytes_bound(mt, out_dim, in_dim, rank, cus));
  return bytes;
}

// Whether the members of a group run as one launch of each prefill kernel:
// bf16, more than kDecodeMaxTokens tokens, and one in_dim and rank for all
// (q, k and v of a layer; gate and up).
bool fused_prefill(int n, const tb_projection* projs, int64_t m, tb_dtype dtype) {
  if (dtype != TB_BF16 || m <= kDecodeMaxTokens || n < 2) return false;
  for (int j = 1; j < n; ++j)
    if (projs[j].in_dim != projs[0].in_dim || projs[j].rank != projs[0].rank) return false;
  return true;
}

GemmPlan fused_prefill_plan(int n, const tb_projection* projs, int64_t m, int cus) {
  int64_t outs[TB_MAX_GROUP];
  for (int j = 0; j < n; ++j) outs[j] = projs[j].out_dim;
  return plan_gemm(n, outs, m, projs[0].in_dim, projs[0].rank, cus);
}

// Data bytes of a group: every member's own buffers one after another (the
// members may run as calls of their own), or the fused launch's buffers if
// they are more.
size_t group_data_bytes(int n, const tb_projection* projs, int64_t m, tb_dtype dtype, int cus) {
  size_t total = 0;
  for (int j = 0; j < n; ++j)
    total += forward_data_bytes(m, projs[j].out_dim, projs[j].in_dim, projs[j].rank, dtype, cus);
  if (fused_prefill(n, projs, m, dtype)) total = std::max(total, fused_prefill_plan(n, projs, m, cus).bytes);
  return total;
}

}  // namespace

tb_status tb_linear_forward_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype,
                                           size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  tb_status st = check_dims(m, out_dim, in_dim, rank);
  if (st != TB_OK) return st;
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  *bytes_out = kControlBytes + forward_data_bytes(m, out_dim, in_dim, rank, dtype, cus);
  return ok();
}

static_assert(TB_MAX_GROUP == kMaxProjections, "one launch takes every member of a group");

namespace {

// Argument checks shared by tb_linear_forward and each member of a group.
tb_status check_projection(const void* x, const void* s, const void* w0, const void* u, const void* v, const void* y,
                           int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  tb_status st = check_dims(m, out_dim, in_dim, rank);
  if (st != TB_OK) return st;
  if (!x || !w0 || !y) return fail(TB_ERR_INVALID_ARGUMENT, "x, w0 and y must be non-NULL");
  if (rank > 0 && (!u || !v)) return fail(TB_ERR_INVALID_ARGUMENT, "u and v must be non-NULL when rank > 0");
  if (!aligned16(x) || !aligned16(w0) || (rank > 0 && (!aligned16(u) || !aligned16(v))))
    return fail(TB_ERR_UNSUPPORTED, "x, w0, u and v must be 16-byte aligned");
  if (!aligned_to(s, esize(dtype)) || !aligned_to(y, esize(dtype)))
    return fail(TB_ERR_UNSUPPORTED, "s and y must be aligned to their element size");
  // The few-token path addresses a row block (at most 96 rows) with 32-bit
  // byte offsets.
  const bool decode = !(dtype == TB_BF16 && m > kDecodeMaxTokens);
  if (decode && in_dim * int64_t(esize(dtype)) * 96 >= (int64_t(1) << 32))
    return fail(TB_ERR_UNSUPPORTED, "in_dim %lld is too large for the few-token path", (long long)in_dim);
  return TB_OK;
}

// One projection with checked arguments: the prefill GEMM, or the decode
// kernel over 64-token slices.  ctrl is its control block, data holds
// forward_data_bytes, timeouts are flagged in *err_word.
tb_status forward_one(const void* x, const void* s, const void* w0, const void* u, const void* v, void* y, int64_t m,
                      int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype, unsigned* ctrl, char* data,
                      unsigned* err_word, int cus, hipStream_t hs) {
  if (dtype == TB_BF16 && m > kDecodeMaxTokens) {
    const GemmPlan p = plan_gemm(1, &out_dim, m, in_dim, rank, cus);
    const Projection q{x, s, w0, u, v, y, out_dim, in_dim, rank};
    hipError_t e = launch_forward_gemm(p, &q, m, in_dim, rank, ctrl, data, err_word, hs);
    if (e != hipSuccess) return hip_fail(e, "launching the prefill projection");
    return ok();
  }
  const int64_t mm = m < kDecodeMaxTokens ? m : kDecodeMaxTokens;
  const size_t es = esize(dtype);
  const int64_t w0_elems = out_dim * in_dim;
  const DecodePlan p = plan_decode_spared(mm, out_dim, in_dim, rank, cus, w0_elems);
  for (int64_t t0 = 0; t0 < m; t0 += kDecodeMaxTokens) {
    const int64_t mt = (m - t0) < kDecodeMaxTokens ? (m - t0) : kDecodeMaxTokens;
    const DecodePlan pt = mt == mm ? p : plan_decode_spared(mt, out_dim, in_dim, rank, cus, w0_elems);
    const char* xt = static_cast<const char*>(x) + size_t(t0) * size_t(in_dim) * es;
    char* yt = static_cast<char*>(y) + size_t(t0) * size_t(out_dim) * es;
    hipError_t e =
        launch_forward_decode(pt, dtype, xt, s, w0, u, v, yt, mt, out_dim, in_dim, rank, ctrl, data, err_word, hs);
    if (e != hipSuccess) return hip_fail(e, "launching the decode projection");
  }
  return ok();
}

}  // namespace

tb_status tb_linear_forward(const void* x, const void* s, const void* w0, const void* u, const void* v, void* y,
                            int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  tb_status st = check_projection(x, s, w0, u, v, y, m, out_dim, in_dim, rank, dtype);
  if (st != TB_OK) return st;
  if (!workspace) return fail(TB_ERR_INVALID_ARGUMENT, "workspace must be non-NULL");
  if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const size_t need = kControlBytes + forward_data_bytes(m, out_dim, in_dim, rank, dtype, cus);
  if (workspace_bytes < need)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, need);
  unsigned* ctrl = static_cast<unsigned*>(workspace);
  return forward_one(x, s, w0, u, v, y, m, out_dim, in_dim, rank, dtype, ctrl, static_cast<char*>(workspace) + kControlBytes,
                     ctrl + 2, cus, static_cast<hipStream_t>(stream));
}

}  // extern "C"

// ---- the forward call that allocates nothing --------------------------------
//
// Its workspace is this file-scope device array, one per GPU, laid out as a
// forward workspace: control words first, then the projection's buffers.  In
// host code `scratch` names a host-side stand-in, never the device memory:
// every host use goes through the address hipGetSymbolAddress gives for the
// current device, looked up once per device.
namespace tb {
namespace {

static_assert(TB_NO_ALLOC_SCRATCH_BYTES >= kControlBytes + (size_t(1) << 20), "scratch holds the control words");
static __device__ __align__(256) unsigned char scratch[TB_NO_ALLOC_SCRATCH_BYTES];

struct ScratchSlot {
  std::once_flag once;
  unsigned char* ptr = nullptr;
  hipError_t err = hipSuccess;
};
ScratchSlot g_scratch[kMaxDevices];

// The device address of this device's scratch (set-up on its first use).
hipError_t device_scratch(unsigned char** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  ScratchSlot& slot = g_scratch[dev];
  std::call_once(slot.once, [&slot] {
    void* p = nullptr;
    slot.err = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    slot.ptr = static_cast<unsigned char*>(p);
  });
  if (slot.err != hipSuccess) return slot.err;
  *out = slot.ptr;
  return hipSuccess;
}

// Clears one control block (a small kernel rather than a memset, so that the
// call can be captured into a graph).
__global__ void clear_control_block(unsigned* words) {
  const int i = int(blockIdx.x * blockDim.x + threadIdx.x);
  if (i < int(kCtrlBlockBytes / 4)) words[i] = 0u;
}

}  // namespace
}  // namespace tb

extern "C" {

tb_status tb_linear_forward_no_alloc(const void* x, const void* s, const void* w0, const void* u, const void* v,
                                     void* y, int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank,
                                     tb_dtype dtype, void* stream) {
  tb_status st = check_projection(x, s, w0, u, v, y, m, out_dim, in_dim, rank, dtype);
  if (st != TB_OK) return st;
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const size_t need = kControlBytes + forward_data_bytes(m, out_dim, in_dim, rank, dtype, cus);
  if (need > TB_NO_ALLOC_SCRATCH_BYTES)
    return fail(TB_ERR_UNSUPPORTED, "this call needs %zu bytes of scratch, above the %zu of the static buffer "
                "(tb_linear_forward takes a workspace of any size)", need, size_t(TB_NO_ALLOC_SCRATCH_BYTES));
  unsigned char* base = nullptr;
  if (hipError_t e = device_scratch(&base)) return hip_fail(e, "looking up the static scratch");
  hipStream_t hs = static_cast<hipStream_t>(stream);
  unsigned* ctrl = reinterpret_cast<unsigned*>(base);
  // A single call uses control block 0 only.  It starts from zero every time,
  // so a call whose wait timed out does not poison the ones after it.
  hipLaunchKernelGGL(clear_control_block, dim3(unsigned(kCtrlBlockBytes / 4 / 256)), dim3(256), 0, hs, ctrl);
  if (hipError_t e = hipGetLastError()) return hip_fail(e, "clearing the scratch's control words");
  return forward_one(x, s, w0, u, v, y, m, out_dim, in_dim, rank, dtype, ctrl,
                     reinterpret_cast<char*>(base) + kControlBytes, ctrl + 2, cus, hs);
}

tb_status tb_dense_forward(const void* x, const void* w, void* y, int64_t m, int64_t out_dim, int64_t in_dim,
                           tb_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!w) return fail(TB_ERR_INVALID_ARGUMENT, "w must be non-NULL");
  return tb_linear_forward(x, nullptr, w, nullptr, nullptr, y, m, out_dim, in_dim, 0, dtype, workspace, workspace_bytes,
                           stream);
}

tb_status tb_linear_forward_group_workspace_size(int32_t n, const tb_projection* projs, int64_t m, tb_dtype dtype,
                                                 size_t* bytes_out) {
  if (bytes_out == nullptr || projs == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "projs and bytes_out must be non-NULL");
  if (n < 1 || n > TB_MAX_GROUP) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_GROUP);
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  for (int j = 0; j < n; ++j) {
    tb_status st = check_dims(m, projs[j].out_dim, projs[j].in_dim, projs[j].rank);
    if (st != TB_OK) return st;
  }
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  *bytes_out = kControlBytes + group_data_bytes(n, projs, m, dtype, cus);
  return ok();
}

tb_status tb_linear_forward_group(int32_t n, const tb_projection* projs, int64_t m, tb_dtype dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (projs == nullptr || workspace == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "projs and workspace must be non-NULL");
  if (n < 1 || n > TB_MAX_GROUP) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_GROUP);
  if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  for (int j = 0; j < n; ++j) {
    const tb_projection& q = projs[j];
    tb_status st = check_projection(q.x, q.s, q.w0, q.u, q.v, q.y, m, q.out_dim, q.in_dim, q.rank, dtype);
    if (st != TB_OK) return st;
  }
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  size_t off[TB_MAX_GROUP], at = kControlBytes;
  for (int j = 0; j < n; ++j) {
    const tb_projection& q = projs[j];
    off[j] = at;
    at += forward_data_bytes(m, q.out_dim, q.in_dim, q.rank, dtype, cus);
  }
  const size_t total = kControlBytes + group_data_bytes(n, projs, m, dtype, cus);
  if (workspace_bytes < total)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, total);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  unsigned* ctrl = reinterpret_cast<unsigned*>(ws);
  unsigned* err = ctrl + 2;

  if (m <= kDecodeMaxTokens) {
    // One launch needs every member on the same tile shape.  In order: the
    // members sharing one workgroup per compute unit, then two; each member
    // on the plan that leaves its producers' compute units to them; the
    // plain plans; else one launch per member.
    DecodePlan plans[TB_MAX_GROUP];
    Projection dp[TB_MAX_GROUP];
    int64_t w0_elems = 0;
    for (int j = 0; j < n; ++j) {
      const tb_projection& q = projs[j];
      dp[j] = Projection{q.x, q.s, q.w0, q.u, q.v, q.y, q.out_dim, q.in_dim, q.rank};
      w0_elems += q.out_dim * q.in_dim;
    }
    for (int choice = 0; choice < 4; ++choice) {
      bool same = true;
      if (choice < 2) {
        same = plan_decode_shared(n, dp, m, cus, choice + 1, w0_elems, plans);
        // Two workgroups per compute unit only where the variant's registers
        // allow it (bf16 tiles below 12 = NT x TILES; fp32 holds one).
        if (same && choice == 1 && !decode_fits_two_per_cu(dtype, plans[0].NT, plans[0].TILES)) same = false;
      } else {
        for (int j = 0; j < n; ++j) {
          const tb_projection& q = projs[j];
          plans[j] = choice == 2 ? plan_decode_spared(m, q.out_dim, q.in_dim, q.rank, cus, w0_elems)
                                 : plan_decode(m, q.out_dim, q.in_dim, q.rank, cus, cus, w0_elems);
          same = same && plans[j].NT == plans[0].NT && plans[j].TILES == plans[0].TILES;
        }
      }
      // Each member's buffers fit its share of the workspace (by construction).
      for (int j = 0; j < n && same; ++j)
        same = plans[j].bytes <= forward_data_bytes(m, projs[j].out_dim, projs[j].in_dim, projs[j].rank, dtype, cus);
      if (same) {
        hipError_t e = launch_forward_decode_group(n, plans, dp, dtype, m, ctrl, ws + kControlBytes, err, hs);
        if (e != hipSuccess) return hip_fail(e, "launching the grouped decode projections");
        return ok();
      }
    }
  }
  if (fused_prefill(n, projs, m, dtype)) {
    // One x . V launch and one GEMM launch for every member, in control
    // block 0, with the buffers from the data base.
    Projection gp[TB_MAX_GROUP];
    for (int j = 0; j < n; ++j) {
      const tb_projection& q = projs[j];
      gp[j] = Projection{q.x, q.s, q.w0, q.u, q.v, q.y, q.out_dim, q.in_dim, q.rank};
    }
    const GemmPlan p = fused_prefill_plan(n, projs, m, cus);
    hipError_t e = launch_forward_gemm(p, gp, m, projs[0].in_dim, projs[0].rank, ctrl, ws + kControlBytes, err, hs);
    if (e != hipSuccess) return hip_fail(e, "launching the grouped prefill projections");
    return ok();
  }
  for (int j = 0; j < n; ++j) {
    const tb_projection& q = projs[j];
    tb_status st = forward_one(q.x, q.s, q.w0, q.u, q.v, q.y, m, q.out_dim, q.in_dim, q.rank, dtype,
                               ctrl + j * (kCtrlBlockBytes / 4), ws + off[j], err, cus, hs);
    if (st != TB_OK) return st;
  }
  return ok();
}

tb_status tb_reconstruct_weight(const void* s, const void* w0, const void* u, const void* v, void* w_out,
                                int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype in_dtype, tb_dtype out_dtype,
                                void* stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype");
  tb_status st = check_dims(1, out_dim, in_dim, rank);
  if (st != TB_OK) return st;
  if (!s || !w0 || !w_out) return fail(TB_ERR_INVALID_ARGUMENT, "s, w0 and w_out must be non-NULL");
  if (rank > 0 && (!u || !v)) return fail(TB_ERR_INVALID_ARGUMENT, "u and v must be non-NULL when rank > 0");
  if (!aligned16(w0) || !aligned16(w_out) || (rank > 0 && (!aligned16(u) || !aligned16(v))))
    return fail(TB_ERR_UNSUPPORTED, "w0, w_out, u and v must be 16-byte aligned");
  if (!aligned_to(s, esize(in_dtype))) return fail(TB_ERR_UNSUPPORTED, "s must be aligned to its element size");
  hipError_t e = launch_reconstruct(in_dtype, out_dtype, s, w0, u, v, w_out, out_dim, in_dim, rank,
                                    static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching reconstruct");
  return ok();
}

tb_status tb_reconstruction_error(const void* s, const void* w0, const void* u, const void* v, const void* original,
                                  int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype bundle_dtype,
                                  tb_dtype original_dtype, double* result_device, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!valid_dtype(bundle_dtype) || !valid_dtype(original_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype");
  tb_status st = check_dims(1, out_dim, in_dim, rank);
  if (st != TB_OK) return st;
  if (!s || !w0 || !original || !result_device || !workspace)
    return fail(TB_ERR_INVALID_ARGUMENT, "s, w0, original, result and workspace must be non-NULL");
  if (rank > 0 && (!u || !v)) return fail(TB_ERR_INVALID_ARGUMENT, "u and v must be non-NULL when rank > 0");
  if (!aligned16(w0) || !aligned16(original) || (rank > 0 && (!aligned16(u) || !aligned16(v))))
    return fail(TB_ERR_UNSUPPORTED, "w0, original, u and v must be 16-byte aligned");
  if (!aligned_to(s, esize(bundle_dtype))) return fail(TB_ERR_UNSUPPORTED, "s must be aligned to its element size");
  if (!aligned_to(result_device, 8) || !aligned_to(workspace, 16))
    return fail(TB_ERR_UNSUPPORTED, "result must be 8-byte and workspace 16-byte aligned");
  if (workspace_bytes < TB_FROBENIUS_WORKSPACE_BYTES)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below %d", workspace_bytes,
                TB_FROBENIUS_WORKSPACE_BYTES);
  if (out_dim > (int64_t(1) << 40) / in_dim) return fail(TB_ERR_UNSUPPORTED, "matrix too large");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  hipError_t e = launch_reconstruction_error(bundle_dtype, original_dtype, s, w0, u, v, original, out_dim, in_dim, rank,
                                             result_device, workspace, cus, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the reconstruction error");
  return ok();
}

tb_status tb_rel_frobenius_error(const void* original, const void* reconstructed, int64_t rows, int64_t cols,
                                 tb_dtype dtype, double* result_device, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  if (!original || !reconstructed || !result_device || !workspace)
    return fail(TB_ERR_INVALID_ARGUMENT, "original, reconstructed, result and workspace must be non-NULL");
  if (rows < 1 || cols < 1) return fail(TB_ERR_INVALID_ARGUMENT, "rows and cols must be >= 1");
  if (rows > (int64_t(1) << 40) / cols) return fail(TB_ERR_UNSUPPORTED, "matrix too large");
  if (cols % 8 != 0) return fail(TB_ERR_UNSUPPORTED, "cols %lld is not a multiple of 8", (long long)cols);
  if (!aligned16(original) || !aligned16(reconstructed))
    return fail(TB_ERR_UNSUPPORTED, "original and reconstructed must be 16-byte aligned");
  if (!aligned_to(result_device, 8) || !aligned_to(workspace, 16))
    return fail(TB_ERR_UNSUPPORTED, "result must be 8-byte and workspace 16-byte aligned");
  if (workspace_bytes < TB_FROBENIUS_WORKSPACE_BYTES)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below %d", workspace_bytes, TB_FROBENIUS_WORKSPACE_BYTES);
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  hipError_t e = launch_frobenius(dtype, original, reconstructed, rows * cols, result_device, workspace, cus,
                                  static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the Frobenius reduction");
  return ok();
}

tb_status tb_shared_block(const void* const* weights, int32_t n, int64_t out_dim, int64_t in_dim, tb_dtype weight_dtype,
                          float* w0_out, void* stream) {
  if (!valid_dtype(weight_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(weight_dtype));
  if (!weights || !w0_out) return fail(TB_ERR_INVALID_ARGUMENT, "weights and w0_out must be non-NULL");
  if (n < 1 || n > TB_MAX_BAND_LAYERS) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_BAND_LAYERS);
  if (out_dim < 1 || in_dim < 1) return fail(TB_ERR_INVALID_ARGUMENT, "out_dim and in_dim must be >= 1");
  if (out_dim > kMaxDim / in_dim) return fail(TB_ERR_UNSUPPORTED, "matrix too large");
  for (int j = 0; j < n; ++j) {
    if (!weights[j]) return fail(TB_ERR_INVALID_ARGUMENT, "weights[%d] is NULL", j);
    if (!aligned_to(weights[j], esize(weight_dtype))) return fail(TB_ERR_INVALID_ARGUMENT, "weights[%d] misaligned", j);
  }
  if (!aligned_to(w0_out, 4)) return fail(TB_ERR_INVALID_ARGUMENT, "w0_out misaligned");
  hipError_t e = launch_shared_block(weight_dtype, weights, n, out_dim * in_dim, w0_out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the shared block");
  return ok();
}

tb_status tb_row_scale(const void* weight, const float* w0, int64_t out_dim, int64_t in_dim, tb_dtype weight_dtype,
                       float* s_out, void* stream) {
  if (!valid_dtype(weight_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(weight_dtype));
  if (!weight || !w0 || !s_out) return fail(TB_ERR_INVALID_ARGUMENT, "weight, w0 and s_out must be non-NULL");
  if (out_dim < 1 || in_dim < 1) return fail(TB_ERR_INVALID_ARGUMENT, "out_dim and in_dim must be >= 1");
  if (out_dim > kMaxDim / in_dim || out_dim > 0x7fffffff) return fail(TB_ERR_UNSUPPORTED, "matrix too large");
  if (!aligned_to(weight, esize(weight_dtype)) || !aligned_to(w0, 4) || !aligned_to(s_out, 4))
    return fail(TB_ERR_INVALID_ARGUMENT, "weight, w0 or s_out misaligned");
  hipError_t e = launch_row_scale(weight_dtype, weight, w0, out_dim, in_dim, s_out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the row scale");
  return ok();
}

namespace {

tb_status check_lowrank_dims(int64_t out_dim, int64_t in_dim, int64_t rank, int64_t k) {
  if (out_dim < 1 || in_dim < 1) return fail(TB_ERR_INVALID_ARGUMENT, "out_dim and in_dim must be >= 1");
  if (rank < 0 || k < rank) return fail(TB_ERR_INVALID_ARGUMENT, "need 0 <= rank <= k (got %lld, %lld)", (long long)rank,
                                        (long long)k);
  if (k < 1 || k > out_dim || k > in_dim)
    return fail(TB_ERR_INVALID_ARGUMENT, "k %lld outside [1, min(out_dim, in_dim)]", (long long)k);
  if (k > TB_MAX_PROBE) return fail(TB_ERR_UNSUPPORTED, "k %lld above %d", (long long)k, TB_MAX_PROBE);
  if (out_dim >= (int64_t(1) << 31) / in_dim) return fail(TB_ERR_UNSUPPORTED, "out_dim * in_dim must stay below 2^31");
  return TB_OK;
}

}  // namespace

tb_status tb_lowrank_factors_workspace_size(int64_t out_dim, int64_t in_dim, int64_t rank, int64_t k, size_t* bytes_out) {
  if (!bytes_out) return fail(TB_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  tb_status st = check_lowrank_dims(out_dim, in_dim, rank, k);
  if (st != TB_OK) return st;
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  *bytes_out = lowrank_workspace_bytes(out_dim, in_dim, k, rank, cus);
  return ok();
}

tb_status tb_lowrank_factors(const void* weight, const float* w0, const float* s, int64_t out_dim, int64_t in_dim,
                             int64_t rank, tb_dtype weight_dtype, const float* omega, int64_t k, int32_t power_iters,
                             float* u_out, float* v_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(weight_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(weight_dtype));
  tb_status st = check_lowrank_dims(out_dim, in_dim, rank, k);
  if (st != TB_OK) return st;
  if (power_iters < 0 || power_iters > 16) return fail(TB_ERR_INVALID_ARGUMENT, "power_iters %d outside [0, 16]", power_iters);
  if (!weight || !w0 || !s || !omega || !workspace)
    return fail(TB_ERR_INVALID_ARGUMENT, "weight, w0, s, omega and workspace must be non-NULL");
  if (rank > 0 && (!u_out || !v_out)) return fail(TB_ERR_INVALID_ARGUMENT, "u_out and v_out must be non-NULL");
  if (!aligned_to(weight, esize(weight_dtype)) || !aligned_to(w0, 4) || !aligned_to(s, 4) || !aligned_to(omega, 4) ||
      !aligned_to(u_out, 4) || !aligned_to(v_out, 4))
    return fail(TB_ERR_INVALID_ARGUMENT, "a pointer is misaligned");
  if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const size_t need = lowrank_workspace_bytes(out_dim, in_dim, k, rank, cus);
  if (workspace_bytes < need)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, need);
  if (rank == 0) return ok();
  const char* what = "";
  const void* const weights[1] = {weight};
  const float* const w0s[1] = {w0};
  const int e = launch_lowrank_factors(weight_dtype, weights, 1, w0s, s, out_dim, in_dim, rank, omega, k, power_iters,
                                       u_out, v_out, workspace, cus, static_cast<hipStream_t>(stream), &what);
  if (e == -1) return fail(TB_ERR_HIP, "%s failed", what);
  if (e != 0) return hip_fail(hipError_t(e), what);
  return ok();
}

tb_status tb_lowrank_factors_batch(const void* const* weights, int32_t n, const float* const* w0s, const float* s,
                                   int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype weight_dtype,
                                   const float* omega, int64_t k, int32_t power_iters, float* u_out, float* v_out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(weight_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(weight_dtype));
  if (!weights) return fail(TB_ERR_INVALID_ARGUMENT, "weights must be non-NULL");
  if (n < 1 || n > TB_MAX_BAND_LAYERS) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_BAND_LAYERS);
  tb_status st = check_lowrank_dims(out_dim, in_dim, rank, k);
  if (st != TB_OK) return st;
  if (power_iters < 0 || power_iters > 16) return fail(TB_ERR_INVALID_ARGUMENT, "power_iters %d outside [0, 16]", power_iters);
  if (!w0s || !s || !omega || !workspace)
    return fail(TB_ERR_INVALID_ARGUMENT, "w0s, s, omega and workspace must be non-NULL");
  if (rank > 0 && (!u_out || !v_out)) return fail(TB_ERR_INVALID_ARGUMENT, "u_out and v_out must be non-NULL");
  for (int j = 0; j < n; ++j) {
    if (!weights[j] || !w0s[j]) return fail(TB_ERR_INVALID_ARGUMENT, "weights[%d] or w0s[%d] is NULL", j, j);
    if (!aligned_to(weights[j], esize(weight_dtype)) || !aligned_to(w0s[j], 4))
      return fail(TB_ERR_INVALID_ARGUMENT, "weights[%d] or w0s[%d] misaligned", j, j);
  }
  if (!aligned_to(s, 4) || !aligned_to(omega, 4) || !aligned_to(u_out, 4) || !aligned_to(v_out, 4))
    return fail(TB_ERR_INVALID_ARGUMENT, "a pointer is misaligned");
  if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const size_t need = size_t(n) * lowrank_workspace_bytes(out_dim, in_dim, k, rank, cus);
  if (workspace_bytes < need)
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, need);
  if (rank == 0) return ok();
  const char* what = "";
  const int e = launch_lowrank_factors(weight_dtype, weights, n, w0s, s, out_dim, in_dim, rank, omega, k, power_iters,
                                       u_out, v_out, workspace, cus, static_cast<hipStream_t>(stream), &what);
  if (e == -1) return fail(TB_ERR_HIP, "%s failed", what);
  if (e != 0) return hip_fail(hipError_t(e), what);
  return ok();
}

tb_status tb_refine_shared_block_workspace_size(int64_t out_dim, int64_t in_dim, int32_t n, int64_t rank,
                                                size_t* bytes_out) {
  if (!bytes_out) return fail(TB_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  if (out_dim < 1 || in_dim < 1 || rank < 0) return fail(TB_ERR_INVALID_ARGUMENT, "need out_dim, in_dim >= 1, rank >= 0");
  if (n < 1 || n > TB_MAX_BAND_LAYERS) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_BAND_LAYERS);
  *bytes_out = refine_workspace_bytes(out_dim, in_dim, n, rank);
  return ok();
}

tb_status tb_refine_shared_block(const void* const* weights, const float* const* s, const float* const* u,
                                 const float* const* v, int32_t n, int64_t out_dim, int64_t in_dim, int64_t rank,
                                 tb_dtype weight_dtype, const float* w0_prev, float* w0_out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!valid_dtype(weight_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(weight_dtype));
  if (!weights || !s || !w0_prev || !w0_out || !workspace)
    return fail(TB_ERR_INVALID_ARGUMENT, "weights, s, w0_prev, w0_out and workspace must be non-NULL");
  if (n < 1 || n > TB_MAX_BAND_LAYERS) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_BAND_LAYERS);
  if (out_dim < 1 || in_dim < 1 || rank < 0) return fail(TB_ERR_INVALID_ARGUMENT, "need out_dim, in_dim >= 1, rank >= 0");
  if (out_dim >= (int64_t(1) << 31) / in_dim || rank > TB_MAX_PROBE)
    return fail(TB_ERR_UNSUPPORTED, "out_dim * in_dim must stay below 2^31 and rank at most %d", TB_MAX_PROBE);
  if (rank > 0 && (!u || !v)) return fail(TB_ERR_INVALID_ARGUMENT, "u and v must be non-NULL when rank > 0");
  for (int j = 0; j < n; ++j) {
    if (!weights[j] || !s[j] || (rank > 0 && (!u[j] || !v[j])))
      return fail(TB_ERR_INVALID_ARGUMENT, "member %d has a NULL pointer", j);
    if (!aligned_to(weights[j], esize(weight_dtype)) || !aligned_to(s[j], 4) ||
        (rank > 0 && (!aligned_to(u[j], 4) || !aligned_to(v[j], 4))))
      return fail(TB_ERR_INVALID_ARGUMENT, "member %d is misaligned", j);
  }
  if (!aligned_to(w0_prev, 4) || !aligned_to(w0_out, 4) || !aligned_to(workspace, 256))
    return fail(TB_ERR_INVALID_ARGUMENT, "w0_prev, w0_out or workspace misaligned");
  if (workspace_bytes < refine_workspace_bytes(out_dim, in_dim, n, rank))
    return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes,
                refine_workspace_bytes(out_dim, in_dim, n, rank));
  const char* what = "";
  const int e = launch_refine_shared_block(weight_dtype, weights, s, rank > 0 ? u : nullptr, rank > 0 ? v : nullptr, n,
                                           out_dim, in_dim, rank, w0_prev, w0_out, workspace,
                                           static_cast<hipStream_t>(stream), &what);
  if (e == -1) return fail(TB_ERR_HIP, "%s failed", what);
  if (e != 0) return hip_fail(hipError_t(e), what);
  return ok();
}

tb_status tb_debug_set_wait_polls(int32_t polls) {
  if (polls < 0) return fail(TB_ERR_INVALID_ARGUMENT, "polls %d < 0", polls);
  g_wait_polls.store(polls, std::memory_order_relaxed);
  return ok();
}

const char* tb_status_string(tb_status status) {
  switch (status) {
    case TB_OK: return "ok";
    case TB_ERR_INVALID_ARGUMENT: return "invalid argument";
    case TB_ERR_UNSUPPORTED: return "unsupported layout or size";
    case TB_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char* tb_last_error(void) { return g_last_error; }

}  // extern "C"

// ---- 8-bit blocks and head norms ---------------------------------------------
namespace tb {
namespace {

bool valid_scale(tb_scale s) { return s == TB_SCALE_F32 || s == TB_SCALE_E8M0; }
size_t scale_bytes(tb_scale s) { return s == TB_SCALE_E8M0 ? 1 : 4; }
static_assert(TB_FP8_BLOCK == kFp8Block, "one block size");

// m may be 0 (an empty batch); a launch has one workgroup or more per block.
tb_status check_fp8_dims(int64_t m, int64_t out_dim, int64_t in_dim, int64_t step) {
  if (m < 0 || out_dim < 1 || in_dim < 1)
    return fail(TB_ERR_INVALID_ARGUMENT, "need m >= 0, out_dim >= 1, in_dim >= 1 (got %lld, %lld, %lld)", (long long)m,
                (long long)out_dim, (long long)in_dim);
  if (m > TB_FP8_MAX_TOKENS || out_dim > kMaxDim)
    return fail(TB_ERR_UNSUPPORTED, "m exceeds %d or out_dim 2^30", TB_FP8_MAX_TOKENS);
  if (in_dim > TB_FP8_MAX_IN_DIM)
    return fail(TB_ERR_UNSUPPORTED, "in_dim %lld exceeds %d", (long long)in_dim, TB_FP8_MAX_IN_DIM);
  if (in_dim % step != 0)
    return fail(TB_ERR_UNSUPPORTED, "in_dim %lld is not a multiple of %lld", (long long)in_dim, (long long)step);
  // One launch's workgroups of 256 threads stay below 2^32 threads.
  if (fp8_blocks(out_dim) * fp8_blocks(in_dim) >= (int64_t(1) << 24) ||
      2 * fp8_blocks(out_dim) * fp8_blocks(m) >= (int64_t(1) << 24))
    return fail(TB_ERR_UNSUPPORTED, "matrix too large");
  return TB_OK;
}

// Whether the rows of a [tokens, heads, dim] output of these strides are apart.
bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  if (tokens <= 1 && heads <= 1) return true;
  if (tokens <= 1) return hs >= dim;
  if (heads <= 1) return ts >= dim;
  return (hs >= dim && ts >= (heads - 1) * hs + dim) || (ts >= dim && hs >= (tokens - 1) * ts + dim);
}

// A tensor of heads in bytes: rows at base + t * ts + h * hs.
struct HeadRows {
  int64_t base, heads, ts, hs;
};

HeadRows head_rows(const void* p, int64_t heads, int64_t ts, int64_t hs, tb_dtype dtype) {
  const int64_t es = int64_t(esize(dtype));
  return HeadRows{int64_t(reinterpret_cast<uintptr_t>(p)), heads, ts * es, hs * es};
}

// Whether rows of `row` bytes of two tensors of heads share memory.  Exact where
// both step alike over tokens and heads (views of one packed tensor, whose
// extents interleave); else only tensors whose first rows meet are told from
// ones that interleave without meeting.
bool rows_meet(const HeadRows& a, const HeadRows& b, int64_t tokens, int64_t row) {
  const int64_t delta = a.base - b.base;
  if (delta < row && -delta < row) return true;
  const int64_t ea = (tokens - 1) * a.ts + (a.heads - 1) * a.hs + row, eb = (tokens - 1) * b.ts + (b.heads - 1) * b.hs + row;
  if (delta >= eb || -delta >= ea) return false;
  if ((tokens > 1 && a.ts != b.ts) || (a.heads > 1 && b.heads > 1 && a.hs != b.hs)) return false;
  const int64_t ts = tokens > 1 ? a.ts : 0, hs = a.heads > 1 ? a.hs : b.hs;
  for (int64_t e = 1 - b.heads; e < a.heads; ++e) {
    // Rows d tokens and e heads apart lie v + d * ts bytes apart.
    const int64_t v = delta + e * hs;
    if (ts == 0) {
      if (v < row && -v < row) return true;
      continue;
    }
    // The d that bring them within a row of each other: -v - row < d * ts < row - v.
    const int64_t low = -v - row;
    const int64_t d = (low >= 0 ? low / ts : -((-low + ts - 1) / ts)) + 1;   // the least one past low
    const int64_t least = std::max(d, 1 - tokens);
    if (least < tokens && least * ts < row - v) return true;
  }
  return false;
}

// The same for 8-bit integers, whose sums of in_dim products stay within 32 bits.
tb_status check_int8_dims(int64_t m, int64_t out_dim, int64_t in_dim, int64_t step) {
  if (in_dim > TB_INT8_MAX_IN_DIM)
    return fail(TB_ERR_UNSUPPORTED, "in_dim %lld exceeds %d", (long long)in_dim, TB_INT8_MAX_IN_DIM);
  return check_fp8_dims(m, out_dim, in_dim, step);
}

// The arguments that tb_head_norm_rotate and tb_head_norm_rotate_axes share; *empty: there is nothing to do.
tb_status check_heads(int32_t n, const tb_head_part* parts, int64_t tokens, int64_t head_dim, int64_t rot_dim,
                      const int64_t* positions, const double* freqs, float eps, tb_dtype dtype, bool* empty) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  if (n < 1 || n > TB_MAX_GROUP) return fail(TB_ERR_INVALID_ARGUMENT, "n %d outside [1, %d]", n, TB_MAX_GROUP);
  if (!parts) return fail(TB_ERR_INVALID_ARGUMENT, "parts is NULL");
  if (tokens < 0 || head_dim < 1 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0)
    return fail(TB_ERR_INVALID_ARGUMENT, "need tokens >= 0, head_dim >= 1 and an even rot_dim in [0, head_dim] (got %lld, %lld, %lld)",
                (long long)tokens, (long long)head_dim, (long long)rot_dim);
  if (!(eps >= 0.f)) return fail(TB_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (head_dim > TB_MAX_HEAD_DIM || tokens > TB_MAX_HEAD_TOKENS)
    return fail(TB_ERR_UNSUPPORTED, "head_dim exceeds %d or tokens %d", TB_MAX_HEAD_DIM, TB_MAX_HEAD_TOKENS);
  int64_t heads = 0;
  for (int j = 0; j < n; ++j) {
    const tb_head_part& p = parts[j];
    if (p.heads < 0) return fail(TB_ERR_INVALID_ARGUMENT, "part %d: heads < 0", j);
    if (p.heads > TB_MAX_HEADS || (heads += p.heads) > TB_MAX_HEADS)
      return fail(TB_ERR_UNSUPPORTED, "more than %d heads", TB_MAX_HEADS);
    if (tokens == 0 || p.heads == 0) continue;
    if (!p.x || !p.y) return fail(TB_ERR_INVALID_ARGUMENT, "part %d: x and y must be non-NULL", j);
    const int64_t strides[4] = {p.x_token_stride, p.x_head_stride, p.y_token_stride, p.y_head_stride};
    for (int64_t s : strides) {
      if (s < 0) return fail(TB_ERR_INVALID_ARGUMENT, "part %d: a stride is negative", j);
      if (s > (int64_t(1) << 35)) return fail(TB_ERR_UNSUPPORTED, "part %d: a stride exceeds 2^35", j);
    }
    if (!aligned_to(p.x, esize(dtype)) || !aligned_to(p.y, esize(dtype)) || !aligned_to(p.weight, esize(dtype)))
      return fail(TB_ERR_UNSUPPORTED, "part %d: pointers must be aligned to their element size", j);
    // In place means element for element.
    if (p.x == p.y && ((tokens > 1 && p.x_token_stride != p.y_token_stride) ||
                       (p.heads > 1 && p.x_head_stride != p.y_head_stride)))
      return fail(TB_ERR_INVALID_ARGUMENT, "part %d: y is x, with other strides", j);
    const HeadRows x = head_rows(p.x, p.heads, p.x_token_stride, p.x_head_stride, dtype);
    const HeadRows y = head_rows(p.y, p.heads, p.y_token_stride, p.y_head_stride, dtype);
    const int64_t row = head_dim * int64_t(esize(dtype));
    if (p.x != p.y && rows_meet(x, y, tokens, row))
      return fail(TB_ERR_INVALID_ARGUMENT, "part %d: y overlaps x without being x", j);
    for (int k = 0; k < j; ++k) {
      const tb_head_part& o = parts[k];
      if (o.heads == 0) continue;
      const HeadRows ox = head_rows(o.x, o.heads, o.x_token_stride, o.x_head_stride, dtype);
      const HeadRows oy = head_rows(o.y, o.heads, o.y_token_stride, o.y_head_stride, dtype);
      if (rows_meet(oy, y, tokens, row) || rows_meet(oy, x, tokens, row) || rows_meet(ox, y, tokens, row))
        return fail(TB_ERR_INVALID_ARGUMENT, "parts %d and %d: one writes what the other reads or writes", k, j);
    }
    if (!rows_apart(tokens, p.heads, head_dim, p.y_token_stride, p.y_head_stride))
      return fail(TB_ERR_INVALID_ARGUMENT, "part %d: the rows of y overlap", j);
  }
  *empty = tokens == 0 || heads == 0;
  if (*empty) return TB_OK;
  if (rot_dim > 0 && (!positions || !freqs))
    return fail(TB_ERR_INVALID_ARGUMENT, "positions and freqs must be non-NULL when rot_dim > 0");
  if (rot_dim > 0 && (!aligned_to(positions, 8) || !aligned_to(freqs, 8)))
    return fail(TB_ERR_UNSUPPORTED, "positions and freqs must be 8-byte aligned");
  return TB_OK;
}

// Whether rows of la and lb bytes at steps sa and sb share memory: exact for equal steps, extents else.
bool rows_share(const void* a, int64_t la, int64_t sa, const void* b, int64_t lb, int64_t sb, int64_t m) {
  const int64_t pa = int64_t(reinterpret_cast<uintptr_t>(a)), pb = int64_t(reinterpret_cast<uintptr_t>(b));
  const int64_t ea = pa + (m - 1) * sa + la, eb = pb + (m - 1) * sb + lb;
  if (pa >= eb || pb >= ea) return false;
  if (m == 1 || sa != sb || sa == 0) return true;
  // Rows of b start at multiples of the step from a's first: a's next one must begin behind b's end.
  const int64_t d = ((pb - pa) % sa + sa) % sa;
  return d < la || d + lb > sa;
}

}  // namespace
}  // namespace tb

extern "C" {

tb_status tb_quantize_activations(const void* x, void* q, void* scale, int64_t m, int64_t in_dim, tb_dtype dtype,
                                  tb_scale scale_type, void* stream) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  if (!valid_scale(scale_type)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown scale type %d", int(scale_type));
  tb_status st = check_fp8_dims(m, 1, in_dim, 8);
  if (st != TB_OK) return st;
  if (m == 0) return ok();
  if (!x || !q || !scale) return fail(TB_ERR_INVALID_ARGUMENT, "x, q and scale must be non-NULL");
  if (!aligned16(x) || !aligned16(q)) return fail(TB_ERR_UNSUPPORTED, "x and q must be 16-byte aligned");
  if (!aligned_to(scale, scale_bytes(scale_type)))
    return fail(TB_ERR_UNSUPPORTED, "scale must be aligned to its element size");
  hipError_t e = launch_quantize_rows(dtype, scale_type, x, q, scale, ScaleStrides{fp8_blocks(in_dim), 1}, m, in_dim,
                                      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the activation quantiser");
  return ok();
}

tb_status tb_reconstruct_weight_fp8(const void* s, const void* w0, const void* u, const void* v, void* q, void* scale,
                                    int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype, tb_scale scale_type,
                                    void* stream) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  if (!valid_scale(scale_type)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown scale type %d", int(scale_type));
  tb_status st = check_fp8_dims(1, out_dim, in_dim, 8);
  if (st != TB_OK) return st;
  if (rank < 0) return fail(TB_ERR_INVALID_ARGUMENT, "rank %lld < 0", (long long)rank);
  if (rank > kMaxDim) return fail(TB_ERR_UNSUPPORTED, "a dimension exceeds 2^30");
  if (!w0 || !q || !scale) return fail(TB_ERR_INVALID_ARGUMENT, "w0, q and scale must be non-NULL");
  if (rank > 0 && (!u || !v)) return fail(TB_ERR_INVALID_ARGUMENT, "u and v must be non-NULL when rank > 0");
  if (!aligned16(w0) || !aligned16(q) || (rank > 0 && (!aligned16(u) || !aligned16(v))))
    return fail(TB_ERR_UNSUPPORTED, "w0, u, v and q must be 16-byte aligned");
  if (!aligned_to(s, esize(dtype)) || !aligned_to(scale, scale_bytes(scale_type)))
    return fail(TB_ERR_UNSUPPORTED, "s and scale must be aligned to their element size");
  hipError_t e = launch_rebuild_blocks(dtype, scale_type, s, w0, u, v, q, scale, out_dim, in_dim, rank,
                                       static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the 8-bit rebuild");
  return ok();
}

tb_status tb_dense_forward_fp8_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype,
                                              tb_dtype y_dtype, tb_scale scale_type, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  if (!valid_dtype(x_dtype) && x_dtype != TB_E4M3)
    return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(x_dtype));
  if (!valid_dtype(y_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(y_dtype));
  if (!valid_scale(scale_type)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown scale type %d", int(scale_type));
  tb_status st = check_fp8_dims(m, out_dim, in_dim, 16);
  if (st != TB_OK) return st;
  if (!fp8_decode_fits(m, out_dim)) return fail(TB_ERR_UNSUPPORTED, "out_dim %lld is too large", (long long)out_dim);
  *bytes_out = 0;
  if (m == 0) return ok();
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  *bytes_out = plan_fp8(m, out_dim, in_dim, x_dtype == TB_E4M3, y_dtype, scale_type, cus).bytes;
  return ok();
}

tb_status tb_dense_forward_fp8(const void* x, const void* x_scale, const void* wq, const void* w_scale, void* y,
                               int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype, tb_dtype y_dtype,
                               tb_scale scale_type, void* workspace, size_t workspace_bytes, void* stream) {
  const bool quantised = x_dtype == TB_E4M3;
  if (!valid_dtype(x_dtype) && !quantised) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(x_dtype));
  if (!valid_dtype(y_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(y_dtype));
  if (!valid_scale(scale_type)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown scale type %d", int(scale_type));
  tb_status st = check_fp8_dims(m, out_dim, in_dim, 16);
  if (st != TB_OK) return st;
  if (!fp8_decode_fits(m, out_dim)) return fail(TB_ERR_UNSUPPORTED, "out_dim %lld is too large", (long long)out_dim);
  if (quantised ? (m > 0 && !x_scale) : x_scale != nullptr)
    return fail(TB_ERR_INVALID_ARGUMENT, "x_scale goes with an x in e4m3, and only with one");
  if (m == 0) return ok();
  if (!x || !wq || !w_scale || !y) return fail(TB_ERR_INVALID_ARGUMENT, "x, wq, w_scale and y must be non-NULL");
  if (!aligned16(x) || !aligned16(wq)) return fail(TB_ERR_UNSUPPORTED, "x and wq must be 16-byte aligned");
  if (!aligned_to(x_scale, scale_bytes(scale_type)) || !aligned_to(w_scale, scale_bytes(scale_type)) ||
      !aligned_to(y, esize(y_dtype)))
    return fail(TB_ERR_UNSUPPORTED, "scales and y must be aligned to their element size");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const Fp8Plan p = plan_fp8(m, out_dim, in_dim, quantised, y_dtype, scale_type, cus);
  if (p.bytes > 0) {
    if (!workspace) return fail(TB_ERR_INVALID_ARGUMENT, "workspace must be non-NULL");
    if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    if (workspace_bytes < p.bytes)
      return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, p.bytes);
  }
  hipError_t e = launch_fp8_product(p, x_dtype, y_dtype, scale_type, x, x_scale, wq, w_scale, y, m, out_dim, in_dim,
                                    static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the 8-bit product");
  return ok();
}

tb_status tb_head_norm_rotate(int32_t n, const tb_head_part* parts, int64_t tokens, int64_t head_dim, int64_t rot_dim,
                              int32_t interleaved, const int64_t* positions, const double* freqs, float eps,
                              float weight_offset, tb_dtype dtype, void* stream) {
  bool empty;
  tb_status st = check_heads(n, parts, tokens, head_dim, rot_dim, positions, freqs, eps, dtype, &empty);
  if (st != TB_OK) return st;
  if (empty) return ok();
  hipError_t e = launch_heads(dtype, n, parts, tokens, int(head_dim), int(rot_dim), interleaved != 0, positions, freqs,
                              eps, weight_offset, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the head norms");
  return ok();
}

tb_status tb_head_norm_rotate_axes(int32_t n, const tb_head_part* parts, int64_t tokens, int64_t head_dim,
                                   int64_t rot_dim, tb_pairs pairs, int32_t axes, const int64_t* positions,
                                   const uint8_t* pair_axis, const double* freqs, int32_t norm, float eps,
                                   float weight_offset, tb_dtype dtype, void* stream) {
  if (pairs != TB_PAIRS_HALF && pairs != TB_PAIRS_INTERLEAVED && pairs != TB_PAIRS_AXIS)
    return fail(TB_ERR_INVALID_ARGUMENT, "unknown layout of pairs %d", int(pairs));
  if (axes < 1 || axes > TB_MAX_AXES)
    return fail(TB_ERR_INVALID_ARGUMENT, "axes %d outside [1, %d]", axes, TB_MAX_AXES);
  if (rot_dim < 2) return fail(TB_ERR_INVALID_ARGUMENT, "rot_dim %lld < 2", (long long)rot_dim);
  bool empty;
  tb_status st = check_heads(n, parts, tokens, head_dim, rot_dim, positions, freqs, norm ? eps : 0.f, dtype, &empty);
  if (st != TB_OK) return st;
  if (!pair_axis) return fail(TB_ERR_INVALID_ARGUMENT, "pair_axis is NULL");
  unsigned seen = 0;   // axes whose pairs have begun
  for (int64_t p = 0; p < rot_dim / 2; ++p) {
    const int ax = pair_axis[p];
    if (ax >= axes) return fail(TB_ERR_INVALID_ARGUMENT, "pair %lld: axis %d of %d", (long long)p, ax, axes);
    if (pairs == TB_PAIRS_AXIS && (p == 0 || ax != pair_axis[p - 1]) && (seen >> ax & 1u))
      return fail(TB_ERR_INVALID_ARGUMENT, "pair %lld: the pairs of axis %d are not consecutive", (long long)p, ax);
    seen |= 1u << ax;
  }
  if (!norm)
    for (int j = 0; j < n; ++j)
      if (parts[j].weight) return fail(TB_ERR_INVALID_ARGUMENT, "part %d has a weight, but there is no norm", j);
  if (empty) return ok();
  hipError_t e = launch_heads_axes(dtype, n, parts, tokens, int(head_dim), int(rot_dim),
                                   HeadAxes{pairs, axes, pair_axis, norm != 0}, positions, freqs, eps, weight_offset,
                                   static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the head norms");
  return ok();
}

tb_status tb_quantize_rows_int8(const void* x, void* q, float* scale, int64_t m, int64_t in_dim, tb_dtype dtype,
                                void* stream) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  tb_status st = check_int8_dims(m, 1, in_dim, 8);
  if (st != TB_OK) return st;
  if (m == 0) return ok();
  if (!x || !q || !scale) return fail(TB_ERR_INVALID_ARGUMENT, "x, q and scale must be non-NULL");
  if (!aligned16(x) || !aligned_to(q, 8)) return fail(TB_ERR_UNSUPPORTED, "x must be 16-byte and q 8-byte aligned");
  if (!aligned_to(scale, 4)) return fail(TB_ERR_UNSUPPORTED, "scale must be aligned to its element size");
  hipError_t e = launch_int8_rows(dtype, x, q, scale, m, in_dim, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the row quantiser");
  return ok();
}

tb_status tb_dense_forward_int8_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype,
                                               tb_dtype y_dtype, size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(TB_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  if (!valid_dtype(x_dtype) && x_dtype != TB_INT8)
    return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(x_dtype));
  if (!valid_dtype(y_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(y_dtype));
  tb_status st = check_int8_dims(m, out_dim, in_dim, 16);
  if (st != TB_OK) return st;
  if (!fp8_decode_fits(m, out_dim)) return fail(TB_ERR_UNSUPPORTED, "out_dim %lld is too large", (long long)out_dim);
  *bytes_out = 0;
  if (m == 0) return ok();
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  *bytes_out = plan_int8(m, out_dim, in_dim, x_dtype, cus).bytes;
  return ok();
}

tb_status tb_dense_forward_int8(const void* x, const float* x_scale, const void* wq, const float* w_scale, void* y,
                                int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype, tb_dtype y_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const bool quantised = x_dtype == TB_INT8;
  if (!valid_dtype(x_dtype) && !quantised) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(x_dtype));
  if (!valid_dtype(y_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(y_dtype));
  tb_status st = check_int8_dims(m, out_dim, in_dim, 16);
  if (st != TB_OK) return st;
  if (!fp8_decode_fits(m, out_dim)) return fail(TB_ERR_UNSUPPORTED, "out_dim %lld is too large", (long long)out_dim);
  if (quantised ? (m > 0 && !x_scale) : x_scale != nullptr)
    return fail(TB_ERR_INVALID_ARGUMENT, "x_scale goes with an x in 8-bit integers, and only with one");
  if (m == 0) return ok();
  if (!x || !wq || !w_scale || !y) return fail(TB_ERR_INVALID_ARGUMENT, "x, wq, w_scale and y must be non-NULL");
  if (!aligned16(x) || !aligned16(wq)) return fail(TB_ERR_UNSUPPORTED, "x and wq must be 16-byte aligned");
  if (!aligned_to(x_scale, 4) || !aligned_to(w_scale, 4) || !aligned_to(y, esize(y_dtype)))
    return fail(TB_ERR_UNSUPPORTED, "scales and y must be aligned to their element size");
  int cus = 0;
  if (int e = device_cu_count(&cus)) return hip_fail(hipError_t(e), "querying the compute-unit count");
  const Int8Plan p = plan_int8(m, out_dim, in_dim, x_dtype, cus);
  if (p.bytes > 0) {
    if (!workspace) return fail(TB_ERR_INVALID_ARGUMENT, "workspace must be non-NULL");
    if (!aligned_to(workspace, 256)) return fail(TB_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    if (workspace_bytes < p.bytes)
      return fail(TB_ERR_INVALID_ARGUMENT, "workspace of %zu bytes is below the %zu needed", workspace_bytes, p.bytes);
  }
  hipError_t e = launch_int8_product(p, x_dtype, y_dtype, x, x_scale, wq, w_scale, y, m, out_dim, in_dim,
                                     static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the 8-bit integer product");
  return ok();
}

tb_status tb_residual_norm(const tb_residual* tensors, int64_t m, int64_t n, float residual_scale, float eps,
                           float weight_offset, int32_t post_norm, tb_dtype dtype, tb_dtype h_dtype, tb_dtype z_dtype,
                           tb_scale scale_type, void* stream) {
  if (!valid_dtype(dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(dtype));
  if (!valid_dtype(h_dtype)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown dtype %d", int(h_dtype));
  if (z_dtype != dtype && z_dtype != TB_INT8 && z_dtype != TB_E4M3)
    return fail(TB_ERR_INVALID_ARGUMENT, "z is in dtype or in 8 bits, not %d", int(z_dtype));
  if (!valid_scale(scale_type)) return fail(TB_ERR_INVALID_ARGUMENT, "unknown scale type %d", int(scale_type));
  if (!tensors) return fail(TB_ERR_INVALID_ARGUMENT, "tensors is NULL");
  if (m < 0 || n < 1)
    return fail(TB_ERR_INVALID_ARGUMENT, "need m >= 0 and n >= 1 (got %lld, %lld)", (long long)m, (long long)n);
  if (m > TB_FP8_MAX_TOKENS || n > TB_MAX_NORM_DIM)
    return fail(TB_ERR_UNSUPPORTED, "m exceeds %d or n %d", TB_FP8_MAX_TOKENS, TB_MAX_NORM_DIM);
  if (!(eps >= 0.f)) return fail(TB_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  const tb_residual& r = *tensors;
  const bool held = z_dtype != dtype;
  if (held && n % 8 != 0) return fail(TB_ERR_UNSUPPORTED, "an 8-bit z needs n %% 8 == 0, not %lld", (long long)n);
  if (m == 0) return ok();   // (the tensors may be NULL)
  if (!r.y && (r.gate || post_norm || residual_scale != 1.f))
    return fail(TB_ERR_INVALID_ARGUMENT, "a gate, post_norm and a residual scale go with a y");
  if (r.post_weight && !post_norm) return fail(TB_ERR_INVALID_ARGUMENT, "post_weight goes with post_norm");
  if (r.gate && r.gate_rows < 1) return fail(TB_ERR_INVALID_ARGUMENT, "gate_rows must be >= 1");
  if (r.gate && r.gate_channels != 0 && r.gate_channels != 1)
    return fail(TB_ERR_INVALID_ARGUMENT, "gate_channels is 0 or 1");
  if (!r.h) return fail(TB_ERR_INVALID_ARGUMENT, "h must be non-NULL");
  if (!r.y != !r.h_out) return fail(TB_ERR_INVALID_ARGUMENT, "y and h_out are given together or not at all");
  if (!r.z && (!r.y || r.z_scale || r.weight || held))
    return fail(TB_ERR_INVALID_ARGUMENT, r.y ? "weight and 8 bits go with a z" : "neither y nor z is given");
  if (r.z && held != (r.z_scale != nullptr)) return fail(TB_ERR_INVALID_ARGUMENT, "z_scale goes with an 8-bit z, and only with one");
  const size_t es = esize(dtype), hs = esize(h_dtype);
  const int64_t blocks = fp8_blocks(n), zes = held ? 1 : int64_t(es);
  const size_t ss = z_dtype == TB_INT8 ? 4 : scale_bytes(scale_type);
  struct Rows {
    const char* name;
    const void* p;
    int64_t stride, bytes, size;   // stride and row in bytes
  };
  if (m > 1) {
    const struct { const char* name; const void* p; int64_t s; } strides[4] = {
        {"h", r.h, r.h_stride}, {"y", r.y, r.y_stride}, {"h_out", r.h_out, r.h_out_stride},
        {"z", held ? nullptr : r.z, r.z_stride}};
    for (int j = 0; j < 4; ++j) {
      if (!strides[j].p) continue;
      if (strides[j].s < 0) return fail(TB_ERR_INVALID_ARGUMENT, "the stride of %s is negative", strides[j].name);
      if (strides[j].s > (int64_t(1) << 35)) return fail(TB_ERR_UNSUPPORTED, "the stride of %s exceeds 2^35", strides[j].name);
      if (j >= 2 && strides[j].s < n) return fail(TB_ERR_INVALID_ARGUMENT, "the rows of %s overlap", strides[j].name);
    }
  }
  if (r.gate && (m - 1) / r.gate_rows > 0) {
    if (r.gate_stride < 0) return fail(TB_ERR_INVALID_ARGUMENT, "the stride of gate is negative");
    if (r.gate_stride > (int64_t(1) << 35)) return fail(TB_ERR_UNSUPPORTED, "the stride of gate exceeds 2^35");
  }
  const int64_t step = m > 1;   // (the strides of a single row are not used)
  const Rows in[2] = {{"h", r.h, step * r.h_stride * int64_t(hs), n * int64_t(hs), int64_t(hs)},
                      {"y", r.y, step * r.y_stride * int64_t(es), n * int64_t(es), int64_t(es)}};
  const int64_t scales = z_dtype == TB_INT8 ? 4 : blocks * int64_t(ss);
  const Rows out[3] = {{"h_out", r.h_out, step * r.h_out_stride * int64_t(hs), n * int64_t(hs), int64_t(hs)},
                       {"z", r.z, held ? n : step * r.z_stride * int64_t(es), n * zes, zes},
                       {"z_scale", r.z ? r.z_scale : nullptr, scales, scales, int64_t(ss)}};
  for (const Rows& t : in)
    if (!aligned_to(t.p, size_t(t.size))) return fail(TB_ERR_UNSUPPORTED, "%s must be aligned to its element size", t.name);
  for (const Rows& t : out)
    if (!aligned_to(t.p, size_t(t.size))) return fail(TB_ERR_UNSUPPORTED, "%s must be aligned to its element size", t.name);
  const struct { const char* name; const void* p; int64_t bytes; bool whole; } small[3] = {
      {"post_weight", r.post_weight, n * int64_t(es), true}, {"weight", r.weight, n * int64_t(es), true},
      {"gate", r.gate, r.gate ? ((m - 1) / r.gate_rows * r.gate_stride + (r.gate_channels ? n : 1)) * int64_t(es) : 0,
       r.gate_channels == 1}};
  for (const auto& t : small)
    if (!aligned_to(t.p, es)) return fail(TB_ERR_UNSUPPORTED, "%s must be aligned to its element size", t.name);
  if (held && r.z) {
    bool fits = aligned16(r.h) && aligned16(r.y) && aligned16(r.h_out) && aligned16(r.z);
    for (const auto& t : small) fits = fits && (!t.whole || aligned16(t.p));
    if (m > 1) fits = fits && (r.h_stride * int64_t(hs)) % 16 == 0 && (!r.y || ((r.y_stride * int64_t(es)) % 16 == 0 && (r.h_out_stride * int64_t(hs)) % 16 == 0));
    if (r.gate && r.gate_channels && (m - 1) / r.gate_rows > 0) fits = fits && (r.gate_stride * int64_t(es)) % 16 == 0;
    if (!fits) return fail(TB_ERR_UNSUPPORTED, "an 8-bit z needs rows and weights that are 16-byte aligned");
  }
  for (int j = 0; j < 3; ++j) {
    const Rows& o = out[j];
    if (!o.p) continue;
    for (int k = 0; k < 2; ++k) {
      const Rows& i = in[k];
      if (!i.p) continue;
      const bool same = o.p == i.p && (m == 1 || o.stride == i.stride) && o.size == i.size;
      if (same && j == k && !(j == 1 && held)) continue;   // h_out is h, z is y: element for element
      if (rows_share(o.p, o.bytes, o.stride, i.p, i.bytes, i.stride, m))
        return fail(TB_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, i.name);
    }
    for (int k = 0; k < j; ++k)
      if (out[k].p && rows_share(o.p, o.bytes, o.stride, out[k].p, out[k].bytes, out[k].stride, m))
        return fail(TB_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, out[k].name);
    for (const auto& t : small)
      if (t.p && rows_share(o.p, (m - 1) * o.stride + o.bytes, 0, t.p, t.bytes, 0, 1))
        return fail(TB_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, t.name);
  }
  hipError_t e = launch_residual_norm(r, m, n, residual_scale, eps, weight_offset, post_norm != 0, dtype, h_dtype,
                                      z_dtype, scale_type, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "launching the residual norm");
  return ok();
}

}  // extern "C"
