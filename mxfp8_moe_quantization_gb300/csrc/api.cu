// C-ABI entry points of libfp8moe: argument checks on the host, then launches
// on the caller's stream.  See include/fp8moe.h for the contract of each call.
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "gemm.h"
#include "launch.h"
#include "moe_ops.h"

// Sticky device status word (static device memory: the library allocates
// nothing).  Kernels receive its address; fp8moe_get_device_status takes it
// (reads and clears it in one atomic exchange) into the take slot.
static __device__ int g_fp8moe_status;
static __device__ int g_fp8moe_status_take;

static __global__ void k_take_status(int* status, int* take) { *take = atomicExch(status, 0); }

namespace {

struct DevInfo {
  bool init = false;
  int* status = nullptr;
  int* take = nullptr;
  int num_sms = 0;
  int max_smem = 0;
};

constexpr int kMaxDevices = 128;
DevInfo g_dev[kMaxDevices];
std::mutex g_mu;
std::mutex g_take_mu;

fp8moe_status device_info(DevInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FP8MOE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[dev];
  if (!d.init) {
    if (cudaGetSymbolAddress((void**)&d.status, g_fp8moe_status) != cudaSuccess) return FP8MOE_ERR_CUDA;
    if (cudaGetSymbolAddress((void**)&d.take, g_fp8moe_status_take) != cudaSuccess) return FP8MOE_ERR_CUDA;
    if (cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FP8MOE_ERR_CUDA;
    if (cudaDeviceGetAttribute(&d.max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
      return FP8MOE_ERR_CUDA;
    d.init = true;
  }
  *out = &d;
  return FP8MOE_OK;
}

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline fp8moe_status cuda_result(cudaError_t e) { return e == cudaSuccess ? FP8MOE_OK : FP8MOE_ERR_CUDA; }

inline bool valid_kind(int kind) { return kind == FP8MOE_E4M3FN || kind == FP8MOE_E4M3FNUZ; }

}  // namespace

extern "C" {

const char* fp8moe_status_string(int s) {
  switch (s) {
    case FP8MOE_OK: return "ok";
    case FP8MOE_ERR_INVALID_ARG: return "invalid argument";
    case FP8MOE_ERR_ALIGNMENT: return "misaligned pointer or size";
    case FP8MOE_ERR_UNSUPPORTED: return "unsupported combination";
    case FP8MOE_ERR_CUDA: return "CUDA error";
    case FP8MOE_ERR_DEVICE_OFFSETS: return "invalid routing offsets (device)";
    case FP8MOE_ERR_TIMEOUT: return "device pipeline wait timed out";
    case FP8MOE_ERR_SCRATCH_LIMIT: return "problem needs more scratch than the library's static array holds";
    case FP8MOE_ERR_CONCURRENT: return "launches in flight at once shared a device work counter";
    default: return "unknown status";
  }
}

int fp8moe_version(void) { return (1 << 16) | 0; }

int64_t fp8moe_jagged_t_cols(int64_t M, int64_t E) { return (M + 31 * E + 15) / 16 * 16; }

fp8moe_status fp8moe_quantize_rowwise(const void* x, int64_t R, int64_t C, int64_t ldx, int kind, void* q,
                                      float* scale_inv, fp8moe_stream_t stream) {
  if (R < 0 || C < 0 || ldx < C || !valid_kind(kind)) return FP8MOE_ERR_INVALID_ARG;
  if (R == 0 || C == 0) return FP8MOE_OK;
  if (!x || !q || !scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(q) || C % 16 || ldx % 8 || ((uintptr_t)scale_inv & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (C > (int64_t)1 << 30) return FP8MOE_ERR_INVALID_ARG;
  return cuda_result(fp8moe::launch_quant_rowwise(x, R, C, ldx, kind, q, scale_inv, (cudaStream_t)stream));
}

fp8moe_status fp8moe_quantize_colwise_3d(const void* x, int64_t E, int64_t R, int64_t C, const int32_t* offs,
                                         int transpose_out, int kind, void* q, float* scale_inv,
                                         fp8moe_stream_t stream) {
  if (E < 0 || R < 0 || C < 0 || !valid_kind(kind)) return FP8MOE_ERR_INVALID_ARG;
  if (offs && E == 0) return FP8MOE_ERR_INVALID_ARG;
  if (offs && E > FP8MOE_MAX_GROUPS) return FP8MOE_ERR_INVALID_ARG;
  if (E == 0 || C == 0) return FP8MOE_OK;
  if (!x || !q || !scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(q) || C % 16 || ((uintptr_t)scale_inv & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (!offs && transpose_out && R % 16) return FP8MOE_ERR_ALIGNMENT;
  if (offs && ((uintptr_t)offs & 3)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  const int64_t ldt = offs ? fp8moe_jagged_t_cols(R, E) : 0;
  return cuda_result(fp8moe::launch_colwise(x, E, R, C, offs, transpose_out, kind, ldt, q, scale_inv, d->status,
                                            d->num_sms, (cudaStream_t)stream));
}

fp8moe_status fp8moe_mxfp8_quantize_dim0(const void* x, int64_t B, int64_t R, int64_t C, void* q, uint8_t* scale,
                                         fp8moe_stream_t stream) {
  if (B < 0 || R < 0 || C < 0) return FP8MOE_ERR_INVALID_ARG;
  if (C % 32) return FP8MOE_ERR_ALIGNMENT;
  if (B == 0 || R == 0 || C == 0) return FP8MOE_OK;
  if (!x || !q || !scale) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(q)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_mx_dim0(x, B, R, C, q, scale, FP8MOE_SCALES_ROWMAJOR, nullptr, 0, d->num_sms,
                                            d->status, (cudaStream_t)stream));
}

fp8moe_status fp8moe_mxfp8_quantize_dim1(const void* x, int64_t B, int64_t R, int64_t C, void* qt,
                                         uint8_t* scale, fp8moe_stream_t stream) {
  if (B < 0 || R < 0 || C < 0) return FP8MOE_ERR_INVALID_ARG;
  if (R % 32 || C % 16) return FP8MOE_ERR_ALIGNMENT;
  if (B == 0 || R == 0 || C == 0) return FP8MOE_OK;
  if (!x || !qt || !scale) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(qt)) return FP8MOE_ERR_ALIGNMENT;
  if (C > ((int64_t)1 << 31) || R > ((int64_t)1 << 31) || B > 65535) return FP8MOE_ERR_INVALID_ARG;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_mx_dual(x, B, R, C, nullptr, nullptr, FP8MOE_SCALES_ROWMAJOR, qt, scale,
                                            FP8MOE_SCALES_ROWMAJOR, nullptr, 0, d->num_sms, d->status,
                                            (cudaStream_t)stream));
}

fp8moe_status fp8moe_mxfp8_quantize_dual(const void* x, int64_t B, int64_t R, int64_t C, const int32_t* offs,
                                         int64_t E, void* q0, uint8_t* s0, int s0_layout, void* q1, uint8_t* s1,
                                         int s1_layout, fp8moe_stream_t stream) {
  if (B < 0 || R < 0 || C < 0 || E < 0) return FP8MOE_ERR_INVALID_ARG;
  if (!q0 && !q1) return FP8MOE_ERR_INVALID_ARG;
  if (C % 32 || (q1 && R % 32)) return FP8MOE_ERR_ALIGNMENT;
  if ((q0 && !s0) || (q1 && !s1)) return FP8MOE_ERR_INVALID_ARG;
  const bool ok0 = !q0 || s0_layout == FP8MOE_SCALES_ROWMAJOR || s0_layout == FP8MOE_NO_GROUPS ||
                   s0_layout == FP8MOE_GROUP_ROWS;
  const bool ok1 = !q1 || s1_layout == FP8MOE_SCALES_ROWMAJOR || s1_layout == FP8MOE_NO_GROUPS ||
                   s1_layout == FP8MOE_GROUP_COLS;
  if (!ok0 || !ok1) return FP8MOE_ERR_INVALID_ARG;
  const bool grouped = (q0 && s0_layout == FP8MOE_GROUP_ROWS) || (q1 && s1_layout == FP8MOE_GROUP_COLS);
  if (grouped && (B != 1 || E < 1 || E > 1024 || !offs)) return FP8MOE_ERR_INVALID_ARG;
  if (grouped && ((uintptr_t)offs & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (B == 0 || R == 0 || C == 0) return FP8MOE_OK;
  if (!x || !al16(x) || (q0 && !al16(q0)) || (q1 && !al16(q1))) return x ? FP8MOE_ERR_ALIGNMENT : FP8MOE_ERR_INVALID_ARG;
  if (B > 65535 || R > ((int64_t)1 << 31) || C > ((int64_t)1 << 31)) return FP8MOE_ERR_INVALID_ARG;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  // both directions: one fused launch reading x once (4 bytes moved per
  // element instead of 6); dim1 alone: the same kernel without dim0; dim0
  // alone: its own kernel.  Scales go straight to their final layout.
  const int64_t Eg = grouped ? E : 0;
  cudaError_t e = cudaSuccess;
  if (q1) {
    e = fp8moe::launch_mx_dual(x, B, R, C, q0, s0, q0 ? s0_layout : FP8MOE_SCALES_ROWMAJOR, q1, s1, s1_layout, offs,
                               Eg, d->num_sms, d->status, (cudaStream_t)stream);
  } else {
    e = fp8moe::launch_mx_dim0(x, B, R, C, q0, s0, s0_layout, offs, Eg, d->num_sms, d->status,
                               (cudaStream_t)stream);
  }
  return e == cudaSuccess ? FP8MOE_OK : FP8MOE_ERR_CUDA;
}

int64_t fp8moe_swizzled_scales_bytes(int64_t B, int64_t R, int64_t Cs, int64_t E, int group_axis) {
  if (B < 0 || R < 0 || Cs < 0 || E < 0) return -1;
  if (group_axis != FP8MOE_NO_GROUPS && group_axis != FP8MOE_GROUP_ROWS && group_axis != FP8MOE_GROUP_COLS)
    return -1;
  const fp8moe::SwizzleGeom g = fp8moe::swizzle_geom(R, Cs, group_axis == FP8MOE_NO_GROUPS ? 0 : E, group_axis);
  return B * g.Rp * g.Cp;
}

fp8moe_status fp8moe_swizzle_scales_128x4(const uint8_t* s, int64_t B, int64_t R, int64_t Cs, const int32_t* offs,
                                          int64_t E, int group_axis, uint8_t* out, fp8moe_stream_t stream) {
  if (B < 0 || R < 0 || Cs < 0 || E < 0) return FP8MOE_ERR_INVALID_ARG;
  if (group_axis != FP8MOE_NO_GROUPS && group_axis != FP8MOE_GROUP_ROWS && group_axis != FP8MOE_GROUP_COLS)
    return FP8MOE_ERR_INVALID_ARG;
  if (group_axis != FP8MOE_NO_GROUPS) {
    if (B != 1 || E < 1 || E > 1024 || !offs) return FP8MOE_ERR_INVALID_ARG;
    if ((uintptr_t)offs & 3) return FP8MOE_ERR_ALIGNMENT;
  }
  if (fp8moe_swizzled_scales_bytes(B, R, Cs, E, group_axis) == 0) return FP8MOE_OK;
  if (!out || (!s && R * Cs > 0)) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(out)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_swizzle(s, B, R, Cs, offs, E, group_axis, out, d->status, d->num_sms,
                                            (cudaStream_t)stream));
}

fp8moe_status fp8moe_quantize_tensorwise(const void* x, int64_t E, int64_t R, int64_t C, const int32_t* offs,
                                         int transpose_out, int kind, void* q, float* scale_inv,
                                         fp8moe_stream_t stream) {
  if (E < 0 || R < 0 || C < 0 || !valid_kind(kind)) return FP8MOE_ERR_INVALID_ARG;
  if (offs && E == 0) return FP8MOE_ERR_INVALID_ARG;
  if (offs && transpose_out && E > FP8MOE_MAX_GROUPS) return FP8MOE_ERR_INVALID_ARG;
  if (!scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if ((uintptr_t)scale_inv & 3) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  if (E == 0 || C == 0 || (R == 0 && !(offs && transpose_out))) {
    // nothing to cast (the jagged transposed layout still gets its zero
    // padding below); the scale is that of an all-zero tensor
    return cuda_result(fp8moe::launch_tensorwise(nullptr, 0, 0, 0, nullptr, 0, kind, nullptr, scale_inv,
                                                 d->num_sms, d->status, (cudaStream_t)stream));
  }
  if (!q || (!x && R > 0)) return FP8MOE_ERR_INVALID_ARG;
  if ((x && !al16(x)) || !al16(q)) return FP8MOE_ERR_ALIGNMENT;
  if (transpose_out && (C % 16 || (!offs && R % 16))) return FP8MOE_ERR_ALIGNMENT;
  if (offs && ((uintptr_t)offs & 3)) return FP8MOE_ERR_ALIGNMENT;
  return cuda_result(fp8moe::launch_tensorwise(x, E, R, C, offs, transpose_out, kind, q, scale_inv, d->num_sms,
                                               d->status, (cudaStream_t)stream));
}

fp8moe_status fp8moe_quantize_blockwise_rows(const void* x, int64_t R, int64_t C, int kind, void* q,
                                             float* scale_inv, fp8moe_stream_t stream) {
  if (R < 0 || C < 0 || !valid_kind(kind)) return FP8MOE_ERR_INVALID_ARG;
  if (C % 128) return FP8MOE_ERR_ALIGNMENT;
  if (R == 0 || C == 0) return FP8MOE_OK;
  if (!x || !q || !scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(q) || ((uintptr_t)scale_inv & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (R > ((int64_t)1 << 35)) return FP8MOE_ERR_INVALID_ARG;
  return cuda_result(fp8moe::launch_bw_rows(x, R, C, kind, q, scale_inv, (cudaStream_t)stream));
}

fp8moe_status fp8moe_quantize_blockwise_weight(const void* w, int64_t E, int64_t N, int64_t K, int kind, void* q,
                                               void* qt, float* scale_inv, fp8moe_stream_t stream) {
  if (E < 0 || N < 0 || K < 0 || !valid_kind(kind) || (!q && !qt)) return FP8MOE_ERR_INVALID_ARG;
  if (N % 128 || K % 128) return FP8MOE_ERR_ALIGNMENT;
  if (E == 0 || N == 0 || K == 0) return FP8MOE_OK;
  if (!w || !scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(w) || (q && !al16(q)) || (qt && !al16(qt)) || ((uintptr_t)scale_inv & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (E * (N / 128) * (K / 128) >= ((int64_t)1 << 31)) return FP8MOE_ERR_INVALID_ARG;
  return cuda_result(fp8moe::launch_bw_weight(w, E, N, K, kind, q, qt, scale_inv, (cudaStream_t)stream));
}

int64_t fp8moe_blockwise_token_blocks(int64_t M, int64_t E) {
  if (M < 0 || E < 1) return -1;
  return (M + 127) / 128 + E;
}

fp8moe_status fp8moe_quantize_blockwise_tokens(const void* x, int64_t M, int64_t C, const int32_t* offs, int64_t E,
                                               int kind, void* qt, float* scale_inv, fp8moe_stream_t stream) {
  if (M < 0 || C < 0 || E < 1 || E > FP8MOE_MAX_GROUPS || !valid_kind(kind) || !offs) return FP8MOE_ERR_INVALID_ARG;
  if (M % 32 || C % 16) return FP8MOE_ERR_ALIGNMENT;
  if (((uintptr_t)offs & 3)) return FP8MOE_ERR_ALIGNMENT;
  if (M == 0 || C == 0) return FP8MOE_OK;
  if (!x || !qt || !scale_inv) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(qt) || !al16(scale_inv)) return FP8MOE_ERR_ALIGNMENT;
  if (fp8moe_blockwise_token_blocks(M, E) * ((C + 127) / 128) >= ((int64_t)1 << 31)) return FP8MOE_ERR_INVALID_ARG;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_bw_tokens(x, M, C, offs, E, kind, qt, scale_inv, d->num_sms, d->status,
                                              (cudaStream_t)stream));
}

static fp8moe_status grouped_mm(int mode, int recipe, const void* a, const void* a_scale, const void* b,
                                const void* b_scale, const int32_t* offs, int64_t E, int64_t M, int64_t N,
                                int64_t K, void* out, fp8moe_stream_t stream) {
  if (recipe != FP8MOE_ROWWISE && recipe != FP8MOE_MXFP8 && recipe != FP8MOE_TENSORWISE &&
      recipe != FP8MOE_BLOCKWISE)
    return FP8MOE_ERR_INVALID_ARG;
  if (E < 1 || M < 0 || N < 0 || K < 0 || E > 4096) return FP8MOE_ERR_INVALID_ARG;
  if (!offs || ((uintptr_t)offs & 3)) return FP8MOE_ERR_INVALID_ARG;
  if (N % 16 || K % 16) return FP8MOE_ERR_ALIGNMENT;
  if (recipe == FP8MOE_MXFP8) {
    // the contracting dimension must hold whole 32-element scale blocks
    if (mode == fp8moe::GEMM_FWD && K % 32) return FP8MOE_ERR_ALIGNMENT;
    if (mode == fp8moe::GEMM_DGRAD && N % 32) return FP8MOE_ERR_ALIGNMENT;
    if (mode == fp8moe::GEMM_WGRAD && M % 32) return FP8MOE_ERR_ALIGNMENT;
  }
  if (recipe == FP8MOE_BLOCKWISE) {
    // weight tiles are 128 x 128; wgrad's token tiles are cut at 32-multiple
    // group boundaries
    if (N % 128 || K % 128 || (mode == fp8moe::GEMM_WGRAD && M % 32)) return FP8MOE_ERR_ALIGNMENT;
  }
  if (!a || !b || !out || !a_scale || !b_scale) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(a) || !al16(b) || !al16(out)) return FP8MOE_ERR_ALIGNMENT;
  if (recipe == FP8MOE_TENSORWISE || (recipe == FP8MOE_BLOCKWISE && mode != fp8moe::GEMM_WGRAD)
          ? (((uintptr_t)a_scale | (uintptr_t)b_scale) & 3)
          : (!al16(a_scale) || !al16(b_scale)))
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  fp8moe::GemmArgs g{};
  g.recipe = recipe;
  g.mode = mode;
  g.E = (int)E;
  g.offs = offs;
  g.out = (uint16_t*)out;
  g.status = d->status;
  g.num_sms = d->num_sms;
  g.max_smem = d->max_smem;
  g.M = M;
  g.a = (const uint8_t*)a;
  g.b = (const uint8_t*)b;
  g.a_scale = a_scale;
  g.b_scale = b_scale;
  if (mode == fp8moe::GEMM_FWD) {          // [M,K] x [E,N,K] -> [M,N]
    g.rows = M, g.cols = N, g.kk = K;
  } else if (mode == fp8moe::GEMM_DGRAD) { // [M,N] x [E,K,N] -> [M,K]
    g.rows = M, g.cols = K, g.kk = N;
  } else {                                 // [N,Mt] x [K,Mt] -> [E,N,K]
    g.rows = N, g.cols = K;
    g.kk = recipe == FP8MOE_MXFP8 || recipe == FP8MOE_BLOCKWISE ? M : fp8moe_jagged_t_cols(M, E);
  }
  if (g.rows == 0 || g.cols == 0) return FP8MOE_OK;
  if (g.kk == 0) {
    // nothing to contract (e.g. wgrad of a batch without routed tokens):
    // every output element is an empty sum
    const int64_t n = (mode == fp8moe::GEMM_WGRAD ? E : 1) * g.rows * g.cols;
    return cuda_result(cudaMemsetAsync(out, 0, (size_t)n * 2, (cudaStream_t)stream));
  }
  cudaError_t e = recipe == FP8MOE_BLOCKWISE ? fp8moe::launch_blockwise_mm(g, (cudaStream_t)stream)
                                             : fp8moe::launch_grouped_mm(g, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8MOE_ERR_UNSUPPORTED;
  return cuda_result(e);
}

fp8moe_status fp8moe_scaled_grouped_mm_fwd(int recipe, const void* a, const void* a_scale, const void* w,
                                           const void* w_scale, const int32_t* offs, int64_t E, int64_t M,
                                           int64_t N, int64_t K, void* out, fp8moe_stream_t stream) {
  return grouped_mm(fp8moe::GEMM_FWD, recipe, a, a_scale, w, w_scale, offs, E, M, N, K, out, stream);
}

fp8moe_status fp8moe_scaled_grouped_mm_dgrad(int recipe, const void* dy, const void* dy_scale, const void* wt,
                                             const void* wt_scale, const int32_t* offs, int64_t E, int64_t M,
                                             int64_t N, int64_t K, void* out, fp8moe_stream_t stream) {
  return grouped_mm(fp8moe::GEMM_DGRAD, recipe, dy, dy_scale, wt, wt_scale, offs, E, M, N, K, out, stream);
}

fp8moe_status fp8moe_scaled_grouped_mm_wgrad(int recipe, const void* dyt, const void* dyt_scale, const void* at,
                                             const void* at_scale, const int32_t* offs, int64_t E, int64_t M,
                                             int64_t N, int64_t K, void* out, fp8moe_stream_t stream) {
  return grouped_mm(fp8moe::GEMM_WGRAD, recipe, dyt, dyt_scale, at, at_scale, offs, E, M, N, K, out, stream);
}

static fp8moe_status grouped_mm_quant_a(int mode, const void* a_bf16, const void* b, const void* b_scale,
                                        const int32_t* offs, int64_t E, int64_t M, int64_t N, int64_t K, void* out,
                                        void* a_q, uint8_t* a_s, fp8moe_stream_t stream) {
  if (E < 1 || E > FP8MOE_MAX_GROUPS || M < 0 || N < 0 || K < 0) return FP8MOE_ERR_INVALID_ARG;
  if (!offs || ((uintptr_t)offs & 3)) return FP8MOE_ERR_INVALID_ARG;
  if ((a_q == nullptr) != (a_s == nullptr)) return FP8MOE_ERR_INVALID_ARG;
  const int64_t kk = mode == fp8moe::GEMM_FWD ? K : N;      // the contracting dimension
  const int64_t cols = mode == fp8moe::GEMM_FWD ? N : K;
  if (N % 16 || K % 16 || kk % 32) return FP8MOE_ERR_ALIGNMENT;
  if (!a_bf16 || !b || !b_scale || !out) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(a_bf16) || !al16(b) || !al16(b_scale) || !al16(out) || (a_q && !al16(a_q))) return FP8MOE_ERR_ALIGNMENT;
  if (M == 0 || cols == 0) return FP8MOE_OK;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  fp8moe::GemmArgs g{};
  g.recipe = FP8MOE_MXFP8;
  g.mode = mode;
  g.E = (int)E;
  g.offs = offs;
  g.out = (uint16_t*)out;
  g.status = d->status;
  g.num_sms = d->num_sms;
  g.max_smem = d->max_smem;
  g.M = M;
  g.a = (const uint8_t*)a_bf16;
  g.b = (const uint8_t*)b;
  g.a_scale = nullptr;
  g.b_scale = b_scale;
  g.rows = M, g.cols = cols, g.kk = kk;
  g.quant_a = 1;
  g.qa_out = (uint8_t*)a_q;
  g.sa_out = a_s;
  cudaError_t e = fp8moe::launch_grouped_mm(g, (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return FP8MOE_ERR_UNSUPPORTED;
  return cuda_result(e);
}

fp8moe_status fp8moe_mxfp8_grouped_mm_fwd_quant_a(const void* a, const void* w, const void* w_scale,
                                                  const int32_t* offs, int64_t E, int64_t M, int64_t N, int64_t K,
                                                  void* out, void* a_q, uint8_t* a_s, fp8moe_stream_t stream) {
  return grouped_mm_quant_a(fp8moe::GEMM_FWD, a, w, w_scale, offs, E, M, N, K, out, a_q, a_s, stream);
}

fp8moe_status fp8moe_mxfp8_grouped_mm_dgrad_quant_a(const void* dy, const void* wt, const void* wt_scale,
                                                    const int32_t* offs, int64_t E, int64_t M, int64_t N, int64_t K,
                                                    void* out, void* dy_q, uint8_t* dy_s, fp8moe_stream_t stream) {
  return grouped_mm_quant_a(fp8moe::GEMM_DGRAD, dy, wt, wt_scale, offs, E, M, N, K, out, dy_q, dy_s, stream);
}

int64_t fp8moe_route_rows(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1) return -1;
  return (T * k + 31 * E + 31) / 32 * 32;
}

int64_t fp8moe_route_workspace_bytes(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1) return -1;
  return fp8moe::route_workspace_bytes(T, k, E);
}

fp8moe_status fp8moe_route_permute(const void* x, int64_t T, int64_t H, const int32_t* topk_idx,
                                   const float* topk_w, int64_t k, int64_t E, void* a, int32_t* offs,
                                   int32_t* row_of, void* workspace, int64_t workspace_bytes,
                                   fp8moe_stream_t stream) {
  if (T < 0 || H < 0 || k < 1 || E < 1 || E > 1024) return FP8MOE_ERR_INVALID_ARG;
  if (T * k > ((int64_t)1 << 30)) return FP8MOE_ERR_INVALID_ARG;
  if (!a || !offs || !workspace || (T > 0 && (!x || !topk_idx || !row_of))) return FP8MOE_ERR_INVALID_ARG;
  if (workspace_bytes < fp8moe::route_workspace_bytes(T, k, E)) return FP8MOE_ERR_INVALID_ARG;
  if (H % 8 || (x && !al16(x)) || !al16(a)) return FP8MOE_ERR_ALIGNMENT;
  if (((uintptr_t)topk_idx | (uintptr_t)offs | (uintptr_t)row_of | (uintptr_t)topk_w | (uintptr_t)workspace) & 3)
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_route_permute(x, T, H, topk_idx, topk_w, k, E, fp8moe_route_rows(T, k, E), a,
                                                  offs, row_of, workspace, d->num_sms, d->status,
                                                  (cudaStream_t)stream));
}

fp8moe_status fp8moe_route_permute_noalloc(const void* x, int64_t T, int64_t H, const int32_t* topk_idx,
                                           const float* topk_w, int64_t k, int64_t E, void* a, int32_t* offs,
                                           int32_t* row_of, fp8moe_stream_t stream) {
  if (T < 0 || H < 0 || k < 1 || E < 1 || E > 1024) return FP8MOE_ERR_INVALID_ARG;
  if (T * k > ((int64_t)1 << 30)) return FP8MOE_ERR_INVALID_ARG;
  // the scratch this problem needs must fit the library's static array
  if (fp8moe::route_workspace_bytes(T, k, E) > fp8moe::route_static_scratch_bytes()) return FP8MOE_ERR_SCRATCH_LIMIT;
  if (!a || !offs || (T > 0 && (!x || !topk_idx || !row_of))) return FP8MOE_ERR_INVALID_ARG;
  if (H % 8 || (x && !al16(x)) || !al16(a)) return FP8MOE_ERR_ALIGNMENT;
  if (((uintptr_t)topk_idx | (uintptr_t)offs | (uintptr_t)row_of | (uintptr_t)topk_w) & 3)
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  void* scratch = nullptr;
  if (fp8moe::route_static_scratch(&scratch) != cudaSuccess) return FP8MOE_ERR_CUDA;
  return cuda_result(fp8moe::launch_route_permute(x, T, H, topk_idx, topk_w, k, E, fp8moe_route_rows(T, k, E), a,
                                                  offs, row_of, scratch, d->num_sms, d->status,
                                                  (cudaStream_t)stream));
}

fp8moe_status fp8moe_route_unpermute(const void* y, int64_t T, int64_t N, const int32_t* row_of,
                                     const float* topk_w, int64_t k, void* out, fp8moe_stream_t stream) {
  if (T < 0 || N < 0 || k < 1) return FP8MOE_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return FP8MOE_OK;
  if (!y || !row_of || !out) return FP8MOE_ERR_INVALID_ARG;
  if (N % 8 || !al16(y) || !al16(out) || (((uintptr_t)row_of | (uintptr_t)topk_w) & 3)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_route_unpermute(y, N, row_of, topk_w, T, k, out, (cudaStream_t)stream));
}

fp8moe_status fp8moe_add_rmsnorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* w,
                                     int weight_type, int64_t T, int64_t H, float eps, void* h, void* y, float* rstd,
                                     int recipe, int kind, void* q, void* scale, int scale_layout,
                                     fp8moe_stream_t stream) {
  if (T < 0 || H < 1 || T > INT32_MAX - 128 || H > ((int64_t)1 << 20) || ldx < H || (residual && ldr < H))
    return FP8MOE_ERR_INVALID_ARG;
  if ((weight_type != FP8MOE_BF16 && weight_type != FP8MOE_FP32) || !(eps >= 0.0f) || std::isinf(eps))
    return FP8MOE_ERR_INVALID_ARG;
  if (H % 8 || ldx % 8 || (residual && ldr % 8)) return FP8MOE_ERR_ALIGNMENT;
  if (T == 0) return FP8MOE_OK;
  if ((q == nullptr) != (scale == nullptr) || (h && !residual) || !(h || y || rstd || q)) return FP8MOE_ERR_INVALID_ARG;
  const bool mx = q && recipe == FP8MOE_MXFP8;
  if (q) {
    if (!valid_kind(kind)) return FP8MOE_ERR_INVALID_ARG;
    if (recipe != FP8MOE_MXFP8 && recipe != FP8MOE_ROWWISE) return FP8MOE_ERR_UNSUPPORTED;
    if (mx && kind != FP8MOE_E4M3FN) return FP8MOE_ERR_UNSUPPORTED;
    if (mx && scale_layout != FP8MOE_SCALES_ROWMAJOR && scale_layout != FP8MOE_NO_GROUPS)
      return FP8MOE_ERR_INVALID_ARG;
    if (H % (mx ? 32 : 16)) return FP8MOE_ERR_ALIGNMENT;
  }
  if (!x || !w) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(residual) || !al16(w) || !al16(h) || !al16(y) || !al16(q) || ((uintptr_t)rstd & 3) ||
      (q && !mx && ((uintptr_t)scale & 3)))
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_norm_fwd(x, ldx, residual, ldr, w, weight_type == FP8MOE_FP32, T, H, eps, h, y,
                                             rstd, recipe, kind, q, scale, scale_layout, d->num_sms,
                                             (cudaStream_t)stream));
}

int64_t fp8moe_add_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || H < 1) return -1;
  return (T < fp8moe::NORM_BWD_PARTS ? T : fp8moe::NORM_BWD_PARTS) * H * (int64_t)sizeof(float);
}

// h: bf16, or MXFP8 codes with their scales hs
static fp8moe_status rmsnorm_bwd(const void* dy, const void* h, const uint8_t* hs, const float* rstd, const void* w,
                                 int weight_type, const void* dh, int64_t T, int64_t H, void* dx, float* dw,
                                 void* workspace, int64_t workspace_bytes, fp8moe_stream_t stream) {
  if (T < 0 || H < 1 || T > INT32_MAX - 128 || H > ((int64_t)1 << 20)) return FP8MOE_ERR_INVALID_ARG;
  if (weight_type != FP8MOE_BF16 && weight_type != FP8MOE_FP32) return FP8MOE_ERR_INVALID_ARG;
  if (H % 8) return FP8MOE_ERR_ALIGNMENT;
  if (!dw || (T > 0 && (!dy || !h || !rstd || !w || !dx || !workspace))) return FP8MOE_ERR_INVALID_ARG;
  if (workspace_bytes < fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H)) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(h) || !al16(w) || !al16(dh) || !al16(dx) || !al16(workspace) ||
      (((uintptr_t)rstd | (uintptr_t)dw) & 3))
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  return cuda_result(fp8moe::launch_norm_bwd(dy, h, hs, rstd, w, weight_type == FP8MOE_FP32, dh, T, H, dx, dw, workspace,
                                             d->num_sms, d->max_smem, d->status, (cudaStream_t)stream));
}

fp8moe_status fp8moe_add_rmsnorm_bwd(const void* dy, const void* h, const float* rstd, const void* w,
                                     int weight_type, const void* dh, int64_t T, int64_t H, void* dx, float* dw,
                                     void* workspace, int64_t workspace_bytes, fp8moe_stream_t stream) {
  return rmsnorm_bwd(dy, h, nullptr, rstd, w, weight_type, dh, T, H, dx, dw, workspace, workspace_bytes, stream);
}

fp8moe_status fp8moe_add_rmsnorm_bwd_ckpt(const void* dy, const void* hq, const uint8_t* hs, const float* rstd,
                                          const void* w, int weight_type, const void* dh, int64_t T, int64_t H, void* dx,
                                          float* dw, void* workspace, int64_t workspace_bytes, fp8moe_stream_t stream) {
  if (H > 0 && H % 32) return FP8MOE_ERR_ALIGNMENT;
  if (T > 0 && !hs) return FP8MOE_ERR_INVALID_ARG;
  return rmsnorm_bwd(dy, hq, hs, rstd, w, weight_type, dh, T, H, dx, dw, workspace, workspace_bytes, stream);
}

int64_t fp8moe_router_workspace_bytes(int64_t T, int64_t E) {
  if (T < 0 || E < 1) return -1;
  return (T < fp8moe::ROUTER_MAX_PARTS ? T : fp8moe::ROUTER_MAX_PARTS) * (2 * E + 1) * (int64_t)sizeof(float);
}

// rows of logits that accesses of four experts reach
static bool router_wide(const void* p, int type, int64_t E, int64_t ld) {
  return E % 4 == 0 && ld % 4 == 0 && (uintptr_t)p % (type == FP8MOE_BF16 ? 8 : 16) == 0;
}

// the checks that both directions share
static fp8moe_status router_check(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ldl, int64_t k,
                                  int score) {
  if (T < 0 || E < 1 || E > fp8moe::ROUTER_MAX_E || ldl < E || k < 1 || k > E || k > fp8moe::ROUTER_MAX_K ||
      T > ((int64_t)1 << 30) / k)
    return FP8MOE_ERR_INVALID_ARG;
  if (logits_type != FP8MOE_BF16 && logits_type != FP8MOE_FP32) return FP8MOE_ERR_INVALID_ARG;
  if (score != FP8MOE_SCORE_SOFTMAX && score != FP8MOE_SCORE_SIGMOID) return FP8MOE_ERR_INVALID_ARG;
  if (T > 0 && !logits) return FP8MOE_ERR_INVALID_ARG;
  if ((uintptr_t)logits & (logits_type == FP8MOE_FP32 ? 3 : 1)) return FP8MOE_ERR_ALIGNMENT;
  return FP8MOE_OK;
}

fp8moe_status fp8moe_router_fwd(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ldl, int64_t k,
                                int score, int renormalize, float route_scale, const float* bias,
                                const uint8_t* token_mask, int32_t* topk_idx, float* topk_w, int32_t* counts,
                                float* prob_sum, float* balance_loss, void* workspace, int64_t workspace_bytes,
                                fp8moe_stream_t stream) {
  fp8moe_status st = router_check(logits, logits_type, T, E, ldl, k, score);
  if (st) return st;
  if (T > 0 && (!topk_idx || !topk_w)) return FP8MOE_ERR_INVALID_ARG;
  const int sums = (counts != nullptr) + (prob_sum != nullptr) + (balance_loss != nullptr);
  if (sums != 0 && sums != 3) return FP8MOE_ERR_INVALID_ARG;
  if (sums && T > 0 && (!workspace || workspace_bytes < fp8moe_router_workspace_bytes(T, E)))
    return FP8MOE_ERR_INVALID_ARG;
  if (((uintptr_t)bias | (uintptr_t)topk_idx | (uintptr_t)topk_w | (uintptr_t)counts | (uintptr_t)prob_sum |
       (uintptr_t)balance_loss | (uintptr_t)workspace) & 3)
    return FP8MOE_ERR_ALIGNMENT;
  if (T == 0 && !sums) return FP8MOE_OK;
  DevInfo* d;
  if ((st = device_info(&d))) return st;
  fp8moe::RouterArgs a{};
  a.logits = logits;
  a.bf16 = logits_type == FP8MOE_BF16;
  a.wide = router_wide(logits, logits_type, E, ldl);
  a.T = T, a.ld = ldl, a.E = (int)E, a.k = (int)k;
  a.score = score, a.renorm = renormalize != 0, a.route_scale = route_scale;
  a.bias = bias, a.mask = token_mask;
  a.idx = topk_idx, a.w = topk_w;
  a.counts = counts, a.psum = prob_sum, a.loss = balance_loss, a.workspace = workspace;
  return cuda_result(fp8moe::launch_router_fwd(a, d->num_sms, (cudaStream_t)stream));
}

fp8moe_status fp8moe_router_bwd(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ldl, int64_t k,
                                int score, int renormalize, float route_scale, const uint8_t* token_mask,
                                const int32_t* topk_idx, const int32_t* counts, const float* dtopk_w,
                                const float* dloss, void* dlogits, fp8moe_stream_t stream) {
  fp8moe_status st = router_check(logits, logits_type, T, E, ldl, k, score);
  if (st) return st;
  if (!dtopk_w && !dloss) return FP8MOE_ERR_INVALID_ARG;
  if (T == 0) return FP8MOE_OK;
  if (!dlogits || (dtopk_w && !topk_idx) || (dloss && !counts)) return FP8MOE_ERR_INVALID_ARG;
  if ((((uintptr_t)topk_idx | (uintptr_t)counts | (uintptr_t)dtopk_w | (uintptr_t)dloss) & 3) ||
      ((uintptr_t)dlogits & (logits_type == FP8MOE_FP32 ? 3 : 1)))
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  if ((st = device_info(&d))) return st;
  fp8moe::RouterArgs a{};
  a.logits = logits;
  a.bf16 = logits_type == FP8MOE_BF16;
  a.wide = router_wide(logits, logits_type, E, ldl) && router_wide(dlogits, logits_type, E, E);
  a.T = T, a.ld = ldl, a.E = (int)E, a.k = (int)k;
  a.score = score, a.renorm = renormalize != 0, a.route_scale = route_scale;
  a.mask = token_mask;
  a.idx_in = topk_idx, a.counts_in = counts, a.dw = dtopk_w, a.dloss = dloss, a.dlogits = dlogits;
  return cuda_result(fp8moe::launch_router_bwd(a, d->num_sms, (cudaStream_t)stream));
}

fp8moe_status fp8moe_route_weight_grad_bounded(const void* dout, const void* y, int64_t rows, const int32_t* row_of,
                                               int64_t T, int64_t N, int64_t k, float* dw, fp8moe_stream_t stream) {
  if (rows < 0 || rows > ((int64_t)1 << 31) || T < 0 || N < 0 || k < 1 || T > ((int64_t)1 << 30) / k) return FP8MOE_ERR_INVALID_ARG;
  if (N % 8) return FP8MOE_ERR_ALIGNMENT;
  if (T == 0) return FP8MOE_OK;
  if (!row_of || !dw || (N > 0 && (!dout || (!y && rows > 0)))) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(dout) || !al16(y) || (((uintptr_t)row_of | (uintptr_t)dw) & 3)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status s = device_info(&d);
  if (s) return s;
  return cuda_result(
      fp8moe::launch_route_weight_grad(dout, y, rows, row_of, T, N, k, dw, d->num_sms, (cudaStream_t)stream));
}

fp8moe_status fp8moe_route_weight_grad(const void* dout, const void* y, const int32_t* row_of, int64_t T, int64_t N,
                                       int64_t k, float* dw, fp8moe_stream_t stream) {
  return fp8moe_route_weight_grad_bounded(dout, y, (int64_t)1 << 31, row_of, T, N, k, dw, stream);
}

fp8moe_status fp8moe_route_weight_grad_ckpt(const void* dout, const void* yq, const uint8_t* ys, int64_t rows,
                                            const int32_t* row_of, int64_t T, int64_t N, int64_t k, float* dw,
                                            fp8moe_stream_t stream) {
  if (rows < 0 || rows > ((int64_t)1 << 31) || T < 0 || N < 0 || N > INT32_MAX || k < 1 || T > ((int64_t)1 << 30) / k) return FP8MOE_ERR_INVALID_ARG;
  if (N % 32) return FP8MOE_ERR_ALIGNMENT;
  if (T == 0) return FP8MOE_OK;
  if (!row_of || !dw || (N > 0 && (!dout || (rows > 0 && (!yq || !ys))))) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(dout) || !al16(yq) || (((uintptr_t)row_of | (uintptr_t)dw) & 3)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status s = device_info(&d);
  if (s) return s;
  return cuda_result(fp8moe::launch_route_weight_grad_ckpt(dout, yq, ys, rows, row_of, T, N, k, dw, d->num_sms,
                                                           (cudaStream_t)stream));
}

// What the checkpointed forms add: the codes and scales of h, written (forward) or
// read in place of h (backward), and the activation along its columns.
struct SwigluCkpt {
  void* q;
  uint8_t* s;
  const void* hq;
  const uint8_t* hs;
  void* aq1;
  uint8_t* as1;
};
static fp8moe_status swiglu(bool bwd, const void* dout, const void* h, int64_t ldh, int64_t M, int64_t F,
                            const int32_t* offs, int64_t E, void* out, void* q0, uint8_t* s0, int s0_layout, void* q1,
                            uint8_t* s1, int s1_layout, const SwigluCkpt* ck, fp8moe_stream_t stream) {
  if (M < 0 || F < 1 || M > ((int64_t)1 << 30) || F > ((int64_t)1 << 28) || ldh < 2 * F)
    return FP8MOE_ERR_INVALID_ARG;
  if (F % 32 || ldh % 8) return FP8MOE_ERR_ALIGNMENT;
  if (M == 0) return FP8MOE_OK;
  const bool act = ck && ck->aq1;
  if (!(out || q0 || q1 || act || (ck && !bwd)) || (q0 == nullptr) != (s0 == nullptr) || (q1 == nullptr) != (s1 == nullptr))
    return FP8MOE_ERR_INVALID_ARG;
  const bool ok0 = !q0 || s0_layout == FP8MOE_SCALES_ROWMAJOR || s0_layout == FP8MOE_NO_GROUPS ||
                   s0_layout == FP8MOE_GROUP_ROWS;
  if (act && !ck->as1) return FP8MOE_ERR_INVALID_ARG;
  const bool ok1 = !(q1 || act) || s1_layout == FP8MOE_SCALES_ROWMAJOR || s1_layout == FP8MOE_NO_GROUPS ||
                   s1_layout == FP8MOE_GROUP_COLS;
  if (!ok0 || !ok1) return FP8MOE_ERR_INVALID_ARG;
  const bool g0 = q0 && s0_layout == FP8MOE_GROUP_ROWS, g1 = (q1 || act) && s1_layout == FP8MOE_GROUP_COLS;
  if ((g0 || g1) && (E < 1 || E > FP8MOE_MAX_GROUPS || !offs)) return FP8MOE_ERR_INVALID_ARG;
  if ((q1 || act || g0) && M % 32) return FP8MOE_ERR_ALIGNMENT;
  if ((g0 || g1) && ((uintptr_t)offs & 3)) return FP8MOE_ERR_ALIGNMENT;
  if ((bwd && ck ? !ck->hq || !ck->hs : !h) || (bwd && !dout) || (ck && !bwd && (!ck->q || !ck->s)))
    return FP8MOE_ERR_INVALID_ARG;
  if (ck && (!al16(ck->q) || !al16(ck->hq) || !al16(ck->aq1))) return FP8MOE_ERR_ALIGNMENT;
  if (!al16(h) || !al16(dout) || !al16(out) || !al16(q0) || !al16(q1)) return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  fp8moe::SwigluArgs a{};
  a.dout = (const uint16_t*)(bwd ? dout : nullptr);
  a.h = (const uint16_t*)h;
  a.M = M, a.F = F, a.ldh = ldh;
  a.offs = offs;
  a.E0 = g0 ? (int)E : 0;
  a.E1 = g1 ? (int)E : 0;
  a.out = (uint16_t*)out;
  a.q0 = (uint8_t*)q0, a.s0 = s0, a.q1 = (uint8_t*)q1, a.s1 = s1;
  a.s0_layout = s0_layout, a.s1_layout = s1_layout;
  if (ck) {
    a.ckpt_q = (uint8_t*)ck->q, a.ckpt_s = ck->s;
    a.hq = (const uint8_t*)ck->hq, a.hs = ck->hs;
    a.aq1 = (uint8_t*)ck->aq1, a.as1 = ck->as1;
  }
  a.num_sms = d->num_sms;
  a.status = d->status;
  return cuda_result(fp8moe::launch_swiglu(a, (cudaStream_t)stream));
}

fp8moe_status fp8moe_swiglu_fwd(const void* h, int64_t ldh, int64_t M, int64_t F, const int32_t* offs, int64_t E,
                                void* out, void* q0, uint8_t* s0, int s0_layout, void* q1, uint8_t* s1,
                                int s1_layout, fp8moe_stream_t stream) {
  return swiglu(false, nullptr, h, ldh, M, F, offs, E, out, q0, s0, s0_layout, q1, s1, s1_layout, nullptr, stream);
}

fp8moe_status fp8moe_swiglu_bwd(const void* dout, const void* h, int64_t ldh, int64_t M, int64_t F,
                                const int32_t* offs, int64_t E, void* dh, void* q0, uint8_t* s0, int s0_layout,
                                void* q1, uint8_t* s1, int s1_layout, fp8moe_stream_t stream) {
  return swiglu(true, dout, h, ldh, M, F, offs, E, dh, q0, s0, s0_layout, q1, s1, s1_layout, nullptr, stream);
}

fp8moe_status fp8moe_swiglu_fwd_ckpt(const void* h, int64_t ldh, int64_t M, int64_t F, const int32_t* offs, int64_t E,
                                     void* out, void* q0, uint8_t* s0, int s0_layout, void* q1, uint8_t* s1,
                                     int s1_layout, void* hq, uint8_t* hs, fp8moe_stream_t stream) {
  const SwigluCkpt ck{hq, hs, nullptr, nullptr, nullptr, nullptr};
  return swiglu(false, nullptr, h, ldh, M, F, offs, E, out, q0, s0, s0_layout, q1, s1, s1_layout, &ck, stream);
}

fp8moe_status fp8moe_swiglu_bwd_ckpt(const void* dout, const void* hq, const uint8_t* hs, int64_t M, int64_t F,
                                     const int32_t* offs, int64_t E, void* dh, void* q0, uint8_t* s0, int s0_layout,
                                     void* q1, uint8_t* s1, int s1_layout, void* aq1, uint8_t* as1,
                                     fp8moe_stream_t stream) {
  const SwigluCkpt ck{nullptr, nullptr, hq, hs, aq1, as1};
  if (F > ((int64_t)1 << 28)) return FP8MOE_ERR_INVALID_ARG;
  if ((aq1 == nullptr) != (as1 == nullptr)) return FP8MOE_ERR_INVALID_ARG;
  return swiglu(true, dout, nullptr, 2 * F, M, F, offs, E, dh, q0, s0, s0_layout, q1, s1, s1_layout, &ck, stream);
}

static bool decode_sizes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F) {
  return T >= 0 && k >= 1 && T <= fp8moe::DECODE_MAX_PAIRS / k && E >= 1 && E <= FP8MOE_MAX_GROUPS && H >= 32 && F >= 32 &&
         H <= ((int64_t)1 << 20) && F <= ((int64_t)1 << 20) && fp8moe::decode_fits(T, k, E, H, F);
}

int64_t fp8moe_mxfp8_moe_decode_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F) {
  if (!decode_sizes(T, k, E, H, F) || H % 32 || F % 32) return -1;
  return fp8moe::decode_workspace_bytes(T, k, E, H, F);
}

fp8moe_status fp8moe_mxfp8_moe_decode(const void* x, int64_t ldx, const int32_t* topk_idx, const float* topk_w, int64_t T,
                                      int64_t k, const void* w1, const uint8_t* w1_scale, const void* w2,
                                      const uint8_t* w2_scale, int64_t E, int64_t H, int64_t F, void* out, void* workspace,
                                      int64_t workspace_bytes, fp8moe_stream_t stream) {
  if (!decode_sizes(T, k, E, H, F) || ldx < H) return FP8MOE_ERR_INVALID_ARG;
  if (H % 32 || F % 32 || ldx % 8) return FP8MOE_ERR_ALIGNMENT;
  if (T == 0) return FP8MOE_OK;
  if (!x || !topk_idx || !topk_w || !w1 || !w1_scale || !w2 || !w2_scale || !out || !workspace)
    return FP8MOE_ERR_INVALID_ARG;
  if (workspace_bytes < fp8moe::decode_workspace_bytes(T, k, E, H, F)) return FP8MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(w1) || !al16(w1_scale) || !al16(w2) || !al16(w2_scale) || !al16(out) || !al16(workspace) ||
      (((uintptr_t)topk_idx | (uintptr_t)topk_w) & 3))
    return FP8MOE_ERR_ALIGNMENT;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  fp8moe::DecodeArgs a{};
  a.x = (const uint16_t*)x, a.ldx = ldx;
  a.T = (int)T, a.k = (int)k, a.E = (int)E, a.H = (int)H, a.F = (int)F;
  a.idx = topk_idx, a.w = topk_w;
  a.q1 = (const uint8_t*)w1, a.s1 = w1_scale, a.q2 = (const uint8_t*)w2, a.s2 = w2_scale;
  a.out = (uint16_t*)out;
  a.status = d->status;
  return cuda_result(fp8moe::launch_decode(a, workspace, d->num_sms, d->max_smem, (cudaStream_t)stream));
}

fp8moe_status fp8moe_get_device_status(fp8moe_stream_t stream, int32_t* out_code) {
  if (!out_code) return FP8MOE_ERR_INVALID_ARG;
  DevInfo* d;
  fp8moe_status st = device_info(&d);
  if (st) return st;
  // The read and the clear are one atomic exchange on the device, ordered
  // after the stream's work: a status that a kernel on another stream sets
  // meanwhile is either taken here or stays for the next call.  The mutex
  // keeps concurrent callers from sharing the take slot.
  std::lock_guard<std::mutex> lk(g_take_mu);
  k_take_status<<<1, 1, 0, (cudaStream_t)stream>>>(d->status, d->take);
  if (cudaGetLastError() != cudaSuccess) return FP8MOE_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyAsync(&v, d->take, sizeof(int), cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess)
    return FP8MOE_ERR_CUDA;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return FP8MOE_ERR_CUDA;
  *out_code = v;
  return FP8MOE_OK;
}

fp8moe_status fp8moe_testing_stall_next_gemm(void) {
  fp8moe::arm_gemm_stall_hook();
  return FP8MOE_OK;
}

fp8moe_status fp8moe_testing_stall_next_tensorwise(void) {
  fp8moe::arm_tensorwise_stall_hook();
  return FP8MOE_OK;
}

fp8moe_status fp8moe_testing_stall_next_quant_ring(void) {
  fp8moe::arm_ring_stall_hook();
  return FP8MOE_OK;
}

}  // extern "C"
