// ctx.h -- the handle behind signmuon_t and the host helpers that the files
// implementing the C ABI share (signmuon_api.cu, layers_api.cu): errors,
// device allocation, the device guard, argument checks.
#pragma once
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <string>
#include <vector>

#include "../../include/signmuon.h"
#include "common.cuh"
#include "plan.h"

struct signmuon_ctx {
  sm::Plan plan;
  int M = 0, K = 0, scale = 0, P = 1;
  float beta = 0.f, lambda = 0.f, eps = 0.f;
  float ns_a = 1.5f, ns_b = -0.5f, ns_c = 0.f;
  unsigned flags = 0;
  cudaStream_t stream = nullptr;
  int device = 0, n_sm = 148;
  bool vote_only = false;
  bool u_valid = true;          // U holds the last step's (or polar call's) polar factors
  bool bits_valid = true;       // bits hold the last step's packed signs
  bool t_valid = false;         // sign8 holds the last step's ternary signs
  bool dir_valid = false;       // get_direction can give the last step's D
  bool dir_in_D = false;        // ... and it is in D (else: the majority of the handle's own signs)
  // device plan tables
  sm::MatInfo* d_mats = nullptr;
  sm::GroupInfo* d_groups = nullptr;
  int* d_group_mats = nullptr;
  int64_t* d_mat_off = nullptr;
  sm::Chunk* d_chunks = nullptr;
  int* d_mat_chunk0 = nullptr;
  int* d_mat_nchunks = nullptr;
  int64_t* d_stage_off = nullptr;
  sm::TileGroup* d_tiles[3][2] = {{nullptr}};
  int* d_sched[3][2] = {{nullptr}};   // tensor-core tile schedules (null: round robin)
  sm::PiTile* d_pi_tiles = nullptr;
  sm::PiSlice* d_pi_slices = nullptr;
  int64_t* d_uoff = nullptr;
  int* d_prob_g = nullptr;
  int* d_prob_gld = nullptr;
  int64_t* d_prob_aoff = nullptr;
  void* d_maps = nullptr;
  // device state / workspace
  float* Mom = nullptr;
  void* X[2] = {nullptr, nullptr};
  void* A = nullptr;
  void* B = nullptr;
  void* A2 = nullptr;           // Gram space: the second A buffer and the Q pair
  void* Q[2] = {nullptr, nullptr};
  float* U = nullptr;
  uint8_t* bits = nullptr;
  int8_t* sign8 = nullptr;      // TERNARY: int8 signs, M x dpad bytes
  float* D = nullptr;
  float* partials = nullptr;
  float* scale_v = nullptr;
  float2* coef_apply = nullptr;
  float2* coef_square = nullptr;
  float2* coef_gram = nullptr;  // Gram space: A1 = a T0 + b cc^2 A~ T0
  float* pi_u = nullptr;        // power-iteration iterates of the M-worker problems (warm state)
  float* pi_u1 = nullptr;       // PI_WARM: iterates of the one-problem-set PolarNS (warm state)
  float* pi_y = nullptr;
  float* pi_part = nullptr;     // per-tile partial sums of A v
  float* pi_inv = nullptr;      // per-problem 1/||y|| between passes
  double* pi_sq = nullptr;      // per-slice ||y||^2 or u.y
  int* pi_cnt = nullptr;        // per-problem slice counters (zero between launches)
  int* status = nullptr;        // [0] non-finite flag, [1] kernel error code
  int* h_status = nullptr;      // pinned mirror
  bool pending = false;         // an async step's status not yet read
  // the ternary signs of the step's last Newton-Schulz GEMM (bf16 path): set
  // by local_part around its run_ns, read by gemm() for the final apply
  int8_t* final_sign8 = nullptr;
  int64_t final_sign8_stride = 0;
  // step_host staging: W, and two gradient buffers so that a call's
  // gradients can come in (on the copy stream) while the step before runs
  float* hw_W = nullptr;
  float* hw_G[2] = {nullptr, nullptr};
  int hw_next = 0;                      // the gradient buffer of the next call
  cudaStream_t copy_stream = nullptr;
  cudaEvent_t g_ready[2] = {nullptr, nullptr};   // buffer b holds its call's gradients
  cudaEvent_t g_free[2] = {nullptr, nullptr};    // the step that read buffer b is done
  cudaEvent_t w_ready = nullptr;                 // W of the current call is on the device
  cudaEvent_t w_free = nullptr;                  // the previous call's W has gone back
  // workspace of the layer calls (signmuon_layers.h), as reserved
  int64_t lay_rows = 0, lay_cols = 0;
  uint8_t* lay_ws = nullptr;
  int* lay_status = nullptr;    // [0] an index was out of range; then two counters per worker, zero between calls
  int* h_lay_status = nullptr;  // pinned mirror of [0]
  std::vector<void*> allocs;
  int64_t bytes = 0;
  std::string err;
  // optional per-kernel timing: event pairs recorded around each launch
  bool prof = false;
  std::vector<cudaEvent_t> ev_pool;
  size_t ev_used = 0;
  std::vector<int> ev_kind;           // kind of each recorded pair
  double prof_ms[SIGNMUON_PROF_KINDS] = {0};
  int64_t prof_n[SIGNMUON_PROF_KINDS] = {0};
};

namespace sm {

inline int fail(signmuon_t h, int code, const std::string& msg) {
  if (h) h->err = msg;
  else set_global_error(msg.c_str());
  return code;
}

#define CK(h, call)                                                                   \
  do {                                                                                \
    cudaError_t e_ = (call);                                                          \
    if (e_ != cudaSuccess) {                                                          \
      cudaGetLastError();                                                             \
      return fail((h), e_ == cudaErrorMemoryAllocation ? SIGNMUON_E_NOMEM : SIGNMUON_E_CUDA, \
                  std::string(#call) + ": " + cudaGetErrorString(e_));                \
    }                                                                                 \
  } while (0)

template <typename T>
int dalloc(signmuon_t h, T** p, int64_t count) {
  *p = nullptr;
  if (count <= 0) count = 1;
  void* q = nullptr;
  cudaError_t e = cudaMalloc(&q, (size_t)count * sizeof(T));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(h, SIGNMUON_E_NOMEM, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  }
  h->allocs.push_back(q);
  h->bytes += count * (int64_t)sizeof(T);
  *p = reinterpret_cast<T*>(q);
  return SIGNMUON_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline WorkerPtrs worker_ptrs(const float* const* p, int M) {
  WorkerPtrs w{};
  for (int m = 0; m < M; ++m) w.p[m] = p[m];
  return w;
}

// A host NVTX range for the lifetime of a scope (a no-op unless a tool such
// as ncu --nvtx is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Makes the handle's device current for the duration of one entry point and
// gives the caller's current device back on return, so that a call on a
// handle of another GPU leaves the caller's device selection as it was.
struct DeviceGuard {
  int saved = -1;
  explicit DeviceGuard(signmuon_t h) {
    if (h == nullptr) return;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      dev = -1;
    }
    if (dev != h->device && cudaSetDevice(h->device) == cudaSuccess) saved = dev;
  }
  ~DeviceGuard() {
    if (saved >= 0) cudaSetDevice(saved);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
};

inline int check_handle(signmuon_t h, bool need_step) {
  if (h == nullptr) return fail(nullptr, SIGNMUON_E_INVALID, "null handle");
  if (need_step && h->vote_only) return fail(h, SIGNMUON_E_UNSUPPORTED, "handle was created with SIGNMUON_VOTE_ONLY");
  return SIGNMUON_OK;
}

}  // namespace sm
