// layers_norm.cu -- layer norm forward.
#include "layers.cuh"

namespace sm {
namespace {

constexpr int kStages = 3;

// ---------------------------------------------------------------------------
// Y = (X - mean) * rstd * gamma + beta.  Bound by the bytes (X read once, Y
// written once).  WPR warps hold a row in registers, EPL elements a lane, so
// the variance is summed around the mean without a second read; gamma and
// beta stay in registers too where there is room.  Rows on 16-byte boundaries come in through
// asynchronous copies, kStages rows ahead, into slots that only the copying
// thread reads.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, int WPR, int EPL>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256)
    k_ln_fwd(const T* __restrict__ X, int64_t ldx, T* __restrict__ Y, int64_t ldy, const float* __restrict__ gamma,
             const float* __restrict__ beta, int64_t n, int E, float eps, float* __restrict__ mean,
             float* __restrict__ rstd) {
  constexpr int VL = Elem<T>::V;
  constexpr int CH = EPL / VL;                      // strips per warp
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;                  // rows per block
  constexpr bool KEEP = VEC || EPL <= 24;           // gamma and beta in registers, where there is room
  extern __shared__ uint4 ring[];                   // VEC: [kStages][CH][threads]
  __shared__ float buf[2][WARPS];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % WPR, group = warp / WPR;
  const float inv_E = 1.f / (float)E;
  const int64_t step = (int64_t)gridDim.x * RPB;
  auto fetch = [&](int64_t r, int stage) {
    if (r < n) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * WPR + w) * 32 * VL + lane * VL;
        copy16(&ring[(stage * CH + c) * (WARPS * 32) + threadIdx.x], X + r * ldx + (col < E ? col : 0), col < E);
      }
    }
    copy_commit();
  };
  const int64_t r_first = (int64_t)blockIdx.x * RPB + group;
  if (VEC) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch(r_first + s * step, s);
  }
  float g[KEEP ? CH : 1][VL], b[KEEP ? CH : 1][VL];
  auto weights = [&](int c, float* gc, float* bc) {
    strip_load_f32<T, VEC>(gamma, (c * WPR + w) * 32 * VL, E, lane, gc);
    if (beta != nullptr) {
      strip_load_f32<T, VEC>(beta, (c * WPR + w) * 32 * VL, E, lane, bc);
    } else {
#pragma unroll
      for (int j = 0; j < VL; ++j) bc[j] = 0.f;
    }
  };
  if (KEEP) {
#pragma unroll
    for (int c = 0; c < CH; ++c) weights(c, g[KEEP ? c : 0], b[KEEP ? c : 0]);
  }
  int stage = 0;
  for (int64_t r = r_first; r < n; r += step) {
    float x[CH][VL];
    float s = 0.f;
    if (VEC) {
      copy_wait<kStages - 1>();
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const Pack<T> p = *reinterpret_cast<const Pack<T>*>(&ring[(stage * CH + c) * (WARPS * 32) + threadIdx.x]);
#pragma unroll
        for (int j = 0; j < VL; ++j) x[c][j] = Elem<T>::up(p.v[j]);
      }
      fetch(r + kStages * step, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) strip_load<T, VEC>(X + r * ldx, (c * WPR + w) * 32 * VL, E, lane, x[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VL; ++j) s += x[c][j];
    auto row_sum = [&](float v, float* at) {
      v = warp_sum(v);
      if (WPR == 1) return v;
      if (lane == 0) at[warp] = v;
      group_sync<WPR, WARPS>(group);
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) t += at[group * WPR + i];
      return t;
    };
    const float mu = row_sum(s, buf[0]) * inv_E;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        // (columns beyond E were loaded as zeros and must not count)
        const float d = strip_col<T, VEC>((c * WPR + w) * 32 * VL, lane, j) < E ? x[c][j] - mu : 0.f;
        x[c][j] = d;
        s = fmaf(d, d, s);
      }
    }
    const float rs = 1.f / sqrtf(row_sum(s, buf[1]) * inv_E + eps);
    if (mean != nullptr && w == 0 && lane == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
      if (!KEEP) weights(c, g[0], b[0]);
#pragma unroll
      for (int j = 0; j < VL; ++j) x[c][j] = fmaf(x[c][j] * rs, g[KEEP ? c : 0][j], b[KEEP ? c : 0][j]);
      strip_store<T, VEC>(Y + r * ldy, base, E, lane, x[c]);
    }
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct FwdArgs {
  const float *gamma, *beta;
  int64_t n;
  int E;
  const void* X;
  int64_t ldx;
  void* Y;
  int64_t ldy;
  float eps;
  float *mean, *rstd;
};

template <typename T, bool VEC, int WPR, int EPL>
void run_fwd(cudaStream_t s, const FwdArgs& a) {
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  const size_t smem = VEC ? (size_t)kStages * (EPL / Elem<T>::V) * WARPS * 32 * 16 : 0;
  auto* kernel = k_ln_fwd<T, VEC, WPR, EPL>;
  if (smem > 32 * 1024) cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  const int grid = stream_grid((const void*)kernel, WARPS * 32, smem, (a.n + WARPS / WPR - 1) / (WARPS / WPR), 8);
  count_launch();
  launch_pdl(kernel, dim3(grid), dim3(WARPS * 32), smem, s, reinterpret_cast<const T*>(a.X), a.ldx,
             reinterpret_cast<T*>(a.Y), a.ldy, a.gamma, a.beta, a.n, a.E, a.eps, a.mean, a.rstd);
}

// the fewest warps that hold a row at 32 elements a lane, then the fewest elements
template <typename T, bool VEC>
void pick_fwd(cudaStream_t s, const FwdArgs& a) {
  auto fits = [&](int wpr, int epl) { return a.E <= 32 * wpr * epl; };
  if (fits(1, 8)) run_fwd<T, VEC, 1, 8>(s, a);
  else if (fits(1, 16)) run_fwd<T, VEC, 1, 16>(s, a);
  else if (fits(1, 24)) run_fwd<T, VEC, 1, 24>(s, a);
  else if (fits(1, 32)) run_fwd<T, VEC, 1, 32>(s, a);
  else if (fits(2, 24)) run_fwd<T, VEC, 2, 24>(s, a);
  else if (fits(2, 32)) run_fwd<T, VEC, 2, 32>(s, a);
  else if (fits(4, 24)) run_fwd<T, VEC, 4, 24>(s, a);
  else if (fits(4, 32)) run_fwd<T, VEC, 4, 32>(s, a);
  else if (fits(8, 24)) run_fwd<T, VEC, 8, 24>(s, a);
  else if (fits(8, 32)) run_fwd<T, VEC, 8, 32>(s, a);
  else if (fits(16, 24)) run_fwd<T, VEC, 16, 24>(s, a);
  else run_fwd<T, VEC, 16, 32>(s, a);
}

}  // namespace

void launch_layernorm(cudaStream_t s, const float* gamma, const float* beta, int64_t n, int64_t E, const void* X,
                      int64_t ldx, void* Y, int64_t ldy, int type, float eps, float* mean, float* rstd) {
  if (n == 0) return;
  const int vl = type == LT_F32 ? 4 : 8;
  const bool vec = E % vl == 0 && ldx % vl == 0 && ldy % vl == 0 && on16(X) && on16(Y) && on16(gamma) && on16(beta);
  const FwdArgs a{gamma, beta, n, (int)E, X, ldx, Y, ldy, eps, mean, rstd};
#define SM_RUN(T) (vec ? pick_fwd<T, true>(s, a) : pick_fwd<T, false>(s, a))
  if (type == LT_F32) SM_RUN(float);
  else if (type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

}  // namespace sm
