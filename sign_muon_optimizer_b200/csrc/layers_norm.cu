// layers_norm.cu -- layer norm forward.
#include "layers.cuh"

namespace sm {
namespace {

// rows on their way: four where two blocks' slots still fit an SM
constexpr int stages(int strips, int threads) { return strips * threads * 16 * 4 * 2 <= 226 * 1024 ? 4 : 3; }

// ---------------------------------------------------------------------------
// Y = (X - mean) * rstd * gamma + beta.  Bound by the bytes (X read once, Y
// written once): 131072 x 768 bf16 takes 74 us, 5.4 TB/s, and 32768 x 4096 92 us,
// 5.8 TB/s.  WPR warps hold a row in registers, EPL elements a lane, so the
// variance is summed around the mean without a second read; gamma and beta stay
// in registers too where there is room.  A lane's elements go in pairs (one
// instruction for two), without which the first takes 76 us.  Rows on 16-byte
// boundaries come in through asynchronous copies, three or four rows ahead, into
// slots that only the copying thread reads: the registers hold one row, and the
// 16 warps that fit an SM would not keep enough loads on their way.  Other rows
// are loaded element by element (30000 x 1001 bf16: 41 us, 2.9 TB/s).
// ---------------------------------------------------------------------------
template <typename T, bool VEC, int WPR, int EPL>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256)
    k_ln_fwd(const T* X, int64_t ldx, T* __restrict__ Y, int64_t ldy, const float* gamma,
             const float* beta, int64_t n, int E, float eps, float* __restrict__ mean,
             float* __restrict__ rstd) {
  constexpr int VL = Elem<T>::V;
  constexpr int CH = EPL / VL;                      // strips per warp
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;                  // rows per block
  constexpr bool KEEP = VEC || EPL <= 24;           // gamma and beta in registers, where there is room
  constexpr int kStages = stages(CH, WARPS * 32);
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
  // pairs of columns: the weights of this thread's columns
  F2 g[KEEP ? CH : 1][VL / 2], b[KEEP ? CH : 1][VL / 2];
  auto load_pairs = [&](const float* from, int c, F2* to) {
    float t[VL];
    strip_load_f32<T, VEC>(from, (c * WPR + w) * 32 * VL, E, lane, t);
#pragma unroll
    for (int j = 0; j < VL / 2; ++j) to[j] = pack2(t[2 * j], t[2 * j + 1]);
  };
  auto weights = [&](int c, F2* gc, F2* bc) {
    load_pairs(gamma, c, gc);
    if (beta != nullptr) {
      load_pairs(beta, c, bc);
    } else {
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) bc[j] = 0ull;
    }
  };
  if (KEEP) {
#pragma unroll
    for (int c = 0; c < CH; ++c) weights(c, g[KEEP ? c : 0], b[KEEP ? c : 0]);
  }
  int stage = 0;
  for (int64_t r = r_first; r < n; r += step) {
    F2 x[CH][VL / 2];
    if (VEC) copy_wait<kStages - 1>();
    F2 a = 0ull;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      Pack<T> p;
      if (VEC) p = *reinterpret_cast<const Pack<T>*>(&ring[(stage * CH + c) * (WARPS * 32) + threadIdx.x]);
      else p = strip_raw<T, VEC>(X + r * ldx, (c * WPR + w) * 32 * VL, E, lane);
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        x[c][j] = up2(p, j);
        a = add2(x[c][j], a);
      }
    }
    if (VEC) {
      fetch(r + kStages * step, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
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
    const float mu = row_sum(sum2(a), buf[0]) * inv_E;
    const F2 neg_mu = pack2(-mu, -mu);
    a = 0ull;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        x[c][j] = add2(x[c][j], neg_mu);
        if (base + 32 * VL > E) {  // columns beyond E were loaded as zeros and must not count
          const float2 t = unpack2(x[c][j]);
          x[c][j] = pack2(strip_col<T, VEC>(base, lane, 2 * j) < E ? t.x : 0.f,
                          strip_col<T, VEC>(base, lane, 2 * j + 1) < E ? t.y : 0.f);
        }
        a = fma2(x[c][j], x[c][j], a);
      }
    }
    const float rs = 1.f / sqrtf(row_sum(sum2(a), buf[1]) * inv_E + eps);
    if (mean != nullptr && w == 0 && lane == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    const F2 rs2 = pack2(rs, rs);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
      if (!KEEP) weights(c, g[0], b[0]);
      float o[VL];
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        const float2 t = unpack2(fma2(mul2(x[c][j], rs2), g[KEEP ? c : 0][j], b[KEEP ? c : 0][j]));
        o[2 * j] = t.x;
        o[2 * j + 1] = t.y;
      }
      strip_store<T, VEC>(Y + r * ldy, base, E, lane, o);
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
  constexpr int CH = EPL / Elem<T>::V;
  const size_t smem = VEC ? (size_t)stages(CH, WARPS * 32) * CH * WARPS * 32 * 16 : 0;
  auto* kernel = k_ln_fwd<T, VEC, WPR, EPL>;
  if (smem > 32 * 1024) allow_shared((const void*)kernel);
  const int grid = stream_grid((const void*)kernel, WARPS * 32, smem, (a.n + WARPS / WPR - 1) / (WARPS / WPR), 8);
  count_launch();
  launch_pdl(kernel, dim3(grid), dim3(WARPS * 32), smem, s, reinterpret_cast<const T*>(a.X), a.ldx,
             reinterpret_cast<T*>(a.Y), a.ldy, a.gamma, a.beta, a.n, a.E, a.eps, a.mean, a.rstd);
}

// The fewest warps that hold a row at 32 elements a lane, then the fewest
// elements.  More warps with 8 elements a lane gain nothing where rows are loaded
// element by element either (16000 x 2001 bf16 46 us instead of 43, 8000 x 4001
// 53 instead of 43; 30000 x 1001 fp32 49 instead of 55).
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
