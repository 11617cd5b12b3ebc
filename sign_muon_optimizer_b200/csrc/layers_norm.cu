// layers_norm.cu -- layer norm forward, and backward with the reduction of
// the weights' gradients per worker.
#include "layers.cuh"

namespace sm {
namespace {

// Sum over the 32 * WPR threads that hold a row.  `buf` has one float per
// warp of the block.  Every thread of the block takes part.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = warp_sum(v);
  if (WPR == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[warp] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) t += buf[warp / WPR * WPR + i];
  return t;
}

// ---------------------------------------------------------------------------
// Forward.  A row is held in the registers of WPR warps (32 elements a lane
// at most), so X is read once: mean, then the variance around the mean, then
// the output.  Bound by the bytes (X read, Y written).
// ---------------------------------------------------------------------------
template <typename T, bool VEC, int WPR>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256)
    k_ln_fwd(const T* __restrict__ X, int64_t ldx, T* __restrict__ Y, int64_t ldy, const float* __restrict__ gamma,
             const float* __restrict__ beta, int64_t n, int E, float eps, float* __restrict__ mean,
             float* __restrict__ rstd) {
  constexpr int VL = Elem<T>::V;
  constexpr int CH = 32 / VL;                       // strips per warp
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;                  // rows per block
  __shared__ float buf[2][WARPS];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % WPR;
  const float inv_E = 1.f / (float)E;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < n; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + warp / WPR;
    const bool live = r < n;
    float x[CH][VL];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      strip_load<T, VEC>(X + (live ? r : 0) * ldx, (c * WPR + w) * 32 * VL, live ? E : 0, lane, x[c]);
#pragma unroll
      for (int j = 0; j < VL; ++j) s += x[c][j];
    }
    const float mu = row_sum<WPR>(s, buf[0]) * inv_E;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const float d = strip_col<T, VEC>((c * WPR + w) * 32 * VL, lane, j) < E ? x[c][j] - mu : 0.f;
        s = fmaf(d, d, s);
      }
    const float rs = 1.f / sqrtf(row_sum<WPR>(s, buf[1]) * inv_E + eps);
    if (!live) continue;
    if (mean != nullptr && w == 0 && lane == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
      if (base < E) {
        float g[VL], b[VL];
        strip_load_f32<T, VEC>(gamma, base, E, lane, g);
        if (beta != nullptr) strip_load_f32<T, VEC>(beta, base, E, lane, b);
#pragma unroll
        for (int j = 0; j < VL; ++j) {
          const float xh = (x[c][j] - mu) * rs;
          x[c][j] = beta != nullptr ? fmaf(xh, g[j], b[j]) : xh * g[j];
        }
        strip_store<T, VEC>(Y + r * ldy, base, E, lane, x[c]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  A block takes consecutive rows of one worker, so the sums over
// rows that make the weights' gradients stay in registers, one column per
// thread and strip element (in shared memory for the longest rows); a
// second kernel adds up the blocks' sums of each worker in order.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, int WPR, int EPL>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256)
    k_ln_bwd(const RowMap map, int rows_per_unit, const T* __restrict__ X, int64_t ldx, const T* dY, int64_t ldy,
             const float* __restrict__ gamma, const float* __restrict__ mean, const float* __restrict__ rstd, T* dX,
             int64_t ldd, int E, float* __restrict__ part) {
  constexpr int VL = Elem<T>::V;
  constexpr int CH = EPL / VL;                      // strips per warp: EPL elements a lane
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;
  constexpr bool IN_SMEM = EPL > 16;                // too few registers for the sums as well
  constexpr bool RELOAD = IN_SMEM && sizeof(T) == 4; // ... nor for dY, which is read a second time (from L1)
  constexpr int COLS = WPR * 32 * EPL;              // columns a row group covers
  extern __shared__ float sums[];                   // IN_SMEM: 2 x COLS; else RPB > 1: RPB x COLS
  __shared__ float buf[2][WARPS];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % WPR;
  const int m = worker_of(map.unit, map.M, blockIdx.x);
  const int first = map.start[m] + (blockIdx.x - map.unit[m]) * rows_per_unit;
  const int last = min(first + rows_per_unit, map.start[m + 1]);
  const float inv_E = 1.f / (float)E;
  float ag[IN_SMEM ? 1 : CH][VL], ab[IN_SMEM ? 1 : CH][VL];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      if (IN_SMEM) {
        const int col = strip_col<T, VEC>((c * WPR + w) * 32 * VL, lane, j);
        sums[col] = 0.f;
        sums[COLS + col] = 0.f;
      } else {
        ag[c][j] = 0.f;
        ab[c][j] = 0.f;
      }
    }
  for (int r0 = first; r0 < last; r0 += RPB) {
    const int64_t r = r0 + warp / WPR;
    const bool live = r < last;
    const int64_t rr = live ? r : first;
    const int cols = live ? E : 0;
    Pack<T> x[CH], dy[RELOAD ? 1 : CH];
    float s1 = 0.f, s2 = 0.f;
    const float mu = live ? mean[rr] : 0.f, rs = live ? rstd[rr] : 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
      x[c] = strip_raw<T, VEC>(X + rr * ldx, base, cols, lane);
      if (!RELOAD) dy[RELOAD ? 0 : c] = strip_raw<T, VEC>(dY + rr * ldy, base, cols, lane);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int base = (c * WPR + w) * 32 * VL;
      float ga[VL];
      strip_load_f32<T, VEC>(gamma, base, cols, lane, ga);
      const Pack<T> raw = RELOAD ? strip_raw<T, VEC>(dY + rr * ldy, base, cols, lane) : dy[RELOAD ? 0 : c];
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int col = strip_col<T, VEC>(base, lane, j);
        const float h = col < cols ? (Elem<T>::up(x[c].v[j]) - mu) * rs : 0.f;
        const float d = Elem<T>::up(raw.v[j]);
        if (IN_SMEM) {
          if (col < cols) {
            sums[col] = fmaf(d, h, sums[col]);
            sums[COLS + col] += d;
          }
        } else {
          ag[c][j] = fmaf(d, h, ag[c][j]);
          ab[c][j] += d;
        }
        const float g = d * ga[j];
        s1 += g;
        s2 = fmaf(g, h, s2);
      }
    }
    s1 = row_sum<WPR>(s1, buf[0]) * inv_E;
    s2 = row_sum<WPR>(s2, buf[1]) * inv_E;
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int base = (c * WPR + w) * 32 * VL;
        float ga[VL], o[VL];
        strip_load_f32<T, VEC>(gamma, base, cols, lane, ga);
        const Pack<T> raw = RELOAD ? strip_raw<T, VEC>(dY + rr * ldy, base, cols, lane) : dy[RELOAD ? 0 : c];
#pragma unroll
        for (int j = 0; j < VL; ++j) {
          const float h = (Elem<T>::up(x[c].v[j]) - mu) * rs;
          o[j] = rs * (Elem<T>::up(raw.v[j]) * ga[j] - s1 - h * s2);
        }
        strip_store<T, VEC>(dX + rr * ldd, base, E, lane, o);
      }
    }
  }
  // the block's sums: row groups added up in order through shared memory
  float* out = part + (int64_t)blockIdx.x * 2 * E;
  if (IN_SMEM) {
    __syncthreads();
    for (int col = threadIdx.x; col < E; col += WARPS * 32) {
      out[col] = sums[col];
      out[E + col] = sums[COLS + col];
    }
    return;
  }
  for (int which = 0; which < 2; ++which) {
    if (RPB > 1) __syncthreads();
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int col = strip_col<T, VEC>((c * WPR + w) * 32 * VL, lane, j);
        const float v = which ? ab[c][j] : ag[c][j];
        if (RPB > 1) sums[warp / WPR * COLS + col] = v;
        else if (col < E) out[which * E + col] = v;
      }
    if (RPB > 1) {
      __syncthreads();
      for (int col = threadIdx.x; col < E; col += WARPS * 32) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < RPB; ++i) t += sums[i * COLS + col];
        out[which * E + col] = t;
      }
    }
  }
}

// G[m] (+)= the sum of worker m's blocks, in order: 32 columns a block, 8
// threads a column, each over a fixed share of the blocks
__global__ void __launch_bounds__(256) k_ln_weights(const RowMap map, const GradPtrs G, const float* __restrict__ part,
                                                    int E, int64_t off_gamma, int64_t off_beta, int accumulate) {
  __shared__ float t[8][33];
  griddep_wait();
  griddep_launch();
  const int m = blockIdx.y;
  const int which = blockIdx.z;
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int u0 = map.unit[m], u1 = map.unit[m + 1];
  const int share = (u1 - u0 + 7) / 8;
  float s = 0.f;
  if (col < E) {
    const int b = min(u1, u0 + (k + 1) * share);
    for (int u = u0 + k * share; u < b; ++u) s += part[((int64_t)u * 2 + which) * E + col];
  }
  t[k][lane] = s;
  __syncthreads();
  if (k == 0 && col < E) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += t[i][lane];
    float* g = G.p[m] + (which ? off_beta : off_gamma) + col;
    *g = accumulate ? *g + s : s;
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, bool VEC, int WPR>
void run_fwd(cudaStream_t s, const float* gamma, const float* beta, int64_t n, int E, const void* X, int64_t ldx,
             void* Y, int64_t ldy, float eps, float* mean, float* rstd) {
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  auto* kernel = k_ln_fwd<T, VEC, WPR>;
  const int grid = stream_grid((const void*)kernel, WARPS * 32, 0, (n + WARPS / WPR - 1) / (WARPS / WPR), 8);
  count_launch();
  launch_pdl(kernel, dim3(grid), dim3(WARPS * 32), 0, s, reinterpret_cast<const T*>(X), ldx, reinterpret_cast<T*>(Y),
             ldy, gamma, beta, n, E, eps, mean, rstd);
}

template <typename T, bool VEC, int WPR, int EPL>
void run_bwd(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;
  constexpr int COLS = WPR * 32 * EPL;
  const size_t smem = EPL > 16 ? (size_t)2 * COLS * 4 : (RPB > 1 ? (size_t)RPB * COLS * 4 : 0);
  auto* kernel = k_ln_bwd<T, VEC, WPR, EPL>;
  if (smem > 48 * 1024) cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  const int N = start[M];
  // one wave of blocks; every worker's rows split into units of equal length
  int64_t want = (int64_t)num_sms() * resident_per_sm((const void*)kernel, WARPS * 32, smem);
  if (want > a.max_blocks - M) want = a.max_blocks - M;
  if (want < 1) want = 1;
  int64_t per = (N + want - 1) / want;
  per = (per + RPB - 1) / RPB * RPB;
  if (per < RPB) per = RPB;
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  for (int m = 0; m < M; ++m) map.unit[m + 1] = map.unit[m] + (int)((start[m + 1] - start[m] + per - 1) / per);
  if (map.unit[M] > 0) {
    count_launch();
    launch_pdl(kernel, dim3(map.unit[M]), dim3(WARPS * 32), smem, s, map, (int)per, reinterpret_cast<const T*>(a.X),
               a.ldx, reinterpret_cast<const T*>(a.dY), a.ldy, a.gamma, a.mean, a.rstd, reinterpret_cast<T*>(a.dX),
               a.ldd, (int)a.E, a.part);
  }
  count_launch();
  launch_pdl(k_ln_weights, dim3((unsigned)((a.E + 31) / 32), M, a.off_beta >= 0 ? 2 : 1), dim3(256), 0, s, map, G,
             (const float*)a.part, (int)a.E, a.off_gamma, a.off_beta, a.accumulate);
}

}  // namespace

void launch_layernorm(cudaStream_t s, const float* gamma, const float* beta, int64_t n, int64_t E, const void* X,
                      int64_t ldx, void* Y, int64_t ldy, int type, float eps, float* mean, float* rstd) {
  if (n == 0) return;
  const int vl = type == LT_F32 ? 4 : 8;
  const bool vec = E % vl == 0 && ldx % vl == 0 && ldy % vl == 0 && on16(X) && on16(Y) && on16(gamma) && on16(beta);
#define SM_W(T, VEC, W) run_fwd<T, VEC, W>(s, gamma, beta, n, (int)E, X, ldx, Y, ldy, eps, mean, rstd)
#define SM_E(T, VEC)                         \
  do {                                       \
    if (E <= 1024) SM_W(T, VEC, 1);          \
    else if (E <= 2048) SM_W(T, VEC, 2);     \
    else if (E <= 4096) SM_W(T, VEC, 4);     \
    else if (E <= 8192) SM_W(T, VEC, 8);     \
    else SM_W(T, VEC, 16);                   \
  } while (0)
#define SM_T(T)                  \
  do {                           \
    if (vec) SM_E(T, true);      \
    else SM_E(T, false);         \
  } while (0)
  if (type == LT_F32) SM_T(float);
  else if (type == LT_BF16) SM_T(__nv_bfloat16);
  else SM_T(__half);
#undef SM_E
#undef SM_W
}

void launch_layernorm_grad(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  const int64_t E = a.E;
  const int vl = a.type == LT_F32 ? 4 : 8;
  const bool vec = E % vl == 0 && a.ldx % vl == 0 && a.ldy % vl == 0 && a.ldd % vl == 0 && on16(a.X) && on16(a.dY) &&
                   on16(a.dX) && on16(a.gamma);
#define SM_W(T, VEC, W, EPL) run_bwd<T, VEC, W, EPL>(s, a, start, M, G)
#define SM_E(T, VEC)                         \
  do {                                       \
    if (E <= 512) SM_W(T, VEC, 1, 16);           \
    else if (E <= 1024) SM_W(T, VEC, 2, 16);     \
    else if (E <= 2048) SM_W(T, VEC, 4, 16);     \
    else if (E <= 4096) SM_W(T, VEC, 8, 16);     \
    else if (E <= 8192) SM_W(T, VEC, 16, 16);    \
    else SM_W(T, VEC, 16, 32);                   \
  } while (0)
  if (a.type == LT_F32) SM_T(float);
  else if (a.type == LT_BF16) SM_T(__nv_bfloat16);
  else SM_T(__half);
#undef SM_E
#undef SM_W
#undef SM_T
}

}  // namespace sm
