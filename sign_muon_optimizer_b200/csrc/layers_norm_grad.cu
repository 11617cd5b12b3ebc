// layers_norm_grad.cu -- layer norm backward, with the reduction of the
// weights' gradients per worker.
#include "layers.cuh"

namespace sm {
namespace {

constexpr int kStages = 3;

// ---------------------------------------------------------------------------
// With xh = (X - mean) * rstd and g = dY * gamma, per row
//   dX = rstd * (g - mean_E(g) - xh * mean_E(g * xh)),
// and per worker dgamma = sum of dY * xh, dbeta = sum of dY over its rows.
// WPR warps hold a row, EPL elements a lane.  A block takes consecutive rows of
// one worker, so the sums over rows stay in registers, a column per element of a
// thread; the blocks' sums of each worker are added up in order by k_ln_weights
// (10 us for 16 workers of 4096 columns, of which the launch hides a part).
// Rows on 16-byte boundaries come in through asynchronous copies, kStages rows
// ahead, into slots that only the copying thread reads.
// Should be bound by the bytes (X and dY read once, dX written once), and takes
// 166 us for 32768 x 4096 bf16, 4.9 TB/s, and 100 for 131072 x 768: the weights,
// the sums and the row take 120 registers, so 16 warps fit an SM and issue in
// half of its cycles, each row with a barrier in its middle.  More stages, fewer
// elements a lane and a shorter reduction of the two row sums all take the same
// time or more; pairs of elements in one instruction took it from 206 us to 175,
// and converting 16-bit values in pairs to 166.
// The longest rows (EPL = 32) leave no registers for the sums and the weights
// and no shared memory for the slots: their sums are in shared memory, and the
// second pass loads them again (from L2).  One such block fits an SM, and nothing
// is loaded ahead: 4096 x 16384 bf16 takes 232 us where the bytes need 61.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, int WPR, int EPL, bool FEW>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256, (WPR > 8 ? 1 : 2) + (EPL <= 8 ? 1 : 0))
    k_ln_bwd(const RowMap map, int rows_per_unit, const T* X, int64_t ldx, const T* dY, int64_t ldy,
             const float* gamma, const float* mean, const float* rstd, T* dX,
             int64_t ldd, int E, float* part, int* arrived, const GradPtrs G, int64_t off_gamma, int64_t off_beta,
             int accumulate) {
  constexpr int VL = Elem<T>::V;
  constexpr int CH = EPL / VL;                      // strips per warp
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;                  // rows per block at a time
  constexpr bool WIDE = EPL > 16;
  constexpr bool RING = VEC && !WIDE;
  constexpr int COLS = WPR * 32 * EPL;              // columns a row group covers
  extern __shared__ uint4 dyn[];                    // RING: [kStages][2][CH][threads]; then the sums:
  float* sums = reinterpret_cast<float*>(dyn);      // WIDE: [2][COLS]; RPB > 1, after the loop: [RPB][COLS]
  __shared__ float2 buf[2][WARPS];
  __shared__ float stat[kStages][WARPS][2];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % WPR, group = warp / WPR;
  const int m = worker_of(map.unit, map.M, blockIdx.x);
  const int first = map.start[m] + (blockIdx.x - map.unit[m]) * rows_per_unit;
  const int last = min(first + rows_per_unit, map.start[m + 1]);
  const float inv_E = 1.f / (float)E;
  auto base_of = [&](int c) { return (c * WPR + w) * 32 * VL; };
  auto fetch = [&](int r, int stage) {
    if (r < last) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = base_of(c) + lane * VL;
        const bool in = col < E;
        uint4* to = &dyn[(stage * 2 * CH + c) * (WARPS * 32) + threadIdx.x];
        copy16(to, X + (int64_t)r * ldx + (in ? col : 0), in);
        copy16(to + CH * WARPS * 32, dY + (int64_t)r * ldy + (in ? col : 0), in);
      }
      if (lane < 2) copy4(&stat[stage][warp][lane], (lane ? rstd : mean) + r);
    }
    copy_commit();
  };
  if (RING) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch(first + group + s * RPB, s);
  }
  // pairs of columns: the weights and the sums of this thread's columns
  constexpr int CK = WIDE ? 1 : CH;
  F2 ga[CK][VL / 2], ag[CK][VL / 2], ab[CK][VL / 2];
  auto load_gamma = [&](int c, F2* to) {
    float t[VL];
    strip_load_f32<T, VEC>(gamma, base_of(c), E, lane, t);
#pragma unroll
    for (int j = 0; j < VL / 2; ++j) to[j] = pack2(t[2 * j], t[2 * j + 1]);
  };
  if (WIDE) {
    for (int i = threadIdx.x; i < 2 * COLS; i += WARPS * 32) sums[i] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int c = 0; c < CK; ++c) {
      load_gamma(c, ga[c]);
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) ag[c][j] = ab[c][j] = 0ull;
    }
  }
  int stage = 0, parity = 0;
  for (int r = first + group; r < last; r += RPB) {
    const T* xr = X + (int64_t)r * ldx;
    const T* dr = dY + (int64_t)r * ldy;
    float mu, rs;
    if (RING) {
      copy_wait<kStages - 1>();
      const float own = lane < 2 ? stat[stage][warp][lane] : 0.f;
      mu = __shfl_sync(0xffffffffu, own, 0);
      rs = __shfl_sync(0xffffffffu, own, 1);
    } else {
      mu = mean[r];
      rs = rstd[r];
    }
    const F2 neg_mu = pack2(-mu, -mu), rs2 = pack2(rs, rs);
    // xh and rs * g of this thread's columns; both are 0 times what is kept
    // in columns beyond E, where dY and gamma were loaded as zeros
    F2 h[CK][VL / 2], g[CK][VL / 2];
    auto convert = [&](int c, F2* hc, F2* gc, F2* dc, const F2* gamma_c) {
      Pack<T> px, pd;
      if (RING) {
        const uint4* from = &dyn[(stage * 2 * CH + c) * (WARPS * 32) + threadIdx.x];
        px = *reinterpret_cast<const Pack<T>*>(from);
        pd = *reinterpret_cast<const Pack<T>*>(from + CH * WARPS * 32);
      } else {
        px = strip_raw<T, VEC>(xr, base_of(c), E, lane);
        pd = strip_raw<T, VEC>(dr, base_of(c), E, lane);
      }
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        dc[j] = up2(pd, j);
        hc[j] = mul2(add2(up2(px, j), neg_mu), rs2);
        gc[j] = mul2(dc[j], gamma_c[j]);
      }
    };
    F2 a1 = 0ull, a2 = 0ull;   // sums of g and g * xh
    if (!WIDE) {
#pragma unroll
      for (int c = 0; c < CK; ++c) {
        if (base_of(c) >= E) continue;
        F2 d[VL / 2];
        convert(c, h[c], g[c], d, ga[c]);
#pragma unroll
        for (int j = 0; j < VL / 2; ++j) {
          ag[c][j] = fma2(d[j], h[c][j], ag[c][j]);
          ab[c][j] = add2(d[j], ab[c][j]);
          a1 = add2(g[c][j], a1);
          a2 = fma2(g[c][j], h[c][j], a2);
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < CH; ++c) {
        if (base_of(c) >= E) continue;
        F2 d[VL / 2];
        load_gamma(c, ga[0]);
        convert(c, h[0], g[0], d, ga[0]);
#pragma unroll
        for (int j = 0; j < VL / 2; ++j) {
          const float2 p = unpack2(mul2(d[j], h[0][j])), q = unpack2(d[j]);
          const int c0 = strip_col<T, VEC>(base_of(c), lane, 2 * j), c1 = strip_col<T, VEC>(base_of(c), lane, 2 * j + 1);
          sums[c0] += p.x;
          sums[c1] += p.y;
          sums[COLS + c0] += q.x;
          sums[COLS + c1] += q.y;
          a1 = add2(g[0][j], a1);
          a2 = fma2(g[0][j], h[0][j], a2);
        }
      }
    }
    if (RING) {
      fetch(r + kStages * RPB, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    float s1 = warp_sum(sum2(a1)), s2 = warp_sum(sum2(a2));
    if (WPR > 1) {
      if (lane == 0) buf[parity][warp] = make_float2(s1, s2);
      group_sync<WPR, WARPS>(group);
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        const float2 t = buf[parity][group * WPR + i];
        s1 += t.x;
        s2 += t.y;
      }
      parity ^= 1;
    }
    const float k0 = -rs * (s1 * inv_E), k1 = -rs * (s2 * inv_E);
    const F2 k02 = pack2(k0, k0), k12 = pack2(k1, k1);
#pragma unroll(WIDE ? 1 : CH)
    for (int c = 0; c < CH; ++c) {
      if (base_of(c) >= E) continue;
      if (WIDE) {
        F2 d[VL / 2];
        load_gamma(c, ga[0]);
        convert(c, h[0], g[0], d, ga[0]);
      }
      float o[VL];
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        const float2 t = unpack2(fma2(k12, h[WIDE ? 0 : c][j], fma2(rs2, g[WIDE ? 0 : c][j], k02)));
        o[2 * j] = t.x;
        o[2 * j + 1] = t.y;
      }
      strip_store<T, VEC>(dX + (int64_t)r * ldd, base_of(c), E, lane, o);
    }
  }
  // the block's sums: row groups added up in order through shared memory
  float* out = part + (int64_t)blockIdx.x * 2 * E;
  if (WIDE) {
    __syncthreads();
    for (int col = threadIdx.x; col < E; col += WARPS * 32) {
      out[col] = sums[col];
      out[E + col] = sums[COLS + col];
    }
  }
  if (RING) copy_wait<0>();
  for (int which = 0; which < (WIDE ? 0 : 2); ++which) {
    if (RPB > 1) __syncthreads();
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float v[VL];
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) {
        const float2 t = unpack2(which ? ab[WIDE ? 0 : c][j] : ag[WIDE ? 0 : c][j]);
        v[2 * j] = t.x;
        v[2 * j + 1] = t.y;
      }
      if (RPB > 1) strip_store_f32<T, VEC>(sums + group * COLS, base_of(c), COLS, lane, v);
      else strip_store_f32<T, VEC>(out + which * E, base_of(c), E, lane, v);
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
  if (!FEW) return;
  // few blocks: the one of the worker that is done last adds up their sums
  __shared__ int is_last;
  const int units = map.unit[m + 1] - map.unit[m];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    is_last = atomicAdd(&arrived[m], 1) == units - 1;
    if (is_last) arrived[m] = 0;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  const float* from = part + (int64_t)map.unit[m] * 2 * E;
  for (int which = 0; which < (off_beta >= 0 ? 2 : 1); ++which) {
    float* g = G.p[m] + (which ? off_beta : off_gamma);
    for (int col = threadIdx.x; col < E; col += WARPS * 32) {
      float t = 0.f;
#pragma unroll 4
      for (int u = 0; u < units; ++u) t += __ldcg(from + ((int64_t)u * 2 + which) * E + col);
      g[col] = accumulate ? g[col] + t : t;
    }
  }
}

// G[m] (+)= the sum of worker m's blocks, in order: 32 columns a block, 8
// threads a column, each over a fixed share of the blocks
__global__ void __launch_bounds__(256) k_ln_weights(const RowMap map, const GradPtrs G, const float* part,
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
#pragma unroll 4
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

// Where every worker has at most kFewRows rows they go in at most kFewUnits
// units, and the sums over those are made in the same launch (by one block,
// while the separate kernel takes E / 32): that saves a launch.
constexpr int kFewUnits = 16, kFewRows = 128;

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, bool VEC, int WPR, int EPL, bool FEW>
void run_units(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  constexpr int WARPS = WPR > 8 ? WPR : 8;
  constexpr int RPB = WARPS / WPR;
  constexpr int COLS = WPR * 32 * EPL;
  constexpr bool WIDE = EPL > 16;
  const size_t ring = VEC && !WIDE ? (size_t)kStages * 2 * (EPL / Elem<T>::V) * WARPS * 32 * 16 : 0;
  const size_t sums = WIDE ? (size_t)2 * COLS * 4 : (RPB > 1 ? (size_t)RPB * COLS * 4 : 0);
  const size_t smem = ring > sums ? ring : sums;
  auto* kernel = k_ln_bwd<T, VEC, WPR, EPL, FEW>;
  if (smem > 32 * 1024) allow_shared((const void*)kernel);
  const int N = start[M];
  // one wave of blocks; every worker's rows split into units of equal length
  int64_t want = (int64_t)num_sms() * resident_per_sm((const void*)kernel, WARPS * 32, smem);
  if (want > a.max_blocks - M) want = a.max_blocks - M;
  if (want < 1) want = 1;
  int64_t per = (N + want - 1) / want;
  if (FEW) {
    int longest = 0;
    for (int m = 0; m < M; ++m) longest = longest > start[m + 1] - start[m] ? longest : start[m + 1] - start[m];
    const int64_t least = (longest + kFewUnits - 1) / kFewUnits;
    if (per < least) per = least;
  }
  per = (per + RPB - 1) / RPB * RPB;
  if (per < RPB) per = RPB;
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  for (int m = 0; m < M; ++m) {
    const int units = (int)((start[m + 1] - start[m] + per - 1) / per);
    map.unit[m + 1] = map.unit[m] + (FEW && units == 0 ? 1 : units);   // (FEW: one that writes the zeros)
  }
  if (map.unit[M] > 0) {
    count_launch();
    launch_pdl(kernel, dim3(map.unit[M]), dim3(WARPS * 32), smem, s, map, (int)per, reinterpret_cast<const T*>(a.X),
               a.ldx, reinterpret_cast<const T*>(a.dY), a.ldy, a.gamma, a.mean, a.rstd, reinterpret_cast<T*>(a.dX),
               a.ldd, (int)a.E, a.part, a.arrived, G, a.off_gamma, a.off_beta, a.accumulate);
  }
  if (FEW) return;
  count_launch();
  launch_pdl(k_ln_weights, dim3((unsigned)((a.E + 31) / 32), M, a.off_beta >= 0 ? 2 : 1), dim3(256), 0, s, map, G,
             (const float*)a.part, (int)a.E, a.off_gamma, a.off_beta, a.accumulate);
}

template <typename T, bool VEC, int WPR, int EPL>
void run_bwd(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  bool few = true;
  for (int m = 0; m < M; ++m) few = few && start[m + 1] - start[m] <= kFewRows;
  if (few) run_units<T, VEC, WPR, EPL, true>(s, a, start, M, G);
  else run_units<T, VEC, WPR, EPL, false>(s, a, start, M, G);
}

// The fewest warps that hold a row at 16 elements a lane; without the
// asynchronous copies at 8, which lets a third block wait on its loads too
// (30000 x 1001 fp32 86 us instead of 107, 8000 x 4001 bf16 68 instead of 80;
// with the copies 32768 x 4096 bf16 takes 226 us at 8 and 166 at 16).  Above
// 16 warps at 16, 32.
template <typename T, bool VEC>
void pick_bwd(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  constexpr int MORE = VEC ? 1 : 2, EPL = 16 / MORE;
  if (a.E <= 256) run_bwd<T, VEC, 1, 8>(s, a, start, M, G);
  else if (a.E <= 512) run_bwd<T, VEC, MORE, EPL>(s, a, start, M, G);
  else if (a.E <= 1024) run_bwd<T, VEC, 2 * MORE, EPL>(s, a, start, M, G);
  else if (a.E <= 2048) run_bwd<T, VEC, 4 * MORE, EPL>(s, a, start, M, G);
  else if (a.E <= 4096) run_bwd<T, VEC, 8 * MORE, EPL>(s, a, start, M, G);
  else if (a.E <= 8192) run_bwd<T, VEC, 16, 16>(s, a, start, M, G);
  else run_bwd<T, VEC, 16, 32>(s, a, start, M, G);
}

}  // namespace

void launch_layernorm_grad(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G) {
  const int vl = a.type == LT_F32 ? 4 : 8;
  const bool vec = a.E % vl == 0 && a.ldx % vl == 0 && a.ldy % vl == 0 && a.ldd % vl == 0 && on16(a.X) && on16(a.dY) &&
                   on16(a.dX) && on16(a.gamma);
#define SM_RUN(T) (vec ? pick_bwd<T, true>(s, a, start, M, G) : pick_bwd<T, false>(s, a, start, M, G))
  if (a.type == LT_F32) SM_RUN(float);
  else if (a.type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

}  // namespace sm
