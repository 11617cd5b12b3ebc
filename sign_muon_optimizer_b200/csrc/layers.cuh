// layers.cuh -- device helpers and launch wrappers of the layer calls
// (include/signmuon_layers.h): element types, 16-byte strips, the map from
// work units to workers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace sm {

enum LayerType { LT_F32 = 0, LT_BF16 = 1, LT_F16 = 2 };

// Rows of each worker, and work units (tiles of rows) that never cross a
// worker: worker m has rows [start[m], start[m+1]) and units [unit[m],
// unit[m+1]).  Passed by value (constant bank).
struct RowMap {
  int M;
  int start[kMaxWorkers + 1];
  int unit[kMaxWorkers + 1];
};

struct GradPtrs {     // per-worker gradient vectors, passed by value
  float* p[kMaxWorkers];
};

#ifdef __CUDACC__
// The kernels' read-only pointers are not __restrict__: of such a pointer the
// compiler may read what it likes as early as it likes, before griddep_wait too,
// when the kernel before this one is still writing it.

// the m with pre[m] <= i < pre[m+1] (pre ascending, pre[0] = 0, i < pre[M])
__device__ __forceinline__ int worker_of(const int* pre, int M, int i) {
  int lo = 0, hi = M - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr int V = 4;   // elements in 16 bytes
  static constexpr bool kHalf = false;
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr int V = 8;
  static constexpr bool kHalf = false;
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
  static constexpr int V = 8;
  static constexpr bool kHalf = true;
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};

template <typename T>
struct alignas(16) Pack {
  T v[Elem<T>::V];
};

// Pairs of fp32 operations in one instruction: the kernels over rows are bound
// by the instructions they issue as much as by the bytes.
typedef unsigned long long F2;
__device__ __forceinline__ F2 pack2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  const float2 f = unpack2(a);
  return f.x + f.y;
}

// elements 2j and 2j + 1 of a pack as floats, and back
__device__ __forceinline__ F2 up2(const Pack<float>& p, int j) { return pack2(p.v[2 * j], p.v[2 * j + 1]); }
__device__ __forceinline__ F2 up2(const Pack<__nv_bfloat16>& p, int j) {
  const unsigned u = reinterpret_cast<const unsigned*>(p.v)[j];
  return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ F2 up2(const Pack<__half>& p, int j) {
  const float2 f = __half22float2(reinterpret_cast<const __half2*>(p.v)[j]);
  return pack2(f.x, f.y);
}
__device__ __forceinline__ void down2(Pack<float>& p, int j, float x, float y) {
  p.v[2 * j] = x;
  p.v[2 * j + 1] = y;
}
__device__ __forceinline__ void down2(Pack<__nv_bfloat16>& p, int j, float x, float y) {
  reinterpret_cast<__nv_bfloat162*>(p.v)[j] = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void down2(Pack<__half>& p, int j, float x, float y) {
  reinterpret_cast<__half2*>(p.v)[j] = __floats2half2_rn(x, y);
}

// A strip is what a warp's 32 lanes hold of a row in one step: 32 * V
// elements.  With VEC a lane holds V neighbours (one 16-byte access; the row
// starts on 16 bytes and its length is a multiple of V), else element j of the
// lane is column j * 32 + lane of the strip.
template <typename T, bool VEC>
__device__ __forceinline__ int strip_col(int base, int lane, int j) {
  constexpr int V = Elem<T>::V;
  return VEC ? base + lane * V + j : base + j * 32 + lane;
}

// x[j] = row[col], 0 beyond `cols`
template <typename T, bool VEC>
__device__ __forceinline__ void strip_load(const T* __restrict__ row, int base, int cols, int lane, float* x) {
  constexpr int V = Elem<T>::V;
  if (VEC) {
    const int c = base + lane * V;
    Pack<T> p;
    if (c < cols) p = *reinterpret_cast<const Pack<T>*>(row + c);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = c < cols ? Elem<T>::up(p.v[j]) : 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = base + j * 32 + lane;
      x[j] = c < cols ? Elem<T>::up(row[c]) : 0.f;
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void strip_store(T* __restrict__ row, int base, int cols, int lane, const float* x) {
  constexpr int V = Elem<T>::V;
  if (VEC) {
    const int c = base + lane * V;
    if (c < cols) {
      Pack<T> p;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) down2(p, j, x[2 * j], x[2 * j + 1]);
      *reinterpret_cast<Pack<T>*>(row + c) = p;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = base + j * 32 + lane;
      if (c < cols) row[c] = Elem<T>::down(x[j]);
    }
  }
}

// the strip as it lies in memory (zeros beyond `cols`), to be converted later:
// half the registers of the values for 16-bit types
template <typename T, bool VEC>
__device__ __forceinline__ Pack<T> strip_raw(const T* __restrict__ row, int base, int cols, int lane) {
  constexpr int V = Elem<T>::V;
  Pack<T> p;
  if (VEC) {
    const int c = base + lane * V;
    if (c < cols) {
      p = *reinterpret_cast<const Pack<T>*>(row + c);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) p.v[j] = Elem<T>::down(0.f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = base + j * 32 + lane;
      p.v[j] = c < cols ? row[c] : Elem<T>::down(0.f);
    }
  }
  return p;
}

// the fp32 companion of a T strip (a weight, a sum): same columns
template <typename T, bool VEC>
__device__ __forceinline__ void strip_load_f32(const float* row, int base, int cols, int lane, float* x) {
  constexpr int V = Elem<T>::V;
  if (VEC) {
    const int c = base + lane * V;
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 f = c < cols ? *reinterpret_cast<const float4*>(row + c + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[j] = f.x; x[j + 1] = f.y; x[j + 2] = f.z; x[j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = base + j * 32 + lane;
      x[j] = c < cols ? row[c] : 0.f;
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void strip_store_f32(float* row, int base, int cols, int lane, const float* x) {
  constexpr int V = Elem<T>::V;
  if (VEC) {
    const int c = base + lane * V;
    if (c < cols) {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        *reinterpret_cast<float4*>(row + c + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = base + j * 32 + lane;
      if (c < cols) row[c] = x[j];
    }
  }
}

// 2^x, below 2^-126 zero
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Asynchronous copies of 16 bytes that only the copying thread reads back:
// waiting for its own groups is enough, no barrier.  live = false: zeros.
__device__ __forceinline__ void copy16(void* to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// barrier of the WPR warps that hold a row (group: their number in the block)
template <int WPR, int WARPS>
__device__ __forceinline__ void group_sync(int group) {
  if (WPR == 1) __syncwarp();
  else if (WPR == WARPS) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(WPR * 32) : "memory");
}

__device__ __forceinline__ int64_t load_id(const void* ids, int i64, int64_t i) {
  return i64 ? reinterpret_cast<const int64_t*>(ids)[i] : (int64_t)reinterpret_cast<const int32_t*>(ids)[i];
}
#endif  // __CUDACC__

// ---- launch wrappers (host) ------------------------------------------------
// Lets a kernel be launched with all the dynamic shared memory that its static
// part leaves, on the current device: what launches of more than 32 KB need.  The
// limit belongs to the kernel, for every handle and host thread, so it is set
// once and to the most: lowered to one launch's size it would refuse another
// thread's larger one.
void allow_shared(const void* kernel);

constexpr int kSortTile = 2048;   // tokens of a worker that one block sorts
constexpr int kRadixTile = 2048;  // ... and that a block of the radix sort takes
constexpr int kRadixBins = 512, kRadixSets = 4;
// Sorted tokens that a warp of the table gradient's reduction takes (a unit is
// eight warps'): 32, or where that leaves an SM fewer than about three blocks, 8 --
// 8192 tokens of 8 x 50304 x 768, bf16, 179 us instead of 196, 32768 204 instead
// of 210; 65536 tokens of 64 columns 35 instead of 32, for the longer join.
constexpr int kFewBlocks = 400;
inline int embed_per_warp(int64_t rows, int64_t cols, int type) {
  const int64_t strip = type == LT_F32 ? 128 : 256;
  return rows / 256 * ((cols + strip - 1) / strip) <= kFewBlocks ? 8 : 32;
}

void launch_embed(cudaStream_t s, const float* table, int64_t V, int64_t E, const void* ids, int id64, int64_t n,
                  float scale, void* out, int type, int64_t ld, int* status);
struct EmbedGradArgs {
  const void* ids;
  int id64;
  int64_t V, E;
  float scale;
  const void* dY;
  int type;
  int64_t ld;
  int64_t off;                 // the table's place in G[m]
  int accumulate;
  unsigned long long* keys[2]; // workspace: one (id, row) key per row, twice
  int* counts;                 // workspace: kRadixSets sets of kRadixBins counts per radix tile
  int64_t count_set;           // ints in a set
  float* part;                 // workspace: 2 x E floats per unit of 8 * embed_per_warp tokens
  int* status;
};
void launch_embed_grad(cudaStream_t s, const EmbedGradArgs& a, const int* start, int M, const GradPtrs& G);

void launch_layernorm(cudaStream_t s, const float* gamma, const float* beta, int64_t n, int64_t E, const void* X,
                      int64_t ldx, void* Y, int64_t ldy, int type, float eps, float* mean, float* rstd);
struct NormGradArgs {
  const float* gamma;
  int64_t E;
  const void* X;
  int64_t ldx;
  const void* dY;
  int64_t ldy;
  const float* mean;
  const float* rstd;
  void* dX;
  int64_t ldd;
  int type;
  int64_t off_gamma, off_beta; // off_beta < 0: none
  int accumulate;
  int* arrived;                // workspace: M counters, zero between calls
  float* part;                 // workspace: 2 x E floats per block
  int max_blocks;              // blocks that part has room for, at least M
};
void launch_layernorm_grad(cudaStream_t s, const NormGradArgs& a, const int* start, int M, const GradPtrs& G);

struct DistillArgs {
  const void* Z;
  int type;
  int64_t ldz, V;
  const void* idx;
  int id64;
  const void* t;
  int t_type;
  int64_t ldt;
  int K;
  float temperature, gscale;
  float* loss;
  int32_t* count_out;
  float* row_loss;             // the caller's, or workspace
  void* dZ;
  int64_t ldd;
  int* count;                  // workspace: twice kMaxWorkers counters, zero between calls
  void* scratch;               // workspace: 12 bytes per row
  int* status;
};
void launch_distill(cudaStream_t s, const DistillArgs& a, const int* start, int M);

}  // namespace sm
