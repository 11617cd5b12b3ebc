// layers_embed.cu -- embedding lookup with scaling, and its gradient per
// worker by sorted tokens.
#include <climits>

#include "layers.cuh"

namespace sm {
namespace {

// ---------------------------------------------------------------------------
// Lookup: out[r] = fl(scale * table[ids[r]]).  Bound by the bytes: N * E
// elements written, one 4 * E-byte table row read per token (from L2 where
// tokens repeat).  One warp per (row, slab of kSlab columns).
// ---------------------------------------------------------------------------
constexpr int kSlab = 1024;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed(const float* __restrict__ table, int64_t V, int E,
                                               const void* __restrict__ ids, int id64, int64_t n, int n_slab,
                                               float scale, T* __restrict__ out, int64_t ld, int* status) {
  griddep_wait();
  griddep_launch();
  constexpr int VL = Elem<T>::V;
  const int lane = threadIdx.x & 31;
  const int64_t units = n * n_slab;
  const int64_t step = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t r = u / n_slab;
    const int c0 = (int)(u - r * n_slab) * kSlab;
    const int c1 = min(E, c0 + kSlab);
    const int64_t id = load_id(ids, id64, r);
    if (id >= V && lane == 0) *status = 1;
    const bool real = id >= 0 && id < V;
    const float* src = table + (real ? id : 0) * E;
    T* dst = out + r * ld;
    for (int c = c0; c < c1; c += 32 * VL) {
      float x[VL];
      if (real) {
        strip_load_f32<T, VEC>(src, c, c1, lane, x);
#pragma unroll
        for (int j = 0; j < VL; ++j) x[j] *= scale;
      } else {
#pragma unroll
        for (int j = 0; j < VL; ++j) x[j] = 0.f;
      }
      strip_store<T, VEC>(dst, c, c1, lane, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient: G[m][v] = scale * sum of dY[r] over worker m's tokens v.
//
// The tokens of each worker are sorted by (id, row): tiles of kSortTile in
// shared memory, then 16-way merges by rank (every key is unique, so a key's
// place in the merge is its own index plus its lower bounds in the other
// runs).  A warp then takes kEmbTile = 32 sorted tokens of one worker, one key
// per lane, and adds up their dY rows in registers; a run of equal ids that
// lies inside the unit is written to G, the parts of a run that crosses units
// go to the workspace and are added up in order afterwards.  Work per unit
// does not depend on how often a token occurs.
// Absent tokens (id < 0, id >= V) get the key UINT_MAX and sort to the end.
// ---------------------------------------------------------------------------
typedef unsigned long long Key;  // id in the upper 32 bits, row in the lower

__device__ __forceinline__ unsigned key_id(Key k) { return (unsigned)(k >> 32); }
constexpr unsigned kAbsent = 0xffffffffu;

// one block per unit of `map` (kSortTile rows of one worker): bitonic sort
__global__ void __launch_bounds__(1024) k_sort_tiles(const RowMap map, const void* __restrict__ ids, int id64,
                                                     int64_t V, Key* __restrict__ keys, int* status) {
  __shared__ Key k[kSortTile];
  griddep_wait();
  griddep_launch();
  const int u = blockIdx.x;
  const int m = worker_of(map.unit, map.M, u);
  const int r0 = map.start[m] + (u - map.unit[m]) * kSortTile;
  const int n = min(kSortTile, map.start[m + 1] - r0);
  for (int i = threadIdx.x; i < kSortTile; i += 1024) {
    Key key = ~0ull;
    if (i < n) {
      const int64_t id = load_id(ids, id64, r0 + i);
      if (id >= V) *status = 1;
      const unsigned w = (id >= 0 && id < V) ? (unsigned)id : kAbsent;
      key = ((Key)w << 32) | (unsigned)(r0 + i);
    }
    k[i] = key;
  }
  int top = 2;  // sort no more than the next power of two
  while (top < n) top <<= 1;
  for (int size = 2; size <= top; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      const int i = threadIdx.x;
      const int lo = 2 * i - (i & (stride - 1));
      if (lo + stride < top) {
        const bool up = (lo & size) == 0;
        const Key a = k[lo], b = k[lo + stride];
        if ((a > b) == up) {
          k[lo] = b;
          k[lo + stride] = a;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) keys[r0 + i] = k[i];
}

// one 16-way merge of sorted runs of `run` keys (a thread per key)
__global__ void __launch_bounds__(256) k_merge(const RowMap map, int64_t run, const Key* __restrict__ src,
                                               Key* __restrict__ dst) {
  griddep_wait();
  griddep_launch();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= map.start[map.M]) return;
  const int m = worker_of(map.start, map.M, i);
  const int base = map.start[m], n = map.start[m + 1] - base;
  const int at = i - base;
  const int64_t g0 = at / (16 * run) * (16 * run);
  const int64_t mine = at / run;
  const Key key = src[i];
  int64_t rank = at - mine * run;
  for (int64_t q = g0; q < g0 + 16 * run && q < n; q += run) {
    if (q == mine * run) continue;
    const Key* p = src + base + q;
    int lo = 0, hi = (int)(run < n - q ? run : n - q);  // keys of the run below `key`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p[mid] < key) lo = mid + 1;
      else hi = mid;
    }
    rank += lo;
  }
  dst[base + g0 + rank] = key;
}

// zero the tables' gradients (before the rows with tokens are written)
__global__ void __launch_bounds__(256) k_zero_tables(const GradPtrs G, int64_t off, int64_t n) {
  griddep_wait();
  griddep_launch();
  float* g = G.p[blockIdx.y] + off;
  const int64_t head = min(n, (int64_t)((4 - (off & 3)) & 3));
  const int64_t t0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const int64_t n4 = (n - head) / 4;
  float4* g4 = reinterpret_cast<float4*>(g + head);
  for (int64_t i = t0; i < n4; i += step) g4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t0 < head) g[t0] = 0.f;
  const int64_t tail = head + 4 * n4 + t0;
  if (tail < n) g[tail] = 0.f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void emit(float* row, int c, int E, int lane, const float* acc, float scale, int accumulate) {
  constexpr int VL = Elem<T>::V;
  float x[VL];
  if (accumulate) {
    strip_load_f32<T, VEC>(row, c, E, lane, x);
#pragma unroll
    for (int j = 0; j < VL; ++j) x[j] = fmaf(scale, acc[j], x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VL; ++j) x[j] = scale * acc[j];
  }
  strip_store_f32<T, VEC>(row, c, E, lane, x);
}

// a warp per (unit of 32 sorted tokens, strip of columns)
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed_reduce(const RowMap map, const GradPtrs G, const Key* __restrict__ keys,
                                                      const T* __restrict__ dY, int64_t ld, int E, int n_strip,
                                                      int64_t off, float scale, int accumulate,
                                                      float* __restrict__ part) {
  constexpr int VL = Elem<T>::V;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int u = (int)(w / n_strip);
  if (u >= map.unit[map.M]) return;
  const int c = (int)(w - (int64_t)u * n_strip) * 32 * VL;
  const int m = worker_of(map.unit, map.M, u);
  const int i0 = map.start[m] + (u - map.unit[m]) * kEmbTile;
  const int n = min(kEmbTile, map.start[m + 1] - i0);
  const Key key = lane < n ? keys[i0 + lane] : ~0ull;
  const unsigned id = key_id(key);
  if (__shfl_sync(0xffffffffu, id, 0) == kAbsent) return;
  // the ids beside the unit, to tell whether its first and last run cross it
  const unsigned before = i0 > map.start[m] ? key_id(keys[i0 - 1]) : kAbsent;
  const unsigned after = i0 + n < map.start[m + 1] ? key_id(keys[i0 + n]) : kAbsent;
  float* gm = G.p[m] + off;
  float acc[VL];
#pragma unroll
  for (int j = 0; j < VL; ++j) acc[j] = 0.f;
  bool head = true;
  for (int i = 0; i < n; ++i) {
    const unsigned v = __shfl_sync(0xffffffffu, id, i);
    if (v == kAbsent) break;
    const unsigned r = __shfl_sync(0xffffffffu, (unsigned)key, i);
    float x[VL];
    strip_load<T, VEC>(dY + (int64_t)r * ld, c, E, lane, x);
#pragma unroll
    for (int j = 0; j < VL; ++j) acc[j] += x[j];
    const unsigned next = i + 1 < n ? __shfl_sync(0xffffffffu, id, i + 1) : after;
    if (i + 1 < n ? next != v : true) {
      const bool from_before = head && before == v;
      const bool goes_on = i + 1 == n && after == v;
      if (from_before) strip_store_f32<T, VEC>(part + (int64_t)u * 2 * E, c, E, lane, acc);
      else if (goes_on) strip_store_f32<T, VEC>(part + ((int64_t)u * 2 + 1) * E, c, E, lane, acc);
      else emit<T, VEC>(gm + (int64_t)v * E, c, E, lane, acc, scale, accumulate);
      head = false;
#pragma unroll
      for (int j = 0; j < VL; ++j) acc[j] = 0.f;
    }
  }
}

// a warp per (unit, strip): where a run starts in the unit and goes on, its
// parts are added up in order and written
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed_join(const RowMap map, const GradPtrs G, const Key* __restrict__ keys,
                                                    int E, int n_strip, int64_t off, float scale, int accumulate,
                                                    const float* __restrict__ part) {
  constexpr int VL = Elem<T>::V;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int u = (int)(w / n_strip);
  if (u >= map.unit[map.M]) return;
  const int c = (int)(w - (int64_t)u * n_strip) * 32 * VL;
  const int m = worker_of(map.unit, map.M, u);
  const int s0 = map.start[m], s1 = map.start[m + 1];
  const int i0 = s0 + (u - map.unit[m]) * kEmbTile;
  if (i0 + kEmbTile >= s1) return;
  const unsigned v = key_id(keys[i0 + kEmbTile - 1]);
  if (v == kAbsent || key_id(keys[i0 + kEmbTile]) != v) return;
  if (i0 > s0 && key_id(keys[i0]) == v && key_id(keys[i0 - 1]) == v) return;  // the run starts further left
  float acc[VL];
  strip_load_f32<T, VEC>(part + ((int64_t)u * 2 + 1) * E, c, E, lane, acc);
  int k = u + 1;
  for (int i = i0 + kEmbTile;; i += kEmbTile, ++k) {
    float x[VL];
    strip_load_f32<T, VEC>(part + (int64_t)k * 2 * E, c, E, lane, x);
#pragma unroll
    for (int j = 0; j < VL; ++j) acc[j] += x[j];
    // on as long as the run fills this unit and enters the next
    if (i + kEmbTile >= s1 || key_id(keys[i + kEmbTile - 1]) != v || key_id(keys[i + kEmbTile]) != v) break;
  }
  emit<T, VEC>(G.p[m] + off + (int64_t)v * E, c, E, lane, acc, scale, accumulate);
}

template <typename T, bool VEC>
void run_embed(cudaStream_t s, const float* table, int64_t V, int64_t E, const void* ids, int id64, int64_t n,
               float scale, void* out, int64_t ld, int* status) {
  const int n_slab = (int)((E + kSlab - 1) / kSlab);
  const int grid = stream_grid((const void*)k_embed<T, VEC>, 256, 0, (n * n_slab + 7) / 8, 8);
  count_launch();
  launch_pdl(k_embed<T, VEC>, dim3(grid), dim3(256), 0, s, table, V, (int)E, ids, id64, n, n_slab, scale,
             reinterpret_cast<T*>(out), ld, status);
}

template <typename T, bool VEC>
void run_embed_reduce(cudaStream_t s, const EmbedGradArgs& a, const RowMap& map, const GradPtrs& G, const Key* keys) {
  const int n_strip = (int)((a.E + 32 * Elem<T>::V - 1) / (32 * Elem<T>::V));
  const int64_t warps = (int64_t)map.unit[map.M] * n_strip;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  count_launch();
  launch_pdl(k_embed_reduce<T, VEC>, dim3(grid), dim3(256), 0, s, map, G, keys, reinterpret_cast<const T*>(a.dY), a.ld,
             (int)a.E, n_strip, a.off, a.scale, a.accumulate, a.part);
  count_launch();
  launch_pdl(k_embed_join<T, VEC>, dim3(grid), dim3(256), 0, s, map, G, keys, (int)a.E, n_strip, a.off, a.scale,
             a.accumulate, (const float*)a.part);
}

RowMap make_map(const int* start, int M, int tile) {
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  for (int m = 0; m < M; ++m) map.unit[m + 1] = map.unit[m] + (int)(((int64_t)start[m + 1] - start[m] + tile - 1) / tile);
  return map;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

void launch_embed(cudaStream_t s, const float* table, int64_t V, int64_t E, const void* ids, int id64, int64_t n,
                  float scale, void* out, int type, int64_t ld, int* status) {
  if (n == 0) return;
  const int vl = type == LT_F32 ? 4 : 8;
  const bool vec = E % vl == 0 && ld % vl == 0 && on16(table) && on16(out);
#define SM_RUN(T)                                                                                      \
  (vec ? run_embed<T, true>(s, table, V, E, ids, id64, n, scale, out, ld, status)                      \
       : run_embed<T, false>(s, table, V, E, ids, id64, n, scale, out, ld, status))
  if (type == LT_F32) SM_RUN(float);
  else if (type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

void launch_embed_grad(cudaStream_t s, const EmbedGradArgs& a, const int* start, int M, const GradPtrs& G) {
  if (!a.accumulate) {
    const int64_t n = a.V * a.E;
    const int64_t blocks = (n / 4 + 255) / 256 + 1;
    count_launch();
    launch_pdl(k_zero_tables, dim3((unsigned)(blocks < 1024 ? blocks : 1024), M), dim3(256), 0, s, G, a.off, n);
  }
  const int N = start[M];
  if (N == 0) return;
  const RowMap sort_map = make_map(start, M, kSortTile);
  count_launch();
  launch_pdl(k_sort_tiles, dim3(sort_map.unit[M]), dim3(1024), 0, s, sort_map, a.ids, a.id64, a.V, a.keys[0], a.status);
  int64_t longest = 0;
  for (int m = 0; m < M; ++m) longest = longest > start[m + 1] - start[m] ? longest : start[m + 1] - start[m];
  int at = 0;
  for (int64_t run = kSortTile; run < longest; run *= 16, at ^= 1) {
    count_launch();
    launch_pdl(k_merge, dim3((unsigned)((N + 255LL) / 256)), dim3(256), 0, s, sort_map, run, (const Key*)a.keys[at],
               a.keys[at ^ 1]);
  }
  const RowMap map = make_map(start, M, kEmbTile);
  const int vl = a.type == LT_F32 ? 4 : 8;
  bool vec = a.E % vl == 0 && a.ld % vl == 0 && a.off % 4 == 0 && on16(a.dY);
#define SM_RUN(T) (vec ? run_embed_reduce<T, true>(s, a, map, G, a.keys[at]) : run_embed_reduce<T, false>(s, a, map, G, a.keys[at]))
  if (a.type == LT_F32) SM_RUN(float);
  else if (a.type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

}  // namespace sm
