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
// Gradient: G[m][v] = scale * sum of dY[r] over worker m's tokens v.  Bound by
// the bytes: dY read once, M dense tables written once.
//
// The tokens of each worker are sorted by (id, row): tiles of kSortTile in
// shared memory, then 16-way merges by rank (every key is unique, so a key's
// place in the merge is its own index plus its lower bounds in the other
// runs).  The tables are zeroed by further blocks of the same launches, which
// hides the sort behind those bytes.  A block then takes kEmbUnit = 256 sorted
// tokens of one worker and a strip of columns, a warp 32 of them, one key per
// lane, and adds up their dY rows in registers; parts of a run of equal ids are
// added up in order across the warps through shared memory, and where it goes
// on in other blocks by k_embed_join.  Work per block does not depend on how
// often a token occurs, and every sum has a fixed order.
// Absent tokens (id < 0, id >= V) get the id kAbsent and sort to the end.
// ---------------------------------------------------------------------------
typedef unsigned long long Key;  // id in the upper 32 bits, row in the lower

__device__ __forceinline__ unsigned key_id(Key k) { return (unsigned)(k >> 32); }
constexpr unsigned kAbsent = 0xffffffffu;

// A share of zeroing n floats at G[m] + off, m < M, by `blocks` blocks of 1024
// threads: block b of them, of share [from, to) in 1/1024ths of each table.
struct ZeroShare {
  int64_t off, n;
  int M, blocks, from, to;
};

__device__ __forceinline__ void zero_tables(const GradPtrs& G, const ZeroShare& z, int b) {
  const int per_table = z.blocks / z.M;    // (blocks is a multiple of M)
  const int m = b / per_table;
  float* g = G.p[m] + z.off;
  const int64_t head = min(z.n, (int64_t)((4 - (z.off & 3)) & 3));   // to the first 16-byte boundary
  const int64_t n4 = (z.n - head) / 4;
  const int64_t lo = n4 * z.from / 1024, hi = n4 * z.to / 1024;
  float4* g4 = reinterpret_cast<float4*>(g + head);
  const int64_t t = (int64_t)(b - m * per_table) * blockDim.x + threadIdx.x, step = (int64_t)per_table * blockDim.x;
  for (int64_t i = lo + t; i < hi; i += step) g4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (z.from == 0 && t < head) g[t] = 0.f;
  if (z.to == 1024 && head + 4 * n4 + t < z.n) g[head + 4 * n4 + t] = 0.f;
}

// a block per unit of `map` (kSortTile rows of one worker): bitonic sort; the
// blocks behind them zero the tables
__global__ void __launch_bounds__(1024, 1) k_sort_tiles(const RowMap map, const void* __restrict__ ids, int id64,
                                                     int64_t V, Key* __restrict__ keys, int* status, const GradPtrs G,
                                                     const ZeroShare zero) {
  __shared__ Key k[kSortTile];
  griddep_wait();
  griddep_launch();
  const int u = blockIdx.x;
  if (u >= map.unit[map.M]) {
    zero_tables(G, zero, u - map.unit[map.M]);
    return;
  }
  const int m = worker_of(map.unit, map.M, u);
  const int r0 = map.start[m] + (u - map.unit[m]) * kSortTile;
  const int n = min(kSortTile, map.start[m + 1] - r0);
  int top = 2;  // the power of two that is sorted
  while (top < n) top <<= 1;
  for (int i = threadIdx.x; i < top; i += 1024) {
    Key key = ~0ull;
    if (i < n) {
      const int64_t id = load_id(ids, id64, r0 + i);
      if (id >= V) *status = 1;
      const unsigned w = (id >= 0 && id < V) ? (unsigned)id : kAbsent;
      key = ((Key)w << 32) | (unsigned)(r0 + i);
    }
    k[i] = key;
  }
  __syncthreads();
  const int i = threadIdx.x;
  for (int size = 2; size <= top; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      // pairs at strides up to 32 stay within the 64 keys of a warp
      if (stride >= 32) __syncthreads();
      else __syncwarp();
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
  for (int j = threadIdx.x; j < n; j += 1024) keys[r0 + j] = k[j];
}

// one 16-way merge of sorted runs of `run` keys (a thread per key); the blocks
// behind them zero the tables
__global__ void __launch_bounds__(1024, 1) k_merge(const RowMap map, int64_t run, const Key* __restrict__ src,
                                                Key* __restrict__ dst, const GradPtrs G, const ZeroShare zero) {
  griddep_wait();
  griddep_launch();
  const int n_all = map.start[map.M], mine_blocks = (n_all + 1023) / 1024;
  if ((int)blockIdx.x >= mine_blocks) {
    zero_tables(G, zero, blockIdx.x - mine_blocks);
    return;
  }
  const int i = blockIdx.x * 1024 + threadIdx.x;
  if (i >= n_all) return;
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

// zero alone (no tokens at all)
__global__ void __launch_bounds__(1024) k_zero_tables(const GradPtrs G, const ZeroShare zero) {
  griddep_wait();
  griddep_launch();
  zero_tables(G, zero, blockIdx.x);
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

// a block per (unit of 256 sorted tokens, strip of columns)
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed_reduce(const RowMap map, const GradPtrs G, const Key* __restrict__ keys,
                                                      const T* __restrict__ dY, int64_t ld, int E, int n_strip,
                                                      int64_t off, float scale, int accumulate,
                                                      float* __restrict__ part) {
  constexpr int VL = Elem<T>::V;
  constexpr int AHEAD = 8;                        // rows loaded before the first is added
  __shared__ float head[8][VL][32], tail[8][VL][32];  // a warp's part of a run from before, and of one that goes on
  __shared__ unsigned first_id[9];                // of each warp; [8]: of the unit behind
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int u = blockIdx.x / n_strip;
  const int c = (blockIdx.x - u * n_strip) * 32 * VL;
  const int m = worker_of(map.unit, map.M, u);
  const int s0 = map.start[m], s1 = map.start[m + 1];
  const int i0 = s0 + (u - map.unit[m]) * kEmbUnit + w * 32;
  const int n = max(0, min(32, s1 - i0));
  const Key key = lane < n ? keys[i0 + lane] : ~0ull;
  const unsigned id = key_id(key);
  const unsigned before = n > 0 && i0 > s0 ? key_id(keys[i0 - 1]) : kAbsent;
  const unsigned after = n == 32 && i0 + 32 < s1 ? key_id(keys[i0 + 32]) : kAbsent;
  if (lane == 0) first_id[w] = id;
  if (w == 7 && lane == 0) first_id[8] = after;
  float* gm = G.p[m] + off;
  float acc[VL];
#pragma unroll
  for (int j = 0; j < VL; ++j) acc[j] = 0.f;
  bool at_head = true;                            // still in the warp's first run
  unsigned goes_on = kAbsent;                     // the id of the run in tail[w]
  for (int k = 0; k < n; k += AHEAD) {
    Pack<T> raw[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const unsigned r = __shfl_sync(0xffffffffu, (unsigned)key, k + a);
      const bool real = __shfl_sync(0xffffffffu, id, k + a) != kAbsent;
      raw[a] = strip_raw<T, VEC>(dY + (int64_t)(real ? r : 0) * ld, c, real ? E : 0, lane);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const unsigned v = __shfl_sync(0xffffffffu, id, k + a);
      if (v == kAbsent) break;
#pragma unroll
      for (int j = 0; j < VL; ++j) acc[j] += Elem<T>::up(raw[a].v[j]);
      const unsigned next = k + a == 31 ? after : __shfl_sync(0xffffffffu, id, (k + a + 1) & 31);
      const bool last = k + a == 31;
      if (next != v || last) {
        if (at_head && before == v) {             // (a run over the whole warp too)
#pragma unroll
          for (int j = 0; j < VL; ++j) head[w][j][lane] = acc[j];
        } else if (next == v) {
          goes_on = v;
#pragma unroll
          for (int j = 0; j < VL; ++j) tail[w][j][lane] = acc[j];
        } else {
          emit<T, VEC>(gm + (int64_t)v * E, c, E, lane, acc, scale, accumulate);
        }
        at_head = false;
#pragma unroll
        for (int j = 0; j < VL; ++j) acc[j] = 0.f;
      }
    }
  }
  __syncthreads();
  // runs over several warps: the warp where one starts adds up its parts; the
  // unit's first warp also those of a run from the unit before
  const bool from_before = w == 0 && before != kAbsent && before == first_id[0];
  for (int which = 0; which < 2; ++which) {
    const bool tail_part = which == 1;
    if (tail_part ? goes_on == kAbsent : !from_before) continue;
    const unsigned v = tail_part ? goes_on : before;
    int j0 = w + 1;                               // the next warp whose head may belong to the run
#pragma unroll
    for (int j = 0; j < VL; ++j) acc[j] = tail_part ? tail[w][j][lane] : head[0][j][lane];
    for (; j0 < 8 && first_id[j0] == v; ++j0)
#pragma unroll
      for (int j = 0; j < VL; ++j) acc[j] += head[j0][j][lane];
    const bool beyond = j0 == 8 && first_id[8] == v;
    if (!tail_part) strip_store_f32<T, VEC>(part + (int64_t)u * 2 * E, c, E, lane, acc);
    else if (beyond) strip_store_f32<T, VEC>(part + ((int64_t)u * 2 + 1) * E, c, E, lane, acc);
    else emit<T, VEC>(gm + (int64_t)v * E, c, E, lane, acc, scale, accumulate);
  }
}

// a warp per (unit, strip): where a run starts in the unit and goes on behind
// it, its parts are added up in order and written
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
  const int i0 = s0 + (u - map.unit[m]) * kEmbUnit;
  if (i0 + kEmbUnit >= s1) return;
  const unsigned v = key_id(keys[i0 + kEmbUnit - 1]);
  if (v == kAbsent || key_id(keys[i0 + kEmbUnit]) != v) return;
  if (i0 > s0 && key_id(keys[i0]) == v && key_id(keys[i0 - 1]) == v) return;  // the run starts further left
  float acc[VL];
  strip_load_f32<T, VEC>(part + ((int64_t)u * 2 + 1) * E, c, E, lane, acc);
  for (int k = u + 1;; k += 32) {
    // the units behind whose first token belongs to the run, 32 at a time
    const int64_t at = (int64_t)i0 + (int64_t)(k - u + lane) * kEmbUnit;
    const unsigned in = __ballot_sync(0xffffffffu, at < s1 && key_id(keys[at < s1 ? at : i0]) == v);
    const int n = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      float x[VL];
      strip_load_f32<T, VEC>(part + (int64_t)(k + i) * 2 * E, c, E, lane, x);
#pragma unroll
      for (int j = 0; j < VL; ++j) acc[j] += x[j];
    }
    if (n < 32) break;
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
void run_embed_reduce(cudaStream_t s, const EmbedGradArgs& a, const RowMap& map, int64_t longest, const GradPtrs& G,
                      const Key* keys) {
  const int n_strip = (int)((a.E + 32 * Elem<T>::V - 1) / (32 * Elem<T>::V));
  const int64_t blocks = (int64_t)map.unit[map.M] * n_strip;
  count_launch();
  launch_pdl(k_embed_reduce<T, VEC>, dim3((unsigned)blocks), dim3(256), 0, s, map, G, keys,
             reinterpret_cast<const T*>(a.dY), a.ld, (int)a.E, n_strip, a.off, a.scale, a.accumulate, a.part);
  if (longest <= kEmbUnit) return;   // no run leaves its unit
  count_launch();
  launch_pdl(k_embed_join<T, VEC>, dim3((unsigned)((blocks + 7) / 8)), dim3(256), 0, s, map, G, keys, (int)a.E, n_strip,
             a.off, a.scale, a.accumulate, (const float*)a.part);
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
  const int N = start[M];
  int64_t longest = 0;
  for (int m = 0; m < M; ++m) longest = longest > start[m + 1] - start[m] ? longest : start[m + 1] - start[m];
  int merges = 0;
  for (int64_t run = kSortTile; run < longest; run *= 16) ++merges;
  // the tables are zeroed in equal shares beside the sort and each merge:
  // eight blocks to an SM, so that they even out, but at least 16 KB a block
  ZeroShare z{};
  z.off = a.off;
  z.n = a.V * a.E;
  z.M = M;
  z.to = 1024;
  if (!a.accumulate) {
    const int64_t want = (8 * num_sms() + M - 1) / M, most = (z.n + 4095) / 4096;
    z.blocks = M * (int)(want < most ? want : most);
  }
  if (N == 0) {
    if (z.blocks > 0) {
      count_launch();
      launch_pdl(k_zero_tables, dim3(z.blocks), dim3(1024), 0, s, G, z);
    }
    return;
  }
  const RowMap sort_map = make_map(start, M, kSortTile);
  z.to = 1024 / (merges + 1);
  count_launch();
  launch_pdl(k_sort_tiles, dim3(sort_map.unit[M] + z.blocks), dim3(1024), 0, s, sort_map, a.ids, a.id64, a.V, a.keys[0],
             a.status, G, z);
  int at = 0;
  int64_t run = kSortTile;
  for (int i = 1; i <= merges; ++i, run *= 16, at ^= 1) {
    z.from = z.to;
    z.to = i == merges ? 1024 : 1024 * (i + 1) / (merges + 1);
    count_launch();
    launch_pdl(k_merge, dim3((unsigned)((N + 1023LL) / 1024) + z.blocks), dim3(1024), 0, s, sort_map, run,
               (const Key*)a.keys[at], a.keys[at ^ 1], G, z);
  }
  const RowMap map = make_map(start, M, kEmbUnit);
  const int vl = a.type == LT_F32 ? 4 : 8;
  const bool vec = a.E % vl == 0 && a.ld % vl == 0 && a.off % 4 == 0 && on16(a.dY);
#define SM_RUN(T)                                                             \
  (vec ? run_embed_reduce<T, true>(s, a, map, longest, G, a.keys[at])         \
       : run_embed_reduce<T, false>(s, a, map, longest, G, a.keys[at]))
  if (a.type == LT_F32) SM_RUN(float);
  else if (a.type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

}  // namespace sm
