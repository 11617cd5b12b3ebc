// layers_embed.cu -- embedding lookup with scaling, and its gradient per
// worker by sorted tokens.
#include <climits>

#include "layers.cuh"

namespace sm {
namespace {

// ---------------------------------------------------------------------------
// Lookup: out[r] = fl(scale * table[ids[r]]).  Bound by the bytes: N * E
// elements written, one 4 * E-byte table row read per token (from L2 where
// tokens repeat).  One warp per (row, slab of kSlab columns), so that a short row
// is one warp's few wide loads and a long one spreads.  131072 tokens of a
// 50304 x 768 table to bf16: 60 us, of which its DRAM bytes need 0.90; 8
// tokens: 2.4 us on the device, of which the launch is nearly all.
// ---------------------------------------------------------------------------
constexpr int kSlab = 1024;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed(const float* table, int64_t V, int E,
                                               const void* ids, int id64, int64_t n, int n_slab,
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
// The tokens of each worker are sorted by (id, row): up to kSortTile of them in
// registers, up to kBlockTile by a radix sort of one block, more by one of many
// blocks.  A block then takes a unit of sorted tokens of one worker and a strip
// of columns, a warp an eighth of them, one key per lane, and adds up their dY
// rows in registers; parts of a run of equal ids are added up in order across the
// warps through shared memory, and where it goes on in other blocks by
// k_embed_join.  Work per block does not depend on how often a token occurs, and
// every sum has a fixed order.
//
// A sort waits on itself most of the time, and the zeros are most of the bytes:
// further blocks of its launches zero the tables meanwhile.  Rows with tokens
// are then written twice; zeroing the others alone, beside the sums, writes every
// byte once but waits for the sort: 131072 tokens, 8 tables of 50304 x 768, bf16:
// 258 us against 275 (8192 tokens: 180 against 210); 9001 tokens, 4 tables of
// 8191 x 1001, fp16: 40 against 55.  Where the tokens outnumber the rows it costs
// a little (8192 tokens, 8 x 1000 x 768, fp32: 28 against 26).
// Of the 258 us 178 are the sort and zeros (6.9 TB/s), 70 the sums and 8 the join.
// Absent tokens (id < 0, id >= V) get the id kAbsent and sort to the end.
// ---------------------------------------------------------------------------
typedef unsigned long long Key;  // id in the upper 32 bits, row in the lower

__device__ __forceinline__ unsigned key_id(Key k) { return (unsigned)(k >> 32); }
constexpr unsigned kAbsent = 0xffffffffu;
constexpr int kSortThreads = 512;

template <typename K>
__device__ __forceinline__ K shfl_xor(K v, int lanes) {
  return __shfl_xor_sync(0xffffffffu, v, lanes);
}

// Zeros for whole tables, in chunks: what a launch of the sort writes in the
// blocks behind its own.
struct ZeroTables {
  int chunk;           // entries
  int per_table;       // chunks per table
  int64_t first;       // this launch's first chunk
  int64_t off, size;   // of each table in G[m]
};

__device__ __forceinline__ void zero_chunk(const GradPtrs& G, const ZeroTables& z, int b) {
  const int64_t k = z.first + b;
  const int m = (int)(k / z.per_table);
  const int64_t i0 = (k - (int64_t)m * z.per_table) * z.chunk;
  const int n = (int)min((int64_t)z.chunk, z.size - i0);
  float* g = G.p[m] + z.off + i0;
  const int head = min(n, (int)((4 - (reinterpret_cast<uintptr_t>(g) >> 2 & 3)) & 3));
  const int n4 = (n - head) / 4, tid = threadIdx.x, tail = head + 4 * n4 + tid;
  if (tid < head) g[tid] = 0.f;
  for (int i = tid; i < n4; i += blockDim.x) reinterpret_cast<float4*>(g + head)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (tail < n) g[tail] = 0.f;
}

// a block per unit of `map` (kSortTile rows of one worker): bitonic sort, PER
// keys a thread, with exchanges in registers within a thread, by shuffles
// within a warp and through shared memory beyond.  K = unsigned: the key is
// (id, place in the tile) in 32 bits (V below 2^(32 - kPlaceBits)); else 64.
constexpr int kPlaceBits = 11;
static_assert(kSortTile == 1 << kPlaceBits, "a place in the tile has kPlaceBits bits");
template <typename K>
__global__ void __launch_bounds__(kSortThreads) k_sort_tiles(const RowMap map, const void* ids, int id64,
                                                             int64_t V, Key* __restrict__ keys, int* status,
                                                             const GradPtrs G, const ZeroTables zero) {
  constexpr int THREADS = kSortThreads;
  constexpr int PER = kSortTile / THREADS;
  __shared__ K swap[kSortTile];
  griddep_wait();
  griddep_launch();
  const int u = blockIdx.x;
  if (u >= map.unit[map.M]) {
    zero_chunk(G, zero, u - map.unit[map.M]);
    return;
  }
  const int m = worker_of(map.unit, map.M, u);
  const int r0 = map.start[m] + (u - map.unit[m]) * kSortTile;
  const int n = min(kSortTile, map.start[m + 1] - r0);
  const int tid = threadIdx.x;
  constexpr K kNone = (K)~(K)0;                   // absent tokens and places beyond n
  K k[PER];                                       // the keys of places tid * PER ... + PER - 1
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = j * THREADS + tid;
    K key = kNone;
    if (i < n) {
      const int64_t id = load_id(ids, id64, r0 + i);
      if (id >= V) *status = 1;
      const K w = (id >= 0 && id < V) ? (K)id : (K)(kNone >> kPlaceBits);
      key = (K)(w << kPlaceBits) | (K)i;
    }
    swap[i] = key;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) k[j] = swap[tid * PER + j];
  for (int size = 2; size < n * 2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      if (stride >= PER) {
        K other[PER];
        if (stride < 32 * PER) {
#pragma unroll
          for (int j = 0; j < PER; ++j) other[j] = shfl_xor(k[j], stride / PER);
        } else {
          __syncthreads();
#pragma unroll
          for (int j = 0; j < PER; ++j) swap[j * THREADS + tid] = k[j];
          __syncthreads();
#pragma unroll
          for (int j = 0; j < PER; ++j) other[j] = swap[j * THREADS + (tid ^ (stride / PER))];
        }
        const bool keep_min = ((tid * PER & stride) == 0) == ((tid * PER & size) == 0);
#pragma unroll
        for (int j = 0; j < PER; ++j) k[j] = (k[j] < other[j]) == keep_min ? k[j] : other[j];
      } else {
#pragma unroll
        for (int d = PER / 2; d > 0; d >>= 1) {
          if (d != stride) continue;
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            if (j & d) continue;
            const K a = k[j], b = k[j | d];
            const bool swapped = (a > b) == (((tid * PER + j) & size) == 0);
            k[j] = swapped ? b : a;
            k[j | d] = swapped ? a : b;
          }
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) swap[tid * PER + j] = k[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = j * THREADS + tid;
    if (i >= n) continue;
    const K w = swap[i] >> kPlaceBits;
    const unsigned id = w == (K)(kNone >> kPlaceBits) ? kAbsent : (unsigned)w;
    keys[r0 + i] = ((Key)id << 32) | (unsigned)(r0 + (int)(swap[i] & (K)(kSortTile - 1)));
  }
}

// Radix sort of longer token lists, least significant digit first, kRadixTile
// tokens of one worker a block.  Within a worker digit d of tile u starts at
// (tokens with a smaller digit) + (tokens with d in the tiles before u), from the
// tiles' digit counts; a token's place behind that comes from counting in order:
// warps take 32 tokens at a time and match equal digits.  Two digits of 8 bits
// and the count take about 18 us for 8193 to 131072 tokens: latency, three
// launches in a row.
// The first counts are made by k_radix_count; each scatter makes the next
// digit's by (integer) atomics.  There is a set of counts per digit; a scatter
// block reads all of its worker's, which is nothing at 131072 tokens, but grows with
// the square of a worker's tokens (2^20: 0.5 GB a digit; 2^24: 130 GB).  Absent
// tokens sort as id V.
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
static_assert(kBins == kRadixBins && kRadixSets * kDigitBits >= 31, "the workspace has a set of counts per digit");

__device__ __forceinline__ unsigned radix_id(const void* ids, int id64, int64_t V, int i) {
  const int64_t id = load_id(ids, id64, i);
  return (unsigned)(id >= 0 && id < V ? id : V);
}

__global__ void __launch_bounds__(256) k_radix_count(const RowMap map, const void* ids, int id64, int64_t V,
                                                     int bits, int digits, int* __restrict__ count, int64_t set,
                                                     int* status, const GradPtrs G, const ZeroTables zero) {
  __shared__ int c[kBins];
  griddep_wait();
  griddep_launch();
  const int u = blockIdx.x;
  if (u >= map.unit[map.M]) {
    zero_chunk(G, zero, u - map.unit[map.M]);
    return;
  }
  const int m = worker_of(map.unit, map.M, u);
  const int r0 = map.start[m] + (u - map.unit[m]) * kRadixTile;
  const int n = min(kRadixTile, map.start[m + 1] - r0);
  for (int d = threadIdx.x; d < kBins; d += 256) {
    c[d] = 0;
    for (int k = 1; k < digits; ++k) count[k * set + (int64_t)u * kBins + d] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    if (load_id(ids, id64, r0 + i) >= V) *status = 1;
    atomicAdd(&c[radix_id(ids, id64, V, r0 + i) & ((1u << bits) - 1)], 1);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kBins; d += 256) count[(int64_t)u * kBins + d] = c[d];
}

// src = null: the first digit, keys from the ids; next = null: the last digit
__global__ void __launch_bounds__(256) k_radix_scatter(const RowMap map, const void* ids, int id64,
                                                       int64_t V, int shift, int bits, const Key* src,
                                                       Key* __restrict__ dst, int* __restrict__ count,
                                                       int* __restrict__ next, const GradPtrs G,
                                                       const ZeroTables zero) {
  constexpr int ROUNDS = kRadixTile / 256;
  __shared__ int warp_count[8][kBins];
  __shared__ int base[kBins];
  __shared__ int scan[8];
  griddep_wait();
  griddep_launch();
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (u >= map.unit[map.M]) {
    zero_chunk(G, zero, u - map.unit[map.M]);
    return;
  }
  const int m = worker_of(map.unit, map.M, u);
  const int r0 = map.start[m] + (u - map.unit[m]) * kRadixTile;
  const int n = min(kRadixTile, map.start[m + 1] - r0);
  const unsigned mask = (1u << bits) - 1;
  Key key[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {   // warp w has tokens w * 32 * ROUNDS on, 32 of them a round
    const int i = (w * ROUNDS + j) * 32 + lane;
    key[j] = ~0ull;
    if (i < n) {
      if (src != nullptr) key[j] = src[r0 + i];
      else key[j] = ((Key)radix_id(ids, id64, V, r0 + i) << 32) | (unsigned)(r0 + i);
    }
  }
  for (int d = tid; d < 8 * kBins; d += 256) (&warp_count[0][0])[d] = 0;
  // where each digit of this tile starts: two neighbouring digits a thread
  const int u0 = map.unit[m], u1 = map.unit[m + 1];
  int all0 = 0, all1 = 0, before0 = 0, before1 = 0;
#pragma unroll 4
  for (int k = u0; k < u1; ++k) {
    const int2 c = *reinterpret_cast<const int2*>(count + (int64_t)k * kBins + 2 * tid);
    all0 += c.x;
    all1 += c.y;
    if (k < u) {
      before0 += c.x;
      before1 += c.y;
    }
  }
  int sum = all0 + all1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  if (lane == 31) scan[w] = sum;
  __syncthreads();
  for (int i = 0; i < w; ++i) sum += scan[i];
  base[2 * tid] = sum - all0 - all1 + before0;
  base[2 * tid + 1] = sum - all1 + before1;
  // counts of the warp so far, and each token's place among its digit's
  int place[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const bool live = (w * ROUNDS + j) * 32 + lane < n;
    const unsigned d = live ? (key_id(key[j]) >> shift) & mask : (unsigned)kBins;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int lower = __popc(same & ((1u << lane) - 1));
    place[j] = live ? warp_count[w][d] + lower : 0;
    __syncwarp();
    if (live && lower == 0) warp_count[w][d] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int d = tid; d < kBins; d += 256) {
    int run = base[d];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = warp_count[i][d];
      warp_count[i][d] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    if ((w * ROUNDS + j) * 32 + lane >= n) continue;
    const unsigned id = key_id(key[j]);
    const int at = warp_count[w][(id >> shift) & mask] + place[j];
    if (next != nullptr) {
      dst[map.start[m] + at] = key[j];
      atomicAdd(&next[(int64_t)(u0 + at / kRadixTile) * kBins + ((id >> (shift + bits)) & mask)], 1);
    } else {
      dst[map.start[m] + at] = id == (unsigned)V ? (key[j] | ((Key)kAbsent << 32)) : key[j];
    }
  }
}

// The same sort of up to kBlockTile tokens a worker by one block, which passes
// the keys through shared memory from digit to digit: one launch.  Two digits of
// 2049 tokens take 11 us, of 4096 14, of 8192 21, where the launches of many
// blocks take 18; with zeros beside it, which want one launch too, it is used up
// to 8192, else up to half of that.
constexpr int kBlockTile = 8192, kBlockThreads = 1024;
inline size_t block_smem(int bits) { return kBlockTile * sizeof(Key) + ((size_t)(kBlockThreads / 32) << bits) * sizeof(int); }

__global__ void __launch_bounds__(kBlockThreads) k_radix_block(const RowMap map, const void* ids, int id64, int64_t V,
                                                               int bits, int digits, Key* __restrict__ dst, int* status,
                                                               const GradPtrs G, const ZeroTables zero) {
  constexpr int ROUNDS = kBlockTile / kBlockThreads, WARPS = kBlockThreads / 32;
  extern __shared__ uint4 shared[];
  Key* keys = reinterpret_cast<Key*>(shared);                        // [kBlockTile]
  int* warp_count = reinterpret_cast<int*>(keys + kBlockTile);       // [WARPS][bins]
  __shared__ int base[kBins];
  __shared__ int scan[kBins / 32];
  griddep_wait();
  griddep_launch();
  const int m = blockIdx.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (m >= map.M) {
    zero_chunk(G, zero, m - map.M);
    return;
  }
  const int r0 = map.start[m], n = map.start[m + 1] - r0;
  const int bins = 1 << bits;
  Key key[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {   // warp w has tokens w * 32 * ROUNDS on, 32 of them a round
    const int i = (w * ROUNDS + j) * 32 + lane;
    key[j] = 0ull;
    if (i < n) {
      const int64_t id = load_id(ids, id64, r0 + i);
      if (id >= V) *status = 1;
      key[j] = ((Key)(id >= 0 && id < V ? id : V) << 32) | (unsigned)(r0 + i);
    }
  }
  for (int digit = 0; digit < digits; ++digit) {
    const int shift = 32 + digit * bits;
    for (int i = tid; i < WARPS * bins; i += kBlockThreads) warp_count[i] = 0;
    __syncthreads();
    int* mine = warp_count + w * bins;
    int place[ROUNDS];
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
      const bool live = (w * ROUNDS + j) * 32 + lane < n;
      const unsigned d = live ? (unsigned)(key[j] >> shift) & (bins - 1) : (unsigned)bins;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int lower = __popc(same & ((1u << lane) - 1));
      place[j] = live ? mine[d] + lower : 0;
      __syncwarp();
      if (live && lower == 0) mine[d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // where each digit starts, and each warp's tokens within it
    int run = 0, sum = 0;
    if (tid < bins) {
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        const int c = warp_count[i * bins + tid];
        warp_count[i * bins + tid] = run;
        run += c;
      }
    }
    if (tid < kBins) {
      sum = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      if (lane == 31) scan[w] = sum;
    }
    __syncthreads();
    if (tid < kBins) {
      for (int i = 0; i < w; ++i) sum += scan[i];
      base[tid] = sum - run;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
      if ((w * ROUNDS + j) * 32 + lane >= n) continue;
      const unsigned d = (unsigned)(key[j] >> shift) & (bins - 1);
      keys[base[d] + mine[d] + place[j]] = key[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ROUNDS; ++j) {
      const int i = (w * ROUNDS + j) * 32 + lane;
      if (i < n) key[j] = keys[i];
    }
  }
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int i = (w * ROUNDS + j) * 32 + lane;
    if (i < n) dst[r0 + i] = key_id(key[j]) == (unsigned)V ? (key[j] | ((Key)kAbsent << 32)) : key[j];
  }
}

// zeros alone (no tokens at all)
__global__ void __launch_bounds__(256) k_zero_tables(const GradPtrs G, const ZeroTables zero) {
  griddep_wait();
  griddep_launch();
  zero_chunk(G, zero, blockIdx.x);
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

// a block per (unit of 8 * per_warp sorted tokens, strip of columns)
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_embed_reduce(const RowMap map, const GradPtrs G, const Key* keys,
                                                      const T* dY, int64_t ld, int E, int n_strip,
                                                      int64_t off, float scale, int accumulate,
                                                      float* __restrict__ part, int per_warp) {
  constexpr int VL = Elem<T>::V;
  constexpr int AHEAD = VEC ? 4 : 8;              // rows in a batch
  constexpr int BATCHES = 3;                      // VEC: batches on their way
  extern __shared__ uint4 ring[];                 // VEC: [8 warps][BATCHES * AHEAD][32 lanes]
  __shared__ float head[8][VL][32], tail[8][VL][32];  // a warp's part of a run from before, and of one that goes on
  __shared__ unsigned first_id[9];                // of each warp; [8]: of the unit behind
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int u = blockIdx.x / n_strip;
  const int c = (blockIdx.x - u * n_strip) * 32 * VL;
  const int m = worker_of(map.unit, map.M, u);
  const int s0 = map.start[m], s1 = map.start[m + 1];
  const int i0 = s0 + ((u - map.unit[m]) * 8 + w) * per_warp;
  const int n = max(0, min(per_warp, s1 - i0));
  const Key key = lane < n ? keys[i0 + lane] : ~0ull;
  const unsigned id = key_id(key);
  const unsigned before = n > 0 && i0 > s0 ? key_id(keys[i0 - 1]) : kAbsent;
  const unsigned after = n == per_warp && i0 + n < s1 ? key_id(keys[i0 + n]) : kAbsent;
  if (lane == 0) first_id[w] = id;
  if (w == 7 && lane == 0) first_id[8] = after;
  float* gm = G.p[m] + off;
  F2 sum[VL / 2];
  float acc[VL];
#pragma unroll
  for (int j = 0; j < VL / 2; ++j) sum[j] = 0ull;
  bool at_head = true;                            // still in the warp's first run
  unsigned goes_on = kAbsent;                     // the id of the run in tail[w]
  // the absent tokens are the last ones
  const int real = __popc(__ballot_sync(0xffffffffu, id != kAbsent));
  uint4* slots = &ring[w * (BATCHES * AHEAD * 32) + lane];
  auto fetch = [&](int k, int batch) {            // the rows from token k on
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const unsigned r = __shfl_sync(0xffffffffu, (unsigned)key, (k + a) & 31);
      const int col = c + lane * VL;
      if (k + a < real && col < E) copy16(slots + (batch * AHEAD + a) * 32, dY + (int64_t)r * ld + col, true);
    }
    copy_commit();
  };
  if (VEC) {
#pragma unroll
    for (int b = 0; b < BATCHES; ++b) fetch(b * AHEAD, b);
  }
  int batch = 0;
  for (int k = 0; k < real; k += AHEAD) {
    Pack<T> raw[AHEAD];
    if (VEC) copy_wait<BATCHES - 1>();
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (VEC) {
        raw[a] = *reinterpret_cast<const Pack<T>*>(slots + (batch * AHEAD + a) * 32);
      } else {
        const unsigned r = __shfl_sync(0xffffffffu, (unsigned)key, k + a);
        raw[a] = strip_raw<T, VEC>(dY + (int64_t)(k + a < real ? r : 0) * ld, c, k + a < real ? E : 0, lane);
      }
    }
    if (VEC) fetch(k + BATCHES * AHEAD, batch);
    batch = batch + 1 == BATCHES ? 0 : batch + 1;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (k + a >= real) break;
      const unsigned v = __shfl_sync(0xffffffffu, id, k + a);
#pragma unroll
      for (int j = 0; j < VL / 2; ++j) sum[j] = add2(sum[j], up2(raw[a], j));
      const bool last = k + a == per_warp - 1;
      const unsigned next = last ? after : __shfl_sync(0xffffffffu, id, (k + a + 1) & 31);
      if (next != v || last) {
#pragma unroll
        for (int j = 0; j < VL / 2; ++j) {
          const float2 t = unpack2(sum[j]);
          acc[2 * j] = t.x;
          acc[2 * j + 1] = t.y;
          sum[j] = 0ull;
        }
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
__global__ void __launch_bounds__(256) k_embed_join(const RowMap map, const GradPtrs G, const Key* keys,
                                                    int E, int n_strip, int64_t off, float scale, int accumulate,
                                                    const float* part, int unit) {
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
  const int i0 = s0 + (u - map.unit[m]) * unit;
  if (i0 + unit >= s1) return;
  const unsigned v = key_id(keys[i0 + unit - 1]);
  if (v == kAbsent || key_id(keys[i0 + unit]) != v) return;
  if (i0 > s0 && key_id(keys[i0]) == v && key_id(keys[i0 - 1]) == v) return;  // the run starts further left
  float acc[VL];
  strip_load_f32<T, VEC>(part + ((int64_t)u * 2 + 1) * E, c, E, lane, acc);
  for (int k = u + 1;; k += 32) {
    // the units behind whose first token belongs to the run, 32 at a time
    const int64_t at = (int64_t)i0 + (int64_t)(k - u + lane) * unit;
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
void run_embed_reduce(cudaStream_t s, const EmbedGradArgs& a, const RowMap& map, int per_warp, int64_t longest,
                      const GradPtrs& G, const Key* keys) {
  const int n_strip = (int)((a.E + 32 * Elem<T>::V - 1) / (32 * Elem<T>::V));
  const int64_t blocks = (int64_t)map.unit[map.M] * n_strip;
  auto* reduce = k_embed_reduce<T, VEC>;
  const size_t smem = VEC ? 8 * 3 * 4 * 32 * 16 : 0;
  if (smem > 32 * 1024) allow_shared((const void*)reduce);
  count_launch();
  launch_pdl(reduce, dim3((unsigned)blocks), dim3(256), smem, s, map, G, keys,
             reinterpret_cast<const T*>(a.dY), a.ld, (int)a.E, n_strip, a.off, a.scale, a.accumulate, a.part, per_warp);
  if (longest <= 8 * per_warp) return;   // no run leaves its unit
  count_launch();
  launch_pdl(k_embed_join<T, VEC>, dim3((unsigned)((blocks + 7) / 8)), dim3(256), 0, s, map, G, keys, (int)a.E, n_strip,
             a.off, a.scale, a.accumulate, (const float*)a.part, 8 * per_warp);
}

RowMap make_map(const int* start, int M, int tile) {
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  for (int m = 0; m < M; ++m) map.unit[m + 1] = map.unit[m] + (int)(((int64_t)start[m + 1] - start[m] + tile - 1) / tile);
  return map;
}

// Chunks of zeros, in entries: 64 KB a block keeps the 256-thread blocks many
// and short.  k_radix_block's 1024 threads start too slowly for that: four shares
// an SM, up to 512 KB (4 x 8191 x 1001: 45 us with four, 50 with sixteen; 8 x
// 50304 x 768 of 4096 tokens each 209 with 512 KB, 231 with 2 MB).
constexpr int64_t kZeroChunk = 16384;
constexpr int64_t kZeroMost = 131072;

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
  // the tables' chunks, shared out over the launches of the sort
  ZeroTables zero{0, 0, 0, a.off, a.V * a.E};
  int launches = 1, launched = 0;
  auto with_zeros = [&](int blocks, int64_t chunk) {
    zero.chunk = (int)chunk;
    zero.per_table = (int)((zero.size + chunk - 1) / chunk);
    const int64_t chunks = a.accumulate ? 0 : (int64_t)M * zero.per_table;
    zero.first = chunks * launched / launches;
    ++launched;
    return dim3((unsigned)(blocks + chunks * launched / launches - zero.first));
  };
  if (N == 0) {
    if (a.accumulate) return;
    const dim3 grid = with_zeros(0, kZeroChunk);
    count_launch();
    launch_pdl(k_zero_tables, grid, dim3(256), 0, s, G, zero);
    return;
  }
  int at = 0;
  if (longest <= kSortTile) {
    const RowMap tiles = make_map(start, M, kSortTile);
    const dim3 grid = with_zeros(tiles.unit[M], kZeroChunk);
    count_launch();
    launch_pdl(a.V < (int64_t(1) << (32 - kPlaceBits)) ? k_sort_tiles<unsigned> : k_sort_tiles<Key>, grid,
               dim3(kSortThreads), 0, s, tiles, a.ids, a.id64, a.V, a.keys[0], a.status, G, zero);
  } else {
    const RowMap tiles = make_map(start, M, kRadixTile);
    int width = 1;   // bits of the ids 0 ... V
    while (a.V >> width) ++width;
    const int digits = (width + kDigitBits - 1) / kDigitBits, bits = (width + digits - 1) / digits;
    if (longest <= (a.accumulate ? kBlockTile / 2 : kBlockTile)) {
      const size_t smem = block_smem(bits);
      allow_shared((const void*)k_radix_block);
      int64_t share = zero.size * M / (num_sms() * 4) / kZeroChunk * kZeroChunk;
      share = share < kZeroChunk ? kZeroChunk : share > kZeroMost ? kZeroMost : share;
      const dim3 grid = with_zeros(M, share);
      count_launch();
      launch_pdl(k_radix_block, grid, dim3(kBlockThreads), smem, s, tiles, a.ids, a.id64, a.V, bits, digits, a.keys[0],
                 a.status, G, zero);
    } else {
      launches = digits + 1;
      dim3 grid = with_zeros(tiles.unit[M], kZeroChunk);
      count_launch();
      launch_pdl(k_radix_count, grid, dim3(256), 0, s, tiles, a.ids, a.id64, a.V, bits, digits, a.counts, a.count_set,
                 a.status, G, zero);
      for (int k = 0; k < digits; ++k) {
        at = k & 1;
        grid = with_zeros(tiles.unit[M], kZeroChunk);
        count_launch();
        launch_pdl(k_radix_scatter, grid, dim3(256), 0, s, tiles, a.ids, a.id64, a.V, k * bits, bits,
                   k == 0 ? (const Key*)nullptr : (const Key*)a.keys[at ^ 1], a.keys[at],
                   a.counts + k * a.count_set, k + 1 < digits ? a.counts + (k + 1) * a.count_set : (int*)nullptr, G, zero);
      }
    }
  }
  const int per_warp = embed_per_warp(N, a.E, a.type);
  const RowMap map = make_map(start, M, 8 * per_warp);
  const int vl = a.type == LT_F32 ? 4 : 8;
  const bool vec = a.E % vl == 0 && a.ld % vl == 0 && a.off % 4 == 0 && on16(a.dY);
#define SM_RUN(T)                                                                     \
  (vec ? run_embed_reduce<T, true>(s, a, map, per_warp, longest, G, a.keys[at])    \
       : run_embed_reduce<T, false>(s, a, map, per_warp, longest, G, a.keys[at]))
  if (a.type == LT_F32) SM_RUN(float);
  else if (a.type == LT_BF16) SM_RUN(__nv_bfloat16);
  else SM_RUN(__half);
#undef SM_RUN
}

}  // namespace sm
