// layers_distill.cu -- distillation loss per worker and its gradient with
// respect to the student's logits.
#include "layers.cuh"

namespace sm {
namespace {

__device__ __forceinline__ float load_t(const void* t, int type, int64_t i) {
  if (type == LT_F32) return reinterpret_cast<const float*>(t)[i];
  if (type == LT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(t)[i]);
  return __half2float(reinterpret_cast<const __half*>(t)[i]);
}

// an entry counts when its index is one of the V columns and its logit is not -inf
__device__ __forceinline__ bool counts(int64_t id, int64_t V, float t) {
  return id >= 0 && id < V && !(t == -INFINITY);
}

struct Teacher {
  const void* idx;
  int id64;
  const void* t;
  int t_type;
  int64_t ldt;
  int K;
};

// What a row's entries come to: nothing to learn from, or the softmax of the
// teacher's logits, exp((t - top) / T - log_sum), and whether an index is there
// twice.
struct RowStat {
  float top, log_sum;
};
enum RowKind { ROW_NONE = 0, ROW_ONCE = 1, ROW_TWICE = 2 };

// The rows' stats and kinds, and count[m] += worker m's rows of a kind other
// than none.  A row takes G threads: a warp (K <= 128), or the block.  Repeated
// indices are found by inserting all of them into a hash table of 2 K slots.
// Latency bound: 8192 rows of 64 entries take 12 us, most of it behind the
// rows' first loads, which do not wait for it; the same work at the head of each
// row's own block cost 90 us at 128 entries, since the row then waited for it.
template <int G>
__global__ void __launch_bounds__(256) k_distill_teacher(const RowMap map, const Teacher te, int64_t V, float inv_T,
                                                         RowStat* __restrict__ stat, int* __restrict__ kind, int* count,
                                                         int* status) {
  constexpr int ROWS = 256 / G, SLOTS = G == 32 ? 256 : 2048;
  __shared__ int table[ROWS][SLOTS];
  __shared__ float part[8];
  __shared__ int any_of[ROWS];
  griddep_wait();
  griddep_launch();
  const int in_block = threadIdx.x / G, tid = threadIdx.x % G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int N = map.start[map.M];
  const int64_t r = (int64_t)blockIdx.x * ROWS + in_block;
  const int K = r < N ? te.K : 0;
  auto sync = [&] {
    if (G == 32) __syncwarp();
    else __syncthreads();
  };
  auto over_row = [&](float v, bool maximum) {    // sum or maximum over the row's threads
    v = maximum ? warp_max(v) : warp_sum(v);
    if (G == 32) return v;
    __syncthreads();
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < 8; ++i) v = maximum ? fmaxf(v, part[i]) : v + part[i];
    return v;
  };
  for (int i = tid; i < SLOTS; i += G) table[in_block][i] = -1;
  sync();
  float top = -INFINITY;
  bool any = false, twice = false;
  for (int k = tid; k < K; k += G) {
    const int64_t i = load_id(te.idx, te.id64, r * te.ldt + k);
    const float t = load_t(te.t, te.t_type, r * te.ldt + k);
    if (i >= V) *status = 1;
    if (!counts(i, V, t)) continue;
    any = true;
    top = fmaxf(top, t);
    unsigned at = ((unsigned)i * 2654435761u) >> 16;
    for (int probes = 0; probes < SLOTS; ++probes, ++at) {
      const int old = atomicCAS(&table[in_block][at % SLOTS], -1, (int)i);
      if (old == (int)i) twice = true;
      if (old == -1 || old == (int)i) break;
    }
  }
  any = over_row(any ? 1.f : 0.f, true) != 0.f;
  twice = over_row(twice ? 1.f : 0.f, true) != 0.f;
  top = over_row(top, true);
  float sum = 0.f;
  for (int k = tid; k < K; k += G) {
    const int64_t i = load_id(te.idx, te.id64, r * te.ldt + k);
    const float t = load_t(te.t, te.t_type, r * te.ldt + k);
    if (counts(i, V, t)) sum += expf((t - top) * inv_T);
  }
  sum = over_row(sum, false);
  if (tid == 0) {
    any_of[in_block] = any;
    if (r < N) {
      stat[r] = RowStat{top, logf(sum)};
      kind[r] = any ? (twice ? ROW_TWICE : ROW_ONCE) : ROW_NONE;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  // lane i: row i of the block
  const int m = lane < ROWS && any_of[lane < ROWS ? lane : 0]
                    ? worker_of(map.start, map.M, (int)((int64_t)blockIdx.x * ROWS + lane)) : -1;
  const unsigned same = __match_any_sync(0xffffffffu, m);
  if (m >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[m], __popc(same));
}

// the maximum of a 16-byte pack, as a float (a NaN does not count)
__device__ __forceinline__ float pack_max(const Pack<float>& p) {
  return fmaxf(fmaxf(p.v[0], p.v[1]), fmaxf(p.v[2], p.v[3]));
}
__device__ __forceinline__ float pack_max(const Pack<__nv_bfloat16>& p) {
  const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(p.v);
  const __nv_bfloat162 m = __hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float pack_max(const Pack<__half>& p) {
  const __half2* a = reinterpret_cast<const __half2*>(p.v);
  const __half2 m = __hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

// A running softmax of y = z c (c = log2 e / T): the maximum m of the logits
// and the sum s of 2^(z c - R), with the reference R = fl(m c), one fma a term.
// The rounding of R is common to every term and cancels in p, as long as it is
// small: within |R| <= 2^24 it is at most 1, but at m c = -1.44e10 it reaches
// 512, and 2^512 is infinity.  So R is at least -2^24, and masked logits, at
// -1e10 as well as at -inf, add 0 to s; rows whose own maximum is out of range
// are `far` and done over, term by term.
constexpr float kFar = 16777216.f;
__device__ __forceinline__ float reference(float m, float c) { return fmaxf(m * c, -kFar); }

struct Running {
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ float raise(float top, float c) {   // returns the reference
    const float r = reference(fmaxf(m, top), c);
    if (top > m) {
      s *= ex2(reference(m, c) - r);
      m = top;
    }
    return r;
  }
  __device__ __forceinline__ void one(float z, float c) {
    const float r = raise(z, c);
    s += ex2(fmaf(z, c, -r));
  }
};

// A row's logits as whole 16-byte packs between a head and a tail.
template <typename T>
struct RowView {
  const T* z;
  int mis, head, nv;
  __device__ __forceinline__ RowView(const T* row, int V) : z(row) {
    constexpr int VL = Elem<T>::V;
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    head = min(V, (VL - mis) % VL);
    nv = (V - head) / VL;
  }
  __device__ __forceinline__ int tail() const { return head + nv * Elem<T>::V; }
  __device__ __forceinline__ const Pack<T>* packs() const { return reinterpret_cast<const Pack<T>*>(z + head); }
};

template <typename T>
__device__ __forceinline__ void add_pack(const Pack<T>& p, F2 neg_ref, F2 c2, F2& sum) {
#pragma unroll
  for (int j = 0; j < Elem<T>::V / 2; ++j) {
    const float2 x = unpack2(fma2(up2(p, j), c2, neg_ref));
    sum = add2(pack2(ex2(x.x), ex2(x.y)), sum);
  }
}

// N packs into the running softmax
template <typename T, int N>
__device__ __forceinline__ void add_packs(Running& run, const Pack<T>* p, float c) {
  float t = pack_max(p[0]);
#pragma unroll
  for (int a = 1; a < N; ++a) t = fmaxf(t, pack_max(p[a]));
  const float r = run.raise(t, c);
  F2 sum = 0ull;
#pragma unroll
  for (int a = 0; a < N; ++a) add_pack(p[a], pack2(-r, -r), pack2(c, c), sum);
  run.s += sum2(sum);
}

// packs tid, tid + THREADS, ... of nv into the running softmax; the first `hold`
// packs of the row (a multiple of THREADS * AHEAD) are left in `held` too, each
// in a place that only its thread reads
template <typename T, int THREADS, int AHEAD>
__device__ __forceinline__ void absorb(Running& run, const Pack<T>* packs, int nv, int tid, float c, Pack<T>* held, int hold) {
  int i = tid;
  for (; i < hold && i + (AHEAD - 1) * THREADS < nv; i += AHEAD * THREADS) {
    Pack<T> p[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) p[a] = packs[i + a * THREADS];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) held[i + a * THREADS] = p[a];
    add_packs<T, AHEAD>(run, p, c);
  }
  for (; i + (AHEAD - 1) * THREADS < nv; i += AHEAD * THREADS) {
    Pack<T> p[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) p[a] = packs[i + a * THREADS];
    add_packs<T, AHEAD>(run, p, c);
  }
  for (; i < nv; i += THREADS) {
    const Pack<T> p = packs[i];
    add_packs<T, 1>(run, &p, c);
  }
}

// The row's maximum and sum from its threads' (a sum that is NaN stays);
// WARPS > 1: buf has a float2 per warp, and the block passes a barrier.
__device__ __forceinline__ void join_lanes(float c, float& m, float& s) {
  const float all = warp_max(m);
  s = warp_sum(s * ex2(reference(m, c) - reference(all, c)));
  m = all;
}
template <int WARPS, typename F>
__device__ __forceinline__ void join_row(const Running& run, int tid, float c, float2* buf, F barrier, float& all, float& s) {
  all = run.m;
  s = run.s;
  join_lanes(c, all, s);
  if (WARPS > 1) {
    if ((tid & 31) == 0) buf[tid >> 5] = make_float2(all, s);
    barrier();
    const float2 b = (tid & 31) < WARPS ? buf[tid & 31] : make_float2(-INFINITY, 0.f);
    all = b.x;
    s = b.y;
    join_lanes(c, all, s);
  }
}

// A row's softmax p = e(z) / s and gradient w * p.
template <typename T>
struct Softmax {
  float all, c, r, s;   // r: the reference of all
  bool far;
  __device__ __forceinline__ Softmax(float all_, float s_, float c_)
      : all(all_), c(c_), r(reference(all_, c_)), s(s_), far(!(fabsf(all_ * c_) <= kFar)) {}
  // log2 of e(z); far rows subtract first
  __device__ __forceinline__ float log2_e(float z) const { return far ? (z - all) * c : fmaf(z, c, -r); }
  __device__ __forceinline__ T grad(float z, float w) const { return Elem<T>::down(w / s * ex2(log2_e(z))); }
  // one pack of a row that is not far; ws = w / s
  __device__ __forceinline__ void pack(const Pack<T>& z, float ws, Pack<T>& o) const {
    const F2 neg = pack2(-r, -r), c2 = pack2(c, c), ws2 = pack2(ws, ws);
#pragma unroll
    for (int j = 0; j < Elem<T>::V / 2; ++j) {
      const float2 x = unpack2(fma2(up2(z, j), c2, neg));
      const float2 y = unpack2(mul2(pack2(ex2(x.x), ex2(x.y)), ws2));
      down2(o, j, y.x, y.y);
    }
  }
};

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_pack(const Pack<T>& o, T* to) {
  if (ALIGNED) {
    __stcs(reinterpret_cast<uint4*>(to), reinterpret_cast<const uint4&>(o));   // (not to push logits out of L2)
  } else {
#pragma unroll
    for (int j = 0; j < Elem<T>::V; ++j) to[j] = o.v[j];
  }
}

// the gradient of packs tid, tid + THREADS, ... to out; held and hold as above
template <typename T, int THREADS, int AHEAD, bool ALIGNED>
__device__ __forceinline__ void emit_grad(const Softmax<T>& x, float ws, const Pack<T>* packs, int nv, int tid, T* out,
                                          const Pack<T>* held, int hold) {
  constexpr int VL = Elem<T>::V;
  int i = tid;
  for (; i < hold && i + (AHEAD - 1) * THREADS < nv; i += AHEAD * THREADS) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      Pack<T> o;
      x.pack(held[i + a * THREADS], ws, o);
      store_pack<T, ALIGNED>(o, out + (int64_t)(i + a * THREADS) * VL);
    }
  }
  for (; i + (AHEAD - 1) * THREADS < nv; i += AHEAD * THREADS) {
    Pack<T> p[AHEAD];
    const Pack<T>* from = packs + i;
    T* to = out + (int64_t)i * VL;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {             // (read for the last time)
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(from + a * THREADS));
      p[a] = reinterpret_cast<const Pack<T>&>(u);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      Pack<T> o;
      x.pack(p[a], ws, o);
      store_pack<T, ALIGNED>(o, to + a * THREADS * VL);
    }
  }
  for (; i < nv; i += THREADS) {
    Pack<T> o;
    x.pack(packs[i], ws, o);
    store_pack<T, ALIGNED>(o, out + (int64_t)i * VL);
  }
}

// A far row's sum, from its maximum: (z - all) c cannot overflow upwards
template <typename T, int WARPS, typename F>
__device__ __forceinline__ float far_sum(const T* z, int V, int tid, float all, float c, float2* buf, F barrier) {
  float s = 0.f;
  for (int v = tid; v < V; v += WARPS * 32) s += ex2((Elem<T>::up(z[v]) - all) * c);
  s = warp_sum(s);
  if (WARPS > 1) {
    barrier();                      // buf has been read
    if ((tid & 31) == 0) buf[tid >> 5].y = s;
    barrier();
    s = warp_sum((tid & 31) < WARPS ? buf[tid & 31].y : 0.f);
  }
  return s;
}

// A row's entries in shared memory, K of each: index (-1: absent), probability
// and the student's logit there.
struct Entries {
  float* at;
  int K;
  __device__ __forceinline__ int& id(int k) const { return reinterpret_cast<int*>(at)[k]; }
  __device__ __forceinline__ float& q(int k) const { return at[K + k]; }
  __device__ __forceinline__ float& zk(int k) const { return at[2 * K + k]; }
};

// an entry as it is read: its index, or -1, and its logit
struct Entry {
  int id;
  float t;
};
__device__ __forceinline__ Entry load_entry(const Teacher& te, int r, int k, int V) {
  const int64_t i = load_id(te.idx, te.id64, (int64_t)r * te.ldt + k);
  const float t = load_t(te.t, te.t_type, (int64_t)r * te.ldt + k);
  return Entry{counts(i, V, t) ? (int)i : -1, t};
}

// Entry k's logit in e.q becomes its probability; returns its part q log q of the loss.
__device__ __forceinline__ float weigh_entry(const Entries& e, int k, const RowStat& st, float inv_T) {
  const float lq = (e.q(k) - st.top) * inv_T - st.log_sum;
  const float q = e.id(k) >= 0 ? expf(lq) : 0.f;
  e.q(k) = q;
  return q == 0.f ? 0.f : q * lq;
}

// entry k's part -q log p of the loss (q = 0: nothing, whatever p is)
template <typename T>
__device__ __forceinline__ float cross(const Entries& e, int k, const Softmax<T>& x, float log2_s) {
  const float q = e.q(k);
  return q == 0.f ? 0.f : q * ((log2_s - x.log2_e(e.zk(k))) * 0.6931471805599453f);
}

// The gradient at entry k, w (p - q).  Where an index may be there twice, the
// first of its entries writes for all.
template <typename T>
__device__ __forceinline__ void correct(const Entries& e, int K, int k, bool twice, const Softmax<T>& x, float w, T* dz) {
  const int id = e.id(k);
  if (id < 0) return;
  bool mine = true;
  float sum = e.q(k);
  if (twice) {
    sum = 0.f;
    for (int i = 0; i < K; ++i)
      if (e.id(i) == id) {
        if (i < k) mine = false;
        sum += e.q(i);
      }
  }
  if (mine) dz[id] = Elem<T>::down(w * (ex2(x.log2_e(e.zk(k))) / x.s - sum));
}

template <typename T>
__device__ __forceinline__ void zero_row(T* dz, int V, int tid, int threads) {
  const RowView<T> v(dz, V);
  Pack<T> o;
#pragma unroll
  for (int j = 0; j < Elem<T>::V; ++j) o.v[j] = Elem<T>::down(0.f);
  for (int i = tid; i < v.nv; i += threads) *reinterpret_cast<Pack<T>*>(dz + v.head + (int64_t)i * Elem<T>::V) = o;
  if (tid < v.head) dz[tid] = o.v[0];
  if (v.tail() + tid < V) dz[v.tail() + tid] = o.v[0];
}

// ROW_THREADS threads take a row: a block, or a warp (short rows, four a block).
// Bound by the bytes: the row is read for the maximum and sum of the softmax,
// and a second time, from L2, for the gradient, which is written.  8192 x 50304
// bf16 with 64 entries: 336 us for the call, 310 of them here, 5.3 TB/s of
// DRAM (818 MB read, as if the second reading were free, and 824 written); loss
// only, 3001 x 32003 fp16, 33 entries: 44 for the call.  What counts
// is that there are always loads on their way: several blocks on an SM, in
// different parts of their rows, do better than rows kept in shared memory and
// loaded a row ahead, of which two fit (8192 x 32003 bf16, 64 entries: 217 us
// against 262), because those fall into step, all waiting for memory and then
// all computing.
// The first blocks start before k_distill_teacher is done (everything before it
// is) and wait for it where they need its results; behind them rows without
// entries are known before their logits are read.
constexpr int kBlocks = 5;      // of 256 threads on an SM
// the registers that this leaves are enough (fp16's conversions take more; the
// 512-thread gradient keeps a few bytes elsewhere, for a third block)
template <typename T, int ROW_THREADS>
constexpr int min_blocks() {
  return ROW_THREADS == 512 ? 3 : ROW_THREADS == 32 ? (Elem<T>::kHalf ? 8 : 9) : (kBlocks - (Elem<T>::kHalf ? 1 : 0)) * (256 / ROW_THREADS);
}
// packs a thread loads before it uses the first; the loss alone leaves room for more
constexpr int kAhead = 2;
template <int ROW_THREADS, bool GRAD>
constexpr int first_ahead() {
  return !GRAD && ROW_THREADS == 128 ? 4 : kAhead;
}
template <typename T, int ROW_THREADS, bool GRAD, bool FEW>
__global__ void __launch_bounds__(ROW_THREADS == 32 ? 128 : ROW_THREADS, FEW ? 2 : min_blocks<T, ROW_THREADS>())
    k_distill_rows(const RowMap map, const Teacher te, const RowStat* stat, const int* kinds,
                   const T* Z, int64_t ldz, int V, float temperature, float gscale, int* count, float* row_loss, T* dZ,
                   int64_t ldd, int early, int hold, int* arrived, float* loss_out, int32_t* count_out) {
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1, WARPS = ROW_THREADS / 32;
  extern __shared__ uint4 shared[];               // `hold` packs; per row: 3 arrays of K
  __shared__ float2 buf[WARPS];
  __shared__ float losses[WARPS];
  __shared__ double sums[WARPS];
  __shared__ float4 kept[ROWS];
  __shared__ int is_last;
  const bool first = (int)blockIdx.x < early;
  if (!first) griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x % ROW_THREADS, in_block = threadIdx.x / ROW_THREADS;
  const int r = blockIdx.x * ROWS + in_block;
  const int K = te.K;
  Pack<T>* held = reinterpret_cast<Pack<T>*>(shared);
  float* entries = reinterpret_cast<float*>(shared + hold);
  auto sync = [&] {
    if (ROW_THREADS == 32) __syncwarp();
    else __syncthreads();
  };
  const float inv_T = 1.f / temperature, c = inv_T * 1.4426950408889634f;
  if (r >= map.start[map.M]) {                    // (a whole warp)
    if (first) griddep_wait();
    return;
  }
  const int m = worker_of(map.start, map.M, r);
  // With FEW rows, the one that is done last adds up its worker's losses, in
  // order, and leaves both of the worker's counters at zero.
  auto finish = [&] {
    if (!FEW) return;
    if (blockIdx.x == 0 && in_block == 0)
      for (int i = tid; i < map.M; i += ROW_THREADS)
        if (map.start[i] == map.start[i + 1]) {
          loss_out[i] = 0.f;
          if (count_out != nullptr) count_out[i] = 0;
        }
    int last = 0;
    if (tid == 0) {
      __threadfence();
      last = atomicAdd(&arrived[m], 1) == map.start[m + 1] - map.start[m] - 1;
    }
    if (ROW_THREADS == 32) {
      last = __shfl_sync(0xffffffffu, last, 0);
    } else {
      if (tid == 0) is_last = last;
      __syncthreads();
      last = is_last;
    }
    if (!last) return;
    __threadfence();
    double t = 0.0;
    for (int i = map.start[m] + tid; i < map.start[m + 1]; i += ROW_THREADS) t += (double)__ldcg(row_loss + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (ROW_THREADS > 32) {
      if ((tid & 31) == 0) sums[tid >> 5] = t;
      __syncthreads();
      t = 0.0;
      for (int i = 0; i < WARPS; ++i) t += sums[i];
    }
    if (tid == 0) {
      const int n = count[m];
      count[m] = arrived[m] = 0;
      loss_out[m] = n > 0 ? (float)(t / n) : 0.f;
      if (count_out != nullptr) count_out[m] = n;
    }
  };
  T* dz = GRAD ? dZ + (int64_t)r * ldd : nullptr;
  int kind = first ? (int)ROW_ONCE : kinds[r];
  const RowView<T> v(Z + (int64_t)r * ldz, V);
  const Entries e{entries + in_block * 3 * K, K};
  if (kind != ROW_NONE) {
    for (int k = tid; k < K; k += ROW_THREADS) {
      const Entry x = load_entry(te, r, k, V);
      e.id(k) = x.id;
      e.q(k) = x.t;
      e.zk(k) = x.id >= 0 ? Elem<T>::up(v.z[x.id]) : 0.f;
    }
  }
  Running run;
  if (kind != ROW_NONE) {
    absorb<T, ROW_THREADS, first_ahead<ROW_THREADS, GRAD>()>(run, v.packs(), v.nv, tid, c, held, GRAD ? hold : 0);
    if (tid < v.head) run.one(Elem<T>::up(v.z[tid]), c);
    if (v.tail() + tid < V) run.one(Elem<T>::up(v.z[v.tail() + tid]), c);
  }
  if (first) {
    griddep_wait();
    kind = kinds[r];
  }
  if (kind == ROW_NONE) {
    if (GRAD) zero_row(dz, V, tid, ROW_THREADS);
    if (tid == 0) row_loss[r] = 0.f;
    finish();
    return;
  }
  float loss = 0.f;
  if (tid < K) {
    const RowStat st = stat[r];
    for (int k = tid; k < K; k += ROW_THREADS) loss += weigh_entry(e, k, st, inv_T);
  }
  float all, s;
  join_row<WARPS>(run, tid, c, buf, sync, all, s);
  Softmax<T> x(all, s, c);
  if (x.far) x.s = far_sum<T, WARPS>(v.z, V, tid, all, c, buf, sync);
  if ((tid & ~31) < K) {                          // (warps beyond K have nothing to add)
    const float log2_s = log2f(x.s);
    for (int k = tid; k < K; k += ROW_THREADS) loss += cross(e, k, x, log2_s);
    loss = warp_sum(loss);
  }
  if (WARPS > 1 && (tid & 31) == 0) losses[tid >> 5] = loss;
  if (GRAD) {
    const float w = gscale * temperature / (float)count[m], ws = w / x.s;
    if (tid == 0) kept[in_block] = make_float4(x.all, x.s, w, kind == ROW_TWICE ? 1.f : 0.f);
    if (x.far) {
      for (int i = tid; i < V; i += ROW_THREADS) dz[i] = x.grad(Elem<T>::up(v.z[i]), w);
    } else {
      if (RowView<T>(dz, V).mis == v.mis) emit_grad<T, ROW_THREADS, kAhead, true>(x, ws, v.packs(), v.nv, tid, dz + v.head, held, hold);
      else emit_grad<T, ROW_THREADS, kAhead, false>(x, ws, v.packs(), v.nv, tid, dz + v.head, held, hold);
      if (tid < v.head) dz[tid] = x.grad(Elem<T>::up(v.z[tid]), w);
      if (v.tail() + tid < V) dz[v.tail() + tid] = x.grad(Elem<T>::up(v.z[v.tail() + tid]), w);
    }
    // (what is needed behind the gradient waits in shared memory: its loop has
    // no registers to spare)
    sync();
    const float4 was = kept[in_block];
    const Softmax<T> y(was.x, was.y, c);
    for (int k = tid; k < K; k += ROW_THREADS) correct(e, K, k, was.w != 0.f, y, was.z, dz);
  } else {
    sync();
  }
  if (tid == 0) {
    if (WARPS > 1) {
      loss = 0.f;
      for (int i = 0; i < WARPS; ++i) loss += losses[i];
    }
    row_loss[r] = loss * (temperature * temperature);
  }
  finish();
}

// loss[m], count[m]; leaves the counters at zero for the next call.  A block per
// worker: 5 us, launch included.
__global__ void __launch_bounds__(256) k_distill_loss(const RowMap map, const float* row_loss, int* count,
                                                      float* __restrict__ loss, int32_t* __restrict__ count_out) {
  __shared__ double buf[256];
  griddep_wait();
  griddep_launch();
  const int m = blockIdx.x;
  double s = 0.0;
  for (int r = map.start[m] + threadIdx.x; r < map.start[m + 1]; r += 256) s += (double)row_loss[r];
  buf[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) buf[threadIdx.x] += buf[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int n = count[m];
    count[m] = 0;
    loss[m] = n > 0 ? (float)(buf[0] / n) : 0.f;
    if (count_out != nullptr) count_out[m] = n;
  }
}

struct Scratch {
  RowStat* stat;
  int* kind;
};

// Calls of so few rows add up the losses in the rows' kernel: that saves a
// launch (about 2.5 us), but each row ends a round trip to L2 later.
constexpr int kFewRows = 1024;
constexpr int64_t kL2Bytes = 50'000'000;

template <typename T, int ROW_THREADS, bool GRAD, bool FEW>
void run_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te, const Scratch& x) {
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1;
  size_t smem = (size_t)ROWS * 3 * a.K * 4;
  auto* kernel = k_distill_rows<T, ROW_THREADS, GRAD, FEW>;
  int hold = 0;
  if (GRAD && ROW_THREADS >= 256) {
    // What the rows on their way have in L2 must stay within half of it, or the
    // second reading misses it: where it would not, the rows' first packs are
    // held in shared memory, and the longest rows go with fewer blocks.
    constexpr int BATCH = ROW_THREADS * kAhead;
    const int64_t row = a.V * (int64_t)sizeof(T);
    int blocks = min_blocks<T, ROW_THREADS>();
    if (num_sms() * blocks * row <= kL2Bytes) blocks = 0;
    for (; blocks >= 1; --blocks) {
      const int64_t room = ((int64_t)226 * 1024 / blocks - 1536 - (int64_t)smem) / 16, packs = row / 16;
      hold = (int)((room < 0 ? 0 : room < packs ? room : packs) / BATCH * BATCH);
      if (num_sms() * blocks * (row - hold * (int64_t)16) <= kL2Bytes) break;
    }
    smem += (size_t)hold * 16;
  }
  if (smem > 32 * 1024) allow_shared((const void*)kernel);
  const int blocks = (map.start[map.M] + ROWS - 1) / ROWS;
  const int early = num_sms() * resident_per_sm((const void*)kernel, ROWS * ROW_THREADS, smem);
  count_launch();
  launch_pdl(kernel, dim3(blocks), dim3(ROWS * ROW_THREADS), smem, s, map, te, (const RowStat*)x.stat,
             (const int*)x.kind, reinterpret_cast<const T*>(a.Z), a.ldz, (int)a.V, a.temperature, a.gscale,
             a.count, a.row_loss, reinterpret_cast<T*>(a.dZ), a.ldd, early, hold,
             a.count + kMaxWorkers, a.loss, a.count_out);
}

// Few threads for short rows, so that each has something to load: 16384 rows
// with gradient of 4000 bf16 take 73 / 89 / 131 us with 32 / 128 / 256 threads,
// of 16000 bf16 273 / 202 / 241, of 16000 fp32 551 / 441 / 378; 8192 rows of
// 50304 bf16 351 with 256 and 325 with 512, of 32003 221 and 246, for which
// L2 is large enough either way.  The loss alone does without L2, and better with
// few threads for longer rows too, as long as there are rows for two rounds of
// them: 8192 x 32003 fp16 97 us with 128 and 115 with 256, 8192 x 50304 bf16 139
// and 145, but 1500 x 50304 40 and 38, 4096 x 128256 171 and 168.  (Calls one
// behind the other on two inputs in turn; with more of them the 325 are 336.)
template <typename T, bool GRAD, bool FEW>
void pick_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te, const Scratch& x) {
  const int64_t row = a.V * (int64_t)sizeof(T);
  if (row <= 16 * 1024) run_rows<T, 32, GRAD, FEW>(s, a, map, te, x);
  else if (row <= 48 * 1024 || (!GRAD && row <= 128 * 1024 && map.start[map.M] >= 2 * num_sms() * min_blocks<T, 128>()))
    run_rows<T, 128, GRAD, FEW>(s, a, map, te, x);
  else if (row <= 80 * 1024) run_rows<T, 256, GRAD, FEW>(s, a, map, te, x);
  else run_rows<T, GRAD ? 512 : 256, GRAD, FEW>(s, a, map, te, x);
}

}  // namespace

void launch_distill(cudaStream_t s, const DistillArgs& a, const int* start, int M) {
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  const int N = start[M];
  const Teacher te{a.idx, a.id64, a.t, a.t_type, a.ldt, a.K};
  if (N > 0) {
    const Scratch x{reinterpret_cast<RowStat*>(a.scratch), reinterpret_cast<int*>(a.scratch) + 2 * (int64_t)N};
    const float inv_T = 1.f / a.temperature;
    count_launch();
    if (a.K <= 128)
      launch_pdl(k_distill_teacher<32>, dim3((unsigned)((N + 7LL) / 8)), dim3(256), 0, s, map, te, a.V, inv_T, x.stat,
                 x.kind, a.count, a.status);
    else
      launch_pdl(k_distill_teacher<256>, dim3(N), dim3(256), 0, s, map, te, a.V, inv_T, x.stat, x.kind, a.count,
                 a.status);
#define SM_FEW(T, GRAD) (N <= kFewRows ? pick_rows<T, GRAD, true>(s, a, map, te, x) : pick_rows<T, GRAD, false>(s, a, map, te, x))
#define SM_PICK(T) (a.dZ != nullptr ? SM_FEW(T, true) : SM_FEW(T, false))
    if (a.type == LT_F32) SM_PICK(float);
    else if (a.type == LT_BF16) SM_PICK(__nv_bfloat16);
    else SM_PICK(__half);
#undef SM_PICK
#undef SM_FEW
  }
  if (N > 0 && N <= kFewRows) return;
  count_launch();
  launch_pdl(k_distill_loss, dim3(M), dim3(256), 0, s, map, (const float*)a.row_loss, a.count, a.loss, a.count_out);
}

}  // namespace sm
