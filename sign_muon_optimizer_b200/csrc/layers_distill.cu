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
// The rounding of R is common to every term and cancels in p.  R is at least
// -1e37, so that logits of -inf or of the type's lowest value add 0 to s; rows
// whose own maximum is out of range are `far` and done over, term by term.
constexpr float kFar = 1e37f;
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
  int mis, head, nv, tail, n_tail;   // tail = head + nv * V; n_tail elements from there on
  __device__ __forceinline__ RowView(const T* row, int64_t V) : z(row) {
    constexpr int VL = Elem<T>::V;
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    head = (int)(V < (VL - mis) % VL ? V : (VL - mis) % VL);
    nv = (int)((V - head) / VL);
    tail = head + nv * VL;
    n_tail = (int)(V - tail);
  }
  __device__ __forceinline__ const Pack<T>* packs() const { return reinterpret_cast<const Pack<T>*>(z + head); }
};

constexpr int kAhead = 4;   // packs loaded before the first is used

// Pass 1: packs tid, tid + THREADS, ... of nv into the running softmax;
// after(i, n) follows when n packs from pack i on (THREADS apart) are done.
template <typename T, int THREADS, typename F>
__device__ __forceinline__ void absorb(Running& run, const Pack<T>* packs, int nv, int tid, float c, F after) {
  constexpr int VL = Elem<T>::V;
  const F2 c2 = pack2(c, c);
  auto take = [&](const Pack<T>& p, F2 neg, F2& sum) {
#pragma unroll
    for (int j = 0; j < VL / 2; ++j) {
      const float2 x = unpack2(fma2(up2(p, j), c2, neg));
      sum = add2(pack2(ex2(x.x), ex2(x.y)), sum);
    }
  };
  int i = tid;
  for (; i + (kAhead - 1) * THREADS < nv; i += kAhead * THREADS) {
    Pack<T> p[kAhead];
    const Pack<T>* from = packs + i;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) p[a] = from[a * THREADS];
    float t = pack_max(p[0]);
#pragma unroll
    for (int a = 1; a < kAhead; ++a) t = fmaxf(t, pack_max(p[a]));
    const float r = run.raise(t, c);
    const F2 neg = pack2(-r, -r);
    F2 sum = 0ull;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) take(p[a], neg, sum);
    run.s += sum2(sum);
    after(i, kAhead);
  }
  for (; i < nv; i += THREADS) {
    const Pack<T> p = packs[i];
    const float r = run.raise(pack_max(p), c);
    F2 sum = 0ull;
    take(p, pack2(-r, -r), sum);
    run.s += sum2(sum);
    after(i, 1);
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
    *reinterpret_cast<Pack<T>*>(to) = o;
  } else {
#pragma unroll
    for (int j = 0; j < Elem<T>::V; ++j) to[j] = o.v[j];
  }
}

// Pass 2: the gradient of packs tid, tid + THREADS, ... to out; after as above
template <typename T, int THREADS, bool ALIGNED, typename F>
__device__ __forceinline__ void emit_grad(const Softmax<T>& x, float ws, const Pack<T>* packs, int nv, int tid, T* out,
                                          F after) {
  constexpr int VL = Elem<T>::V;
  int i = tid;
  for (; i + (kAhead - 1) * THREADS < nv; i += kAhead * THREADS) {
    Pack<T> p[kAhead];
    const Pack<T>* from = packs + i;
    T* to = out + (int64_t)i * VL;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) p[a] = from[a * THREADS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      Pack<T> o;
      x.pack(p[a], ws, o);
      store_pack<T, ALIGNED>(o, to + a * THREADS * VL);
    }
    after(i, kAhead);
  }
  for (; i < nv; i += THREADS) {
    Pack<T> o;
    x.pack(packs[i], ws, o);
    store_pack<T, ALIGNED>(o, out + (int64_t)i * VL);
    after(i, 1);
  }
}

// A far row's sum, from its maximum: (z - all) c cannot overflow upwards
template <typename T, int WARPS, typename F>
__device__ __forceinline__ float far_sum(const T* z, int64_t V, int tid, float all, float c, float2* buf, F barrier) {
  float s = 0.f;
  for (int64_t v = tid; v < V; v += WARPS * 32) s += ex2((Elem<T>::up(z[v]) - all) * c);
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
  int* id;
  float *q, *zk;
  __device__ __forceinline__ Entries(float* at, int K) : id(reinterpret_cast<int*>(at)), q(at + K), zk(at + 2 * K) {}
};

// an entry as it is read: its index, or -1, and its logit
struct Entry {
  int id;
  float t;
};
__device__ __forceinline__ Entry load_entry(const Teacher& te, int r, int k, int64_t V) {
  const int64_t i = load_id(te.idx, te.id64, (int64_t)r * te.ldt + k);
  const float t = load_t(te.t, te.t_type, (int64_t)r * te.ldt + k);
  return Entry{counts(i, V, t) ? (int)i : -1, t};
}

// Entry k into shared memory; returns its part q log q of the loss.
__device__ __forceinline__ float put_entry(const Entries& e, int k, const Entry& x, float zk, const RowStat& st, float inv_T) {
  const float lq = (x.t - st.top) * inv_T - st.log_sum;
  const float q = x.id >= 0 ? expf(lq) : 0.f;
  e.id[k] = x.id;
  e.q[k] = q;
  e.zk[k] = zk;
  return q == 0.f ? 0.f : q * lq;
}

// entry k's part -q log p of the loss (q = 0: nothing, whatever p is)
template <typename T>
__device__ __forceinline__ float cross(const Entries& e, int k, const Softmax<T>& x, float log2_s) {
  const float q = e.q[k];
  return q == 0.f ? 0.f : q * ((log2_s - x.log2_e(e.zk[k])) * 0.6931471805599453f);
}

// The gradient at entry k, w (p - q).  Where an index may be there twice, the
// first of its entries writes for all.
template <typename T>
__device__ __forceinline__ void correct(const Entries& e, int K, int k, bool twice, const Softmax<T>& x, float w, T* dz) {
  const int id = e.id[k];
  if (id < 0) return;
  bool mine = true;
  float sum = e.q[k];
  if (twice) {
    sum = 0.f;
    for (int i = 0; i < K; ++i)
      if (e.id[i] == id) {
        if (i < k) mine = false;
        sum += e.q[i];
      }
  }
  if (mine) dz[id] = Elem<T>::down(w * (ex2(x.log2_e(e.zk[k])) / x.s - sum));
}

template <typename T>
__device__ __forceinline__ void zero_row(T* dz, int64_t V, int tid, int threads) {
  const RowView<T> v(dz, V);
  Pack<T> o;
#pragma unroll
  for (int j = 0; j < Elem<T>::V; ++j) o.v[j] = Elem<T>::down(0.f);
  for (int i = tid; i < v.nv; i += threads) *reinterpret_cast<Pack<T>*>(dz + v.head + (int64_t)i * Elem<T>::V) = o;
  if (tid < v.head) dz[tid] = o.v[0];
  if (tid < v.n_tail) dz[v.tail + tid] = o.v[0];
}

// ROW_THREADS threads hold a row: a block (rows too long for shared memory), or
// a warp (short rows, four a block).  The row is read twice, for the maximum
// and sum of the softmax and for the gradient (the second time from L2).
template <typename T, int ROW_THREADS>
__global__ void __launch_bounds__(ROW_THREADS == 32 ? 128 : ROW_THREADS, ROW_THREADS == 32 ? 6 : 3)
    k_distill_rows(const RowMap map, const Teacher te, const RowStat* __restrict__ stat, const int* __restrict__ kinds,
                   const T* Z, int64_t ldz, int64_t V, float temperature, float gscale, const int* __restrict__ count,
                   float* __restrict__ row_loss, T* dZ, int64_t ldd) {
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1, WARPS = ROW_THREADS / 32;
  extern __shared__ float entries[];              // per row: 3 arrays of K
  __shared__ float2 buf[WARPS];
  __shared__ float losses[WARPS];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x % ROW_THREADS, in_block = threadIdx.x / ROW_THREADS;
  const int r = blockIdx.x * ROWS + in_block;
  if (r >= map.start[map.M]) return;              // (a whole warp)
  const Entries e(entries + (int64_t)in_block * 3 * te.K, te.K);
  auto sync = [&] {
    if (ROW_THREADS == 32) __syncwarp();
    else __syncthreads();
  };
  const float inv_T = 1.f / temperature, c = inv_T * 1.4426950408889634f;
  const RowView<T> v(Z + (int64_t)r * ldz, V);
  T* dz = dZ != nullptr ? dZ + (int64_t)r * ldd : nullptr;
  const int kind = kinds[r];
  if (kind == ROW_NONE) {
    if (dz != nullptr) zero_row(dz, V, tid, ROW_THREADS);
    if (tid == 0) row_loss[r] = 0.f;
    return;
  }
  float loss = 0.f;
  {
    const RowStat st = stat[r];
    for (int k = tid; k < te.K; k += ROW_THREADS) {
      const Entry x = load_entry(te, r, k, V);
      loss += put_entry(e, k, x, x.id >= 0 ? Elem<T>::up(v.z[x.id]) : 0.f, st, inv_T);
    }
  }
  Running run;
  absorb<T, ROW_THREADS>(run, v.packs(), v.nv, tid, c, [](int, int) {});
  if (tid < v.head) run.one(Elem<T>::up(v.z[tid]), c);
  if (tid < v.n_tail) run.one(Elem<T>::up(v.z[v.tail + tid]), c);
  float all, s;
  join_row<WARPS>(run, tid, c, buf, sync, all, s);
  Softmax<T> x(all, s, c);
  if (x.far) x.s = far_sum<T, WARPS>(v.z, V, tid, all, c, buf, sync);
  const float log2_s = log2f(x.s);
  for (int k = tid; k < te.K; k += ROW_THREADS) loss += cross(e, k, x, log2_s);
  loss = warp_sum(loss);
  if (WARPS > 1 && (tid & 31) == 0) losses[tid >> 5] = loss;
  if (dz != nullptr) {
    const float w = gscale * temperature / (float)count[worker_of(map.start, map.M, r)], ws = w / x.s;
    if (x.far) {
      for (int64_t i = tid; i < V; i += ROW_THREADS) dz[i] = x.grad(Elem<T>::up(v.z[i]), w);
    } else {
      if (RowView<T>(dz, V).mis == v.mis) emit_grad<T, ROW_THREADS, true>(x, ws, v.packs(), v.nv, tid, dz + v.head, [](int, int) {});
      else emit_grad<T, ROW_THREADS, false>(x, ws, v.packs(), v.nv, tid, dz + v.head, [](int, int) {});
      if (tid < v.head) dz[tid] = x.grad(Elem<T>::up(v.z[tid]), w);
      if (tid < v.n_tail) dz[v.tail + tid] = x.grad(Elem<T>::up(v.z[v.tail + tid]), w);
    }
    sync();
    for (int k = tid; k < te.K; k += ROW_THREADS) correct(e, te.K, k, kind == ROW_TWICE, x, w, dz);
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
}

// A block stays and takes row after row, each in shared memory: the next row
// comes in through asynchronous copies while this one's gradient goes out (or,
// for the loss alone, while its sum is made), pack by pack into the places that
// the same thread has just read.  The next row's entries are loaded a row ahead
// too, the logits there at the row's start.  Two blocks on an SM.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 128 ? 2 : 6)
    k_distill_resident(const RowMap map, const Teacher te, const RowStat* __restrict__ stat,
                       const int* __restrict__ kinds, const T* Z, int64_t ldz, int64_t V, int slots, float temperature,
                       float gscale, const int* __restrict__ count, float* __restrict__ row_loss, T* dZ, int64_t ldd) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ uint4 row_at[];               // `slots` packs, then twice 3 arrays of K
  __shared__ float2 buf[2][WARPS];
  __shared__ float losses[2][WARPS];
  griddep_wait();
  griddep_launch();
  float* entries = reinterpret_cast<float*>(row_at + slots);
  const int N = map.start[map.M], step = gridDim.x;
  const int tid = threadIdx.x, K = te.K;
  const float inv_T = 1.f / temperature, c = inv_T * 1.4426950408889634f;
  const Pack<T>* packs = reinterpret_cast<const Pack<T>*>(row_at);
  auto sync = [] { __syncthreads(); };
  const unsigned slot = (unsigned)__cvta_generic_to_shared(row_at);
  // packs i, i + THREADS, ..., n of them, of the next row
  auto fetch = [&](const Pack<T>* from, int nv, int i, int n) {
    from += i;
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (a < n && i + a * THREADS < nv)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + (i + a * THREADS) * 16), "l"(from + a * THREADS)
                     : "memory");
  };
  auto finish_loss = [&](int r, int b) {          // thread 0, behind a barrier
    float t = 0.f;
    for (int i = 0; i < WARPS; ++i) t += losses[b][i];
    row_loss[r] = t * (temperature * temperature);
  };
  int b = 0, r = blockIdx.x;
  // this row's and the next one's kind; this row's first entry of the thread
  int kind = kinds[r], kind1 = r + step < N ? kinds[r + step] : ROW_NONE;
  Entry x0 = tid < K ? load_entry(te, r, tid, V) : Entry{-1, 0.f};
  RowStat st = stat[r];
  if (kind != ROW_NONE) {
    const RowView<T> v(Z + (int64_t)r * ldz, V);
    for (int i = tid; i < v.nv; i += THREADS) fetch(v.packs(), v.nv, i, 1);
  }
  for (; r < N; r += step) {
    const RowView<T> v(Z + (int64_t)r * ldz, V);
    const Entries e(entries + b * 3 * K, K);
    // loads whose results are wanted later: the logits at the entries, the
    // row's edges, the worker's count; the next row's first entries, the kind
    // of the row behind it
    const float zk = kind != ROW_NONE && x0.id >= 0 ? Elem<T>::up(v.z[x0.id]) : 0.f;
    const float edge0 = tid < v.head ? Elem<T>::up(v.z[tid]) : -INFINITY;
    const float edge1 = tid < v.n_tail ? Elem<T>::up(v.z[v.tail + tid]) : -INFINITY;
    const float n = dZ != nullptr ? (float)count[worker_of(map.start, map.M, r)] : 1.f;
    const int64_t r1 = (int64_t)r + step, r2 = r1 + step;
    Entry x1{-1, 0.f};
    RowStat st1 = st;
    if (r1 < N) {
      if (tid < K) x1 = load_entry(te, (int)r1, tid, V);
      st1 = stat[r1];
    }
    const int kind2 = r2 < N ? kinds[r2] : ROW_NONE;
    const RowView<T> next(Z + (r1 < N ? r1 : (int64_t)r) * ldz, V);
    const Pack<T>* next_packs = next.packs();
    const int next_nv = kind1 != ROW_NONE ? next.nv : 0;
    auto after = [&](int i, int k) { fetch(next_packs, next_nv, i, k); };
    T* dz = dZ != nullptr ? dZ + (int64_t)r * ldd : nullptr;
    if (kind != ROW_NONE) {
      copy_commit();
      copy_wait<0>();
      Running run;
      if (dz != nullptr) absorb<T, THREADS>(run, packs, v.nv, tid, c, [](int, int) {});
      else absorb<T, THREADS>(run, packs, v.nv, tid, c, after);
      if (tid < v.head) run.one(edge0, c);
      if (tid < v.n_tail) run.one(edge1, c);
      float loss = 0.f;
      if (tid < K) loss = put_entry(e, tid, x0, zk, st, inv_T);
      for (int k = tid + THREADS; k < K; k += THREADS) {
        const Entry y = load_entry(te, r, k, V);
        loss += put_entry(e, k, y, y.id >= 0 ? Elem<T>::up(v.z[y.id]) : 0.f, st, inv_T);
      }
      float all, s;
      join_row<WARPS>(run, tid, c, buf[b], sync, all, s);
      Softmax<T> x(all, s, c);
      if (x.far) x.s = far_sum<T, WARPS>(v.z, V, tid, all, c, buf[b], sync);
      const float log2_s = log2f(x.s);
      for (int k = tid; k < K; k += THREADS) loss += cross(e, k, x, log2_s);
      loss = warp_sum(loss);
      if ((tid & 31) == 0) losses[b][tid >> 5] = loss;
      int done = tid;                             // the first pack of this thread's that is not yet sent for
      while (done < v.nv) done += THREADS;
      if (dz != nullptr) {
        const float w = gscale * temperature / n, ws = w / x.s;
        if (x.far) {
          for (int64_t i = tid; i < V; i += THREADS) dz[i] = x.grad(Elem<T>::up(v.z[i]), w);
          done = tid;
        } else {
          if (RowView<T>(dz, V).mis == v.mis) emit_grad<T, THREADS, true>(x, ws, packs, v.nv, tid, dz + v.head, after);
          else emit_grad<T, THREADS, false>(x, ws, packs, v.nv, tid, dz + v.head, after);
          if (tid < v.head) dz[tid] = x.grad(edge0, w);
          if (tid < v.n_tail) dz[v.tail + tid] = x.grad(edge1, w);
        }
        for (; done < next_nv; done += THREADS) fetch(next_packs, next_nv, done, 1);
        __syncthreads();                          // the row's gradient is written
        for (int k = tid; k < K; k += THREADS) correct(e, K, k, kind == ROW_TWICE, x, w, dz);
      } else {
        for (; done < next_nv; done += THREADS) fetch(next_packs, next_nv, done, 1);
        __syncthreads();                          // the row's losses are in place
      }
      if (tid == 0) finish_loss(r, b);
      b ^= 1;                                     // two barriers lie before these buffers are used again
    } else {
      if (dz != nullptr) zero_row(dz, V, tid, THREADS);
      if (tid == 0) row_loss[r] = 0.f;
      for (int i = tid; i < next_nv; i += THREADS) fetch(next_packs, next_nv, i, 1);
    }
    kind = kind1;
    kind1 = kind2;
    x0 = x1;
    st = st1;
  }
}

// loss[m], count[m]; leaves the counters at zero for the next call
__global__ void __launch_bounds__(256) k_distill_loss(const RowMap map, const float* __restrict__ row_loss, int* count,
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

template <typename T, int ROW_THREADS>
void run_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te, const Scratch& x) {
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1;
  const size_t smem = (size_t)ROWS * 3 * a.K * 4;
  auto* kernel = k_distill_rows<T, ROW_THREADS>;
  if (smem > 32 * 1024) cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  count_launch();
  launch_pdl(kernel, dim3((map.start[map.M] + ROWS - 1) / ROWS), dim3(ROWS * ROW_THREADS), smem, s, map, te,
             (const RowStat*)x.stat, (const int*)x.kind, reinterpret_cast<const T*>(a.Z), a.ldz, a.V, a.temperature,
             a.gscale, (const int*)a.count, a.row_loss, reinterpret_cast<T*>(a.dZ), a.ldd);
}

int resident_slots(const DistillArgs& a, int elem, int threads) {
  const int64_t packs = a.V * elem / 16;
  return (int)((packs + threads - 1) / threads * threads);
}

template <typename T, int THREADS>
void run_resident(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te, const Scratch& x) {
  auto* kernel = k_distill_resident<T, THREADS>;
  const int slots = resident_slots(a, sizeof(T), THREADS);
  const size_t smem = (size_t)slots * 16 + (size_t)2 * 3 * a.K * 4;
  if (smem > 32 * 1024) cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  const int grid = stream_grid((const void*)kernel, THREADS, smem, map.start[map.M], 16);
  count_launch();
  launch_pdl(kernel, dim3(grid), dim3(THREADS), smem, s, map, te, (const RowStat*)x.stat, (const int*)x.kind,
             reinterpret_cast<const T*>(a.Z), a.ldz, a.V, slots, a.temperature, a.gscale, (const int*)a.count,
             a.row_loss, reinterpret_cast<T*>(a.dZ), a.ldd);
}

// A warp for the shortest rows, so that most of it has something to load; rows
// of which two fit an SM's shared memory stay there; longer ones are read twice.
constexpr int64_t kResidentBytes = 112 * 1024;
constexpr int kLong = 256;
template <typename T>
void pick_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te, const Scratch& x) {
  const int64_t fixed = (int64_t)2 * 3 * a.K * 4 + 512;
  if (a.V <= 1024) run_rows<T, 32>(s, a, map, te, x);
  else if (a.V <= 8192) run_resident<T, 128>(s, a, map, te, x);
  else if (a.V * (int64_t)sizeof(T) + 16 * kLong + fixed <= kResidentBytes) run_resident<T, kLong>(s, a, map, te, x);
  else run_rows<T, kLong>(s, a, map, te, x);
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
    if (a.type == LT_F32) pick_rows<float>(s, a, map, te, x);
    else if (a.type == LT_BF16) pick_rows<__nv_bfloat16>(s, a, map, te, x);
    else pick_rows<__half>(s, a, map, te, x);
  }
  count_launch();
  launch_pdl(k_distill_loss, dim3(M), dim3(256), 0, s, map, (const float*)a.row_loss, a.count, a.loss, a.count_out);
}

}  // namespace sm
