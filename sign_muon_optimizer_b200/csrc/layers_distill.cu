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

// count[m] += rows of worker m with an entry that counts (a warp per row)
__global__ void __launch_bounds__(256) k_distill_count(const RowMap map, const Teacher te, int64_t V, int* count) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= map.start[map.M]) return;
  bool any = false;
  for (int k = lane; k < te.K; k += 32)
    any |= counts(load_id(te.idx, te.id64, (int64_t)r * te.ldt + k), V, load_t(te.t, te.t_type, (int64_t)r * te.ldt + k));
  any = __any_sync(0xffffffffu, any);
  if (lane == 0 && any) atomicAdd(&count[worker_of(map.start, map.M, r)], 1);
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

// A running softmax: the maximum m of the logits so far and the sum s of
// 2^((z - m) c).  Without a finite logit m is -inf and s is 0 (or NaN).
struct Running {
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ static float ref(float m) { return m == -INFINITY ? 0.f : m; }
  __device__ __forceinline__ void raise(float top, float c) {
    if (top > m) {
      if (m != -INFINITY) s *= ex2((m - top) * c);
      m = top;
    }
  }
  __device__ __forceinline__ void one(float z, float c) {
    raise(z, c);
    s += ex2((z - ref(m)) * c);
  }
};

// ROW_THREADS threads hold a row: a block, or a warp (four rows a block).  The
// row is read twice, for the maximum and sum of the softmax and for the
// gradient (the second time from L2).  Every warp works out the teacher's
// softmax for itself, the first one leaves its entries in shared memory.
template <typename T, int ROW_THREADS>
__global__ void __launch_bounds__(ROW_THREADS == 32 ? 128 : ROW_THREADS)
    k_distill_rows(const RowMap map, const Teacher te, const T* Z, int64_t ldz, int64_t V, float temperature,
                   float gscale, int* count, int count_here, float* __restrict__ row_loss, T* dZ, int64_t ldd,
                   int* status) {
  constexpr int VL = Elem<T>::V;
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1, WARPS = ROW_THREADS / 32;
  constexpr int AHEAD = 4;                        // packs loaded before the first is used
  extern __shared__ float entries[];              // per row: q, z and index of the K entries
  __shared__ float2 buf[WARPS];
  griddep_wait();
  griddep_launch();
  const int K = te.K;
  const int lane = threadIdx.x & 31, tid = threadIdx.x % ROW_THREADS;
  const int in_block = threadIdx.x / ROW_THREADS;
  const int r = blockIdx.x * ROWS + in_block;
  if (r >= map.start[map.M]) return;              // (a whole warp)
  float* q = entries + (int64_t)in_block * 3 * K;
  float* zk = q + K;
  int* id = reinterpret_cast<int*>(q + 2 * K);
  auto sync = [&] {
    if (ROW_THREADS == 32) __syncwarp();
    else __syncthreads();
  };
  const T* z = Z + (int64_t)r * ldz;
  T* dz = dZ != nullptr ? dZ + (int64_t)r * ldd : nullptr;
  const int m = worker_of(map.start, map.M, r);
  // the teacher's softmax
  const float inv_T = 1.f / temperature;
  float top = -INFINITY;
  bool any = false;
  for (int k = lane; k < K; k += 32) {
    const int64_t i = load_id(te.idx, te.id64, (int64_t)r * te.ldt + k);
    const float t = load_t(te.t, te.t_type, (int64_t)r * te.ldt + k);
    const bool c = counts(i, V, t);
    any |= c;
    if (c) top = fmaxf(top, t);
    if (tid < 32) {
      if (i >= V) *status = 1;
      id[k] = c ? (int)i : -1;
      q[k] = t;
      if (c) zk[k] = Elem<T>::up(z[i]);
    }
  }
  if (!__any_sync(0xffffffffu, any)) {            // the same in every warp of the row
    if (dz != nullptr)
      for (int64_t v = tid; v < V; v += ROW_THREADS) dz[v] = Elem<T>::down(0.f);
    if (tid == 0) row_loss[r] = 0.f;
    return;
  }
  if (count_here && tid == 0) atomicAdd(&count[m], 1);
  top = warp_max(top);
  // the student's maximum and sum: whole 16-byte packs between a head and a tail
  const float c = inv_T * 1.4426950408889634f;
  const int mis = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
  const int head = (int)(V < (VL - mis) % VL ? V : (VL - mis) % VL);
  const int nv = (int)((V - head) / VL);
  const int tail = head + nv * VL, n_tail = (int)(V - tail);
  const Pack<T>* zp = reinterpret_cast<const Pack<T>*>(z + head);
  Running run;
  const F2 c2 = pack2(c, c);
  auto take = [&](const Pack<T>& p, F2 neg_m, F2& sum) {
#pragma unroll
    for (int j = 0; j < VL; j += 2) {
      const float2 x = unpack2(mul2(add2(up2(p, j / 2), neg_m), c2));
      sum = add2(pack2(ex2(x.x), ex2(x.y)), sum);
    }
  };
  int i = tid;
  for (; i + (AHEAD - 1) * ROW_THREADS < nv; i += AHEAD * ROW_THREADS) {
    Pack<T> p[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) p[a] = zp[i + a * ROW_THREADS];
    float t = pack_max(p[0]);
#pragma unroll
    for (int a = 1; a < AHEAD; ++a) t = fmaxf(t, pack_max(p[a]));
    run.raise(t, c);
    const float neg = -Running::ref(run.m);
    F2 sum = 0ull;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) take(p[a], pack2(neg, neg), sum);
    run.s += sum2(sum);
  }
  for (; i < nv; i += ROW_THREADS) {
    const Pack<T> p = zp[i];
    run.raise(pack_max(p), c);
    const float neg = -Running::ref(run.m);
    F2 sum = 0ull;
    take(p, pack2(neg, neg), sum);
    run.s += sum2(sum);
  }
  if (tid < head) run.one(Elem<T>::up(z[tid]), c);
  if (tid < n_tail) run.one(Elem<T>::up(z[tail + tid]), c);
  // over the row's threads (a sum without a finite logit is 0 or NaN and is kept)
  float all = warp_max(run.m);
  float s = warp_sum(run.m == -INFINITY ? run.s : run.s * ex2((run.m - all) * c));
  if (ROW_THREADS > 32) {
    if (lane == 0) buf[tid >> 5] = make_float2(all, s);
    __syncthreads();
    const float2 b = lane < WARPS ? buf[lane] : make_float2(-INFINITY, 0.f);
    all = warp_max(b.x);
    s = warp_sum(b.x == -INFINITY ? b.y : b.y * ex2((b.x - all) * c));
  } else {
    __syncwarp();
  }
  const float log2_s = log2f(s);
  if (tid < 32) {
    // the row's loss, and the teacher's probabilities
    float sum = 0.f;
    for (int k = lane; k < K; k += 32)
      if (id[k] >= 0) sum += expf((q[k] - top) * inv_T);
    const float log_sum_t = logf(warp_sum(sum));
    const float log_s = log2_s * 0.6931471805599453f;
    float loss = 0.f;
    for (int k = lane; k < K; k += 32) {
      if (id[k] < 0) continue;
      const float lq = (q[k] - top) * inv_T - log_sum_t;
      const float qk = expf(lq);
      if (!(qk == 0.f)) loss += qk * (lq - ((zk[k] - all) * inv_T - log_s));
      q[k] = qk;
    }
    loss = warp_sum(loss);
    if (tid == 0) row_loss[r] = loss * (temperature * temperature);
  }
  if (dz == nullptr) return;
  // the gradient: w * p everywhere, then the teacher's entries
  const float w = gscale * temperature / (float)count[m];
  const F2 neg_all = pack2(-all, -all), neg_log = pack2(-log2_s, -log2_s), w2 = pack2(w, w);
  const bool vec_out = ((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T)) == mis;
  auto grad = [&](float x) { return Elem<T>::down(w * ex2(fmaf(x - all, c, -log2_s))); };
  auto give = [&](const Pack<T>& p, int at) {
    Pack<T> o;
#pragma unroll
    for (int j = 0; j < VL; j += 2) {
      const float2 x = unpack2(fma2(add2(up2(p, j / 2), neg_all), c2, neg_log));
      const float2 y = unpack2(mul2(pack2(ex2(x.x), ex2(x.y)), w2));
      down2(o, j / 2, y.x, y.y);
    }
    T* to = dz + head + (int64_t)at * VL;
    if (vec_out) {
      *reinterpret_cast<Pack<T>*>(to) = o;
    } else {
#pragma unroll
      for (int j = 0; j < VL; ++j) to[j] = o.v[j];
    }
  };
  i = tid;
  for (; i + (AHEAD - 1) * ROW_THREADS < nv; i += AHEAD * ROW_THREADS) {
    Pack<T> p[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) p[a] = zp[i + a * ROW_THREADS];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) give(p[a], i + a * ROW_THREADS);
  }
  for (; i < nv; i += ROW_THREADS) give(zp[i], i);
  if (tid < head) dz[tid] = grad(Elem<T>::up(z[tid]));
  if (tid < n_tail) dz[tail + tid] = grad(Elem<T>::up(z[tail + tid]));
  sync();
  for (int k = tid; k < K; k += ROW_THREADS) {
    if (id[k] < 0) continue;
    bool mine = true;   // the first of the entries with this index writes for all of them
    float sum_q = 0.f;
    for (int e = 0; e < K; ++e)
      if (id[e] == id[k]) {
        if (e < k) mine = false;
        sum_q += q[e];
      }
    if (mine) dz[id[k]] = Elem<T>::down(w * (ex2(fmaf(zk[k] - all, c, -log2_s)) - sum_q));
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

template <typename T, int ROW_THREADS>
void run_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te) {
  constexpr int ROWS = ROW_THREADS == 32 ? 4 : 1;
  const size_t smem = (size_t)ROWS * 3 * a.K * 4;
  auto* kernel = k_distill_rows<T, ROW_THREADS>;
  if (smem > 32 * 1024) cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  count_launch();
  launch_pdl(kernel, dim3((map.start[map.M] + ROWS - 1) / ROWS), dim3(ROWS * ROW_THREADS), smem, s, map, te,
             reinterpret_cast<const T*>(a.Z), a.ldz, a.V, a.temperature, a.gscale, a.count, a.dZ == nullptr ? 1 : 0,
             a.row_loss, reinterpret_cast<T*>(a.dZ), a.ldd, a.status);
}

// a warp for the shortest rows, so that most of it has something to load
template <typename T>
void pick_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te) {
  if (a.V <= 1024) run_rows<T, 32>(s, a, map, te);
  else if (a.V <= 8192) run_rows<T, 128>(s, a, map, te);
  else run_rows<T, 512>(s, a, map, te);
}

}  // namespace

void launch_distill(cudaStream_t s, const DistillArgs& a, const int* start, int M) {
  RowMap map{};
  map.M = M;
  for (int m = 0; m <= M; ++m) map.start[m] = start[m];
  const int N = start[M];
  const Teacher te{a.idx, a.id64, a.t, a.t_type, a.ldt, a.K};
  if (N > 0) {
    // the gradient needs the worker's row count before its first row is done
    if (a.dZ != nullptr) {
      count_launch();
      launch_pdl(k_distill_count, dim3((unsigned)((N + 7LL) / 8)), dim3(256), 0, s, map, te, a.V, a.count);
    }
    if (a.type == LT_F32) pick_rows<float>(s, a, map, te);
    else if (a.type == LT_BF16) pick_rows<__nv_bfloat16>(s, a, map, te);
    else pick_rows<__half>(s, a, map, te);
  }
  count_launch();
  launch_pdl(k_distill_loss, dim3(M), dim3(256), 0, s, map, (const float*)a.row_loss, a.count, a.loss, a.count_out);
}

}  // namespace sm
