// layers_distill.cu -- distillation loss per worker and its gradient with
// respect to the student's logits.
#include "layers.cuh"

namespace sm {
namespace {

constexpr int kMaxK = 1024;       // teacher entries of a row
constexpr int kThreads = 512;

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

// sum (or maximum) over the block; every thread gets it.  buf: one float per warp
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += buf[i];
  __syncthreads();
  return t;
}
__device__ __forceinline__ float block_max(float v, float* buf) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = buf[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) t = fmaxf(t, buf[i]);
  __syncthreads();
  return t;
}

// running maximum m (of z) and sum s of exp2((z - m) * c); exact for m = -inf
__device__ __forceinline__ void online(float& m, float& s, float z, float c) {
  if (z > m) {
    s = s * exp2f((m - z) * c) + 1.f;
    m = z;
  } else if (z != -INFINITY) {
    s += exp2f((z - m) * c);   // a NaN comes here and stays in the sum
  }
}

// A block per row.  The row is read twice, for the maximum and sum of the
// softmax and for the gradient (the second time from L2).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_distill_rows(const RowMap map, const Teacher te, const T* Z, int64_t ldz, int64_t V, float temperature,
                   float gscale, int* count, int count_here, float* __restrict__ row_loss, T* dZ, int64_t ldd,
                   int* status) {
  constexpr int VL = Elem<T>::V;
  __shared__ float q[kMaxK], zk[kMaxK];
  __shared__ int id[kMaxK];
  __shared__ float buf[kThreads / 32];
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x, tid = threadIdx.x;
  const int K = te.K;
  const T* z = Z + (int64_t)r * ldz;
  T* dz = dZ != nullptr ? dZ + (int64_t)r * ldd : nullptr;
  const int m = worker_of(map.start, map.M, r);
  // the teacher's entries
  float top = -INFINITY;
  bool any = false;
  for (int k = tid; k < K; k += kThreads) {
    const int64_t i = load_id(te.idx, te.id64, (int64_t)r * te.ldt + k);
    const float t = load_t(te.t, te.t_type, (int64_t)r * te.ldt + k);
    if (i >= V) *status = 1;
    const bool c = counts(i, V, t);
    id[k] = c ? (int)i : -1;
    q[k] = t;
    any |= c;
    if (c) top = fmaxf(top, t);
  }
  any = __syncthreads_or(any);
  if (!any) {  // block-uniform: nothing to learn from this row
    if (dz != nullptr)
      for (int64_t v = tid; v < V; v += kThreads) dz[v] = Elem<T>::down(0.f);
    if (tid == 0) row_loss[r] = 0.f;
    return;
  }
  if (count_here && tid == 0) atomicAdd(&count[m], 1);
  top = block_max(top, buf);
  const float inv_T = 1.f / temperature;
  float sum = 0.f;
  for (int k = tid; k < K; k += kThreads)
    if (id[k] >= 0) sum += expf((q[k] - top) * inv_T);
  const float log_sum_t = logf(block_sum(sum, buf));
  // the student's maximum and sum: whole 16-byte vectors between a head and a tail
  const float c = inv_T * 1.4426950408889634f;
  const int mis = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
  const int64_t head = V < (VL - mis) % VL ? V : (VL - mis) % VL;
  const int64_t nv = (V - head) / VL;
  const int64_t tail = head + nv * VL;
  float mx = -INFINITY, s = 0.f;
  if (tid < head) online(mx, s, Elem<T>::up(z[tid]), c);
  for (int64_t i = tid; i < nv; i += kThreads) {
    const Pack<T> p = *reinterpret_cast<const Pack<T>*>(z + head + i * VL);
#pragma unroll
    for (int j = 0; j < VL; ++j) online(mx, s, Elem<T>::up(p.v[j]), c);
  }
  if (tail + tid < V) online(mx, s, Elem<T>::up(z[tail + tid]), c);
  const float all = block_max(mx, buf);
  // a thread without finite logits has s = 0 (or NaN, which must stay)
  s = block_sum(mx == -INFINITY ? s : s * exp2f((mx - all) * c), buf);
  const float log2_s = log2f(s);
  const float log_s = log2_s * 0.6931471805599453f;
  // the row's loss
  float loss = 0.f;
  for (int k = tid; k < K; k += kThreads) {
    if (id[k] < 0) continue;
    const float lq = (q[k] - top) * inv_T - log_sum_t;
    const float qk = expf(lq);
    const float zz = Elem<T>::up(z[id[k]]);
    if (!(qk == 0.f)) loss += qk * (lq - ((zz - all) * inv_T - log_s));
    q[k] = qk;
    zk[k] = zz;
  }
  loss = block_sum(loss, buf);
  if (tid == 0) row_loss[r] = loss * (temperature * temperature);
  if (dz == nullptr) return;
  // the gradient: w * p everywhere, then the teacher's entries
  const float w = gscale * temperature / (float)count[m];
  if (tid < head) dz[tid] = Elem<T>::down(w * exp2f(fmaf(Elem<T>::up(z[tid]) - all, c, -log2_s)));
  const bool vec_out = ((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T)) == mis;
  for (int64_t i = tid; i < nv; i += kThreads) {
    Pack<T> p = *reinterpret_cast<const Pack<T>*>(z + head + i * VL);
#pragma unroll
    for (int j = 0; j < VL; ++j) p.v[j] = Elem<T>::down(w * exp2f(fmaf(Elem<T>::up(p.v[j]) - all, c, -log2_s)));
    T* o = dz + head + i * VL;
    if (vec_out) {
      *reinterpret_cast<Pack<T>*>(o) = p;
    } else {
#pragma unroll
      for (int j = 0; j < VL; ++j) o[j] = p.v[j];
    }
  }
  if (tail + tid < V) dz[tail + tid] = Elem<T>::down(w * exp2f(fmaf(Elem<T>::up(z[tail + tid]) - all, c, -log2_s)));
  __syncthreads();
  for (int k = tid; k < K; k += kThreads) {
    if (id[k] < 0) continue;
    bool mine = true;   // the first of the entries with this index writes for all of them
    float sum_q = 0.f;
    for (int i = 0; i < K; ++i)
      if (id[i] == id[k]) {
        if (i < k) mine = false;
        sum_q += q[i];
      }
    if (mine) dz[id[k]] = Elem<T>::down(w * (exp2f(fmaf(zk[k] - all, c, -log2_s)) - sum_q));
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

template <typename T>
void run_rows(cudaStream_t s, const DistillArgs& a, const RowMap& map, const Teacher& te) {
  count_launch();
  launch_pdl(k_distill_rows<T>, dim3(map.start[map.M]), dim3(kThreads), 0, s, map, te, reinterpret_cast<const T*>(a.Z),
             a.ldz, a.V, a.temperature, a.gscale, a.count, a.dZ == nullptr ? 1 : 0, a.row_loss,
             reinterpret_cast<T*>(a.dZ), a.ldd, a.status);
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
    if (a.type == LT_F32) run_rows<float>(s, a, map, te);
    else if (a.type == LT_BF16) run_rows<__nv_bfloat16>(s, a, map, te);
    else run_rows<__half>(s, a, map, te);
  }
  count_launch();
  launch_pdl(k_distill_loss, dim3(M), dim3(256), 0, s, map, (const float*)a.row_loss, a.count, a.loss, a.count_out);
}

}  // namespace sm
