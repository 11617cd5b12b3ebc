// cpu_layers_launch.cpp -- the library's host code over a CUDA runtime that only
// keeps books (no GPU): what a launch asks for, what a kernel's limits are, what
// is cleared.  Linked with the library's own objects in place of libcudart.
//   cpu_layers_launch limits     a kernel's shared-memory limit is never lowered
//   cpu_layers_launch counters   a call that fails between its launches leaves
//                                the handle's counters cleared
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <vector>

#include "../include/signmuon_layers.h"

namespace {
constexpr int kMost = 232448, kStatic = 1024, kDefault = 48 * 1024;
std::map<const void*, int> limit;          // of dynamic shared memory, where it was set
std::map<const void*, size_t> largest;     // dynamic shared memory of any launch so far
int lowered = 0, beyond = 0, launches = 0, fail_at = -1;
cudaError_t last = cudaSuccess;
struct Cleared {
  void* p;
  int value;
  size_t bytes;
  int after;                               // launches before it
};
std::vector<Cleared> cleared;

cudaError_t done(cudaError_t e) {
  if (e != cudaSuccess) last = e;
  return e;
}
}  // namespace

extern "C" {
cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const int at = launches++;
  const int most = limit.count(f) ? limit[f] : kDefault;
  if ((int)c->dynamicSmemBytes > most) {
    ++beyond;
    return done(cudaErrorInvalidValue);
  }
  if (c->dynamicSmemBytes > largest[f]) largest[f] = c->dynamicSmemBytes;
  return done(at == fail_at ? cudaErrorInvalidValue : cudaSuccess);
}
cudaError_t CUDARTAPI cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) {
  ++launches;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  if (v < 0 || v > kMost - kStatic) return done(cudaErrorInvalidValue);
  // what another thread's launch, made ready before this, may need
  if (v < (int)largest[f]) ++lowered;
  limit[f] = v;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaFuncGetAttributes(cudaFuncAttributes* a, const void* f) {
  memset(a, 0, sizeof *a);
  a->sharedSizeBytes = kStatic;
  a->maxDynamicSharedSizeBytes = limit.count(f) ? limit[f] : kDefault;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) {
  *n = 3;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 148 : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? kMost : 0;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaSetDevice(int) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return "made by the test"; }
cudaError_t CUDARTAPI cudaMalloc(void** p, size_t n) {
  *p = aligned_alloc(256, (n + 255) / 256 * 256);
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t CUDARTAPI cudaFree(void* p) {
  free(p);
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaHostAlloc(void** p, size_t n, unsigned) { return cudaMalloc(p, n); }
cudaError_t CUDARTAPI cudaMallocHost(void** p, size_t n) { return cudaMalloc(p, n); }
cudaError_t CUDARTAPI cudaFreeHost(void* p) { return cudaFree(p); }
cudaError_t CUDARTAPI cudaMemset(void* p, int v, size_t n) {
  memset(p, v, n);
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) {
  cleared.push_back({p, v, n, launches});
  return cudaMemset(p, v, n);
}
cudaError_t CUDARTAPI cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind) {
  memcpy(to, from, n);
  return cudaSuccess;
}
cudaError_t CUDARTAPI cudaMemcpyAsync(void* to, const void* from, size_t n, cudaMemcpyKind k, cudaStream_t) {
  return cudaMemcpy(to, from, n, k);
}
cudaError_t CUDARTAPI cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventCreate(cudaEvent_t*) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaEventCreateWithFlags(cudaEvent_t*, unsigned) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaEventElapsedTime(float*, cudaEvent_t, cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaIpcCloseMemHandle(void*) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaIpcGetMemHandle(cudaIpcMemHandle_t*, void*) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaIpcOpenMemHandle(void**, cudaIpcMemHandle_t, unsigned) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaGetSymbolAddress(void**, const void*) { return cudaErrorNotSupported; }
cudaError_t CUDARTAPI cudaGetDriverEntryPoint(const char*, void**, unsigned long long, cudaDriverEntryPointQueryResult*) {
  return cudaErrorNotSupported;
}
void** CUDARTAPI __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void CUDARTAPI __cudaRegisterFatBinaryEnd(void**) {}
void CUDARTAPI __cudaUnregisterFatBinary(void**) {}
void CUDARTAPI __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void CUDARTAPI __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned CUDARTAPI __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t CUDARTAPI __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
}

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      printf("line %d: %s is not so\n", __LINE__, #x);       \
      return 1;                                              \
    }                                                        \
  } while (0)

// (device memory is host memory here and no kernel reads it: one address does for all)
alignas(256) static float room[4096];

static signmuon_t handle(int64_t rows, int64_t cols, int64_t max_rows) {
  const int64_t shapes[4] = {rows, cols, 1, cols};
  signmuon_t h = nullptr;
  if (signmuon_init(&h, shapes, 2, 1, 0.f, 0.f, 0, 1e-7f, SIGNMUON_SCALE_FRO, 1, SIGNMUON_VOTE_ONLY, nullptr)) return nullptr;
  if (signmuon_layers_reserve(h, max_rows, cols)) return nullptr;
  return h;
}

static int distill(signmuon_t h, int type, int64_t V, int K, int64_t n, bool grad) {
  return signmuon_distill(h, room, type, V, V, room, SIGNMUON_I32, room, SIGNMUON_F32, K, K, &n, 1.f, 1.f, room, nullptr,
                          nullptr, grad ? (void*)(room + 1024) : nullptr, V);
}

static int limits() {
  float* G[1] = {room};
  signmuon_t h = handle(600, 8, 70000);
  CHECK(h != nullptr);
  // long rows, then shorter ones, then long ones again, in every kind of call
  const int64_t lengths[] = {128256, 64000, 300000, 50304, 30000, 12000, 1000, 128256};
  for (int type = 0; type < 3; ++type)
    for (int grad = 0; grad < 2; ++grad)
      for (int64_t n : {2, 2000})
        for (int K : {1024, 1, 700, 64})
          for (int64_t V : lengths) CHECK(distill(h, type, V, K, n, grad) == SIGNMUON_OK);
  for (int64_t rows : {400, 600, 300, 400}) {
    signmuon_t t = handle(rows, 8, 70000);
    CHECK(t != nullptr);
    for (int type = 0; type < 3; ++type)
      for (int64_t n : {10, 2500, 9000, 70000})
        CHECK(signmuon_embed_grad(t, 0, room, SIGNMUON_I32, &n, 1.f, room, type, 8, G, 0) == SIGNMUON_OK);
    signmuon_destroy(t);
  }
  for (int64_t cols : {16384, 768, 5000, 2000, 1001, 64, 16384}) {
    signmuon_t t = handle(1, cols, 2000);
    CHECK(t != nullptr);
    for (int type = 0; type < 3; ++type)
      for (int64_t n : {1, 2000}) {
        CHECK(signmuon_layernorm(t, room, 0, 1, n, room, cols, room, cols, type, 1e-5f, nullptr, nullptr) == SIGNMUON_OK);
        CHECK(signmuon_layernorm_grad(t, room, 0, 1, &n, room, cols, room, cols, room, room, room, cols, type, G, 0) ==
              SIGNMUON_OK);
      }
    signmuon_destroy(t);
  }
  signmuon_destroy(h);
  CHECK(launches > 500);
  CHECK(beyond == 0);
  CHECK(lowered == 0);
  return 0;
}

// A distillation whose n-th launch fails: its first kernel has counted rows, which
// the next call would add to.
static int counters() {
  cleared.clear();
  signmuon_t h = handle(4, 8, 2000);
  CHECK(h != nullptr && cleared.size() == 1);
  const char* from = (const char*)cleared[0].p + sizeof(int);   // behind the status
  const char* to = (const char*)cleared[0].p + cleared[0].bytes;
  for (int64_t n : {2, 2000})
    for (int grad = 0; grad < 2; ++grad) {
      int before = launches;
      CHECK(distill(h, SIGNMUON_BF16, 5000, 4, n, grad) == SIGNMUON_OK);
      const int count = launches - before;
      CHECK(count == (n == 2 ? 2 : 3));
      for (int k = 0; k < count; ++k) {
        before = launches;
        cleared.clear();
        fail_at = launches + k;
        CHECK(distill(h, SIGNMUON_BF16, 5000, 4, n, grad) == SIGNMUON_E_CUDA);
        CHECK(strstr(signmuon_last_error(h), "made by the test") != nullptr);
        fail_at = -1;
        bool all = false;
        for (const Cleared& c : cleared)
          all = all || (c.value == 0 && (char*)c.p <= from && (char*)c.p + c.bytes >= to && c.after == launches);
        CHECK(all || k == 0);
        CHECK(distill(h, SIGNMUON_BF16, 5000, 4, n, grad) == SIGNMUON_OK);   // and is usable
      }
    }
  signmuon_destroy(h);
  return 0;
}

int main(int argc, char** argv) {
  int rc = 2;
  if (argc == 2 && !strcmp(argv[1], "limits")) rc = limits();
  if (argc == 2 && !strcmp(argv[1], "counters")) rc = counters();
  printf(rc ? "failed\n" : "layer launches ok\n");
  return rc;
}
