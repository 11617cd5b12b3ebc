// layers_api.cu -- the C ABI of include/signmuon_layers.h: argument checks,
// the workspace, and the launches on the handle's stream.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <mutex>
#include <set>
#include <utility>

#include "../../include/signmuon_layers.h"
#include "ctx.h"
#include "layers.cuh"

using sm::DeviceGuard;
using sm::NvtxRange;
using sm::aligned16;
using sm::check_handle;
using sm::dalloc;
using sm::fail;

void sm::allow_shared(const void* kernel) {
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> allowed;
  int dev = 0, most = 0;
  cudaFuncAttributes own{};
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  if (allowed.count({kernel, dev})) return;
  if (cudaFuncGetAttributes(&own, kernel) == cudaSuccess &&
      cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) == cudaSuccess &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)own.sharedSizeBytes) == cudaSuccess)
    allowed.insert({kernel, dev});     // (else the launch reports it)
}

namespace {

// No C++ exception crosses the C boundary (a message may fail to allocate).
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return SIGNMUON_E_NOMEM;
  }
}

int ready(signmuon_t h) {
  const int rc = check_handle(h, false);
  if (rc) return rc;
  if (h->lay_rows == 0) return fail(h, SIGNMUON_E_UNSUPPORTED, "call signmuon_layers_reserve first");
  return SIGNMUON_OK;
}

int elem_bytes(int type) { return type == SIGNMUON_F32 ? 4 : 2; }

int check_type(signmuon_t h, int type) {
  if (type != SIGNMUON_F32 && type != SIGNMUON_BF16 && type != SIGNMUON_F16)
    return fail(h, SIGNMUON_E_INVALID, "unknown element type");
  return SIGNMUON_OK;
}

int check_ids(signmuon_t h, const void* ids, int id_type, int64_t n) {
  if (id_type != SIGNMUON_I32 && id_type != SIGNMUON_I64) return fail(h, SIGNMUON_E_INVALID, "unknown index type");
  const uintptr_t mask = id_type == SIGNMUON_I64 ? 7 : 3;
  if (n > 0 && (ids == nullptr || (reinterpret_cast<uintptr_t>(ids) & mask)))
    return fail(h, SIGNMUON_E_INVALID, "indices null or misaligned");
  return SIGNMUON_OK;
}

// an n x cols matrix of `type` with row stride ld
int check_matrix(signmuon_t h, const char* name, const void* p, int type, int64_t n, int64_t cols, int64_t ld) {
  if (ld < cols) return fail(h, SIGNMUON_E_INVALID, std::string(name) + ": row stride below the number of columns");
  if (n > 0 && ld > INT64_MAX / 8 / n) return fail(h, SIGNMUON_E_INVALID, std::string(name) + ": row stride too large");
  if (n > 0 && (p == nullptr || reinterpret_cast<uintptr_t>(p) % elem_bytes(type)))
    return fail(h, SIGNMUON_E_INVALID, std::string(name) + " null or misaligned");
  return SIGNMUON_OK;
}

int check_floats(signmuon_t h, const char* name, const void* p, int64_t n) {
  if (n > 0 && (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3)))
    return fail(h, SIGNMUON_E_INVALID, std::string(name) + " null or misaligned");
  return SIGNMUON_OK;
}

int check_mat(signmuon_t h, int mat) {
  if (mat < 0 || mat >= h->plan.n_mats) return fail(h, SIGNMUON_E_INVALID, "matrix index out of range");
  return SIGNMUON_OK;
}

int64_t mat_size(signmuon_t h, int mat) { return (int64_t)h->plan.mats[mat].rows * h->plan.mats[mat].cols; }

int check_rows(signmuon_t h, const int64_t* rows, int* start) {
  if (rows == nullptr) return fail(h, SIGNMUON_E_INVALID, "null row counts");
  int64_t n = 0;
  for (int m = 0; m < h->M; ++m) {
    start[m] = (int)n;
    if (rows[m] < 0 || rows[m] > INT_MAX) return fail(h, SIGNMUON_E_INVALID, "row counts must be in [0, 2^31)");
    n += rows[m];
    if (n > h->lay_rows) return fail(h, SIGNMUON_E_INVALID, "more rows than signmuon_layers_reserve made room for");
  }
  start[h->M] = (int)n;
  return SIGNMUON_OK;
}

int check_grads(signmuon_t h, float* const* G, sm::GradPtrs* out) {
  if (G == nullptr) return fail(h, SIGNMUON_E_INVALID, "null G");
  for (int m = 0; m < h->M; ++m) {
    if (G[m] == nullptr || !aligned16(G[m])) return fail(h, SIGNMUON_E_INVALID, "G[m] null or misaligned");
    out->p[m] = G[m];
  }
  // outputs of different workers: no two may share memory
  float* sorted[sm::kMaxWorkers];
  std::copy(G, G + h->M, sorted);
  std::sort(sorted, sorted + h->M);
  for (int m = 1; m < h->M; ++m)
    if (sorted[m] - sorted[m - 1] < h->plan.d) return fail(h, SIGNMUON_E_INVALID, "two gradient vectors overlap");
  return SIGNMUON_OK;
}

#define TRY(call)                     \
  do {                                \
    const int rc_ = (call);           \
    if (rc_ != SIGNMUON_OK) return rc_; \
  } while (0)

// rows of a call, and entries of a table's row: leaves room in 32-bit indices
constexpr int64_t kMaxSize = int64_t(1) << 30;

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// blocks of the layer norm backward pass: at most 8 per SM, and one more per
// worker, whose last unit may be short
int norm_blocks(signmuon_t h) { return h->n_sm * 8 + h->M; }

// workspace layout, in bytes: embed_grad has two key arrays, digit counts and
// the parts of cut runs, layernorm_grad the blocks' sums, distill the
// rows' losses and stats
// Parts of cut runs: units x columns.  Units of 64 rows are taken where
// (rows / 256) * strips <= kFewBlocks, with strips >= columns / 256, so that
// (rows / 64) * columns <= (kFewBlocks + strips) * 1024.
int64_t embed_parts(signmuon_t h, int64_t rows, int64_t cols) {
  const int64_t few = std::min(rows / 64 * cols, sm::kFewBlocks * 1024 + 4 * cols + 1024);
  return std::max(rows / 256 * cols, few) + (h->M + 1) * cols;
}
int64_t count_set(signmuon_t h, int64_t rows) { return (rows / sm::kRadixTile + h->M + 1) * sm::kRadixBins; }
int64_t embed_bytes(signmuon_t h, int64_t rows, int64_t cols) {
  return 2 * align256(rows * 8) + sm::kRadixSets * count_set(h, rows) * 4 + embed_parts(h, rows, cols) * 2 * 4;
}
int64_t norm_bytes(signmuon_t h, int64_t cols) {
  return cols <= SIGNMUON_LAYERNORM_MAX_COLS ? (int64_t)norm_blocks(h) * 2 * cols * 4 : 0;
}

}  // namespace

extern "C" {

int signmuon_layers_reserve(signmuon_t h, int64_t max_rows, int64_t max_cols) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(check_handle(h, false));
    if (max_rows < 1 || max_rows > kMaxSize || max_cols < 1 || max_cols > kMaxSize)
      return fail(h, SIGNMUON_E_INVALID, "max_rows and max_cols must be in [1, 2^30]");
    if (max_rows <= h->lay_rows && max_cols <= h->lay_cols) return SIGNMUON_OK;
    if (max_rows < h->lay_rows) max_rows = h->lay_rows;
    if (max_cols < h->lay_cols) max_cols = h->lay_cols;
    int64_t n = embed_bytes(h, max_rows, max_cols);
    const int64_t b = norm_bytes(h, max_cols < SIGNMUON_LAYERNORM_MAX_COLS ? max_cols : SIGNMUON_LAYERNORM_MAX_COLS);
    if (b > n) n = b;
    if (max_rows * 16 > n) n = max_rows * 16;   // distill: the rows' losses, and 12 bytes of scratch
    uint8_t* ws = nullptr;
    TRY(dalloc(h, &ws, n));
    if (h->lay_status == nullptr) {
      int* p = nullptr;
      TRY(dalloc(h, &p, 1 + 2 * sm::kMaxWorkers));
      if (h->h_lay_status == nullptr) CK(h, cudaMallocHost(&h->h_lay_status, sizeof(int)));
      CK(h, cudaMemsetAsync(p, 0, (1 + 2 * sm::kMaxWorkers) * sizeof(int), h->stream));
      CK(h, cudaStreamSynchronize(h->stream));
      h->lay_status = p;
    }
    h->lay_ws = ws;
    h->lay_rows = max_rows;
    h->lay_cols = max_cols;
    return SIGNMUON_OK;
  });
}

int signmuon_layers_sync(signmuon_t h) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    CK(h, cudaMemcpyAsync(h->h_lay_status, h->lay_status, sizeof(int), cudaMemcpyDeviceToHost, h->stream));
    CK(h, cudaMemsetAsync(h->lay_status, 0, sizeof(int), h->stream));
    CK(h, cudaStreamSynchronize(h->stream));
    if (*h->h_lay_status)
      return fail(h, SIGNMUON_E_INVALID, "an index was at or above the number of rows or columns it points into");
    return SIGNMUON_OK;
  });
}

int signmuon_embed(signmuon_t h, const float* W, int mat, const void* ids, int id_type, int64_t n, float scale,
                   void* out, int type, int64_t ld) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    TRY(check_type(h, type));
    TRY(check_mat(h, mat));
    if (n < 0 || n > kMaxSize) return fail(h, SIGNMUON_E_INVALID, "n must be in [0, 2^30]");
    if (W == nullptr || !aligned16(W)) return fail(h, SIGNMUON_E_INVALID, "W null or misaligned");
    const sm::MatInfo& mi = h->plan.mats[mat];
    if (mi.cols > kMaxSize) return fail(h, SIGNMUON_E_UNSUPPORTED, "table rows have at most 2^30 entries");
    TRY(check_ids(h, ids, id_type, n));
    TRY(check_matrix(h, "out", out, type, n, mi.cols, ld));
    NvtxRange range("signmuon embed");
    sm::launch_embed(h->stream, W + mi.off, mi.rows, mi.cols, ids, id_type == SIGNMUON_I64, n, scale, out, type, ld,
                     h->lay_status);
    CK(h, cudaGetLastError());
    return SIGNMUON_OK;
  });
}

int signmuon_embed_grad(signmuon_t h, int mat, const void* ids, int id_type, const int64_t* rows, float scale,
                        const void* dY, int type, int64_t ld, float* const* G, int accumulate) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    TRY(check_type(h, type));
    TRY(check_mat(h, mat));
    int start[sm::kMaxWorkers + 1];
    TRY(check_rows(h, rows, start));
    const int64_t n = start[h->M];
    const sm::MatInfo& mi = h->plan.mats[mat];
    if (mi.cols > h->lay_cols) return fail(h, SIGNMUON_E_INVALID, "wider rows than signmuon_layers_reserve made room for");
    TRY(check_ids(h, ids, id_type, n));
    TRY(check_matrix(h, "dY", dY, type, n, mi.cols, ld));
    sm::GradPtrs gp{};
    TRY(check_grads(h, G, &gp));
    sm::EmbedGradArgs a{};
    a.ids = ids;
    a.id64 = id_type == SIGNMUON_I64;
    a.V = mi.rows;
    a.E = mi.cols;
    a.scale = scale;
    a.dY = dY;
    a.type = type;
    a.ld = ld;
    a.off = mi.off;
    a.accumulate = accumulate != 0;
    a.keys[0] = reinterpret_cast<unsigned long long*>(h->lay_ws);
    a.keys[1] = reinterpret_cast<unsigned long long*>(h->lay_ws + align256(h->lay_rows * 8));
    a.counts = reinterpret_cast<int*>(h->lay_ws + 2 * align256(h->lay_rows * 8));
    a.count_set = count_set(h, h->lay_rows);
    a.part = reinterpret_cast<float*>(a.counts + sm::kRadixSets * a.count_set);
    a.status = h->lay_status;
    NvtxRange range("signmuon embed_grad");
    sm::launch_embed_grad(h->stream, a, start, h->M, gp);
    CK(h, cudaGetLastError());
    return SIGNMUON_OK;
  });
}

// gamma and beta of a layer norm: the row length, and beta's offset or -1
static int norm_mats(signmuon_t h, int gamma, int beta, int64_t* E) {
  TRY(check_mat(h, gamma));
  if (beta != -1) TRY(check_mat(h, beta));
  *E = mat_size(h, gamma);
  if (beta != -1 && mat_size(h, beta) != *E) return fail(h, SIGNMUON_E_INVALID, "gamma and beta have different sizes");
  if (beta == gamma) return fail(h, SIGNMUON_E_INVALID, "gamma and beta are the same matrix");
  if (*E > SIGNMUON_LAYERNORM_MAX_COLS)
    return fail(h, SIGNMUON_E_UNSUPPORTED, "layer norm rows have at most " +
                                               std::to_string(SIGNMUON_LAYERNORM_MAX_COLS) + " entries");
  return SIGNMUON_OK;
}

int signmuon_layernorm(signmuon_t h, const float* W, int gamma, int beta, int64_t n, const void* X, int64_t ldx,
                       void* Y, int64_t ldy, int type, float eps, float* mean, float* rstd) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    TRY(check_type(h, type));
    int64_t E = 0;
    TRY(norm_mats(h, gamma, beta, &E));
    if (n < 0 || n > kMaxSize) return fail(h, SIGNMUON_E_INVALID, "n must be in [0, 2^30]");
    if (W == nullptr || !aligned16(W)) return fail(h, SIGNMUON_E_INVALID, "W null or misaligned");
    if (!(eps > 0.f)) return fail(h, SIGNMUON_E_INVALID, "eps must be > 0");
    TRY(check_matrix(h, "X", X, type, n, E, ldx));
    TRY(check_matrix(h, "Y", Y, type, n, E, ldy));
    if ((mean == nullptr) != (rstd == nullptr)) return fail(h, SIGNMUON_E_INVALID, "mean and rstd: both or neither");
    if (mean != nullptr) {
      TRY(check_floats(h, "mean", mean, n));
      TRY(check_floats(h, "rstd", rstd, n));
    }
    const auto& mats = h->plan.mats;
    NvtxRange range("signmuon layernorm");
    sm::launch_layernorm(h->stream, W + mats[gamma].off, beta < 0 ? nullptr : W + mats[beta].off, n, E, X, ldx, Y, ldy,
                         type, eps, mean, rstd);
    CK(h, cudaGetLastError());
    return SIGNMUON_OK;
  });
}

int signmuon_layernorm_grad(signmuon_t h, const float* W, int gamma, int beta, const int64_t* rows, const void* X,
                            int64_t ldx, const void* dY, int64_t ldy, const float* mean, const float* rstd, void* dX,
                            int64_t ldd, int type, float* const* G, int accumulate) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    TRY(check_type(h, type));
    int64_t E = 0;
    TRY(norm_mats(h, gamma, beta, &E));
    if (E > h->lay_cols) return fail(h, SIGNMUON_E_INVALID, "wider rows than signmuon_layers_reserve made room for");
    int start[sm::kMaxWorkers + 1];
    TRY(check_rows(h, rows, start));
    const int64_t n = start[h->M];
    if (W == nullptr || !aligned16(W)) return fail(h, SIGNMUON_E_INVALID, "W null or misaligned");
    TRY(check_matrix(h, "X", X, type, n, E, ldx));
    TRY(check_matrix(h, "dY", dY, type, n, E, ldy));
    TRY(check_matrix(h, "dX", dX, type, n, E, ldd));
    TRY(check_floats(h, "mean", mean, n));
    TRY(check_floats(h, "rstd", rstd, n));
    if (n > 0 && dX == dY && ldd != ldy)
      return fail(h, SIGNMUON_E_INVALID, "dX may be dY only with the same row stride");
    sm::GradPtrs gp{};
    TRY(check_grads(h, G, &gp));
    sm::NormGradArgs a{};
    a.gamma = W + h->plan.mats[gamma].off;
    a.E = E;
    a.X = X;
    a.ldx = ldx;
    a.dY = dY;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.dX = dX;
    a.ldd = ldd;
    a.type = type;
    a.off_gamma = h->plan.mats[gamma].off;
    a.off_beta = beta < 0 ? -1 : h->plan.mats[beta].off;
    a.accumulate = accumulate != 0;
    a.arrived = h->lay_status + 1 + sm::kMaxWorkers;
    a.part = reinterpret_cast<float*>(h->lay_ws);
    a.max_blocks = norm_blocks(h);
    NvtxRange range("signmuon layernorm_grad");
    sm::launch_layernorm_grad(h->stream, a, start, h->M, gp);
    CK(h, cudaGetLastError());
    return SIGNMUON_OK;
  });
}

int signmuon_distill(signmuon_t h, const void* Z, int type, int64_t ldz, int64_t V, const void* idx, int id_type,
                     const void* t, int t_type, int64_t ldt, int K, const int64_t* rows, float temperature,
                     float gscale, float* loss, int32_t* count, float* row_loss, void* dZ, int64_t ldd) {
  return guarded([&]() -> int {
    DeviceGuard dev_guard(h);
    TRY(ready(h));
    TRY(check_type(h, type));
    TRY(check_type(h, t_type));
    if (V < 1 || V > kMaxSize) return fail(h, SIGNMUON_E_INVALID, "V must be in [1, 2^30]");
    if (K < 1) return fail(h, SIGNMUON_E_INVALID, "K must be >= 1");
    if (K > SIGNMUON_DISTILL_MAX_K)
      return fail(h, SIGNMUON_E_UNSUPPORTED, "at most " + std::to_string(SIGNMUON_DISTILL_MAX_K) + " teacher entries a row");
    if (!(temperature >= 1e-18f && temperature <= 1e18f))   // its square and its inverse times log2 e stay in range
      return fail(h, SIGNMUON_E_INVALID, "temperature must be in [1e-18, 1e18]");
    int start[sm::kMaxWorkers + 1];
    TRY(check_rows(h, rows, start));
    const int64_t n = start[h->M];
    TRY(check_matrix(h, "Z", Z, type, n, V, ldz));
    TRY(check_matrix(h, "t", t, t_type, n, K, ldt));
    TRY(check_ids(h, idx, id_type, n));
    TRY(check_floats(h, "loss", loss, h->M));
    TRY(check_floats(h, "count", count, count ? h->M : 0));
    TRY(check_floats(h, "row_loss", row_loss, row_loss ? n : 0));
    if (dZ != nullptr) {
      TRY(check_matrix(h, "dZ", dZ, type, n, V, ldd));
      if (n > 0 && dZ == Z && ldd != ldz) return fail(h, SIGNMUON_E_INVALID, "dZ may be Z only with the same row stride");
    }
    sm::DistillArgs a{};
    a.Z = Z;
    a.type = type;
    a.ldz = ldz;
    a.V = V;
    a.idx = idx;
    a.id64 = id_type == SIGNMUON_I64;
    a.t = t;
    a.t_type = t_type;
    a.ldt = ldt;
    a.K = K;
    a.temperature = temperature;
    a.gscale = gscale;
    a.loss = loss;
    a.count_out = count;
    a.row_loss = row_loss != nullptr ? row_loss : reinterpret_cast<float*>(h->lay_ws);
    a.dZ = n > 0 ? dZ : nullptr;
    a.ldd = ldd;
    a.count = h->lay_status + 1;
    a.scratch = h->lay_ws + h->lay_rows * 4;
    a.status = h->lay_status;
    NvtxRange range("signmuon distill");
    sm::launch_distill(h->stream, a, start, h->M);
    const cudaError_t launches = cudaGetLastError();
    if (launches != cudaSuccess) {
      // the launches that did go may have counted rows, to which the next call would add
      cudaMemsetAsync(a.count, 0, 2 * sm::kMaxWorkers * sizeof(int), h->stream);
      CK(h, launches);
    }
    return SIGNMUON_OK;
  });
}

}  // extern "C"
