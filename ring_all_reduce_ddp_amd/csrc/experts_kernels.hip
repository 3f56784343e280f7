// Linear layers of several experts over rows sorted by expert (ddp_train.h):
// the linear layer's products (linear_device.h) of one expert's rows each.
//
// One launch covers all experts. Their bounds are on the device, so nothing
// waits for the host: the grid is what the worst bounds would need, and each
// block finds its expert by a scan over the bounds, 64 a wave at a time.
//
// What bounds it: with some 100 to 300 rows an expert the weights' bytes, and the rows of
// tiles that are not full. bf16, 16384 rows of 64 experts, 4096 x 2048: forward with
// z kept 440 us (1.75 GB read, of 1.14 needed, and 0.27 written: 4.6 TB/s; the matrix
// units busy 38 %), weight gradient added to fp32 870 (2.8 GB read and 2.2 written,
// 5.7 TB/s). 16 rows of 32: 30 us, 168 MB of weights at 5.5 TB/s.
#include "linear_host.h"

namespace ddp {
namespace {

constexpr int32_t kMostExperts = 1 << 16;

int check_experts(const char* fn, int64_t T, int64_t E, int64_t N, int64_t K, int32_t dtype, int32_t act) {
  int st = check_common(fn, T, N, K, dtype, act);
  if (st != DDP_OK) return st;
  if (E < 1 || E > kMostExperts) return fail(DDP_EINVAL, std::string(fn) + ": E must lie in [1, 65536]");
  if (K < 1) return fail(DDP_EINVAL, std::string(fn) + ": K must be at least 1");
  if (E * N >= (int64_t(1) << 31)) return fail(DDP_EINVAL, std::string(fn) + ": E * N must be below 2^31");
  return DDP_OK;
}

// The bounds, as a matrix argument of 8-byte elements.
Matrix bounds_of(const int64_t* offsets, int64_t E) { return {offsets, 1, E + 1, E + 1, 8, "offsets", false, false}; }

// How the weight gradient is cut, with or without direct loads.
Cut weight_cut(int64_t T, int64_t E, int64_t N, int64_t K, int32_t dtype, bool direct) {
  return cut_of(DDP_LINEAR_BACKWARD_WEIGHT, N, K, T, dtype, direct, int32_t(E));
}

// How a product of rows is cut.
Cut rows_cut(int dir, int64_t T, int64_t E, int64_t J, int64_t K, int32_t dtype, bool direct) {
  return cut_of(dir, T, J, K, dtype, direct, int32_t(E));
}

template <int DT, int DIR>
int launch_rows(LinearArgs& g, void* workspace, const char* fn, hipStream_t s) {
  const bool direct = whole_chunks(g.a, g.lda, g.I, g.K, DT) &&
                      whole_chunks(g.b, g.ldb, b_along(DIR) ? g.J : g.K, b_along(DIR) ? g.K : g.J, DT);
  g.partial = static_cast<float*>(workspace);
  int st = launch_groups<DT, DIR>(g, rows_cut(DIR, g.I, g.groups, g.J, g.K, DT, direct), direct, fn, s);
  if (st != DDP_OK || g.parts == 1) return st;
  g.bias = nullptr;  // the first part's sums have it
  hipLaunchKernelGGL((k_linear_join<DT, DIR, true>), dim3(unsigned(div_up(g.I * div_up(g.J, 8), kThreads))), dim3(kThreads), 0, s, g);
  DDP_HIP_TRY(hipGetLastError(), fn);
  return DDP_OK;
}

template <int DT>
int launch_weight(LinearArgs& g, void* db, int32_t grad_dtype, void* workspace, const char* fn, hipStream_t s) {
  const bool direct = whole_chunks(g.a, g.lda, g.K, g.I, DT) && whole_chunks(g.b, g.ldb, g.K, g.J, DT);
  const Cut c = weight_cut(g.K, g.groups, g.I, g.J, DT, direct);
  const int64_t N = g.groups * g.I;  // of dw, as one matrix
  g.stream_c = streams(N * g.J, grad_dtype);
  g.partial = static_cast<float*>(workspace);
  if (db != nullptr) g.row_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + partial_bytes(c, N, g.J));
  int st = launch_groups<DT, DDP_LINEAR_BACKWARD_WEIGHT>(g, c, direct, fn, s);
  if (st != DDP_OK) return st;
  if (g.parts > 1) {
    LinearArgs j = g;
    j.I = N;
    hipLaunchKernelGGL((k_linear_join<DT, DDP_LINEAR_BACKWARD_WEIGHT>), dim3(unsigned(div_up(N * div_up(g.J, 8), kThreads))),
                       dim3(kThreads), 0, s, j);
    DDP_HIP_TRY(hipGetLastError(), fn);
  }
  if (db == nullptr) return DDP_OK;
  return launch_column_sums<DDP_FP32>(g.row_sums, N, int64_t(g.parts) * g.tiles_j, N, db, grad_dtype, g.accumulate, fn, s);
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" int ddp_experts_workspace(int32_t direction, int64_t T, int64_t E, int64_t N, int64_t K, int32_t dtype,
                                     int64_t* bytes) {
  const char* fn = "ddp_experts_workspace";
  if (bytes == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": bytes is NULL");
  *bytes = 0;
  if (direction < DDP_LINEAR_FORWARD || direction > DDP_LINEAR_BACKWARD_WEIGHT)
    return fail(DDP_EINVAL, std::string(fn) + ": unknown direction");
  int st = check_experts(fn, T, E, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  if (N == 0) return DDP_OK;
  for (bool direct : {false, true}) {
    if (direction == DDP_LINEAR_BACKWARD_WEIGHT) {
      const Cut c = weight_cut(T, E, N, K, dtype, direct);
      *bytes = std::max(*bytes, partial_bytes(c, E * N, K) + bias_bytes(c, E * N, K));
    } else {
      const int64_t J = direction == DDP_LINEAR_FORWARD ? N : K;
      *bytes = std::max(*bytes, partial_bytes(rows_cut(direction, T, E, J, N + K - J, dtype, direct), T, J));
    }
  }
  return DDP_OK;
}

extern "C" int ddp_experts_tiling(int32_t direction, int64_t T, int64_t E, int64_t N, int64_t K, int32_t dtype, int32_t direct,
                                  int32_t* rows, int32_t* columns, int32_t* parts) {
  const char* fn = "ddp_experts_tiling";
  if (rows == nullptr || columns == nullptr || parts == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": an output is NULL");
  *rows = *columns = *parts = 0;
  if (direction < DDP_LINEAR_FORWARD || direction > DDP_LINEAR_BACKWARD_WEIGHT)
    return fail(DDP_EINVAL, std::string(fn) + ": unknown direction");
  if (direct != 0 && direct != 1) return fail(DDP_EINVAL, std::string(fn) + ": direct must be 0 or 1");
  int st = check_experts(fn, T, E, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  const int64_t J = direction == DDP_LINEAR_FORWARD ? N : K;
  const Cut c = direction == DDP_LINEAR_BACKWARD_WEIGHT ? weight_cut(T, E, N, K, dtype, direct != 0)
                                                        : rows_cut(direction, T, E, J, N + K - J, dtype, direct != 0);
  *rows = c.rows();
  *columns = c.tile;
  *parts = c.parts;
  return DDP_OK;
}

extern "C" int ddp_experts_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                   const int64_t* offsets, void* y, int64_t ldy, void* z, int64_t ldz, int64_t T, int64_t E,
                                   int64_t N, int64_t K, int32_t dtype, int32_t act, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_experts_forward";
  int st = check_experts(fn, T, E, N, K, dtype, act);
  if (st != DDP_OK) return st;
  if (T == 0 || N == 0) return DDP_OK;
  const int eb = elem_bytes(dtype);
  int64_t need = 0;
  st = ddp_experts_workspace(DDP_LINEAR_FORWARD, T, E, N, K, dtype, &need);
  if (st == DDP_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  const Matrix m[] = {{x, T, K, ldx, eb, "x", false, false},     {w, E * N, K, ldw, eb, "w", false, false},
                      {bias, 1, E * N, E * N, eb, "bias", false, true}, bounds_of(offsets, E),
                      {y, T, N, ldy, eb, "y", true, false},      {z, T, N, ldz, eb, "z", true, true},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_matrices(fn, m, 7, -1, -1);
  if (st != DDP_OK) return st;
  LinearArgs g{};
  g.a = x, g.lda = ldx, g.b = w, g.ldb = ldw, g.b_group = N * ldw;
  g.I = T, g.J = N, g.K = K;
  g.c = y, g.ldc = ldy, g.z = z, g.ldz = ldz, g.bias = bias;
  g.act = act;
  g.bounds = offsets, g.groups = int32_t(E), g.rows = T;
  return dtype == DDP_BF16 ? launch_rows<DDP_BF16, DDP_LINEAR_FORWARD>(g, workspace, fn, as_stream(stream))
                           : launch_rows<DDP_FP32, DDP_LINEAR_FORWARD>(g, workspace, fn, as_stream(stream));
}

extern "C" int ddp_experts_backward_input(const void* dz, int64_t lddz, const void* w, int64_t ldw, const int64_t* offsets,
                                          const void* z, int64_t ldz, void* dx, int64_t lddx, int64_t T, int64_t E, int64_t N,
                                          int64_t K, int32_t dtype, int32_t act, void* workspace, int64_t workspace_bytes,
                                          void* stream) {
  const char* fn = "ddp_experts_backward_input";
  int st = check_experts(fn, T, E, N, K, dtype, act);
  if (st != DDP_OK) return st;
  if (z == nullptr && act != DDP_ACT_NONE) return fail(DDP_EINVAL, std::string(fn) + ": an activation's slope needs z");
  if (T == 0) return DDP_OK;
  const int eb = elem_bytes(dtype);
  int64_t need = 0;
  st = ddp_experts_workspace(DDP_LINEAR_BACKWARD_INPUT, T, E, N, K, dtype, &need);
  if (st == DDP_OK) st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  const Matrix m[] = {{dz, T, N, lddz, eb, "dz", false, false}, {w, E * N, K, ldw, eb, "w", false, false},
                      bounds_of(offsets, E),                    {z, T, K, ldz, eb, "z", false, true},
                      {dx, T, K, lddx, eb, "dx", true, false},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_matrices(fn, m, 6, -1, -1);
  if (st != DDP_OK) return st;
  LinearArgs g{};
  g.a = dz, g.lda = lddz, g.b = w, g.ldb = ldw, g.b_group = N * ldw;
  g.I = T, g.J = K, g.K = N;
  g.c = dx, g.ldc = lddx, g.z = const_cast<void*>(z), g.ldz = ldz;
  g.act = act;
  g.bounds = offsets, g.groups = int32_t(E), g.rows = T;
  return dtype == DDP_BF16 ? launch_rows<DDP_BF16, DDP_LINEAR_BACKWARD_INPUT>(g, workspace, fn, as_stream(stream))
                           : launch_rows<DDP_FP32, DDP_LINEAR_BACKWARD_INPUT>(g, workspace, fn, as_stream(stream));
}

extern "C" int ddp_experts_backward_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx, const int64_t* offsets,
                                           void* dw, int64_t lddw, void* db, int64_t T, int64_t E, int64_t N, int64_t K,
                                           int32_t dtype, int32_t grad_dtype, int32_t accumulate, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_experts_backward_weight";
  int st = check_experts(fn, T, E, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  if (grad_dtype != dtype && grad_dtype != DDP_FP32)
    return fail(DDP_EINVAL, std::string(fn) + ": grad_dtype must be the data's or fp32");
  if (accumulate != 0 && accumulate != 1) return fail(DDP_EINVAL, std::string(fn) + ": accumulate must be 0 or 1");
  if (N == 0) return DDP_OK;
  const int eb = elem_bytes(dtype), gb = elem_bytes(grad_dtype);
  int64_t need = 0;
  st = ddp_experts_workspace(DDP_LINEAR_BACKWARD_WEIGHT, T, E, N, K, dtype, &need);
  if (st != DDP_OK) return st;
  const Matrix m[] = {{dz, T, N, lddz, eb, "dz", false, false},    {x, T, K, ldx, eb, "x", false, false},
                      bounds_of(offsets, E),                       {dw, E * N, K, lddw, gb, "dw", true, false},
                      {db, 1, E * N, E * N, gb, "db", true, true},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  st = check_matrices(fn, m, 6, -1, -1);
  if (st != DDP_OK) return st;
  LinearArgs g{};
  g.a = dz, g.lda = lddz, g.b = x, g.ldb = ldx;
  g.I = N, g.J = K, g.K = T;
  g.c = dw, g.ldc = lddw;
  g.grad32 = grad_dtype == DDP_FP32, g.accumulate = accumulate;
  g.bounds = offsets, g.groups = int32_t(E), g.rows = T;
  return dtype == DDP_BF16 ? launch_weight<DDP_BF16>(g, db, grad_dtype, workspace, fn, as_stream(stream))
                           : launch_weight<DDP_FP32>(g, db, grad_dtype, workspace, fn, as_stream(stream));
}
