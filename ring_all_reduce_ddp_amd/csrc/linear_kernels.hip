// A linear layer's entry points (ddp_train.h): its three products
// (linear_device.h), the forward product of a few rows, and the activations'
// slopes by themselves.
#include "linear_host.h"

namespace ddp {
namespace {

// ---------------------------------------------------------------- few rows

// The forward product for up to kFewRows rows of x (tokens of an answer): w
// is read once and each value meets every row's, so the bound is w's bytes. A
// block takes 4 rows of w, its waves every fourth kilobyte of each; x stays in
// the caches. (1 row, 8192 x 2048 bf16: 6 us, 5.6 TB/s with w in the Infinity
// Cache. The whole call, without and with tiles: 1 and 2 rows 7.0 us and 10.4
// there, 7.0 and 10.8 at 4096 x 4096, fp32 12 and 26. 4 rows gain where outputs are
// few, 9.9 and 14.0 at 2048 x 8192, fp32 16 and 26 at 4096 x 4096, and lose where
// they are many, 16.5 and 10.5 at 8192 x 2048, 50 and 12.5 at 32000 x 1024.)
constexpr int kFewOuts = 4;

// V = 16 / element size values of a row from k on, zeros past K.
template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const void* p, int64_t at, int64_t k, int64_t K) {
  constexpr int V = DT == DDP_BF16 ? 8 : 4;
  if constexpr (DT == DDP_BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (k + V <= K) return load_at<false, u32x4_at2>(q, 0);
    u32x4 r{};
    for (int e = 0; e < V; ++e)
      if (k + e < K) r[e >> 1] |= uint32_t(q[e]) << ((e & 1) * 16);
    return r;
  } else {
    const float* q = static_cast<const float*>(p) + at;
    if (k + V <= K) return load_at<false, u32x4_at4>(q, 0);
    u32x4 r{};
    for (int e = 0; e < V; ++e)
      if (k + e < K) r[e] = __float_as_uint(q[e]);
    return r;
  }
}
template <int DT>
__device__ __forceinline__ float dot_chunk(u32x4 a, u32x4 b, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == DDP_BF16)
      s = fmaf(bf16_hi(a[e]), bf16_hi(b[e]), fmaf(bf16_lo(a[e]), bf16_lo(b[e]), s));
    else
      s = fmaf(__uint_as_float(a[e]), __uint_as_float(b[e]), s);
  }
  return s;
}

template <int DT, int M>
__global__ __launch_bounds__(kThreads) void k_linear_few(LinearArgs g) {
  constexpr int V = DT == DDP_BF16 ? 8 : 4, OUTS = kFewOuts * M;
  __shared__ float sums[4][OUTS];
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  const int64_t j0 = (int64_t(g.begin) + blockIdx.x) * kFewOuts;
  float acc[OUTS] = {};  // [r * M + m]
#pragma unroll 1
  for (int64_t k = int64_t(threadIdx.x) * V; k < g.K; k += kThreads * V) {
    u32x4 w[kFewOuts], x[M];
#pragma unroll
    for (int r = 0; r < kFewOuts; ++r) w[r] = load_chunk<DT>(g.b, (j0 + r < g.J ? j0 + r : g.J - 1) * g.ldb + k, k, g.K);
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = load_chunk<DT>(g.a, (m < g.I ? m : g.I - 1) * g.lda + k, k, g.K);
#pragma unroll
    for (int r = 0; r < kFewOuts; ++r)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[r * M + m] = dot_chunk<DT>(w[r], x[m], acc[r * M + m]);
  }
  // Across the wave, halving the values a lane holds at each exchange: OUTS + 4
  // exchanges or so instead of 6 OUTS. Lane bit d decides which half it keeps.
  int kept = OUTS, index = 0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    if (kept > 1) {
      kept /= 2;
      const bool upper = (lane & d) != 0;
      index += upper ? kept : 0;
#pragma unroll
      for (int v = 0; v < OUTS / 2; ++v) {
        if (v >= kept) continue;
        const float keep = upper ? acc[v + kept] : acc[v], give = upper ? acc[v] : acc[v + kept];
        acc[v] = keep + __shfl_xor(give, d);
      }
    } else {
      acc[0] += __shfl_xor(acc[0], d);
    }
  }
  if (lane % (64 / OUTS) == 0) sums[wave][index] = acc[0];
  __syncthreads();
  const int r = int(threadIdx.x) / M, m = int(threadIdx.x) % M;
  if (r >= kFewOuts || m >= g.I || j0 + r >= g.J) return;
  const int64_t j = j0 + r;
  float z = (sums[0][r * M + m] + sums[1][r * M + m]) + (sums[2][r * M + m] + sums[3][r * M + m]);
  if (g.bias != nullptr) z += Ops<DT>::load1(g.bias, j);
  const auto rounded = [](float v) { return DT == DDP_BF16 ? round_bf16(v) : v; };
  if (g.z != nullptr) Ops<DT>::store1(g.z, m * g.ldz + j, rounded(z));
  float y = z;
  switch (g.act) {
    case DDP_ACT_RELU:
      y = act_value<DT, DDP_ACT_RELU>(z);
      break;
    case DDP_ACT_GELU:
      y = act_value<DT, DDP_ACT_GELU>(z);
      break;
    case DDP_ACT_GELU_TANH:
      y = act_value<DT, DDP_ACT_GELU_TANH>(z);
      break;
    case DDP_ACT_SILU:
      y = act_value<DT, DDP_ACT_SILU>(z);
      break;
  }
  if (g.e != nullptr) y += Ops<DT>::load1(g.e, m * g.lde + j);
  Ops<DT>::store1(g.c, m * g.ldc + j, rounded(y));
}

// ---------------------------------------------------------------- element by element

template <int DT, int ACT>
__global__ __launch_bounds__(kThreads) void k_act_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz,
                                                           void* dz, int64_t lddz, int64_t M, int64_t N) {
  const int64_t nv = (N + 7) / 8;
  for (int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x; at < M * nv; at += int64_t(gridDim.x) * kThreads) {
    const int64_t m = at / nv, j = at % nv * 8;
    const int n = N - j >= 8 ? 8 : int(N - j);
    float g[8], x[8];
    load8<DT>(dy, m * lddy + j, n, g);
    load8<DT>(z, m * ldz + j, n, x);
    for (int k = 0; k < 8; ++k) g[k] *= act_slope<DT, ACT>(x[k]);
    store8<DT>(dz, m * lddz + j, n, g);
  }
}

// ---------------------------------------------------------------- host side

template <int DT>
void launch_act_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz, int64_t M,
                         int64_t N, int32_t act, hipStream_t s) {
  const dim3 grid(unsigned(std::min<int64_t>(div_up(M * div_up(N, 8), kThreads), 1 << 16))), block(kThreads);
  switch (act) {
#define DDP_ACT_CASE(A)                                                                                     \
  case A:                                                                                                   \
    hipLaunchKernelGGL((k_act_backward<DT, A>), grid, block, 0, s, dy, lddy, z, ldz, dz, lddz, M, N);        \
    break;
    DDP_ACT_CASE(DDP_ACT_NONE)
    DDP_ACT_CASE(DDP_ACT_RELU)
    DDP_ACT_CASE(DDP_ACT_GELU)
    DDP_ACT_CASE(DDP_ACT_GELU_TANH)
    DDP_ACT_CASE(DDP_ACT_SILU)
#undef DDP_ACT_CASE
  }
}


// Scratch of a product: for either loader, as the sizes alone do not tell which.
int64_t scratch_bytes(int dir, int64_t I, int64_t J, int64_t K, int dtype, bool bias) {
  int64_t most = 0;
  for (bool direct : {false, true}) {
    const Cut c = cut_of(dir, I, J, K, dtype, direct);
    most = std::max(most, partial_bytes(c, I, J) + (bias ? bias_bytes(c, I, J) : 0));
  }
  return most;
}

// The sizes of a direction as those of C = A B^T.
void product_sizes(int dir, int64_t M, int64_t N, int64_t K, int64_t* I, int64_t* J, int64_t* S) {
  if (dir == DDP_LINEAR_FORWARD)
    *I = M, *J = N, *S = K;
  else if (dir == DDP_LINEAR_BACKWARD_INPUT)
    *I = M, *J = K, *S = N;
  else
    *I = N, *J = K, *S = M;
}

template <int DT, int DIR, int T, int WI, int WJ, int LOAD>
int launch_tiles(LinearArgs& g, hipStream_t s) {
  const int64_t ti = div_up(g.I, T), tj = div_up(g.J, T);
  if (ti * tj * g.parts >= (int64_t(1) << 30)) return fail(DDP_EINVAL, "ddp_linear: too many tiles for one launch");
  g.tiles_i = int32_t(ti);
  g.tiles_j = int32_t(tj);
  launch_blocks(round_up(ti * tj * g.parts, 8), [&](int64_t begin, dim3 grid) {
    g.begin = int32_t(begin);
    hipLaunchKernelGGL((k_linear<DT, DIR, T, T, WI, WJ, LOAD>), grid, dim3(WI * WJ * 64), 0, s, g);
  });
  DDP_HIP_TRY(hipGetLastError(), "ddp_linear: launch");
  return DDP_OK;
}

// The product of g's operands; the workspace starts with the parts' sums, and
// with want_rows has the row sums behind them.
template <int DT, int DIR>
int launch_product(LinearArgs& g, void* workspace, bool want_rows, hipStream_t s) {
  constexpr int V = 16 / (DT == DDP_BF16 ? 2 : 4);
  const bool direct = whole_chunks(g.a, g.lda, a_along(DIR) ? g.I : g.K, a_along(DIR) ? g.K : g.I, DT) &&
                      whole_chunks(g.b, g.ldb, b_along(DIR) ? g.J : g.K, b_along(DIR) ? g.K : g.J, DT);
  const Cut c = cut_of(DIR, g.I, g.J, g.K, DT, direct);
  const bool shorter = (a_along(DIR) ? g.K : g.I) < V || (b_along(DIR) ? g.K : g.J) < V;  // rows than a chunk
  if constexpr (DIR == DDP_LINEAR_FORWARD) {
    if (c.few) {
      launch_blocks(div_up(g.J, kFewOuts), [&](int64_t begin, dim3 grid) {
        g.begin = int32_t(begin);
        if (g.I == 1)
          hipLaunchKernelGGL((k_linear_few<DT, 1>), grid, dim3(kThreads), 0, s, g);
        else if (g.I == 2)
          hipLaunchKernelGGL((k_linear_few<DT, 2>), grid, dim3(kThreads), 0, s, g);
        else
          hipLaunchKernelGGL((k_linear_few<DT, kFewRows>), grid, dim3(kThreads), 0, s, g);
      });
      DDP_HIP_TRY(hipGetLastError(), "ddp_linear: launch");
      return DDP_OK;
    }
  }
  // z waits for the backward pass, the rest of what the call touches does not:
  // where all of it is much for the Infinity Cache, z leaves it to y. A layer and
  // the one after it, rows x inputs x outputs and back, with z cached and streamed,
  // forward and, in brackets, with the backward pass, which reads z from further away:
  // 8192 x 2048 x 8192 512 and 467 us (1501 and 1485), 8192 x 1536 x 6144, 244 MB,
  // 327 and 293 (1047 and 1025), 4096 x 2048 x 8192, 184 MB, 275 and 257 (830 and
  // 818), 16384 x 1024 x 4096 284 and 267 (876 and 865). At 159 MB, 8192 x 1024 x
  // 4096, nothing is gained: 144 and 144 (480 and 484). C streamed too is better
  // for the whole step at some sizes (1464, 862; 476 at 159 MB) and worse at others
  // (1044; 8 to 10 % at 4096 x 1024 x 4096 and 8192 x 512 x 2048), and the forward
  // pass by itself is slower with it: 487, 325, 267, 281.
  if (DIR == DDP_LINEAR_FORWARD && g.z != nullptr)
    g.stream_z = (g.I * g.K + g.J * g.K + g.I * g.J * (g.e != nullptr ? 3 : 2)) * elem_bytes(DT) > kInfinityCacheBytes / 3 * 2;
  g.parts = c.parts;
  g.part_k = c.part_k;
  g.partial = static_cast<float*>(workspace);
  if (want_rows) g.row_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + partial_bytes(c, g.I, g.J));
  int st = DDP_OK;
  if constexpr (DT == DDP_BF16) {
    if (c.tile == 256) st = launch_tiles<DT, DIR, 256, 2, 4, kDirect>(g, s);
  }
  if (shorter)
    st = launch_tiles<DT, DIR, 64, 2, 2, kShort>(g, s);
  else if (c.tile == 128)
    st = direct ? launch_tiles<DT, DIR, 128, 2, 2, kDirect>(g, s) : launch_tiles<DT, DIR, 128, 2, 2, kAny>(g, s);
  else if (c.tile == 64)
    st = direct ? launch_tiles<DT, DIR, 64, 2, 2, kDirect>(g, s) : launch_tiles<DT, DIR, 64, 2, 2, kAny>(g, s);
  if (st != DDP_OK || g.parts == 1) return st;
  const int64_t blocks = div_up(g.I * div_up(g.J, 8), kThreads);  // parts come with few tiles: one launch
  hipLaunchKernelGGL((k_linear_join<DT, DIR>), dim3(unsigned(blocks)), dim3(kThreads), 0, s, g);
  DDP_HIP_TRY(hipGetLastError(), "ddp_linear: join launch");
  return DDP_OK;
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" int ddp_linear_workspace(int32_t direction, int64_t M, int64_t N, int64_t K, int32_t dtype, int64_t* bytes) {
  const char* fn = "ddp_linear_workspace";
  if (bytes == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": bytes is NULL");
  *bytes = 0;
  if (direction < DDP_LINEAR_FORWARD || direction > DDP_LINEAR_BACKWARD_WEIGHT)
    return fail(DDP_EINVAL, std::string(fn) + ": unknown direction");
  int st = check_common(fn, M, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  int64_t I, J, S;
  product_sizes(direction, M, N, K, &I, &J, &S);
  *bytes = scratch_bytes(direction, I, J, S, dtype, direction == DDP_LINEAR_BACKWARD_WEIGHT);
  return DDP_OK;
}

extern "C" int ddp_linear_tiling(int32_t direction, int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t direct,
                                 int32_t* tile, int32_t* parts) {
  const char* fn = "ddp_linear_tiling";
  if (tile == nullptr || parts == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": an output is NULL");
  *tile = *parts = 0;
  if (direction < DDP_LINEAR_FORWARD || direction > DDP_LINEAR_BACKWARD_WEIGHT)
    return fail(DDP_EINVAL, std::string(fn) + ": unknown direction");
  if (direct != 0 && direct != 1) return fail(DDP_EINVAL, std::string(fn) + ": direct must be 0 or 1");
  int st = check_common(fn, M, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  int64_t I, J, S;
  product_sizes(direction, M, N, K, &I, &J, &S);
  const Cut c = cut_of(direction, I, J, S, dtype, direct != 0);
  *tile = c.few ? 0 : c.tile;
  *parts = c.parts;
  return DDP_OK;
}

extern "C" int ddp_linear_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                  const void* residual, int64_t ldr, void* y, int64_t ldy, void* z, int64_t ldz,
                                  int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_linear_forward";
  int st = check_common(fn, M, N, K, dtype, act);
  if (st != DDP_OK) return st;
  if (M == 0 || N == 0) return DDP_OK;
  const int eb = elem_bytes(dtype);
  const int64_t need = scratch_bytes(DDP_LINEAR_FORWARD, M, N, K, dtype, false);
  const Matrix m[] = {{x, M, K, ldx, eb, "x", false, false},       {w, N, K, ldw, eb, "w", false, false},
                      {bias, 1, N, N, eb, "bias", false, true},    {residual, M, N, ldr, eb, "residual", false, true},
                      {y, M, N, ldy, eb, "y", true, false},        {z, M, N, ldz, eb, "z", true, true},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  st = check_matrices(fn, m, 7, 3, 4);
  if (st != DDP_OK) return st;
  LinearArgs g{};
  g.a = x, g.lda = ldx, g.b = w, g.ldb = ldw;
  g.I = M, g.J = N, g.K = K;
  g.c = y, g.ldc = ldy, g.z = z, g.ldz = ldz, g.e = residual, g.lde = ldr, g.bias = bias;
  g.act = act;
  return dtype == DDP_BF16 ? launch_product<DDP_BF16, DDP_LINEAR_FORWARD>(g, workspace, false, as_stream(stream))
                           : launch_product<DDP_FP32, DDP_LINEAR_FORWARD>(g, workspace, false, as_stream(stream));
}

extern "C" int ddp_linear_backward_input(const void* dz, int64_t lddz, const void* w, int64_t ldw, const void* z,
                                         int64_t ldz, const void* add, int64_t ldadd, void* dx, int64_t lddx,
                                         int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_linear_backward_input";
  int st = check_common(fn, M, N, K, dtype, act);
  if (st != DDP_OK) return st;
  if (z == nullptr && act != DDP_ACT_NONE) return fail(DDP_EINVAL, std::string(fn) + ": an activation's slope needs z");
  if (M == 0 || K == 0) return DDP_OK;
  const int eb = elem_bytes(dtype);
  const int64_t need = scratch_bytes(DDP_LINEAR_BACKWARD_INPUT, M, K, N, dtype, false);
  const Matrix m[] = {{dz, M, N, lddz, eb, "dz", false, false}, {w, N, K, ldw, eb, "w", false, false},
                      {z, M, K, ldz, eb, "z", false, true},     {add, M, K, ldadd, eb, "add", false, true},
                      {dx, M, K, lddx, eb, "dx", true, false},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  st = check_matrices(fn, m, 6, 3, 4);
  if (st != DDP_OK) return st;
  LinearArgs g{};
  g.a = dz, g.lda = lddz, g.b = w, g.ldb = ldw;
  g.I = M, g.J = K, g.K = N;
  g.c = dx, g.ldc = lddx, g.z = const_cast<void*>(z), g.ldz = ldz, g.e = add, g.lde = ldadd;
  g.act = act;
  return dtype == DDP_BF16 ? launch_product<DDP_BF16, DDP_LINEAR_BACKWARD_INPUT>(g, workspace, false, as_stream(stream))
                           : launch_product<DDP_FP32, DDP_LINEAR_BACKWARD_INPUT>(g, workspace, false, as_stream(stream));
}

extern "C" int ddp_linear_backward_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx, void* dw,
                                          int64_t lddw, void* db, int64_t M, int64_t N, int64_t K, int32_t dtype,
                                          int32_t grad_dtype, int32_t accumulate, void* workspace,
                                          int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_linear_backward_weight";
  int st = check_common(fn, M, N, K, dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  if (grad_dtype != dtype && grad_dtype != DDP_FP32)
    return fail(DDP_EINVAL, std::string(fn) + ": grad_dtype must be the data's or fp32");
  if (accumulate != 0 && accumulate != 1) return fail(DDP_EINVAL, std::string(fn) + ": accumulate must be 0 or 1");
  if (N == 0) return DDP_OK;
  const int eb = elem_bytes(dtype), gb = elem_bytes(grad_dtype);
  const int64_t need = scratch_bytes(DDP_LINEAR_BACKWARD_WEIGHT, N, K, M, dtype, db != nullptr);
  const Matrix m[] = {{dz, M, N, lddz, eb, "dz", false, false}, {x, M, K, ldx, eb, "x", false, false},
                      {dw, N, K, lddw, gb, "dw", true, false},  {db, 1, N, N, gb, "db", true, true},
                      {need > 0 ? workspace : nullptr, 1, need, need, 1, "workspace", true, true}};
  st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  st = check_matrices(fn, m, 5, -1, -1);
  if (st != DDP_OK) return st;
  hipStream_t s = as_stream(stream);
  const void* sums = dz;  // what the bias gradient is summed from: without inputs, dz itself
  int64_t sums_ld = lddz, sums_rows = M;
  if (K > 0) {
    LinearArgs g{};
    g.a = dz, g.lda = lddz, g.b = x, g.ldb = ldx;
    g.I = N, g.J = K, g.K = M;
    g.c = dw, g.ldc = lddw;
    g.grad32 = grad_dtype == DDP_FP32, g.accumulate = accumulate;
    st = dtype == DDP_BF16 ? launch_product<DDP_BF16, DDP_LINEAR_BACKWARD_WEIGHT>(g, workspace, db != nullptr, s)
                           : launch_product<DDP_FP32, DDP_LINEAR_BACKWARD_WEIGHT>(g, workspace, db != nullptr, s);
    if (st != DDP_OK) return st;
    sums = g.row_sums, sums_ld = N, sums_rows = int64_t(g.parts) * g.tiles_j;
  }
  if (db == nullptr) return DDP_OK;
  const char* where = "ddp_linear_backward_weight: bias launch";
  return K == 0 && dtype == DDP_BF16 ? launch_column_sums<DDP_BF16>(sums, sums_ld, sums_rows, N, db, grad_dtype, accumulate, where, s)
                                     : launch_column_sums<DDP_FP32>(sums, sums_ld, sums_rows, N, db, grad_dtype, accumulate, where, s);
}

extern "C" int ddp_act_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz,
                                int64_t M, int64_t N, int32_t dtype, int32_t act, void* stream) {
  const char* fn = "ddp_act_backward";
  int st = check_common(fn, M, N, 0, dtype, act);
  if (st != DDP_OK) return st;
  if (M == 0 || N == 0) return DDP_OK;
  const int eb = elem_bytes(dtype);
  const Matrix m[] = {{dy, M, N, lddy, eb, "dy", false, false}, {z, M, N, ldz, eb, "z", false, false},
                      {dz, M, N, lddz, eb, "dz", true, false}};
  st = check_matrices(fn, m, 3, 0, 2);
  if (st != DDP_OK) return st;
  hipStream_t s = as_stream(stream);
  if (dtype == DDP_BF16)
    launch_act_backward<DDP_BF16>(dy, lddy, z, ldz, dz, lddz, M, N, act, s);
  else
    launch_act_backward<DDP_FP32>(dy, lddy, z, ldz, dz, lddz, M, N, act, s);
  DDP_HIP_TRY(hipGetLastError(), "ddp_act_backward: launch");
  return DDP_OK;
}
