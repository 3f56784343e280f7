// The AdamW step on fp32 master weights, all tensors in one launch:
//
//   g = f grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
//
// with the clipping factor f read from the gradients' norm on the device. Per
// element it reads p, m, v and the gradient and writes p, m, v (and the bf16
// weights): 28 bytes in fp32 against about 16 flops, so memory is the bound.
// Applying f here saves clipping's own pass (8 bytes an element in fp32).
#include <algorithm>
#include <cmath>
#include <new>

#include "train_internal.h"

namespace ddp {
namespace {

struct AdamTile {
  const void* g;
  float* p;
  float* m;
  float* v;
  uint16_t* c;     // bf16 weights, or NULL
  int32_t count;   // elements, kAdamTile but for a tensor's last tile
  int32_t decays;
};
// 512 elements: with 256 M elements and more, the 1 to 2 KB runs of each array
// that a block of this size touches kept HBM busier than longer ones (300M
// elements, bf16 gradients and weights: 1.46 ms at 512, 1.54 at 1024, 1.72 at
// 256).
constexpr int kAdamTile = 512;

// Step constants; those near 1 or 0 are taken from fp64 (1 - 0.999 in fp32 is
// off by 1e-5).
struct AdamArgs {
  float b1, c1;      // beta1, 1 - beta1
  float b2, c2;
  float keep;        // 1 - lr * weight_decay
  float eps;
  float lr;
  double log_b1, log_b2;
  float max_norm;
  const float* norm;   // NULL: no clipping
  long long* step;
  unsigned int* tickets;
  int32_t begin;       // the launch's first tile
  int32_t last;        // whether the step's last launch: it moves the count on
};

// 1 - b^t = -expm1(t ln b). The product is made in fp64 and rounded once, and
// expm1 keeps the relative precision of a small one, so fp32 is enough from
// there; b^t by itself would need fp64 (1 - 0.999 in fp32 is off by 1e-5).
__device__ __forceinline__ float correction(double log_b, double t) { return -expm1f(float(log_b * t)); }

struct AdamElem {
  float p, m, v;
};

__device__ __forceinline__ AdamElem adam(float g, float p, float m, float v, const AdamArgs& a, float keep, float rate,
                                         float root) {
  m = fmaf(a.b1, m, a.c1 * g);
  v = fmaf(a.b2, v, a.c2 * (g * g));
  const float denom = fmaf(sqrtf(v), root, a.eps);
  p = fmaf(-rate, m / denom, keep * p);
  return {p, m, v};
}

// One block per tile and one wave per array: wave 0 streams the gradient (and
// the bf16 weights), waves 1 to 3 p, m and v; they meet in LDS, where each
// thread updates two elements. A wave that reads and writes one array keeps
// each array's accesses together; threads that each took 4 elements of every
// array ran the 300M-element step in 1.62 ms against 1.54. Blocks go to the 8
// XCDs in turn, so block b takes tile b / 8 of the part b % 8 of the tiles:
// each XCD walks a run of memory of its own (1.46 against 1.54 ms, 5.8 TB/s).
//
// NT: accesses stream past the caches, for tensors that exceed the Infinity
// Cache together (1.46 against 1.84 ms with cached loads).
template <int DT, bool NT>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamTile* tiles, int64_t n_tiles, AdamArgs a) {
  constexpr int U = kAdamTile / 256;   // vectors of four per lane
  __shared__ float st[4][kAdamTile];
  AdamTile tile{};
  const unsigned int at = unsigned(a.begin) + blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;  // the grid is a multiple of 8
  if (at < n_tiles) tile = table_entry(tiles, at);  // else an empty one
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 64), lane = int(threadIdx.x) % 64;
  float x[U][4];
  if (tile.count == kAdamTile) {
    if (wave == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) load4<DT, NT>(tile.g, u * 64 + lane, x[u]);
    } else {
      const float* p = wave == 1 ? tile.p : wave == 2 ? tile.m : tile.v;
#pragma unroll
      for (int u = 0; u < U; ++u) load4<DDP_FP32, NT>(p, u * 64 + lane, x[u]);
    }
  }
  float f = 1.0f;
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(fabsf(norm) < INFINITY)) return;  // the step is skipped, by every block alike
    const float q = a.max_norm / (norm + 1e-6f);
    f = q >= 1.0f ? 1.0f : q;
  }
  const long long t = *a.step + 1;
  const float rate = a.lr / correction(a.log_b1, double(t));
  const float root = 1.0f / sqrtf(correction(a.log_b2, double(t)));  // sqrt(v / (1 - b2^t)) = root * sqrt(v)
  const float keep = tile.decays ? a.keep : 1.0f;
  if (tile.count == kAdamTile) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      *reinterpret_cast<float4*>(&st[wave][(u * 64 + lane) * 4]) = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = u * kThreads + int(threadIdx.x);
      const AdamElem y = adam(f * st[0][e], st[1][e], st[2][e], st[3][e], a, keep, rate, root);
      st[1][e] = y.p, st[2][e] = y.m, st[3][e] = y.v;
    }
    __syncthreads();
    if (wave == 0) {
      if (tile.c != nullptr)
#pragma unroll
        for (int u = 0; u < U; ++u) store4<DDP_BF16, NT>(tile.c, u * 64 + lane, &st[1][(u * 64 + lane) * 4]);
    } else {
      float* p = wave == 1 ? tile.p : wave == 2 ? tile.m : tile.v;
#pragma unroll
      for (int u = 0; u < U; ++u) store4<DDP_FP32, NT>(p, u * 64 + lane, &st[wave][(u * 64 + lane) * 4]);
    }
  } else {
    for (int e = threadIdx.x; e < tile.count; e += kThreads) {
      const AdamElem y = adam(f * Ops<DT>::load1(tile.g, e), tile.p[e], tile.m[e], tile.v[e], a, keep, rate, root);
      tile.p[e] = y.p;
      tile.m[e] = y.m;
      tile.v[e] = y.v;
      if (tile.c != nullptr) Ops<DDP_BF16>::store1(tile.c, e, round_bf16(y.p));
    }
  }
  // The step count moves on when every block has read it: the last block of
  // the last launch to finish writes it.
  if (!a.last) return;
  __syncthreads();
  if (threadIdx.x == 0 && is_last_block(a.tickets)) *a.step = t;
}

template <int DT>
void launch_adamw(const AdamTile* tiles, int64_t n_tiles, int64_t bytes, AdamArgs a, hipStream_t s) {
  int64_t t = 0;
  do {  // no tiles: one launch, which counts the step
    a.begin = int32_t(t);
    a.last = t + kMaxGrid >= n_tiles;
    const dim3 grid(unsigned(std::max<int64_t>(8, round_up(std::min(n_tiles - t, kMaxGrid), 8)))), block(kThreads);
    if (bytes > kInfinityCacheBytes)
      hipLaunchKernelGGL((k_adamw<DT, true>), grid, block, 0, s, tiles, n_tiles, a);
    else
      hipLaunchKernelGGL((k_adamw<DT, false>), grid, block, 0, s, tiles, n_tiles, a);
    t += kMaxGrid;
  } while (t < n_tiles);
}

}  // namespace
}  // namespace ddp

struct ddp_adamw {
  int32_t dtype = DDP_FP32;  // the gradients'
  int dev = 0;
  int64_t n_tiles = 0;
  int64_t bytes = 0;       // of all the tensors
  void* memory = nullptr;  // tiles, then the tickets
  ddp::AdamTile* tiles = nullptr;
  unsigned int* tickets = nullptr;
  int64_t* step = nullptr;
  std::vector<ddp::Span> written;  // everything but the gradients, by address
};

using namespace ddp;

extern "C" int ddp_adamw_create(const ddp_grads* grads, void* const* params, void* const* exp_avg,
                                void* const* exp_avg_sq, void* const* params_bf16, const uint8_t* decay,
                                int64_t* step_dev, ddp_adamw** out) {
  const char* fn = "ddp_adamw_create";
  if (out == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": out is NULL");
  *out = nullptr;
  if (grads == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": grads is NULL");
  const size_t n = grads->numels.size();
  if (n > 0 && (params == nullptr || exp_avg == nullptr || exp_avg_sq == nullptr))
    return fail(DDP_EINVAL, std::string(fn) + ": an array is NULL");
  int st = check_device(grads->dev, fn);
  if (st != DDP_OK) return st;
  st = check_scalar(step_dev, 8, fn, "step_dev");
  if (st != DDP_OK) return st;
  ddp_adamw* o = nullptr;
  try {
    std::vector<Span> spans{{step_dev, 8, "step_dev", -1}};
    std::vector<AdamTile> tiles;
    for (size_t i = 0; i < n; ++i) {
      const int64_t numel = grads->numels[i];
      if (numel == 0) continue;
      spans.push_back({grads->ptrs[i], numel * elem_bytes(grads->dtype), "grads", int32_t(i)});
      const struct {
        void* p;
        int eb;
        const char* what;
      } arrays[4] = {{params[i], 4, "params"},
                     {exp_avg[i], 4, "exp_avg"},
                     {exp_avg_sq[i], 4, "exp_avg_sq"},
                     {params_bf16 == nullptr ? nullptr : params_bf16[i], 2, "params_bf16"}};
      for (int k = 0; k < (params_bf16 == nullptr ? 3 : 4); ++k) {
        const std::string what = std::string(arrays[k].what) + "[" + std::to_string(i) + "]";
        if (reinterpret_cast<uintptr_t>(arrays[k].p) % uintptr_t(arrays[k].eb) != 0)
          return fail(DDP_EINVAL, std::string(fn) + ": " + what + " is not aligned to its element");
        st = check_range(arrays[k].p, numel * arrays[k].eb, fn, what.c_str());
        if (st != DDP_OK) return st;
        spans.push_back({arrays[k].p, numel * arrays[k].eb, arrays[k].what, int32_t(i)});
      }
      for (int64_t e = 0; e < numel; e += kAdamTile)
        tiles.push_back({static_cast<const char*>(grads->ptrs[i]) + e * elem_bytes(grads->dtype),
                         static_cast<float*>(params[i]) + e, static_cast<float*>(exp_avg[i]) + e,
                         static_cast<float*>(exp_avg_sq[i]) + e,
                         params_bf16 == nullptr ? nullptr : static_cast<uint16_t*>(params_bf16[i]) + e,
                         int32_t(std::min<int64_t>(kAdamTile, numel - e)), decay == nullptr || decay[i] != 0});
    }
    st = check_disjoint(spans, fn);
    if (st != DDP_OK) return st;
    if (tiles.size() >= (size_t(1) << 31)) return fail(DDP_EINVAL, std::string(fn) + ": too many elements");
    o = new ddp_adamw;
    o->dtype = grads->dtype;
    o->dev = grads->dev;
    o->n_tiles = int64_t(tiles.size());
    o->bytes = grads->total * (elem_bytes(grads->dtype) + 12 + (params_bf16 == nullptr ? 0 : 2));
    o->step = step_dev;
    for (const Span& w : spans)
      if (w.what != std::string("grads")) o->written.push_back(w);
    const size_t table = size_t(round_up(int64_t(sizeof(AdamTile) * tiles.size()), 256));
    hipError_t e = hipMalloc(&o->memory, table + kTicketBytes);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      delete o;
      return fail(DDP_ENOMEM, std::string(fn) + ": hipMalloc: " + hipGetErrorString(e));
    }
    char* base = static_cast<char*>(o->memory);
    const std::vector<char> zeros(kTicketBytes, 0);
    if (!tiles.empty()) e = hipMemcpy(base, tiles.data(), sizeof(AdamTile) * tiles.size(), hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipMemcpy(base + table, zeros.data(), zeros.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
      (void)hipFree(o->memory);
      delete o;
      return hip_fail(e, "ddp_adamw_create: tables");
    }
    o->tiles = reinterpret_cast<AdamTile*>(base);
    o->tickets = reinterpret_cast<unsigned int*>(base + table);
    *out = o;
    return DDP_OK;
  } catch (const std::bad_alloc&) {
    if (o != nullptr && o->memory != nullptr) (void)hipFree(o->memory);
    delete o;
    return fail(DDP_ENOMEM, std::string(fn) + ": out of host memory");
  }
}

extern "C" void ddp_adamw_free(ddp_adamw* o) {
  if (o == nullptr) return;
  (void)hipFree(o->memory);
  delete o;
}

extern "C" int ddp_adamw_step(ddp_adamw* o, double lr, double beta1, double beta2, double eps, double weight_decay,
                              double max_norm, const float* norm_dev, void* stream) {
  const char* fn = "ddp_adamw_step";
  if (o == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": opt is NULL");
  if (!(lr >= 0.0 && std::isfinite(lr) && eps >= 0.0 && std::isfinite(eps) && weight_decay >= 0.0 &&
        std::isfinite(weight_decay)))
    return fail(DDP_EINVAL, std::string(fn) + ": lr, eps and weight_decay must be finite and not negative");
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
    return fail(DDP_EINVAL, std::string(fn) + ": beta1 and beta2 must lie in [0, 1)");
  int st = check_device(o->dev, fn);
  if (st != DDP_OK) return st;
  if (norm_dev != nullptr) {
    if (!(max_norm >= 0.0)) return fail(DDP_EINVAL, std::string(fn) + ": max_norm is negative or not a number");
    st = check_scalar(norm_dev, 4, fn, "norm_dev");
    if (st != DDP_OK) return st;
    st = check_norm_apart(norm_dev, o->written, fn);
    if (st != DDP_OK) return st;
  }
  AdamArgs a{};
  a.b1 = float(beta1), a.c1 = float(1.0 - beta1);
  a.b2 = float(beta2), a.c2 = float(1.0 - beta2);
  a.keep = float(1.0 - lr * weight_decay);
  a.eps = float(eps);
  a.lr = float(lr);
  a.log_b1 = std::log(beta1), a.log_b2 = std::log(beta2);  // -inf for 0: b^t = 0
  a.max_norm = float(max_norm);
  a.norm = norm_dev;
  a.step = reinterpret_cast<long long*>(o->step);
  a.tickets = o->tickets;
  if (o->dtype == DDP_FP32)
    launch_adamw<DDP_FP32>(o->tiles, o->n_tiles, o->bytes, a, as_stream(stream));
  else
    launch_adamw<DDP_BF16>(o->tiles, o->n_tiles, o->bytes, a, as_stream(stream));
  DDP_HIP_TRY(hipGetLastError(), "ddp_adamw_step: launch");
  return DDP_OK;
}
