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
constexpr int kAdamTile = 2048;

// Step constants; those near 1 or 0 are taken from fp64 (1 - 0.999 in fp32 is
// off by 1e-5).
struct AdamArgs {
  float b1, c1;      // beta1, 1 - beta1
  float b2, c2;
  float keep;        // 1 - lr * weight_decay
  float eps;
  double lr, beta1, beta2;
  float max_norm;
  const float* norm;   // NULL: no clipping
  long long* step;
  unsigned int* ticket;
};

// b^t in fp64 by squaring: at most 2 log2(t) products.
__device__ __forceinline__ double power(double b, long long t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

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

template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float x[4]) {
  if constexpr (DT == DDP_FP32) {
    const u32x4 w = reinterpret_cast<const u32x4_at4*>(p)[i];
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
  } else {
    const u32x2 w = reinterpret_cast<const u32x2_at2*>(p)[i];
    x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  }
}

__device__ __forceinline__ void store4(float* p, int64_t i, const float x[4]) {
  reinterpret_cast<u32x4_at4*>(p)[i] =
      u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamTile* tiles, int64_t n_tiles, AdamArgs a) {
  float f = 1.0f;
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(fabsf(norm) < INFINITY)) return;  // the step is skipped, by every block alike
    const float q = a.max_norm / (norm + 1e-6f);
    f = q >= 1.0f ? 1.0f : q;
  }
  const long long t = *a.step + 1;
  const float rate = float(a.lr / (1.0 - power(a.beta1, t)));
  const float root = float(sqrt(1.0 / (1.0 - power(a.beta2, t))));  // sqrt(v / (1 - b2^t)) = root * sqrt(v)
  for (int64_t i = blockIdx.x; i < n_tiles; i += gridDim.x) {
    const AdamTile tile = tiles[i];
    const float keep = tile.decays ? a.keep : 1.0f;
    const int vecs = tile.count / 4;
    for (int k = threadIdx.x; k < vecs; k += kThreads) {
      float g[4], p[4], m[4], v[4];
      load4<DT>(tile.g, k, g);
      load4<DDP_FP32>(tile.p, k, p);
      load4<DDP_FP32>(tile.m, k, m);
      load4<DDP_FP32>(tile.v, k, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const AdamElem e = adam(f * g[j], p[j], m[j], v[j], a, keep, rate, root);
        p[j] = e.p, m[j] = e.m, v[j] = e.v;
      }
      store4(tile.p, k, p);
      store4(tile.m, k, m);
      store4(tile.v, k, v);
      if (tile.c != nullptr)
        reinterpret_cast<u32x2_at2*>(tile.c)[k] = u32x2{round_bf16x2(p[0], p[1]), round_bf16x2(p[2], p[3])};
    }
    const int e = vecs * 4 + int(threadIdx.x);
    if (e < tile.count) {
      const AdamElem x = adam(f * Ops<DT>::load1(tile.g, e), tile.p[e], tile.m[e], tile.v[e], a, keep, rate, root);
      tile.p[e] = x.p;
      tile.m[e] = x.m;
      tile.v[e] = x.v;
      if (tile.c != nullptr) Ops<DDP_BF16>::store1(tile.c, e, round_bf16(x.p));
    }
  }
  // The step count moves on when every block has read it: the block with the
  // last ticket writes it, and clears the ticket for the next launch.
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned int k = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (k == gridDim.x - 1) {
      __hip_atomic_store(a.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *a.step = t;
    }
  }
}

}  // namespace
}  // namespace ddp

struct ddp_adamw {
  int32_t dtype = DDP_FP32;  // the gradients'
  int dev = 0;
  int64_t n_tiles = 0;
  void* memory = nullptr;  // tiles, then the ticket
  ddp::AdamTile* tiles = nullptr;
  unsigned int* ticket = nullptr;
  int64_t* step = nullptr;
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
    o = new ddp_adamw;
    o->dtype = grads->dtype;
    o->dev = grads->dev;
    o->n_tiles = int64_t(tiles.size());
    o->step = step_dev;
    const size_t table = size_t(round_up(int64_t(sizeof(AdamTile) * tiles.size()), 256));
    hipError_t e = hipMalloc(&o->memory, table + 256);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      delete o;
      return fail(DDP_ENOMEM, std::string(fn) + ": hipMalloc: " + hipGetErrorString(e));
    }
    char* base = static_cast<char*>(o->memory);
    const char zeros[256] = {};
    if (!tiles.empty()) e = hipMemcpy(base, tiles.data(), sizeof(AdamTile) * tiles.size(), hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipMemcpy(base + table, zeros, sizeof(zeros), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
      (void)hipFree(o->memory);
      delete o;
      return hip_fail(e, "ddp_adamw_create: tables");
    }
    o->tiles = reinterpret_cast<AdamTile*>(base);
    o->ticket = reinterpret_cast<unsigned int*>(base + table);
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
  }
  AdamArgs a{};
  a.b1 = float(beta1), a.c1 = float(1.0 - beta1);
  a.b2 = float(beta2), a.c2 = float(1.0 - beta2);
  a.keep = float(1.0 - lr * weight_decay);
  a.eps = float(eps);
  a.lr = lr, a.beta1 = beta1, a.beta2 = beta2;
  a.max_norm = float(max_norm);
  a.norm = norm_dev;
  a.step = reinterpret_cast<long long*>(o->step);
  a.ticket = o->ticket;
  const dim3 grid(unsigned(std::max<int64_t>(1, std::min<int64_t>(o->n_tiles, 4096)))), block(kThreads);
  if (o->dtype == DDP_FP32)
    hipLaunchKernelGGL(k_adamw<DDP_FP32>, grid, block, 0, as_stream(stream), o->tiles, o->n_tiles, a);
  else
    hipLaunchKernelGGL(k_adamw<DDP_BF16>, grid, block, 0, as_stream(stream), o->tiles, o->n_tiles, a);
  DDP_HIP_TRY(hipGetLastError(), "ddp_adamw_step: launch");
  return DDP_OK;
}
