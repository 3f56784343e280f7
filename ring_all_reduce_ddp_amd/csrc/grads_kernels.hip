// The global norm of a set of gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)   (or max |g|)
//   clip: g <- rnd(g * min(1, max_norm / (norm + 1e-6)))
//
// Both stream the gradients: two flops a byte at most, so the bound is memory.
// The set's tile table maps a block to a run of one tensor with one scalar
// load (no search over tensors, no launch per tensor).
#include <algorithm>
#include <cmath>
#include <new>

#include "train_internal.h"

namespace ddp {

bool spans_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return abytes > 0 && bbytes > 0 && x < y + uint64_t(bbytes) && y < x + uint64_t(abytes);
}

namespace {

std::string span_name(const Span& s) {
  return s.index < 0 ? std::string(s.what) : std::string(s.what) + "[" + std::to_string(s.index) + "]";
}

unsigned stream_grid(int64_t tiles, int64_t most) { return unsigned(std::max<int64_t>(1, std::min(tiles, most))); }

template <int DT, bool NT>
__device__ __forceinline__ u32x4 load16(const void* p, int64_t i) {
  if constexpr (DT == DDP_FP32)
    return load_at<NT, u32x4_at4>(p, i);
  else
    return load_at<NT, u32x4_at2>(p, i);
}

// Running sum of squares, or largest magnitude, of one thread.
//
// The squares are added in fp64: an fp32 square overflows from 1.8e19 and
// vanishes below 1e-23, and a sum of 1e9 of them loses digits. fp64 runs at
// half the fp32 rate here, far from the bound of a stream.
template <int KIND>
struct Norm;
template <>
struct Norm<DDP_NORM_L2> {
  double s[2] = {0.0, 0.0};
  __device__ __forceinline__ void add(float x, int k) { s[k & 1] = fma(double(x), double(x), s[k & 1]); }
  __device__ __forceinline__ double value() const { return s[0] + s[1]; }
  static __device__ __forceinline__ double join(double a, double b) { return a + b; }
  static __device__ __forceinline__ float finish(double s) { return float(sqrt(s)); }
};
// Magnitudes compare as the integers of their bits, NaN above infinity, so a
// NaN survives every comparison. The partial travels as the double of that
// integer, which is exact.
template <>
struct Norm<DDP_NORM_MAX> {
  uint32_t m[2] = {0u, 0u};
  __device__ __forceinline__ void add(float x, int k) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    m[k & 1] = b > m[k & 1] ? b : m[k & 1];
  }
  __device__ __forceinline__ double value() const { return double(m[0] > m[1] ? m[0] : m[1]); }
  static __device__ __forceinline__ double join(double a, double b) { return a > b ? a : b; }
  static __device__ __forceinline__ float finish(double s) { return __uint_as_float(uint32_t(s)); }
};

// The block's 256 values joined in a fixed order; valid in thread 0.
template <int KIND>
__device__ __forceinline__ double block_join(double v) {
  __shared__ double wave[kThreads / 64];
  for (int d = 32; d > 0; d >>= 1) v = Norm<KIND>::join(v, __shfl_down(v, d));
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = wave[0];
  for (int w = 1; w < kThreads / 64; ++w) v = Norm<KIND>::join(v, wave[w]);
  __syncthreads();
  return v;
}

// One launch: every block leaves one fp64 partial, and the block whose ticket
// is the last joins them, in index order whichever block that is, so the
// result does not depend on the order of arrival.
//
// Blocks walk the tiles with 32 KB in flight each (8192 elements of fp32, 16
// KB of bf16), 1024 blocks at most: 157 us over 1 GiB of fp32 (6.9 TB/s)
// against 165 with 2048 blocks; 300M bf16 91 us against 97.
// NT: loads stream past the caches, for a set that exceeds the Infinity Cache
// (157 against 170 us cached at 1 GiB; at 300M bf16 the clip that follows gains
// 1 us from what cached loads leave behind, less than the norm loses).
template <int DT, int KIND, bool NT>
__global__ __launch_bounds__(kThreads) void k_grads_norm(const GradTile* tiles, int64_t n_tiles, double* partials,
                                                         unsigned int* tickets, float* norm) {
  constexpr int V = Ops<DT>::V;
  constexpr int U = kGradTile / (kThreads * V);
  Norm<KIND> acc;
  for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x) {
    const GradTile tile = table_entry(tiles, t);
    if (tile.count == kGradTile) {
      u32x4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = load16<DT, NT>(tile.p, u * kThreads + int(threadIdx.x));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const typename Ops<DT>::Acc a = Ops<DT>::from(x[u]);
#pragma unroll
        for (int i = 0; i < V; ++i) acc.add(a.v[i], i);
      }
    } else {
      const int vecs = tile.count / V;
      for (int i = threadIdx.x; i < vecs; i += kThreads) {
        const typename Ops<DT>::Acc a = Ops<DT>::from(load16<DT, NT>(tile.p, i));
#pragma unroll
        for (int j = 0; j < V; ++j) acc.add(a.v[j], j);
      }
      const int e = vecs * V + int(threadIdx.x);
      if (e < tile.count) acc.add(Ops<DT>::load1(tile.p, e), 0);
    }
  }
  const double mine = block_join<KIND>(acc.value());
  if (gridDim.x == 1) {
    if (threadIdx.x == 0) *norm = Norm<KIND>::finish(mine);
    return;
  }
  __shared__ bool last;
  if (threadIdx.x == 0) {
    // The partial goes by an exchange whose old value is waited for: it has
    // then been performed where every XCD sees it, before the block counts
    // in. (A release fence would write back this XCD's whole L2 instead, once
    // per block.)
    const unsigned long long old = __hip_atomic_exchange(reinterpret_cast<unsigned long long*>(&partials[blockIdx.x]),
                                                         static_cast<unsigned long long>(__double_as_longlong(mine)),
                                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::"v"(old) : "memory");
    last = is_last_block(tickets);
  }
  __syncthreads();
  if (!last) return;
  double s = 0.0;
  for (unsigned int i = threadIdx.x; i < gridDim.x; i += kThreads)
    s = Norm<KIND>::join(s, __hip_atomic_load(&partials[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  s = block_join<KIND>(s);
  if (threadIdx.x == 0) *norm = Norm<KIND>::finish(s);
}

constexpr int kClipParts = 4;

// kClipParts blocks share a tile, 2048 elements each (300M bf16 into fp32: 302
// us with 4, 354 with 1, 362 with 8). Blocks go to the 8 XCDs in turn, so block b
// takes part b / 8 of eighth b % 8: each XCD walks memory of its own (302
// against 309 us; 1.8 GB, 6.0 TB/s). A launch's parts begin with `begin`.
template <int SRC, int DST, bool NTL, bool NTS>
__global__ __launch_bounds__(kThreads) void k_grads_clip(const GradTile* src, const GradTile* dst,
                                                         unsigned int begin, unsigned int n_parts, float max_norm,
                                                         const float* norm) {
  constexpr int kPart = kGradTile / kClipParts;
  constexpr int U = kPart / (kThreads * 4);
  const unsigned int at = begin + blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;  // the grid is a multiple of 8
  if (at >= n_parts) return;
  const GradTile a = table_entry(src, at / kClipParts);
  void* const to = table_entry(dst, at / kClipParts).p;
  const int first = at % kClipParts * kPart;
  const int count = a.count - first < kPart ? a.count - first : kPart;
  if (count == kPart) {
    float x[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) load4<SRC, NTL>(a.p, first / 4 + u * kThreads + int(threadIdx.x), x[u]);
    const float q = max_norm / (*norm + 1e-6f);
    const float f = q >= 1.0f ? 1.0f : q;  // a NaN stays
    if (src == dst && f == 1.0f) return;   // in place, nothing to do
#pragma unroll
    for (int u = 0; u < U; ++u) {
      for (int j = 0; j < 4; ++j) x[u][j] *= f;
      store4<DST, NTS>(to, first / 4 + u * kThreads + int(threadIdx.x), x[u]);
    }
    return;
  }
  if (count <= 0) return;
  const float q = max_norm / (*norm + 1e-6f);
  const float f = q >= 1.0f ? 1.0f : q;
  if (src == dst && f == 1.0f) return;
  const int vecs = count / 4;
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    float x[4];
    load4<SRC, NTL>(a.p, first / 4 + i, x);
    for (int j = 0; j < 4; ++j) x[j] *= f;
    store4<DST, NTS>(to, first / 4 + i, x);
  }
  const int e = first + vecs * 4 + int(threadIdx.x);
  if (e < first + count) {
    const float x = Ops<SRC>::load1(a.p, e) * f;
    Ops<DST>::store1(to, e, DST == DDP_BF16 ? round_bf16(x) : x);
  }
}

template <int DT, int KIND>
void launch_norm(const ddp_grads* g, float* norm, hipStream_t s) {
  const dim3 grid(stream_grid(g->n_tiles, kNormBlocks)), block(kThreads);
  if (g->total * elem_bytes(DT) > kInfinityCacheBytes)
    hipLaunchKernelGGL((k_grads_norm<DT, KIND, true>), grid, block, 0, s, g->tiles, g->n_tiles, g->partials, g->tickets, norm);
  else
    hipLaunchKernelGGL((k_grads_norm<DT, KIND, false>), grid, block, 0, s, g->tiles, g->n_tiles, g->partials, g->tickets, norm);
}

template <int SRC, int DST>
void launch_clip(const ddp_grads* g, const ddp_grads* into, float max_norm, const float* norm, hipStream_t s) {
  const int64_t parts = g->n_tiles * kClipParts;
  const auto launch = [&](auto kernel) {
    for (int64_t p = 0; p < parts; p += kMaxGrid) {
      const dim3 grid(unsigned(round_up(std::min(parts - p, kMaxGrid), 8))), block(kThreads);
      hipLaunchKernelGGL(kernel, grid, block, 0, s, g->tiles, into->tiles, unsigned(p), unsigned(parts), max_norm, norm);
    }
  };
  // Stores stream past the caches into another set, which leaves the cache to the
  // gradients that the norm has just read (25.6M fp32, 102 MB: both 51 us
  // against 62; whoever reads the result next pays 2 us of it back); loads, and
  // stores in place, from the Infinity Cache's size on.
  if (g->total * (elem_bytes(SRC) + elem_bytes(DST)) > kInfinityCacheBytes) return launch(k_grads_clip<SRC, DST, true, true>);
  if constexpr (SRC == DST) {
    if (into == g) return launch(k_grads_clip<SRC, DST, false, false>);
  }
  launch(k_grads_clip<SRC, DST, false, true>);
}

// The sets' tensors against each other: at once if the sets lie apart as
// wholes (two arenas), else tensor by tensor.
int check_sets_disjoint(const ddp_grads& a, const ddp_grads& b, const char* fn) {
  if (a.hi <= b.lo || b.hi <= a.lo) return DDP_OK;
  try {
    std::vector<Span> spans;
    for (size_t i = 0; i < a.ptrs.size(); ++i) {
      spans.push_back({a.ptrs[i], a.numels[i] * elem_bytes(a.dtype), "grads", int32_t(i)});
      spans.push_back({b.ptrs[i], b.numels[i] * elem_bytes(b.dtype), "into", int32_t(i)});
    }
    return check_disjoint(spans, fn);
  } catch (const std::bad_alloc&) {
    return fail(DDP_ENOMEM, std::string(fn) + ": out of host memory");
  }
}

}  // namespace

int check_disjoint(std::vector<Span>& spans, const char* fn) {
  spans.erase(std::remove_if(spans.begin(), spans.end(), [](const Span& s) { return s.bytes == 0; }), spans.end());
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) {
    return reinterpret_cast<uintptr_t>(a.p) < reinterpret_cast<uintptr_t>(b.p);
  });
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans_overlap(spans[i - 1].p, spans[i - 1].bytes, spans[i].p, spans[i].bytes))
      return fail(DDP_EINVAL, std::string(fn) + ": " + span_name(spans[i - 1]) + " and " + span_name(spans[i]) + " overlap");
  return DDP_OK;
}

int check_norm_apart(const float* norm_dev, const std::vector<Span>& written, const char* fn) {
  // the first span that ends behind the norm's start
  const auto s = std::partition_point(written.begin(), written.end(), [&](const Span& w) {
    return reinterpret_cast<uintptr_t>(w.p) + uint64_t(w.bytes) <= reinterpret_cast<uintptr_t>(norm_dev);
  });
  if (s != written.end() && spans_overlap(norm_dev, sizeof(float), s->p, s->bytes))
    return fail(DDP_EINVAL, std::string(fn) + ": norm_dev and " + span_name(*s) + " overlap");
  return DDP_OK;
}

int check_scalar(const void* p, int64_t bytes, const char* fn, const char* what) {
  int st = check_range(p, bytes, fn, what);
  if (st != DDP_OK) return st;
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes) != 0)
    return fail(DDP_EINVAL, std::string(fn) + ": " + what + " is not " + std::to_string(bytes) + "-byte aligned");
  return DDP_OK;
}

int check_device(int dev, const char* fn) {
  int now = 0;
  DDP_HIP_TRY(hipGetDevice(&now), fn);
  if (now != dev) return fail(DDP_EINVAL, std::string(fn) + ": the current device is not the one it was created on");
  return DDP_OK;
}

}  // namespace ddp

using namespace ddp;

extern "C" int ddp_grads_create(void* const* grads, const int64_t* numels, int32_t n, int32_t dtype, ddp_grads** out) {
  const char* fn = "ddp_grads_create";
  if (out == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": out is NULL");
  *out = nullptr;
  if (!valid_dtype(dtype)) return fail(DDP_EINVAL, std::string(fn) + ": unknown dtype");
  if (n < 0) return fail(DDP_EINVAL, std::string(fn) + ": n is negative");
  if (n > 0 && (grads == nullptr || numels == nullptr)) return fail(DDP_EINVAL, std::string(fn) + ": an array is NULL");
  const int eb = elem_bytes(dtype);
  ddp_grads* g = nullptr;
  try {
    std::vector<Span> spans;
    for (int32_t i = 0; i < n; ++i) {
      if (numels[i] < 0 || numels[i] > (int64_t(1) << 48))
        return fail(DDP_EINVAL, std::string(fn) + ": numels[" + std::to_string(i) + "] out of range");
      const std::string what = "grads[" + std::to_string(i) + "]";
      if (reinterpret_cast<uintptr_t>(grads[i]) % uintptr_t(eb) != 0 && numels[i] > 0)
        return fail(DDP_EINVAL, std::string(fn) + ": " + what + " is not aligned to its element");
      int st = check_range(grads[i], numels[i] * eb, fn, what.c_str());
      if (st != DDP_OK) return st;
      spans.push_back({grads[i], numels[i] * eb, "grads", i});
    }
    int st = check_disjoint(spans, fn);
    if (st != DDP_OK) return st;
    std::vector<GradTile> tiles;
    int64_t total = 0;
    uintptr_t lo = UINTPTR_MAX, hi = 0;
    for (int32_t i = 0; i < n; ++i) {
      if (numels[i] == 0) continue;
      total += numels[i];
      lo = std::min(lo, reinterpret_cast<uintptr_t>(grads[i]));
      hi = std::max(hi, reinterpret_cast<uintptr_t>(grads[i]) + uintptr_t(numels[i] * eb));
      for (int64_t e = 0; e < numels[i]; e += kGradTile)
        tiles.push_back({static_cast<char*>(grads[i]) + e * eb, int32_t(std::min<int64_t>(kGradTile, numels[i] - e)), i});
    }
    if (tiles.size() >= (size_t(1) << 31) / kClipParts)
      return fail(DDP_EINVAL, std::string(fn) + ": too many elements");
    g = new ddp_grads;
    g->dtype = dtype;
    if (n > 0) {
      g->ptrs.assign(grads, grads + n);
      g->numels.assign(numels, numels + n);
    }
    g->spans = std::move(spans);
    g->total = total;
    g->lo = lo;
    g->hi = hi;
    g->n_tiles = int64_t(tiles.size());
    const size_t table = size_t(round_up(int64_t(sizeof(GradTile) * tiles.size()), 256));
    const size_t scratch = sizeof(double) * kNormBlocks + kTicketBytes;
    hipError_t e = hipGetDevice(&g->dev);
    if (e == hipSuccess) {
      e = hipMalloc(&g->memory, table + scratch);
      if (e != hipSuccess) {
        (void)hipGetLastError();
        delete g;
        return fail(DDP_ENOMEM, std::string(fn) + ": hipMalloc: " + hipGetErrorString(e));
      }
    }
    char* base = static_cast<char*>(g->memory);
    if (e == hipSuccess && !tiles.empty())
      e = hipMemcpy(base, tiles.data(), sizeof(GradTile) * tiles.size(), hipMemcpyHostToDevice);
    if (e == hipSuccess) {
      const std::vector<char> zeros(scratch, 0);
      e = hipMemcpy(base + table, zeros.data(), scratch, hipMemcpyHostToDevice);
    }
    if (e != hipSuccess) {
      if (g->memory != nullptr) (void)hipFree(g->memory);
      delete g;
      return hip_fail(e, "ddp_grads_create: tables");
    }
    g->tiles = reinterpret_cast<GradTile*>(base);
    g->partials = reinterpret_cast<double*>(base + table);
    g->tickets = reinterpret_cast<unsigned int*>(base + table + sizeof(double) * kNormBlocks);
    *out = g;
    return DDP_OK;
  } catch (const std::bad_alloc&) {
    if (g != nullptr && g->memory != nullptr) (void)hipFree(g->memory);
    delete g;
    return fail(DDP_ENOMEM, std::string(fn) + ": out of host memory");
  }
}

extern "C" void ddp_grads_free(ddp_grads* g) {
  if (g == nullptr) return;
  (void)hipFree(g->memory);
  delete g;
}

extern "C" int ddp_grads_norm(ddp_grads* g, int32_t kind, float* norm_dev, void* stream) {
  const char* fn = "ddp_grads_norm";
  if (g == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": grads is NULL");
  if (kind != DDP_NORM_L2 && kind != DDP_NORM_MAX) return fail(DDP_EINVAL, std::string(fn) + ": unknown kind");
  int st = check_device(g->dev, fn);
  if (st != DDP_OK) return st;
  st = check_scalar(norm_dev, 4, fn, "norm_dev");
  if (st != DDP_OK) return st;
  st = check_norm_apart(norm_dev, g->spans, fn);
  if (st != DDP_OK) return st;
  hipStream_t s = as_stream(stream);
  if (g->dtype == DDP_FP32)
    kind == DDP_NORM_L2 ? launch_norm<DDP_FP32, DDP_NORM_L2>(g, norm_dev, s) : launch_norm<DDP_FP32, DDP_NORM_MAX>(g, norm_dev, s);
  else
    kind == DDP_NORM_L2 ? launch_norm<DDP_BF16, DDP_NORM_L2>(g, norm_dev, s) : launch_norm<DDP_BF16, DDP_NORM_MAX>(g, norm_dev, s);
  DDP_HIP_TRY(hipGetLastError(), "ddp_grads_norm: launch");
  return DDP_OK;
}

extern "C" int ddp_grads_clip(const ddp_grads* g, const ddp_grads* into, float max_norm, const float* norm_dev,
                              void* stream) {
  const char* fn = "ddp_grads_clip";
  if (g == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": grads is NULL");
  if (!(max_norm >= 0.0f)) return fail(DDP_EINVAL, std::string(fn) + ": max_norm is negative or not a number");
  int st = check_device(g->dev, fn);
  if (st != DDP_OK) return st;
  if (into == nullptr) into = g;
  if (into != g) {
    if (into->dev != g->dev) return fail(DDP_EINVAL, std::string(fn) + ": the sets are on different devices");
    if (into->numels != g->numels) return fail(DDP_EINVAL, std::string(fn) + ": the sets' element counts differ");
    st = check_sets_disjoint(*g, *into, fn);
    if (st != DDP_OK) return st;
  }
  st = check_scalar(norm_dev, 4, fn, "norm_dev");
  if (st != DDP_OK) return st;
  st = check_norm_apart(norm_dev, into->spans, fn);
  if (st != DDP_OK) return st;
  if (g->n_tiles == 0) return DDP_OK;
  hipStream_t s = as_stream(stream);
  const bool to32 = into->dtype == DDP_FP32;
  if (g->dtype == DDP_FP32)
    to32 ? launch_clip<DDP_FP32, DDP_FP32>(g, into, max_norm, norm_dev, s) : launch_clip<DDP_FP32, DDP_BF16>(g, into, max_norm, norm_dev, s);
  else
    to32 ? launch_clip<DDP_BF16, DDP_FP32>(g, into, max_norm, norm_dev, s) : launch_clip<DDP_BF16, DDP_BF16>(g, into, max_norm, norm_dev, s);
  DDP_HIP_TRY(hipGetLastError(), "ddp_grads_clip: launch");
  return DDP_OK;
}
