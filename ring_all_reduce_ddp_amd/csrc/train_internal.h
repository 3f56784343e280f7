// Declarations shared by the sources of the operators around the sync
// (ddp_train.h).
#pragma once

#include <cstdint>
#include <vector>

#include "ddp_train.h"
#include "hip_common.h"

namespace ddp {

// A tile of a gradient set: `count` consecutive elements from p, all of one
// tensor. Every tile but a tensor's last has kGradTile elements.
struct GradTile {
  void* p;
  int32_t count;
  int32_t tensor;
};
constexpr int kGradTile = 8192;
// Blocks of the norm's launch at most, one fp64 partial sum each.
constexpr int kNormBlocks = 1024;

// Vectors at the alignment of one element: tensors may start anywhere. gfx950
// runs in unaligned access mode, so these are single wide loads and stores.
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Pointers that come from a table are generic to the compiler; these say that
// they are global, so that accesses become global_load / global_store (a
// generic access also occupies the LDS counter), and the table itself is read
// with scalar loads.
#define DDP_GLOBAL __attribute__((address_space(1)))
#define DDP_CONST __attribute__((address_space(4)))
template <class T>
__device__ __forceinline__ T table_entry(const T* table, int64_t i) {
  struct Words {
    uint64_t w[sizeof(T) / 8];
  } e;
  const DDP_CONST uint64_t* q = (const DDP_CONST uint64_t*)(table + i);
  for (size_t k = 0; k < sizeof(T) / 8; ++k) e.w[k] = q[k];
  return __builtin_bit_cast(T, e);
}
// 16 or 8 bytes at any element's alignment; NT: streamed past the caches.
template <bool NT, class T>
__device__ __forceinline__ T load_at(const void* p, int64_t i) {
  const DDP_GLOBAL T* q = (const DDP_GLOBAL T*)p + i;
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool NT, class T>
__device__ __forceinline__ void store_at(void* p, int64_t i, T v) {
  DDP_GLOBAL T* q = (DDP_GLOBAL T*)p + i;
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}
// Four consecutive elements of a tensor, i in units of four.
template <int DT, bool NT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float x[4]) {
  if constexpr (DT == DDP_FP32) {
    const u32x4 w = load_at<NT, u32x4_at4>(p, i);
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
  } else {
    const u32x2 w = load_at<NT, u32x2_at2>(p, i);
    x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  }
}
template <int DT, bool NT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float x[4]) {
  if constexpr (DT == DDP_FP32)
    store_at<NT, u32x4_at4>(p, i, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
  else
    store_at<NT, u32x2_at2>(p, i, u32x2{round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3])});
}

// Which block of a launch finishes last. Device-wide atomics on one address
// take their turns, about 11 ns each on MI355X (2048 blocks on one counter:
// 20 us), so blocks count in on kTicketLines counters, on lines of their own,
// and the last of each line counts in on the top one.
// All counters are 0 between launches. Called by one thread of each block.
constexpr int kTicketLines = 64;
constexpr int kTicketStride = 32;  // words: 128 bytes
constexpr size_t kTicketBytes = size_t(kTicketLines + 1) * kTicketStride * 4;
__device__ __forceinline__ bool is_last_block(unsigned int* tickets) {
  const unsigned int blocks = gridDim.x, line = blockIdx.x % kTicketLines;
  const unsigned int lines = blocks < unsigned(kTicketLines) ? blocks : unsigned(kTicketLines);
  const unsigned int members = (blocks - line + kTicketLines - 1) / kTicketLines;
  unsigned int* const mine = tickets + (1 + line) * kTicketStride;
  if (__hip_atomic_fetch_add(mine, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != members - 1) return false;
  __hip_atomic_store(mine, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__hip_atomic_fetch_add(tickets, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != lines - 1) return false;
  __hip_atomic_store(tickets, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}

// A range that a call touches, for the checks of overlap.
struct Span {
  const void* p;
  int64_t bytes;
  const char* what;
  int32_t index;
};
// DDP_EINVAL, naming both, if two of the spans overlap (empty ones do not).
int check_disjoint(std::vector<Span>& spans, const char* fn);
bool spans_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes);
// DDP_EINVAL if the norm's place overlaps one of `written`: sorted, disjoint
// spans (as check_disjoint leaves them) that the call's blocks write while others
// read the norm, or read until it is written.
int check_norm_apart(const float* norm_dev, const std::vector<Span>& written, const char* fn);
// DDP_EINVAL unless `dev` is the current device.
int check_device(int dev, const char* fn);
// p: a device pointer to an aligned scalar of `bytes` bytes.
int check_scalar(const void* p, int64_t bytes, const char* fn, const char* what);

}  // namespace ddp

struct ddp_grads {
  int32_t dtype = DDP_FP32;
  int dev = 0;
  std::vector<void*> ptrs;
  std::vector<int64_t> numels;
  std::vector<ddp::Span> spans;   // of the tensors that are not empty, by address
  int64_t total = 0;              // elements
  uintptr_t lo = 0, hi = 0;       // addresses from the lowest tensor's start to the highest one's end
  int64_t n_tiles = 0;
  void* memory = nullptr;         // the one allocation: tiles, then scratch
  ddp::GradTile* tiles = nullptr;
  double* partials = nullptr;     // kNormBlocks
  unsigned int* tickets = nullptr;  // is_last_block's counters
};
