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
constexpr int kNormBlocks = 2048;

// Vectors at the alignment of one element: tensors may start anywhere. gfx950
// runs in unaligned access mode, so these are single wide loads and stores.
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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
  int64_t total = 0;              // elements
  uintptr_t lo = 0, hi = 0;       // addresses from the lowest tensor's start to the highest one's end
  int64_t n_tiles = 0;
  void* memory = nullptr;         // the one allocation: tiles, then scratch
  ddp::GradTile* tiles = nullptr;
  double* partials = nullptr;     // kNormBlocks
  unsigned int* ticket = nullptr; // 0 between launches
};
