// Host side of the products (linear_device.h): how they are cut and launched,
// and the checks of their arguments.
#pragma once

#include <algorithm>
#include <cmath>
#include <string>

#include "linear_device.h"

namespace ddp {
namespace {

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }


// `blocks` blocks in launches of kMaxGrid at most: launch(first block, grid).
template <class F>
void launch_blocks(int64_t blocks, F&& launch) {
  for (int64_t b = 0; b < blocks; b += kMaxGrid) launch(b, dim3(unsigned(std::min(blocks - b, kMaxGrid))));
}

// Up to so many rows a forward product goes without tiles (linear_kernels.hip).
constexpr int kFewRows = 4;

// Flat tiles are for few rows, which read the other operand from memory: 32 rows,
// 128 columns and four steps of 128 bytes in LDS or on their way, two blocks a CU.
// (Cross entropy of 8 rows, 64000 columns of 2048 bf16 from memory: forward 53 us, with three steps 53.5, two
// 55, in tiles of 64 54; with the backward pass 270, 264, 269 and 306.)
constexpr int kFlatRows = 32, kFlatStages = 4;

// How a product is cut: the tile's side (256 needs direct loads), and in how
// many parts the sum. Up to kFewRows rows of a forward product go without
// tiles.
struct Cut {
  bool few = false;
  bool flat = false;  // 32 rows
  bool deep = false;  // 32 rows and columns, four waves along the sum
  bool half = false;  // 128 rows, of 256 columns
  int tile = 128;
  int32_t parts = 1;
  int64_t part_k = 0;
  int32_t rows() const { return flat ? 32 : half ? 128 : tile; }
};

// The cut with the least time by a rough model in cycles. Its constants were
// fitted to the times of 250 products of 5 to 8192 rows, 64 to 8192 columns
// and terms, odd and even, on MI355X, each cut in up to 27 ways: the cut it
// picks takes 1.9 % longer than the best of them in the mean, 31 % at worst. Those
// products are the linear layer's. The shapes that came with groups and losses (flat,
// deep, half) have constants set by hand: over 400 drawn products (8 to 16384 rows in up to 128 groups, 1 to 4096
// of losses, 64 to 4096 columns and terms), each also in every other tile, the pick takes longer than the best by
// 6 % in the mean (experts forward; 60 % at worst), 7 (input gradient; 36), 7 to 13 (weight gradient; 88) and
// 15 (z of losses; 149: 40 to 230 rows of some 2000 columns and terms, which deep tiles would take in half the time).
// A tile's step (128 bytes of k) takes `step` cycles of a CU that its blocks
// fill and `alone` of a block by itself, its outputs `ends`; parts cost a
// launch, a round each, and their bytes. With `groups`, of I rows or K terms in all,
// the groups count as equally long, a group of rows as half a tile longer.
Cut cut_by_model(int dir, int32_t I, int32_t J, int32_t K, int dtype, bool direct, int32_t groups, int32_t most_parts) {
  Cut best;
  if (dir == DDP_LINEAR_FORWARD && groups == 0 && I <= kFewRows) {
    best.few = true;
    return best;
  }
  struct Shape {
    int32_t tile, fit;  // `fit` blocks share a CU
    float step, alone, ends;
  };
  static const Shape shapes[2][2][3] = {
      // fp32: loads at any alignment, direct loads
      {{{64, 5, 1160, 1880, 1500}, {128, 2, 3840, 4670, 5400}, {}}, {{64, 5, 1050, 1140, 1230}, {128, 2, 3920, 3700, 2970}, {}}},
      // bf16
      {{{64, 5, 620, 1150, 1050}, {128, 2, 1850, 2040, 3350}, {}},
       {{64, 5, 440, 850, 2190}, {128, 2, 920, 1010, 4340}, {256, 1, 2100, 2290, 10160}}}};
  constexpr float kStart = 2000, kJoin = 13100, kPart = 320, kBytesPerCycle = 3160;
  constexpr int32_t kCus = 256;
  const auto up = [](int64_t a, int64_t b) { return int32_t((a + b - 1) / b); };
  const int32_t row = std::min(a_along(dir) ? K : I, b_along(dir) ? K : J);  // the operands' shorter rows
  const int n_shapes = row < 16 / elem_bytes(dtype) ? 1 : dtype == DDP_BF16 && direct ? 3 : 2;
  // Few rows: the other operand's bytes are what counts, whatever the type. (By the mean of the groups: where
  // one group has nearly all rows, they are read again for every 32 of them. 2048 rows of 64 groups, 4096 x 2048
  // bf16, evenly and so: 195 and 279 us; in half tiles, a row more, 195 and 202.)
  const Shape flat = direct ? Shape{128, 4, 1000, 600, 1000} : Shape{128, 4, 1500, 1100, 1000};
  // Groups of some 100 rows leave much of a tile of 256 empty: half tiles of 128 rows and 256 columns,
  // three steps in LDS or on their way. (4096 rows of 32 groups, 4096 x 2048: 162 us, in tiles of
  // 256 188; 16384 rows of 64: 480 and 461.)
  static const Shape half{256, 1, 1350, 1450, 5500};
  const bool half_rows = groups > 1 && !is_weight(dir) && n_shapes == 3;
  const bool flat_rows = (groups > 0 || dir >= kRowStats) && !is_weight(dir) && row >= 16 / elem_bytes(dtype) && I <= kFlatRows * std::max(groups, 1);
  const bool sums = groups > 0 && is_weight(dir);  // the groups are of terms
  const int32_t step = 128 / elem_bytes(dtype), steps = std::max(1, up(sums ? up(K, groups) : K, step));
  const float busy = float(std::min(groups, I));   // groups that have rows
  float least = INFINITY;
  const Shape deep{32, 2, 2600, direct ? 1100.0f : 1400.0f, 1500};  // of four steps
  for (int k = 0; k < (flat_rows ? b_along(dir) ? 2 : 1 : n_shapes + int(half_rows)); ++k) {
    const bool is_deep = flat_rows && k == 1;
    const Shape& sh = is_deep ? deep : flat_rows ? flat : k == 3 ? half : shapes[dtype == DDP_BF16][direct][k];
    const int32_t rows = flat_rows ? kFlatRows : k == 3 ? 128 : sh.tile;
    // Short sums are a matter of the outputs' bytes, in which two blocks a CU overlap better
    // than one (64 experts of 256 rows, 2048 x 4096, added to fp32: 950 us against 1070). Of 65 drawn
    // bf16 products with so short sums the 256 tile was the better one, by 2 to 14 %, in 3, all with
    // nothing added; in the mean it took 1.7 times as long (fp32 and bf16 outputs alike), 2 where they are added to.
    if (sh.tile == 256 && is_weight(dir) && (groups > 0 || dir >= kRowStats) && steps <= 8) continue;
    int64_t tiles = int64_t(up(I, rows)) * up(J, sh.tile);
    if (sums)
      tiles *= groups;
    else if (groups > 1)
      tiles = int64_t(std::max(busy, float(I) / float(rows) + 0.5f * busy)) * up(J, sh.tile);
    for (int32_t want : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32, 48, 64, 96, 128}) {
      if (want > most_parts) break;
      if (want > 1 && (want > steps / 2 || tiles * want > 4 * kCus * sh.fit)) break;
      const int32_t per = up(steps, want), parts = up(steps, per), on_cu = up(tiles * parts, kCus);
      const int32_t rounds = is_deep ? up(per, 4) : per;
      float t = std::max(float(up(on_cu, sh.fit)) * (kStart + float(rounds) * sh.alone),
                         kStart + float(on_cu) * (float(rounds) * sh.step + sh.ends));
      if (parts > 1) t += kJoin + float(parts) * kPart + float(parts + 2) * float(I) * float(J) * (4 / kBytesPerCycle);
      if (t >= least) continue;
      least = t;
      best.flat = flat_rows;
      best.deep = is_deep;
      best.half = k == 3;
      best.tile = sh.tile;
      best.parts = parts;
      best.part_k = int64_t(per) * step;
    }
  }
  return best;
}

// The same, remembered per thread for the sizes seen last: the model takes a
// microsecond or two, and a call asks it three times.
Cut cut_of(int dir, int64_t I, int64_t J, int64_t K, int dtype, bool direct, int32_t groups = 0, int32_t most_parts = 32) {
  struct Seen {
    int64_t key[4] = {-1, -1, -1, -1};
    Cut cut;
  };
  static thread_local Seen seen[64];
  const int64_t key[4] = {I, J, K, (int64_t(groups) * 256 + most_parts) * 32 + dir * 4 + dtype * 2 + int(direct)};
  const uint64_t h = (uint64_t(I) * 31 + uint64_t(J) * 7 + uint64_t(K)) * 8 + uint64_t(key[3]);
  Seen& s = seen[(h ^ (h >> 7)) % 64];
  if (!std::equal(key, key + 4, s.key)) {
    s.cut = cut_by_model(dir, int32_t(I), int32_t(J), int32_t(K), dtype, direct, groups, most_parts);
    std::copy(key, key + 4, s.key);
  }
  return s.cut;
}

int64_t partial_bytes(const Cut& c, int64_t I, int64_t J) {
  return c.parts > 1 ? round_up(int64_t(c.parts) * I * round_up(J, 8) * 4, 256) : 0;
}

// The bias gradient's partial rows, one per part and tile column.
int64_t bias_bytes(const Cut& c, int64_t I, int64_t J) { return round_up(c.parts * div_up(J, c.tile) * I * 4, 256); }

// Direct loads need whole, aligned chunks: the contiguous index of an
// operand (with what lies behind it) a multiple of a chunk, offsets within a
// tile below 2^32 bytes and the whole operand below 2^31 chunks.
bool whole_chunks(const void* p, int64_t ld, int64_t rows, int64_t contiguous, int dtype) {
  const int64_t V = 16 / elem_bytes(dtype);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % V == 0 && contiguous % V == 0 && ld <= (int64_t(1) << 21) &&
         rows * (ld / V) < (int64_t(1) << 31);
}

// Whether a weight gradient of so many elements passes the caches: it would
// push out what the other products read again.
bool streams(int64_t elements, int32_t grad_dtype) { return elements * elem_bytes(grad_dtype) > kInfinityCacheBytes / 3 * 2; }

// The tiles of g's groups, in as many blocks as any bounds can ask for.
template <int DT, int DIR, int TI, int TJ, int WI, int WJ, int LOAD, int STAGES = 2, int WK = 1>
int launch_group_tiles(LinearArgs& g, const char* fn, hipStream_t s) {
  const int64_t ti = div_up(g.I, TI) + (is_weight(DIR) ? 0 : g.groups - 1), tj = div_up(g.J, TJ);
  const int64_t blocks = is_weight(DIR) ? round_up(ti * tj * g.parts, 8) * g.groups : round_up(ti * tj * g.parts, 8);
  if (blocks >= (int64_t(1) << 30)) return fail(DDP_EINVAL, std::string(fn) + ": too many tiles for one launch");
  g.tiles_i = int32_t(ti);
  g.tiles_j = int32_t(tj);
  g.spread = g.I <= 2 * TI * g.groups;  // else blocks share what they read of A while they read it
  launch_blocks(blocks, [&](int64_t begin, dim3 grid) {
    g.begin = int32_t(begin);
    hipLaunchKernelGGL((k_linear<DT, DIR, TI, TJ, WI, WJ, LOAD, true, STAGES, WK>), grid, dim3(WI * WJ * WK * 64), 0, s, g);
  });
  DDP_HIP_TRY(hipGetLastError(), fn);
  return DDP_OK;
}

// The same for a cut, and how its operands are loaded.
template <int DT, int DIR>
int launch_groups(LinearArgs& g, const Cut& c, bool direct, const char* fn, hipStream_t s) {
  constexpr int V = 16 / (DT == DDP_BF16 ? 2 : 4);
  g.parts = c.parts;
  g.part_k = c.part_k;
  if constexpr (DIR == kWeightTerms) {  // operands in the library's own room: always whole chunks
    if (c.tile == 128) return launch_group_tiles<DT, DIR, 128, 128, 2, 2, kDirect>(g, fn, s);
    if constexpr (DT == DDP_BF16) {
      if (c.tile == 256) return launch_group_tiles<DT, DIR, 256, 256, 2, 4, kDirect>(g, fn, s);
    }
    return launch_group_tiles<DT, DIR, 64, 64, 2, 2, kDirect>(g, fn, s);
  } else {
    if ((a_along(DIR) ? g.K : g.I) < V || (b_along(DIR) ? g.K : g.J) < V)  // rows shorter than a chunk
      return launch_group_tiles<DT, DIR, 64, 64, 2, 2, kShort>(g, fn, s);
    if constexpr (b_along(DIR)) {
      if (c.deep)
        return direct ? launch_group_tiles<DT, DIR, kFlatRows, 32, 1, 1, kDirect, 2, 4>(g, fn, s)
                      : launch_group_tiles<DT, DIR, kFlatRows, 32, 1, 1, kAny, 2, 4>(g, fn, s);
    }
    if constexpr (!is_weight(DIR)) {
      if (c.flat)
        return direct ? launch_group_tiles<DT, DIR, kFlatRows, 128, 1, 4, kDirect, kFlatStages>(g, fn, s)
                      : launch_group_tiles<DT, DIR, kFlatRows, 128, 1, 4, kAny>(g, fn, s);
    }
    if constexpr (DT == DDP_BF16) {
      if constexpr (!one_group(DIR) && !is_weight(DIR)) {
        if (c.half) return launch_group_tiles<DT, DIR, 128, 256, 2, 4, kDirect, 3>(g, fn, s);
      }
      if (c.tile == 256) return launch_group_tiles<DT, DIR, 256, 256, 2, 4, kDirect>(g, fn, s);
    }
    if (c.tile == 128)
      return direct ? launch_group_tiles<DT, DIR, 128, 128, 2, 2, kDirect>(g, fn, s) : launch_group_tiles<DT, DIR, 128, 128, 2, 2, kAny>(g, fn, s);
    return direct ? launch_group_tiles<DT, DIR, 64, 64, 2, 2, kDirect>(g, fn, s) : launch_group_tiles<DT, DIR, 64, 64, 2, 2, kAny>(g, fn, s);
  }
}

// db (+)= the column sums of `rows` rows of `from`.
template <int SRC>
int launch_column_sums(const void* from, int64_t ld, int64_t rows, int64_t N, void* db, int32_t grad_dtype, int32_t accumulate,
                       const char* fn, hipStream_t s) {
  launch_blocks(div_up(N, 64), [&](int64_t begin, dim3 grid) {
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, from, ld, rows, N, db, accumulate, begin * 64);
    };
    grad_dtype == DDP_BF16 ? launch(k_column_sums<SRC, DDP_BF16>) : launch(k_column_sums<SRC, DDP_FP32>);
  });
  DDP_HIP_TRY(hipGetLastError(), fn);
  return DDP_OK;
}

// A matrix argument: rows x cols, leading dimension ld, NULL where allowed.
struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
  int eb;
  const char* what;
  bool written;
  bool may_be_null;
  int64_t bytes() const { return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * eb : 0; }
};

// Whether two matrices share a byte. Of one pitch (or one of them a single
// row, which has none), they may lie side by side as column blocks.
bool matrices_overlap(const Matrix& a, const Matrix& b) {
  if (!spans_overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const uint64_t pa = uint64_t(a.ld) * a.eb, pb = uint64_t(b.ld) * b.eb;
  if (a.rows > 1 && b.rows > 1 && pa != pb) return true;
  const uint64_t pitch = a.rows > 1 ? pa : pb;
  const uint64_t wa = uint64_t(a.cols) * a.eb, wb = uint64_t(b.cols) * b.eb;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t ahead = y >= x ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;  // of b's columns, before a's begin again
  return ahead < wa || ahead + wb > pitch;
}

// Every matrix lies in its allocation, and what is written overlaps nothing
// else, except that matrix `in_place` may be matrix `out` (the same place and rows).
int check_matrices(const char* fn, const Matrix* m, int n, int in_place, int out) {
  for (int k = 0; k < n; ++k) {
    const Matrix& x = m[k];
    if (x.p == nullptr && x.may_be_null) continue;
    if (x.ld < x.cols) return fail(DDP_EINVAL, std::string(fn) + ": the leading dimension of " + x.what + " is less than its columns");
    if (x.rows > 1 && x.ld > (int64_t(1) << 30))  // so that bytes() fits 63 bits
      return fail(DDP_EINVAL, std::string(fn) + ": the leading dimension of " + x.what + " is over 2^22");
    if (x.bytes() == 0) continue;
    if (x.p == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": " + x.what + " is NULL");
    if (reinterpret_cast<uintptr_t>(x.p) % uintptr_t(x.eb) != 0)
      return fail(DDP_EINVAL, std::string(fn) + ": " + x.what + " is not aligned to its element");
  }
  for (int k = 0; k < n; ++k) {
    if (!m[k].written || m[k].p == nullptr) continue;
    for (int o = 0; o < n; ++o) {
      if (o == k || m[o].p == nullptr) continue;
      if (k == out && o == in_place && m[o].p == m[k].p && m[o].ld == m[k].ld) continue;
      if (matrices_overlap(m[k], m[o]))
        return fail(DDP_EINVAL, std::string(fn) + ": " + m[k].what + " overlaps " + m[o].what);
    }
  }
  for (int k = 0; k < n; ++k) {  // asks the runtime, so last
    if (m[k].p == nullptr) continue;
    int st = check_range(m[k].p, m[k].bytes(), fn, m[k].what);
    if (st != DDP_OK) return st;
    if (m[k].rows > 1 && m[k].ld > (int64_t(1) << 22))  // offsets within a tile are 32 bits wide
      return fail(DDP_EINVAL, std::string(fn) + ": the leading dimension of " + m[k].what + " is over 2^22");
  }
  return DDP_OK;
}

int check_common(const char* fn, int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act) {
  if (!valid_dtype(dtype)) return fail(DDP_EINVAL, std::string(fn) + ": unknown dtype");
  if (act < DDP_ACT_NONE || act > DDP_ACT_SILU) return fail(DDP_EINVAL, std::string(fn) + ": unknown activation");
  const int64_t most = int64_t(1) << 31;  // sums and rows are counted in 32 bits
  if (M < 0 || N < 0 || K < 0 || M >= most || N >= most || K >= most)
    return fail(DDP_EINVAL, std::string(fn) + ": M, N and K must lie in [0, 2^31)");
  return DDP_OK;
}

int check_workspace(const char* fn, const void* p, int64_t have, int64_t need) {
  if (need == 0) return DDP_OK;
  if (p == nullptr || have < need)
    return fail(DDP_EINVAL, std::string(fn) + ": the workspace needs " + std::to_string(need) + " bytes");
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return fail(DDP_EINVAL, std::string(fn) + ": the workspace is not 16-byte aligned");
  return DDP_OK;
}

}  // namespace
}  // namespace ddp
