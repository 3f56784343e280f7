// Losses of an output layer z = x w^T over a large vocabulary, without a
// matrix of z (ddp_train.h): cross entropy with a target a row, and the
// divergence from a teacher's top logits.
//
//   forward    lse = log sum exp(z), loss from lse and z of the row's entries
//   backward   dz = dloss (exp(z - lse) - q), dx = dz w, dw (+)= dz^T x
//
// The rows that count are gathered first, by index and by value: rows that do
// not (padding, a prompt) cost nothing, and what they hold, NaN too, reaches
// nothing. The products then have one group of rows, whose length is on the
// device (linear_device.h). Forward is one product whose tiles leave a maximum
// and a sum a row. Backward makes z again, a piece of the vocabulary at a time:
// dz of the piece, then its part of dx, kept in fp32 from piece to piece, and
// its rows of dw.
//
// What bounds it: the matrix instructions of four products, six with bf16 data, whose
// dz is taken in two terms of bf16: off by 2^-16, where one term's 2^-8 left bf16 gradients
// 1.8 to 2.2 thousandths off instead of the 1.66 of their own rounding. 8192 rows (2 % of
// them not counted), 128000 columns of 4096, bf16: z and its statistics 6.3 ms
// (1340 TFLOP/s, the matrix units busy 78 %; the library's bare product 1420), then by
// pieces of 16128 columns dz 0.87 (1220), dx 1.76 (1200) and dw 1.72 (1230), both
// in two terms: 41 ms in all. Making z again costs 7 of them; kept in bf16 it would take
// 2 GiB. Few rows: the weights' bytes. Small sizes: seven launches of 4 to 8 us.
#include <climits>

#include "linear_host.h"

namespace ddp {
namespace {

constexpr int32_t kMostTop = 1024;
constexpr float kLeastTemperature = 0x1p-20f, kMostTemperature = 0x1p20f;
// Operands of direct loads have leading dimensions up to 2^21 and fewer than
// 2^31 chunks of 16 bytes, and those in the scratch are always loaded so: the
// gathered rows, and dz, whose pieces have 4096 columns where the rows are most.
constexpr int64_t kCopyRows = 2048;  // of a forward pass; backward two products read the copy
constexpr int64_t kCopyProducts = int64_t(12000000000);  // M V K
constexpr int64_t kMostRows = int64_t(1) << 20, kMostIns = int64_t(1) << 21;

// ---------------------------------------------------------------- a teacher's top logits

// One wave takes a row: the softmax of its logits / T over the entries that are
// kept, then these in ascending order, and where each column tile's start.
struct TopArgs {
  const int64_t* ids;
  const void* logits;
  int64_t ld_ids, ld_logits, vocabulary;
  int32_t top, width, tiles;  // column tiles
  float inverse;              // 1 / T
  int32_t* out_ids;
  float* out_weights;
  uint16_t* out_starts;
  float* own_terms;           // sum of q log q, NaN where an entry is not valid
  int32_t* counted;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <int DT>
__global__ __launch_bounds__(64) void k_top(TopArgs g) {
  extern __shared__ __attribute__((aligned(16))) int32_t lds[];
  const int padded = (g.top + 3) / 4 * 4;
  int32_t* const ids = lds;                                    // of the kept entries, else INT_MAX
  float* const weights = reinterpret_cast<float*>(lds + padded);
  int32_t* const sorted = lds + 2 * padded;
  const int lane = int(threadIdx.x);
  const int64_t row = blockIdx.x;
  const int64_t* const id_row = g.ids + row * g.ld_ids;
  bool bad = false, any = false;
  float most = -INFINITY;
  for (int k = lane; k < g.top; k += 64) {
    const int64_t id = id_row[k];
    const float t = Ops<DT>::load1(g.logits, row * g.ld_logits + k);
    const bool kept = id >= 0 && t != -INFINITY;
    if (kept) {
      any = true;
      bad |= id >= g.vocabulary || !(t < INFINITY);
      most = fmaxf(most, t);
    }
    ids[k] = !kept ? INT_MAX : id < g.vocabulary ? int32_t(id) : INT_MAX - 1;
    weights[k] = t;
  }
  if (lane < padded - g.top) ids[g.top + lane] = INT_MAX;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
  bad = __any(bad);
  any = __any(any);
  __syncthreads();
  float sum = 0.0f;
  for (int k = lane; k < g.top; k += 64) sum += ids[k] < INT_MAX ? expf((weights[k] - most) * g.inverse) : 0.0f;
  sum = wave_sum(sum);
  const float log_sum = logf(sum);
  float own = 0.0f;
  for (int k = lane; k < g.top; k += 64) {
    const float log_q = (weights[k] - most) * g.inverse - log_sum;
    const float q = ids[k] < INT_MAX ? expf((weights[k] - most) * g.inverse) / sum : 0.0f;
    if (q > 0.0f) own += q * log_q;
    weights[k] = q;
  }
  own = wave_sum(own);
  if (lane == 0) {
    g.own_terms[row] = bad ? NAN : own;
    g.counted[row] = any;
  }
  if (!any) return;
  __syncthreads();
  // The kept entries in ascending order of their ids, by counting for each those
  // before it, four at a time.
  int count = 0;
  for (int k0 = 0; k0 < padded; k0 += 64) {
    const int k = k0 + lane;
    const int id = k < padded ? ids[k] : INT_MAX;
    const bool kept = id < INT_MAX;
    count += int(__popcll(__ballot(kept)));
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < padded; o += 4) {
      const int4 v = *reinterpret_cast<const int4*>(ids + o);
      rank += (v.x < id || (v.x == id && o < k)) + (v.y < id || (v.y == id && o + 1 < k)) + (v.z < id || (v.z == id && o + 2 < k)) +
              (v.w < id || (v.w == id && o + 3 < k));
    }
    if (!kept) continue;
    sorted[rank] = id;
    g.out_ids[row * g.top + rank] = id;
    g.out_weights[row * g.top + rank] = weights[k];
  }
  __syncthreads();
  for (int t = lane; t <= g.tiles; t += 64) {
    const int64_t column = int64_t(t) * g.width;
    int lo = 0, hi = count;   // the first entry not below the tile's first column
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (sorted[mid] < column)
        lo = mid + 1;
      else
        hi = mid;
    }
    g.out_starts[row * (g.tiles + 1) + t] = uint16_t(lo);
  }
}

// ---------------------------------------------------------------- the rows that count

struct RowsArgs {
  const int64_t* targets;  // a row counts if its target is not negative,
  const int32_t* counted;  // or (targets NULL) where this is not 0
  const void* x;
  int64_t ldx, M, K, ld_out;
  int32_t rows;            // of a block, at most kThreads
  int64_t* bounds;         // receives 0 and the rows' number
  int32_t* row_of;
  void* out;               // [number][ld_out], zeros from K on
  float* loss;             // forward: zeros where rows do not count
  float* lse;
  void* dx;                // backward: likewise (NULL: not wanted)
  int64_t lddx;
  const float* dloss;      // backward: of every row
  float* factor;           // receives the largest magnitude of those that count (1 if that is 0 or not finite)
  __device__ __forceinline__ bool counts(int64_t i) const { return targets != nullptr ? targets[i] >= 0 : counted[i] != 0; }
};

// A block counts the rows before its own by itself, and the last one finds the largest dloss: up to some
// 10000 rows, reading a flag each costs less than a launch that would sum them. The reads grow with the square of the rows:
// of a call with little else to do (64 columns, 8 inputs), forward, 4096 rows take 18 us, 16384 24, 65536 58, 2^18 340 and
// 2^20 1440, the last of which read 17 GB of flags.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_rows(RowsArgs g) {
  __shared__ int32_t waves[2][4];
  __shared__ int32_t here[kThreads];
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  const int64_t first = int64_t(blockIdx.x) * g.rows, end = first + g.rows < g.M ? first + g.rows : g.M;
  const bool last = blockIdx.x == gridDim.x - 1;
  if (last && g.factor != nullptr) {
    __shared__ float most[4];
    float m = 0.0f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < g.M; i += kThreads) {
      const float d = fabsf(g.dloss[i]);
      if (g.counts(i)) m = fmaxf(m, d);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if (lane == 0) most[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    if (threadIdx.x == 0) *g.factor = m > 0.0f && m < INFINITY ? m : 1.0f;
  }
  int32_t before = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < first; i += kThreads) before += g.counts(i) ? 1 : 0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d);
  const int64_t row = first + threadIdx.x;
  const bool inside = row < end, mine = inside && g.counts(row);
  const uint64_t votes = __ballot(mine);
  if (lane == 0) {
    waves[0][wave] = before;
    waves[1][wave] = int32_t(__popcll(votes));
  }
  __syncthreads();
  before = waves[0][0] + waves[0][1] + waves[0][2] + waves[0][3];
  int32_t place = int32_t(__popcll(votes & ((uint64_t(1) << lane) - 1))), number = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) place += waves[1][w];
    number += waves[1][w];
  }
  if (mine) {
    here[place] = int32_t(row);
    g.row_of[before + place] = int32_t(row);
  } else if (inside) {
    if (g.loss != nullptr) g.loss[row] = g.lse[row] = 0.0f;
  }
  if (last && threadIdx.x == 0) {
    g.bounds[0] = 0;
    g.bounds[1] = before + number;
  }
  __syncthreads();
  constexpr int ES = DT == DDP_BF16 ? 2 : 4;
  for (int32_t r = wave; r < number; r += 4) {
    const int64_t from = here[r] * g.ldx;
    char* const to = static_cast<char*>(g.out) + (before + r) * g.ld_out * ES;
    for (int64_t j = lane * 8; j < g.ld_out; j += 512) {
      const Raw8 v = load_raw8<DT>(g.x, from + j, g.K - j >= 8 ? 8 : g.K > j ? int(g.K - j) : 0);
      u32x4* const p = reinterpret_cast<u32x4*>(to + j * ES);
      p[0] = v.a;
      if (DT == DDP_FP32) p[1] = v.b;
    }
  }
  if (g.dx == nullptr || number == end - first) return;
  const float zeros[8] = {};
  for (int64_t i = first + wave; i < end; i += 4) {
    if (g.counts(i)) continue;
    for (int64_t j = lane * 8; j < g.K; j += 512) store8<DT>(g.dx, i * g.lddx + j, g.K - j >= 8 ? 8 : int(g.K - j), zeros);
  }
}

// ---------------------------------------------------------------- weights whose rows are not whole chunks

// Rows of w, of 8 elements and more, in whole chunks of 16 bytes with zeros from K on:
// what direct loads need. Four chunks a lane, all under way at once: a row's last chunk
// is loaded from where it is whole, and shifted. Memory bounds it.
constexpr int kCopied = 4;

__global__ __launch_bounds__(kThreads) void k_whole_rows(const uint16_t* w, int64_t ldw, uint32_t chunks, uint32_t per_row, int32_t K,
                                                         u32x4* out) {
  const uint32_t first = blockIdx.x * uint32_t(kCopied * kThreads) + threadIdx.x;
  u32x4 v[kCopied];
  int32_t past[kCopied];  // elements of the chunk behind the row
#pragma unroll
  for (int u = 0; u < kCopied; ++u) {
    const uint32_t q = first + u * kThreads < chunks ? first + u * kThreads : chunks - 1;
    const uint32_t row = q / per_row;
    const int32_t j = int32_t(q - row * per_row) * 8;
    past[u] = j + 8 > K ? j + 8 - K : 0;
    v[u] = load_at<false, u32x4_at2>(w + (int64_t(row) * ldw + j - past[u]), 0);
  }
#pragma unroll
  for (int u = 0; u < kCopied; ++u) {
    uint64_t lo = v[u].x | uint64_t(v[u].y) << 32, hi = v[u].z | uint64_t(v[u].w) << 32;
    const int bits = 16 * past[u];
    if (bits >= 64) {
      lo = hi >> (bits - 64);
      hi = 0;
    } else if (bits > 0) {
      lo = lo >> bits | hi << (64 - bits);
      hi >>= bits;
    }
    if (first + u * kThreads < chunks) out[first + u * kThreads] = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
  }
}

// ---------------------------------------------------------------- the rows' losses

struct JoinArgs {
  const int64_t* bounds;
  const int32_t* row_of;
  int64_t M;
  int32_t column_tiles;
  HeadArgs head;
  float factor;   // of the loss
  float* loss;
  float* lse;
};

constexpr int kJoinRows = 8, kJoinSlices = kThreads / kJoinRows;

// 8 rows a block, 32 threads a row: each a share of the column tiles, then of
// the row's entries, joined in a fixed order.
__global__ __launch_bounds__(kThreads) void k_loss_join(JoinArgs g) {
  __shared__ float part[kJoinSlices][kJoinRows + 1];
  const HeadArgs& h = g.head;
  const int in = int(threadIdx.x) % kJoinRows, slice = int(threadIdx.x) / kJoinRows;
  const bool in_place = g.row_of == nullptr;  // all rows are here, also those that do not count
  const int64_t number = in_place ? g.M : g.bounds[1], i = int64_t(blockIdx.x) * kJoinRows + in;
  if (int64_t(blockIdx.x) * kJoinRows >= number) return;
  const int64_t row = i >= number ? 0 : in_place ? i : g.row_of[i];
  const bool counts = i < number && (!in_place || (h.targets != nullptr ? h.targets[row] >= 0 : h.counted[row] != 0));
  const auto joined = [&](float mine, auto&& join) {
    part[slice][in] = mine;
    __syncthreads();
#pragma unroll
    for (int n = kJoinSlices / 2; n > 0; n /= 2) {
      if (slice < n) part[slice][in] = join(part[slice][in], part[slice + n][in]);
      __syncthreads();
    }
    const float v = part[0][in];
    __syncthreads();
    return v;
  };
  const auto add = [](float a, float b) { return a + b; };
  float mine = -INFINITY, sum = 0.0f;
  if (counts) {
    for (int t = slice; t < g.column_tiles; t += 4 * kJoinSlices) {
      float m[4], s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // past the last tile: the last again, unused
        const int at = t + u * kJoinSlices < g.column_tiles ? t + u * kJoinSlices : g.column_tiles - 1;
        m[u] = h.stats[int64_t(at) * 2 * g.M + i];
        s[u] = h.stats[(int64_t(at) * 2 + 1) * g.M + i];
        if (t + u * kJoinSlices >= g.column_tiles) m[u] = -INFINITY, s[u] = 0.0f;
      }
      const float most = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), mine);
      const float base = most == -INFINITY ? 0.0f : most;
      sum *= expf((mine == -INFINITY ? base : mine) - base);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += s[u] * expf((m[u] == -INFINITY ? base : m[u]) - base);
      mine = most;
    }
  }
  const float most = joined(mine, [](float a, float b) { return fmaxf(a, b); });
  const float base = most == -INFINITY ? 0.0f : most;
  sum *= expf((mine == -INFINITY ? base : mine) - base);
  const float lse = base + logf(joined(sum, add));
  float loss = 0.0f;
  if (h.targets != nullptr) {
    if (counts) loss = h.targets[row] < h.vocabulary ? lse - h.picked[row] : NAN;
  } else {
    if (counts) {
      const int entries = h.starts[row * (h.tiles + 1) + h.tiles];
      for (int k = slice; k < entries; k += kJoinSlices) {
        const float q = h.weights[row * h.top + k];
        if (q > 0.0f) loss += q * (lse - h.picked[row * h.top + k]);
      }
    }
    loss = joined(loss, add);
    if (counts) loss = g.factor * (loss + h.own_terms[row]);
  }
  if (i >= number || slice != 0) return;
  g.loss[row] = loss;
  g.lse[row] = counts ? lse : 0.0f;
}

// ---------------------------------------------------------------- host side

// What a call works on: sizes, types and the rows' targets or entries.
struct Head {
  int64_t M, V, K;
  int32_t top;           // 0: targets
  int32_t dtype, grad_dtype;
  bool backward;
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const int64_t* targets;
  const int64_t* ids;
  int64_t ld_ids;
  const void* teacher;
  int64_t ld_teacher;
  int32_t teacher_dtype;
  float temperature;

  int64_t ldg() const { return round_up(K, 8); }   // of the gathered rows
  // bf16 data: dz in two terms, as one would be as coarse as the gradients' own rounding.
  int32_t terms() const { return dtype == DDP_BF16 ? 2 : 1; }
  bool w_whole() const { return whole_chunks(w, ldw, V, K, dtype); }
  // Whether the weights are copied to whole chunks, a piece at a time: those of a width that has none, where
  // rows are many enough that the copy costs less than what loads at any alignment and smaller tiles do.
  // Forward, without and with it: 32003 columns of 2047, 1030 rows 206 us and 215, 2050 370 and 327, 4100 701
  // and 558; 5003 of 501, 2050 37 and 41, 4100 60 and 64, 8000 95 and 86; 1003 of 1001, 2050 31 and 36, 8000 50 and 49; 12003 of
  // 135, 4100 70 and 64: so by the rows and the product's length. Backward: 32003 of 2047, 520 rows 569
  // and 517, 1030 959 and 796, 4100 3340 and 2786; 5003 of 501, 1030 103 and 96, 4100 227 and 200; 1003 of 135,
  // 1030 49 and 50, 2050 54 and 58, 8000 86 and 81: by the rows, as what small vocabularies lose is a few us.
  // (Rows mean all of them: how many count is on the device. 1037 rows, of which half count, 32003 of
  // 1001, backward: 206 and 200. Rows of a whole width that begin at odd places are not copied.)
  bool copies() const {
    if (dtype != DDP_BF16 || K % 8 == 0 || K < 128) return false;
    if (backward) return M >= kCopyRows / 2;
    return M >= kCopyRows && (M * V >= int64_t(25000000) || M * V >= kCopyProducts / K);
  }
};

// Columns of a piece, and pieces. A piece of dz, 4 bytes a value, should lie in the
// Infinity Cache for the two products that read it, but be long enough that dx's
// sum over it is worth the pass over dx in fp32 that each piece costs: 128 MiB, or 4096
// columns. (Backward, bf16, in pieces of 128, 256 and 512 MiB: 8192 rows, 128000 columns of
// 4096, 35.0, 35.7 and 35.8 ms; 4096 x 64000 x 2048 4.59, 4.72 and 4.73. 32768 x 32000 x 1024, in
// pieces of 4096 columns and 1024, 10.4 and 12.5.) With an fp32 dw of bf16 data 512 MiB,
// which takes 3 % longer (36.0 ms and 34.9; 4.77 and 4.62): the width that test_tilings holds. Never more than 512 MiB, or
// 1024 columns: beyond 32768 rows, room counts more than time (65536 x 16000 x 1024, 2048 columns and 4096:
// 11.3 and 10.3 ms; 131072 x 8000 x 512, 1024 and 4096: 7.4 and 6.3). A copy of the weights has
// 128 MiB, or 4096 rows.
struct Pieces {
  int64_t columns, number;
};
Pieces pieces_of(const Head& h) {
  int64_t most = h.V;
  if (h.backward) {
    const int64_t M = std::max<int64_t>(h.M, 1);
    most = std::min<int64_t>(1 << 20, std::max<int64_t>(1024, (int64_t(1) << 27) / M));
    if (h.dtype != DDP_BF16 || h.grad_dtype != DDP_FP32) most = std::min(most, std::max<int64_t>(4096, (int64_t(1) << 25) / M));
  }
  if (h.copies()) most = std::min(most, std::max<int64_t>(4096, (int64_t(1) << 26) / h.ldg()));
  const int64_t columns = round_up(div_up(h.V, div_up(h.V, most)), 256);
  return {columns, div_up(h.V, columns)};
}

// How the products that make z are cut, with or without direct loads.
Cut z_cut(const Head& h, bool direct) {
  return cut_of(kRowStats, h.M, std::min(pieces_of(h).columns, h.V), h.K, h.dtype, direct || h.copies(), 0, 1);
}

// Where a call's scratch lies; with base NULL, only its size.
struct Scratch {
  int64_t* bounds;   // of the one group, then the gradients' factor
  int32_t* row_of;
  char* rows;
  int32_t* counted;
  float* own_terms;
  int32_t* ids;
  float* weights;
  uint16_t* starts;
  char* whole;       // the weights' copy
  float* stats;
  float* picked;
  char* dz;
  int64_t lddz;
  float* sums;
  float* partial;
  int64_t bytes;
};
Scratch scratch_of(const Head& h, void* base) {
  Scratch s{};
  int64_t at = 0;
  const auto take = [&](auto*& p, int64_t bytes) {
    p = base == nullptr ? nullptr : reinterpret_cast<std::remove_reference_t<decltype(p)>>(static_cast<char*>(base) + at);
    at += round_up(bytes, 256);
  };
  const int64_t eb = elem_bytes(h.dtype), tiles = div_up(h.V, std::min(z_cut(h, false).tile, z_cut(h, true).tile));
  take(s.bounds, 24);
  take(s.row_of, h.M * 4);
  take(s.rows, h.M * h.ldg() * eb);
  if (h.top > 0) {
    take(s.counted, h.M * 4);
    take(s.own_terms, h.M * 4);
    take(s.ids, h.M * h.top * 4);
    take(s.weights, h.M * h.top * 4);
    take(s.starts, h.M * (tiles + 1) * 2);
  }
  if (h.copies()) take(s.whole, pieces_of(h).columns * h.ldg() * eb);
  if (!h.backward) {
    take(s.stats, tiles * 2 * h.M * 4);
    take(s.picked, h.M * std::max(h.top, 1) * 4);
  } else {
    const Pieces p = pieces_of(h);
    s.lddz = std::min(p.columns, round_up(h.V, 8));
    take(s.dz, h.terms() * h.M * s.lddz * eb);
    if (p.number > 1) take(s.sums, h.M * h.K * 4);
    int64_t most = 0;
    for (int64_t v0 = 0; v0 < h.V; v0 += p.columns) {
      const int64_t n = std::min(p.columns, h.V - v0);
      for (bool direct : {false, true})
        most = std::max(most, partial_bytes(cut_of(kInputPiece, h.M, h.K, n, h.dtype, direct, 0, 128), h.M, h.K));
      most = std::max(most, partial_bytes(cut_of(kWeightTerms, n, h.K, h.M * h.terms(), h.dtype, true), n, h.K));
    }
    take(s.partial, most);
  }
  s.bytes = at;
  return s;
}

int check_head(const char* fn, const Head& h) {
  int st = check_common(fn, h.M, h.V, h.K, h.dtype, DDP_ACT_NONE);
  if (st != DDP_OK) return st;
  if (h.V < 1 || h.K < 1) return fail(DDP_EINVAL, std::string(fn) + ": V and K must be at least 1");
  if (h.M > kMostRows || h.K > kMostIns || h.M * h.K > kMostRows * 4096)
    return fail(DDP_EINVAL, std::string(fn) + ": M may be 2^20 at most, K 2^21, M * K 2^32");
  if (h.M > 0 && h.V >= (int64_t(1) << 42) / h.M) return fail(DDP_EINVAL, std::string(fn) + ": M * V must be below 2^42");
  if (h.grad_dtype != h.dtype && h.grad_dtype != DDP_FP32)
    return fail(DDP_EINVAL, std::string(fn) + ": grad_dtype must be the data's or fp32");
  return DDP_OK;
}
int check_top(const char* fn, const Head& h) {
  if (h.top < 1 || h.top > kMostTop) return fail(DDP_EINVAL, std::string(fn) + ": C must lie in [1, 1024]");
  return DDP_OK;
}

// The rows that count (not gathered where they are in_place), and a teacher's
// entries; g: the products' arguments that all have in common.
template <int DT>
int launch_rows_that_count(const Head& h, const Scratch& w, int width, bool in_place, RowsArgs r, LinearArgs& g, const char* fn,
                           hipStream_t s) {
  const int32_t tiles = int32_t(div_up(h.V, width));
  if (h.top > 0 && h.M > 0) {
    TopArgs t{h.ids, h.teacher, h.ld_ids, h.ld_teacher, h.V, h.top, width, tiles, 1.0f / h.temperature,
              w.ids, w.weights, w.starts, w.own_terms, w.counted};
    const size_t lds = size_t(round_up(h.top, 4)) * 12;
    if (h.teacher_dtype == DDP_BF16)
      hipLaunchKernelGGL((k_top<DDP_BF16>), dim3(unsigned(h.M)), dim3(64), lds, s, t);
    else
      hipLaunchKernelGGL((k_top<DDP_FP32>), dim3(unsigned(h.M)), dim3(64), lds, s, t);
    DDP_HIP_TRY(hipGetLastError(), fn);
  }
  if (!in_place) {
    r.targets = h.targets, r.counted = w.counted;
    r.x = h.x, r.ldx = h.ldx, r.M = h.M, r.K = h.K, r.ld_out = h.ldg();
    r.rows = int32_t(std::min<int64_t>(kThreads, std::max<int64_t>(8, div_up(h.M, 1024))));
    r.bounds = w.bounds, r.row_of = w.row_of, r.out = w.rows;
    hipLaunchKernelGGL((k_rows<DT>), dim3(unsigned(std::max<int64_t>(1, div_up(h.M, r.rows)))), dim3(kThreads), 0, s, r);
    DDP_HIP_TRY(hipGetLastError(), fn);
    g.a = w.rows, g.lda = h.ldg(), g.a_room = int32_t(h.ldg() - h.K);
    g.bounds = w.bounds, g.row_of = w.row_of;
  } else {
    g.a = h.x, g.lda = h.ldx;
  }
  g.ldb = h.ldw;
  g.I = h.M, g.K = h.K;
  g.groups = 1, g.rows = h.M;
  HeadArgs& a = g.head;
  a.scale = 1.0f / h.temperature;
  a.slope = h.temperature;
  a.vocabulary = h.V;
  a.targets = h.targets;
  a.top = std::max(h.top, 1), a.tiles = tiles;
  a.ids = w.ids, a.weights = w.weights, a.starts = w.starts, a.own_terms = w.own_terms, a.counted = w.counted;
  return DDP_OK;
}

// Columns v0 .. v0 + n of the vocabulary as an operand of g, copied to whole chunks or in place.
template <int DT>
int launch_weights(const Head& h, const Scratch& w, int64_t v0, int64_t n, LinearArgs& g, const char* fn, hipStream_t s) {
  g.b = static_cast<const char*>(h.w) + v0 * h.ldw * elem_bytes(DT);
  if (!h.copies()) return DDP_OK;
  const int64_t per_row = h.ldg() / 8, chunks = n * per_row;
  hipLaunchKernelGGL(k_whole_rows, dim3(unsigned(div_up(chunks, kCopied * kThreads))), dim3(kThreads), 0, s,
                     static_cast<const uint16_t*>(g.b), h.ldw, uint32_t(chunks), uint32_t(per_row), int32_t(h.K), reinterpret_cast<u32x4*>(w.whole));
  DDP_HIP_TRY(hipGetLastError(), fn);
  g.b = w.whole, g.ldb = h.ldg(), g.b_room = int32_t(h.ldg() - h.K);
  return DDP_OK;
}

template <int DT>
int loss_forward(const Head& h, float* loss, float* lse, void* workspace, const char* fn, hipStream_t s) {
  const Scratch w = scratch_of(h, workspace);
  // Few rows are a tile or two whether they count or not, and a launch less counts.
  const bool in_place = h.M <= 64;
  const bool direct = h.copies() || (h.w_whole() && (!in_place || whole_chunks(h.x, h.ldx, h.M, h.K, DT)));
  const Pieces p = pieces_of(h);
  const Cut c = z_cut(h, direct);
  LinearArgs all{};
  RowsArgs r{};
  r.loss = loss, r.lse = lse;
  int st = launch_rows_that_count<DT>(h, w, c.tile, in_place, r, all, fn, s);
  if (st != DDP_OK) return st;
  all.head.stats = w.stats, all.head.picked = w.picked;
  for (int64_t v0 = 0; v0 < h.V; v0 += p.columns) {
    LinearArgs g = all;
    g.J = std::min(p.columns, h.V - v0);
    st = launch_weights<DT>(h, w, v0, g.J, g, fn, s);
    if (st != DDP_OK) return st;
    g.head.j_base = v0;
    g.head.stats += v0 / c.tile * 2 * h.M;
    st = launch_groups<DT, kRowStats>(g, c, direct, fn, s);
    if (st != DDP_OK) return st;
  }
  const int32_t tiles = int32_t(div_up(h.V, c.tile));
  const JoinArgs j{all.bounds, all.row_of, h.M, tiles, all.head, h.temperature * h.temperature, loss, lse};
  hipLaunchKernelGGL(k_loss_join, dim3(unsigned(div_up(h.M, kJoinRows))), dim3(kThreads), 0, s, j);
  DDP_HIP_TRY(hipGetLastError(), fn);
  return DDP_OK;
}

// The product of g cut like c, its parts joined.
template <int DT, int DIR>
int launch_joined(LinearArgs& g, const Cut& c, bool direct, const char* fn, hipStream_t s) {
  int st = launch_groups<DT, DIR>(g, c, direct, fn, s);
  if (st != DDP_OK || g.parts == 1) return st;
  hipLaunchKernelGGL((k_linear_join<DT, DIR, !is_weight(DIR)>), dim3(unsigned(div_up(g.I * div_up(g.J, 8), kThreads))), dim3(kThreads),
                     0, s, g);
  DDP_HIP_TRY(hipGetLastError(), fn);
  return DDP_OK;
}

template <int DT>
int loss_backward(const Head& h, const float* lse, const float* dloss, void* dx, int64_t lddx, void* dw, int64_t lddw,
                  int32_t accumulate, void* workspace, const char* fn, hipStream_t s) {
  const Scratch w = scratch_of(h, workspace);
  const Pieces p = pieces_of(h);
  const bool w_whole = h.copies() || h.w_whole();
  const Cut c = z_cut(h, w_whole);
  constexpr int64_t ES = DT == DDP_BF16 ? 2 : 4;
  LinearArgs all{};
  RowsArgs r{};
  r.dx = dx, r.lddx = lddx;
  r.dloss = dloss, r.factor = reinterpret_cast<float*>(w.bounds + 2);
  int st = launch_rows_that_count<DT>(h, w, c.tile, false, r, all, fn, s);
  if (st != DDP_OK) return st;
  all.head.lse = lse, all.head.dloss = dloss;
  all.factor = r.factor;
  all.terms = h.terms();
  if (h.M == 0) dx = nullptr;
  for (int64_t v0 = 0; v0 < h.V; v0 += p.columns) {
    const int64_t n = std::min(p.columns, h.V - v0);
    LinearArgs piece = all;
    st = launch_weights<DT>(h, w, v0, n, piece, fn, s);
    if (st != DDP_OK) return st;
    // dz of the piece
    LinearArgs g = piece;
    g.J = n;
    g.c = w.dz, g.ldc = w.lddz, g.term = h.M * w.lddz;
    g.head.j_base = v0;
    st = launch_groups<DT, kRowSlopes>(g, c, w_whole, fn, s);
    if (st != DDP_OK) return st;
    const int32_t room = int32_t(round_up(n, 8) - n);
    if (dx != nullptr) {
      g = piece;
      g.a = w.dz, g.lda = w.lddz, g.a_room = room, g.term = h.M * w.lddz * ES;
      g.J = h.K, g.K = n;
      g.c = dx, g.ldc = lddx;
      g.sums = w.sums, g.first = v0 == 0, g.last = v0 + n == h.V;
      g.partial = w.partial;
      st = launch_joined<DT, kInputPiece>(g, cut_of(kInputPiece, h.M, h.K, n, DT, w_whole, 0, 128), w_whole, fn, s);
      if (st != DDP_OK) return st;
    }
    if (dw != nullptr) {
      g = all;
      g.a = w.dz, g.lda = w.lddz, g.a_room = room, g.term = h.M * w.lddz * ES;
      g.b = w.rows, g.ldb = h.ldg(), g.b_room = int32_t(h.ldg() - h.K);
      g.I = n, g.J = h.K, g.K = h.M;
      g.c = static_cast<char*>(dw) + v0 * lddw * elem_bytes(h.grad_dtype), g.ldc = lddw;
      g.grad32 = h.grad_dtype == DDP_FP32, g.accumulate = accumulate;
      g.stream_c = streams(h.V * h.K, h.grad_dtype);
      g.partial = w.partial;
      st = launch_joined<DT, kWeightTerms>(g, cut_of(kWeightTerms, n, h.K, h.M * all.terms, DT, true), true, fn, s);
      if (st != DDP_OK) return st;
    }
  }
  return DDP_OK;
}

// The matrices that every call reads, and its scratch.
struct Checked {
  Matrix m[12];
  int n = 0;
  void add(const Matrix& x) { m[n++] = x; }
};
Checked common_matrices(const Head& h) {
  Checked c;
  const int eb = elem_bytes(h.dtype);
  c.add({h.x, h.M, h.K, h.ldx, eb, "x", false, false});
  c.add({h.w, h.V, h.K, h.ldw, eb, "w", false, false});
  if (h.top > 0) {
    c.add({h.ids, h.M, h.top, h.ld_ids, 8, "ids", false, false});
    c.add({h.teacher, h.M, h.top, h.ld_teacher, elem_bytes(h.teacher_dtype), "teacher", false, false});
  } else {
    c.add({h.targets, 1, h.M, h.M, 8, "targets", false, false});
  }
  return c;
}

int forward_call(const char* fn, const Head& h, float* loss, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  if (h.M == 0) return DDP_OK;
  const int64_t need = scratch_of(h, nullptr).bytes;
  int st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  Checked c = common_matrices(h);
  c.add({loss, 1, h.M, h.M, 4, "loss", true, false});
  c.add({lse, 1, h.M, h.M, 4, "lse", true, false});
  c.add({workspace, 1, need, need, 1, "workspace", true, false});
  st = check_matrices(fn, c.m, c.n, -1, -1);
  if (st != DDP_OK) return st;
  return h.dtype == DDP_BF16 ? loss_forward<DDP_BF16>(h, loss, lse, workspace, fn, as_stream(stream))
                             : loss_forward<DDP_FP32>(h, loss, lse, workspace, fn, as_stream(stream));
}

int backward_call(const char* fn, const Head& h, const float* lse, const float* dloss, void* dx, int64_t lddx, void* dw, int64_t lddw,
                  int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  if (accumulate != 0 && accumulate != 1) return fail(DDP_EINVAL, std::string(fn) + ": accumulate must be 0 or 1");
  if (dx == nullptr && dw == nullptr) return DDP_OK;
  const int64_t need = scratch_of(h, nullptr).bytes;
  int st = check_workspace(fn, workspace, workspace_bytes, need);
  if (st != DDP_OK) return st;
  Checked c = common_matrices(h);
  c.add({lse, 1, h.M, h.M, 4, "lse", false, false});
  c.add({dloss, 1, h.M, h.M, 4, "dloss", false, false});
  c.add({dx, h.M, h.K, lddx, elem_bytes(h.dtype), "dx", true, true});
  c.add({dw, h.V, h.K, lddw, elem_bytes(h.grad_dtype), "dw", true, true});
  c.add({workspace, 1, need, need, 1, "workspace", true, false});
  st = check_matrices(fn, c.m, c.n, -1, -1);
  if (st != DDP_OK) return st;
  return h.dtype == DDP_BF16 ? loss_backward<DDP_BF16>(h, lse, dloss, dx, lddx, dw, lddw, accumulate, workspace, fn, as_stream(stream))
                             : loss_backward<DDP_FP32>(h, lse, dloss, dx, lddx, dw, lddw, accumulate, workspace, fn, as_stream(stream));
}

Head head_of(int64_t M, int64_t V, int64_t K, int32_t C, int32_t dtype, int32_t grad_dtype, bool backward) {
  Head h{};
  h.M = M, h.V = V, h.K = K, h.top = C;
  h.dtype = dtype, h.grad_dtype = grad_dtype;
  h.backward = backward;
  h.temperature = 1.0f;
  return h;
}

int workspace_call(const char* fn, int32_t direction, const Head& h, int64_t* bytes) {
  if (bytes == nullptr) return fail(DDP_EINVAL, std::string(fn) + ": bytes is NULL");
  *bytes = 0;
  if (direction != DDP_LOSS_FORWARD && direction != DDP_LOSS_BACKWARD) return fail(DDP_EINVAL, std::string(fn) + ": unknown direction");
  int st = check_head(fn, h);
  if (st != DDP_OK) return st;
  *bytes = scratch_of(h, nullptr).bytes;
  return DDP_OK;
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" int ddp_cross_entropy_workspace(int32_t direction, int64_t M, int64_t V, int64_t K, int32_t dtype, int32_t grad_dtype,
                                           int64_t* bytes) {
  return workspace_call("ddp_cross_entropy_workspace", direction,
                        head_of(M, V, K, 0, dtype, grad_dtype, direction == DDP_LOSS_BACKWARD), bytes);
}

extern "C" int ddp_loss_tiling(int32_t product, int64_t M, int64_t V, int64_t K, int32_t dtype, int32_t grad_dtype, int32_t direct,
                               int32_t* rows, int32_t* columns, int32_t* parts, int64_t* piece) {
  const char* fn = "ddp_loss_tiling";
  if (rows == nullptr || columns == nullptr || parts == nullptr || piece == nullptr)
    return fail(DDP_EINVAL, std::string(fn) + ": an output is NULL");
  *rows = *columns = *parts = 0;
  *piece = 0;
  if (product < 0 || product > 3) return fail(DDP_EINVAL, std::string(fn) + ": unknown product");
  if (direct != 0 && direct != 1) return fail(DDP_EINVAL, std::string(fn) + ": direct must be 0 or 1");
  const Head h = head_of(M, V, K, 0, dtype, grad_dtype, product > 0);
  int st = check_head(fn, h);
  if (st != DDP_OK) return st;
  const int64_t n = std::min(pieces_of(h).columns, V);
  const bool whole = direct != 0 || h.copies();
  const Cut c = product < 2    ? z_cut(h, whole)
                : product == 2 ? cut_of(kInputPiece, M, K, n, dtype, whole, 0, 128)
                               : cut_of(kWeightTerms, n, K, M * h.terms(), dtype, true);
  *rows = c.rows();
  *columns = c.tile;
  *parts = c.parts;
  *piece = n;
  return DDP_OK;
}

extern "C" int ddp_cross_entropy_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* targets, float* loss,
                                         float* lse, int64_t M, int64_t V, int64_t K, int32_t dtype, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_cross_entropy_forward";
  Head h = head_of(M, V, K, 0, dtype, dtype, false);
  h.x = x, h.ldx = ldx, h.w = w, h.ldw = ldw, h.targets = targets;
  int st = check_head(fn, h);
  if (st != DDP_OK) return st;
  return forward_call(fn, h, loss, lse, workspace, workspace_bytes, stream);
}

extern "C" int ddp_cross_entropy_backward(const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* targets,
                                          const float* lse, const float* dloss, void* dx, int64_t lddx, void* dw, int64_t lddw,
                                          int64_t M, int64_t V, int64_t K, int32_t dtype, int32_t grad_dtype, int32_t accumulate,
                                          void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_cross_entropy_backward";
  Head h = head_of(M, V, K, 0, dtype, grad_dtype, true);
  h.x = x, h.ldx = ldx, h.w = w, h.ldw = ldw, h.targets = targets;
  int st = check_head(fn, h);
  if (st != DDP_OK) return st;
  return backward_call(fn, h, lse, dloss, dx, lddx, dw, lddw, accumulate, workspace, workspace_bytes, stream);
}

extern "C" int ddp_distill_workspace(int32_t direction, int64_t M, int64_t V, int64_t K, int32_t C, int32_t dtype,
                                     int32_t grad_dtype, int64_t* bytes) {
  const char* fn = "ddp_distill_workspace";
  const Head h = head_of(M, V, K, C, dtype, grad_dtype, direction == DDP_LOSS_BACKWARD);
  if (bytes != nullptr) *bytes = 0;
  int st = check_top(fn, h);
  if (st != DDP_OK) return st;
  return workspace_call(fn, direction, h, bytes);
}

namespace ddp {
namespace {
int distill_head(const char* fn, Head& h, const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* ids, int64_t ld_ids,
                 const void* teacher, int64_t ld_teacher, int32_t teacher_dtype, float temperature) {
  h.x = x, h.ldx = ldx, h.w = w, h.ldw = ldw;
  h.ids = ids, h.ld_ids = ld_ids, h.teacher = teacher, h.ld_teacher = ld_teacher, h.teacher_dtype = teacher_dtype;
  h.temperature = temperature;
  int st = check_top(fn, h);
  if (st == DDP_OK) st = check_head(fn, h);
  if (st != DDP_OK) return st;
  if (!valid_dtype(teacher_dtype)) return fail(DDP_EINVAL, std::string(fn) + ": unknown teacher_dtype");
  // T^2 and logits / T have to keep clear of fp32's ends: the exponent of a power of z / T is off by 2^-24 of it,
  // which beyond 2^31 is a factor that overflows.
  if (!(temperature >= kLeastTemperature) || !(temperature <= kMostTemperature))
    return fail(DDP_EINVAL, std::string(fn) + ": temperature must lie in [2^-20, 2^20]");
  return DDP_OK;
}
}  // namespace
}  // namespace ddp

extern "C" int ddp_distill_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* ids, int64_t ld_ids,
                                   const void* teacher, int64_t ld_teacher, int32_t teacher_dtype, float temperature, float* loss,
                                   float* lse, int64_t M, int64_t V, int64_t K, int32_t C, int32_t dtype, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_distill_forward";
  Head h = head_of(M, V, K, C, dtype, dtype, false);
  int st = distill_head(fn, h, x, ldx, w, ldw, ids, ld_ids, teacher, ld_teacher, teacher_dtype, temperature);
  if (st != DDP_OK) return st;
  return forward_call(fn, h, loss, lse, workspace, workspace_bytes, stream);
}

extern "C" int ddp_distill_backward(const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* ids, int64_t ld_ids,
                                    const void* teacher, int64_t ld_teacher, int32_t teacher_dtype, float temperature,
                                    const float* lse, const float* dloss, void* dx, int64_t lddx, void* dw, int64_t lddw, int64_t M,
                                    int64_t V, int64_t K, int32_t C, int32_t dtype, int32_t grad_dtype, int32_t accumulate,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "ddp_distill_backward";
  Head h = head_of(M, V, K, C, dtype, grad_dtype, true);
  int st = distill_head(fn, h, x, ldx, w, ldw, ids, ld_ids, teacher, ld_teacher, teacher_dtype, temperature);
  if (st != DDP_OK) return st;
  return backward_call(fn, h, lse, dloss, dx, lddx, dw, lddw, accumulate, workspace, workspace_bytes, stream);
}
