// A linear layer's products on the matrix instructions, each with what
// follows it in the same pass (ddp_train.h):
//
//   forward          z = x w^T + bias,  y = act(z) + residual
//   input gradient   dx = (dz w) * act'(z) + add
//   weight gradient  dw (+)= dz^T x,  db (+)= sum of dz's rows
//
// and, of the other operators that are products,

//   row statistics   of z = x w^T: each row's maximum and sum of exponentials (the losses of an output layer)
//   row slopes       the loss's gradient with respect to z, from z made again
//   input pieces     dx += (dz1 + dz2) w over a piece of dz's columns, kept in fp32 between pieces
//   weight terms     dw (+)= (dz1 + dz2)^T x
//
// (dz in two terms of 16 bits, or in fp32 one)
//
// each of the rows of one group or of several (experts) whose bounds are on the device.
//
// All are C[i][j] = sum_k A(i, k) B(j, k). What differs is how an
// operand lies in memory: with the sum's index k contiguous ("along": x and w
// in the forward product), or with k going from row to row ("across": w in
// the input gradient, both operands of the weight gradient).
//
// A block computes a tile of C in steps of 128 bytes of k. Both operands' parts
// of a step lie in LDS as they lie in memory, in 16-byte chunks, the next
// step's on their way while this one's are multiplied. A lane of a 32 x 32
// matrix instruction needs one row's k values 8h .. 8h+7 (h: its half of the
// wave): 16 bytes of an "along" row, or, of an "across" operand, eight rows'
// values of one column, which the transposing LDS read gathers (bf16), or four
// single reads (fp32).
//
// What bounds it: a 256 x 256 tile's step of bf16 is 2048 cycles of the matrix
// instructions and, at 128 bytes a cycle, 2031 of LDS (196 KB read by 8 waves,
// 64 KB written), so the two have to overlap throughout, and a wave's other
// instructions have to fit between its products. Measured, 8192 rows, 8192
// inputs and 2048 outputs on random data: forward 202 us (1360 TFLOP/s), weight
// gradient 208 (216 added to fp32 gradients, 221 with the bias's); input gradient of
// the layer with inputs and outputs exchanged 202; a 256 x 256 tile's outputs take
// 7 to 15 us more, in which its CU multiplies nothing. Power takes part of it: on
// zeros the same products run a fifth faster. fp32: 148 TFLOP/s at 4096 x 4096 x
// 4096 in all directions, the instructions' rate.
#pragma once

#include <type_traits>

#include "train_internal.h"

namespace ddp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define DDP_LDS __attribute__((address_space(3)))

// What the losses of an output layer need besides the product. Rows are those
// of the caller; the product has only those that count.
struct HeadArgs {
  float scale;             // z = scale * x w^T
  float slope;             // row slopes: dz = slope * dloss * (p - q)
  int64_t vocabulary;
  int64_t j_base;          // the piece's first column, a multiple of the tile
  const int64_t* targets;  // a row's target; or NULL, and its entries:
  int32_t top;             // as many a row at most (1 with targets)
  int32_t tiles;           // column tiles of the vocabulary
  const int32_t* ids;      // [row][top], ascending
  const float* weights;    // [row][top]
  const uint16_t* starts;  // [row][tiles + 1], the first entry of a column tile or a later one
  const float* own_terms;  // [row], NaN where an entry is not valid
  const int32_t* counted;  // [row], 0 where a row has no entry
  float* stats;            // row statistics: [column tile][2][compact row]: maximum, sum of exp(z - maximum)
  float* picked;           // row statistics: [row][top], z of the entries
  const float* lse;        // row slopes: [row]
  const float* dloss;      // row slopes: [row]; dz is relative to the largest of them, `factor`
};

struct LinearArgs {
  const void* a;    // operand of the rows of C
  const void* b;    // operand of the columns of C
  int64_t lda, ldb; // elements
  int64_t I, J, K;  // C is I x J, the sum has K terms
  void* c;          // y, dx or dw
  int64_t ldc;
  void* z;          // forward: kept z (NULL: not); input gradient: z (NULL: no activation)
  int64_t ldz;
  const void* e;    // forward: residual; input gradient: add (NULL: none)
  int64_t lde;
  const void* bias; // forward (NULL: none)
  int32_t act;
  int32_t grad32;      // weight gradient: dw is fp32
  int32_t accumulate;  // weight gradient: add to dw
  int32_t stream_z;    // forward: z's stores pass the caches
  int32_t parts;       // blocks that share a tile's sum
  int64_t part_k;      // terms of one part (whole steps)
  float* partial;      // parts > 1: [part][I][round_up(J, 8)]
  float* row_sums;     // weight gradient: [part * tiles_j + tile_j][I], sums of A's rows (NULL: not wanted)
  int32_t tiles_i, tiles_j;
  int32_t begin;    // the launch's first block

  // Groups: group e has the rows bounds[e] .. bounds[e + 1] of x and dz, and
  // its own w, bias, dw and db, one after the other's.
  const int64_t* bounds;  // groups + 1, on the device
  int32_t groups;
  int64_t rows;           // of x and dz: no bound counts beyond them
  int64_t b_group;        // elements from one group's w to the next one's
  int32_t spread;         // begin the sums at different steps,
  int32_t spread_from;    // from the group's on

  // Operands with room behind their rows, which holds zeros.
  int32_t a_room, b_room;  // elements of it that belong to the last chunk
  int32_t stream_c;        // weight gradients: C passes the caches
  int32_t terms;           // input pieces, weight terms, row slopes: of dz, 1 or 2
  int64_t term;            // bytes from A's first term to its second, or elements of C (row slopes)
  float* sums;             // input pieces: the sum over pieces, fp32 (NULL: one piece)
  int32_t first, last;     // input pieces: whether this is the first, the last piece
  const int32_t* row_of;   // where the compact rows come from (row statistics: NULL, bounds too: all rows, in place)
  const float* factor;     // input pieces, weight terms: the sums' factor, on the device
  HeadArgs head;
};

// Products beside the linear layer's three directions.
constexpr int kRowStats = 3, kRowSlopes = 4, kInputPiece = 5, kWeightTerms = 6;
constexpr bool one_group(int dir) { return dir >= kRowStats; }  // of grouped products, those that have only one
constexpr bool has_terms(int dir) { return dir == kInputPiece || dir == kWeightTerms; }
constexpr bool is_weight(int dir) { return dir == DDP_LINEAR_BACKWARD_WEIGHT || dir == kWeightTerms; }
constexpr bool is_head(int dir) { return dir == kRowStats || dir == kRowSlopes; }
constexpr bool a_along(int dir) { return !is_weight(dir); }
constexpr bool b_along(int dir) { return dir == DDP_LINEAR_FORWARD || is_head(dir); }

// ---------------------------------------------------------------- activations

// The outputs' last step takes the vector units while the matrix units wait, so
// its length counts where the products are short, in bf16. There, quotients
// come from the reciprocal instruction (1 ulp) and exponentials from the
// exponential instruction (relative error 2^-24 times its argument and 2 ulp): errors
// far below the outputs' rounding. fp32 data gets the library's functions.
template <int DT>
__device__ __forceinline__ float quotient(float x, float y) {
  return DT == DDP_BF16 ? x * __builtin_amdgcn_rcpf(y) : x / y;
}
template <int DT>
__device__ __forceinline__ float exponential(float x) {
  return DT == DDP_BF16 ? __expf(x) : expf(x);
}

// 2 sqrt(2/pi) (z + 0.044715 z^3) = z (kTanh1 + kTanh3 z^2); 1 + tanh(u) = 2 / (1 + exp(-2u))
constexpr float kTanh1 = 1.59576912f, kTanh3 = 0.0713548163f;

// The normal distribution function (1 + erf(z / sqrt 2)) / 2 and exp(-z^2 / 2).
// With x = |z| / sqrt 2, it is erfc(x) / 2 or 1 less that: 1 + erf would cancel
// for negative z.
//
// bf16: by formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions: erfc(x) = t (a1 + ... + a5 t^4) exp(-x^2), t = 1 / (1 + p x), off by
// 1.5e-7 at most. That is 2e-4 of the function itself at z = -3.5 and 1.6e-3 at
// -5, where it still rounds to bf16 about as well as the exact one, and 3e-2 at -10, of
// values near 1e-23. One exponential and one reciprocal serve value and slope; the
// library's erff is several times as long (8192 x 8192 x 2048 forward with z
// kept: 263 us against 286).
//
// fp32: the library's erfc, good to 4 ulp, and x's rounding: 2^-24 (1.3 z^2 +
// 9.3) of the function at most. Its length shows where little else is done (4096 x 4096
// slopes alone 41 us against 29, a forward product of 64 terms 51 against 40) and
// not in longer products (1037 x 1023 x 2049 60 us either way).
struct Normal {
  float cdf, bell;
};
template <int DT>
__device__ __forceinline__ Normal normal(float z) {
  const float x = fabsf(z) * 0.70710678f;
  float q, bell;
  if constexpr (DT == DDP_BF16) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
    bell = __expf(-x * x);
    q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    q *= 0.5f * t * bell;
  } else {
    q = 0.5f * erfcf(x);
    bell = expf(-0.5f * z * z);
  }
  return {z < 0.0f ? q : 1.0f - q, bell};
}

template <int DT, int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == DDP_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays
  if constexpr (ACT == DDP_ACT_GELU) return z * normal<DT>(z).cdf;
  if constexpr (ACT == DDP_ACT_GELU_TANH)
    return quotient<DT>(z, 1.0f + exponential<DT>(-z * fmaf(kTanh3, z * z, kTanh1)));
  if constexpr (ACT == DDP_ACT_SILU) return quotient<DT>(z, 1.0f + exponential<DT>(-z));
  return z;
}

// The slopes are flat to the last bit beyond |z| = 16 (silu: 104), where their
// factors would become infinity times zero. A NaN stays.
__device__ __forceinline__ float within(float z, float most) { return z > most ? most : z < -most ? -most : z; }

template <int DT, int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == DDP_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == DDP_ACT_GELU) {
    z = within(z, 16.0f);
    const Normal d = normal<DT>(z);
    return fmaf(z * 0.39894228f, d.bell, d.cdf);
  }
  if constexpr (ACT == DDP_ACT_GELU_TANH) {
    z = within(z, 16.0f);
    const float z2 = z * z;
    const float s = quotient<DT>(1.0f, 1.0f + exponential<DT>(-z * fmaf(kTanh3, z2, kTanh1)));  // (1 + tanh u) / 2
    return fmaf(z * s * (1.0f - s), fmaf(3.0f * kTanh3, z2, kTanh1), s);                          // s + z s (1 - s) 2u'
  }
  if constexpr (ACT == DDP_ACT_SILU) {
    z = within(z, 104.0f);
    const float s = quotient<DT>(1.0f, 1.0f + exponential<DT>(-z));
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  return 1.0f;
}

// ---------------------------------------------------------------- eight outputs of a row

// Eight elements of a row as they lie in memory: bf16 in `a`, fp32 in both.
struct Raw8 {
  u32x4 a, b;
};
// Elements [0, n) of eight at p (element-aligned), the rest zero.
template <int DT>
__device__ __forceinline__ Raw8 load_raw8(const void* p, int64_t at, int n) {
  Raw8 r{};
  if constexpr (DT == DDP_FP32) {
    const float* q = static_cast<const float*>(p) + at;
    if (n == 8) {
      r.a = load_at<false, u32x4_at4>(q, 0);
      r.b = load_at<false, u32x4_at4>(q, 1);
    } else {
      for (int k = 0; k < 4; ++k)
        if (k < n) r.a[k] = __float_as_uint(q[k]);
      for (int k = 4; k < 8; ++k)
        if (k < n) r.b[k - 4] = __float_as_uint(q[k]);
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (n == 8) {
      r.a = load_at<false, u32x4_at2>(q, 0);
    } else {
      for (int k = 0; k < 8; ++k)
        if (k < n) r.a[k >> 1] |= uint32_t(q[k]) << ((k & 1) * 16);
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8& r, float v[8]) {
  if constexpr (DT == DDP_FP32) {
    for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(r.a[k]), v[4 + k] = __uint_as_float(r.b[k]);
  } else {
    for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(r.a[k]), v[2 * k + 1] = bf16_hi(r.a[k]);
  }
}
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, float v[8]) {
  unpack8<DT>(load_raw8<DT>(p, at, n), v);
}

template <int DT, bool NT>
__device__ __forceinline__ void store_all8(void* p, int64_t at, const float v[8]) {
  if constexpr (DT == DDP_FP32) {
    float* q = static_cast<float*>(p) + at;
    store4<DDP_FP32, NT>(q, 0, v);
    store4<DDP_FP32, NT>(q, 1, v + 4);
  } else {
    store_at<NT, u32x4_at2>(static_cast<uint16_t*>(p) + at, 0,
                            u32x4{round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]), round_bf16x2(v[4], v[5]),
                                  round_bf16x2(v[6], v[7])});
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, int n, const float v[8], bool streamed = false) {
  if (n == 8) {
    if (streamed) {  // between marks, or the compiler makes the two stores one, and that not a streamed one
      asm volatile("; streamed");
      store_all8<DT, true>(p, at, v);
      asm volatile("; to here");
    } else {
      store_all8<DT, false>(p, at, v);
    }
  } else {
    for (int k = 0; k < 8; ++k)
      if (k < n) Ops<DT>::store1(p, at + k, DT == DDP_BF16 ? round_bf16(v[k]) : v[k]);
  }
}

// What eight outputs need besides their sums, as it lies in memory: the
// residual, add and z, or the old gradient. Loaded ahead of their use.
struct Extra {
  Raw8 e, z;
};

template <int DT, int DIR>
__device__ __forceinline__ void load_extra(const LinearArgs& g, int64_t i, int64_t j, int n, Extra& x) {
  if constexpr (DIR == kInputPiece) {
    if (!g.first) x.e = load_raw8<DDP_FP32>(g.sums, i * g.J + j, n);
  } else if constexpr (is_weight(DIR)) {
    if (g.accumulate) x.e = g.grad32 ? load_raw8<DDP_FP32>(g.c, i * g.ldc + j, n) : load_raw8<DT>(g.c, i * g.ldc + j, n);
  } else {
    if (g.e != nullptr) x.e = load_raw8<DT>(g.e, i * g.lde + j, n);
    if (DIR == DDP_LINEAR_BACKWARD_INPUT && g.act != DDP_ACT_NONE) x.z = load_raw8<DT>(g.z, i * g.ldz + j, n);
  }
}

// Eight sums of row i from column j on (n of them inside C) become outputs:
// what is done before the store of C, z's store with it ...
template <int DT, int DIR, int ACT>
__device__ __forceinline__ void before_store(const LinearArgs& g, int64_t i, int64_t j, int n, float v[8], const Extra& x,
                                             const float bias[8]) {
  float e[8];
  if constexpr (DIR == kInputPiece) {
    if (!g.first) {
      unpack8<DDP_FP32>(x.e, e);
      for (int k = 0; k < 8; ++k) v[k] += e[k];
    }
    if (g.last) {
      const float factor = *g.factor;
      for (int k = 0; k < 8; ++k) v[k] *= factor;
    }
  } else if constexpr (is_weight(DIR)) {
    if constexpr (DIR == kWeightTerms) {
      const float factor = *g.factor;
      for (int k = 0; k < 8; ++k) v[k] *= factor;
    }
    if (g.accumulate) {
      if (g.grad32)
        unpack8<DDP_FP32>(x.e, e);
      else
        unpack8<DT>(x.e, e);
      for (int k = 0; k < 8; ++k) v[k] += e[k];
    }
  } else {
    if constexpr (DIR == DDP_LINEAR_FORWARD) {
      for (int k = 0; k < 8; ++k) v[k] += bias[k];  // zeros without a bias
      if (g.z != nullptr) store8<DT>(g.z, i * g.ldz + j, n, v, g.stream_z != 0);
      for (int k = 0; k < 8; ++k) v[k] = act_value<DT, ACT>(v[k]);
    } else if constexpr (ACT != DDP_ACT_NONE) {
      float z[8];
      unpack8<DT>(x.z, z);
#pragma unroll  // else z goes to scratch memory
      for (int k = 0; k < 8; ++k) v[k] *= act_slope<DT, ACT>(z[k]);
    }
    if (g.e != nullptr) {
      unpack8<DT>(x.e, e);
      for (int k = 0; k < 8; ++k) v[k] += e[k];
    }
  }
}
// ... and the store.
template <int DT, int DIR>
__device__ __forceinline__ void store_output(const LinearArgs& g, int64_t i, int64_t j, int n, const float v[8]) {
  if (DIR == kInputPiece && !g.last)
    store8<DDP_FP32>(g.sums, i * g.J + j, n, v);
  else if (DIR == kInputPiece)
    store8<DT>(g.c, g.row_of[i] * g.ldc + j, n, v);
  else if (is_weight(DIR) && g.grad32)
    store8<DDP_FP32>(g.c, i * g.ldc + j, n, v);
  else
    store8<DT>(g.c, i * g.ldc + j, n, v);
}
// Both, for any activation.
template <int DT, int DIR>
__device__ __forceinline__ void finish(const LinearArgs& g, int64_t i, int64_t j, int n, float v[8], const Extra& x,
                                       const float bias[8]) {
  switch (g.act) {
#define DDP_ACT_CASE(A)                                   \
  case A:                                                 \
    before_store<DT, DIR, A>(g, i, j, n, v, x, bias);     \
    break;
    DDP_ACT_CASE(DDP_ACT_RELU)
    DDP_ACT_CASE(DDP_ACT_GELU)
    DDP_ACT_CASE(DDP_ACT_GELU_TANH)
    DDP_ACT_CASE(DDP_ACT_SILU)
#undef DDP_ACT_CASE
    default:
      before_store<DT, DIR, DDP_ACT_NONE>(g, i, j, n, v, x, bias);
  }
  store_output<DT, DIR>(g, i, j, n, v);
}

// ---------------------------------------------------------------- an operand's tile

// T rows of C's side (i or j) by SB bytes of k, in LDS as 16-byte chunks.
// "along": T rows of SB bytes. A read takes the same chunk of 16 neighbouring
// rows at a time; 256 / SB rows fill the 64 banks, so chunk c of row r is kept
// at c ^ (r / (256 / SB)) and the reads touch every bank once.
// "across": one row of T elements per k. The transposing read takes 64 bytes
// of 4 neighbouring rows at a time, which are kept apart by exchanging chunks
// by the row's low bits.
// (Exchanges made for 32 banks ran 2 to 3 % slower.)
// (The exchange is applied to the address that a lane loads from: a direct
// load to LDS writes the wave's 64 chunks in lane order.)
template <int DT, bool ALONG, int T, int SB, int THREADS>
struct Tile {
  static constexpr int ES = DT == DDP_BF16 ? 2 : 4;
  static constexpr int V = 16 / ES;             // elements per chunk
  static constexpr int STEP = SB / ES;          // k per step
  static constexpr int BYTES = T * SB;
  static constexpr int ROW = ALONG ? SB : T * ES;
  static constexpr int CPR = ROW / 16;
  static constexpr int N = BYTES / 16 / THREADS;  // chunks per thread
  static_assert(BYTES % (16 * THREADS) == 0, "whole chunks per thread");

  static __device__ __forceinline__ int swizzle(int row) {
    if (ALONG) return SB > 256 ? row & 15 : (row / (256 / (SB > 256 ? 256 : SB))) & (CPR - 1);
    if (DT != DDP_BF16) return 0;
    return CPR > 8 ? (row & 3) << 2 : (row >> 1 & 1) << 2;  // rows of 128 bytes: two fill the banks as they lie
  }
  // Chunk q of the tile in LDS: its row, and the chunk of memory it holds.
  static __device__ __forceinline__ int row_of(int q) { return q / CPR; }
  static __device__ __forceinline__ int col_of(int q) { return (q % CPR) ^ swizzle(q / CPR); }

  // This lane's part of the fragment for rows [32 * t, 32 * t + 32) from
  // `base` on and the s-th 32 bytes of the step.
  static __device__ __forceinline__ u32x4 fragment(const char* lds, int base, int t, int s, int lane) {
    if constexpr (ALONG) {
      const int row = base + 32 * t + (lane & 31);
      const int c = (2 * s + (lane >> 5)) ^ swizzle(lane & 31);  // as of `row`: base and 32 t are multiples of 32
      return *reinterpret_cast<const u32x4*>(lds + row * SB + c * 16);
    } else if constexpr (DT == DDP_BF16) {
      const int group = lane >> 4, in = lane & 15;
      const int k = 16 * s + 8 * (group >> 1) + (in >> 2);
      const int i = base + 32 * t + 16 * (group & 1) + 4 * (in & 3);
      const int c = (i >> 3) ^ swizzle(k);
      const char* p = lds + k * ROW + c * 16 + (i & 7) * 2;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DDP_LDS i16x4*)p);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DDP_LDS i16x4*)(p + 4 * ROW));  // rows k+4..k+7: the same exchange
      const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
      return u32x4{a.x, a.y, b.x, b.y};
    } else {
      const int k = 8 * s + 4 * (lane >> 5);
      const int i = base + 32 * t + (lane & 31);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(lds + k * ROW + i * 4);
      return u32x4{p[0], p[ROW / 4], p[2 * (ROW / 4)], p[3 * (ROW / 4)]};
    }
  }
};

// The 32 x 32 product of two fragments, added to d: lane l holds column l & 31
// (of `col`'s rows), rows 8 q + 4 (l >> 5) + r in element 4 q + r.
template <int DT>
__device__ __forceinline__ f32x16 multiply(u32x4 row, u32x4 col, f32x16 d) {
  if constexpr (DT == DDP_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, row), __builtin_bit_cast(bf16x8, col), d, 0, 0, 0);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      d = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(row[k]), __uint_as_float(col[k]), d, 0, 0, 0);
    return d;
  }
}

// The sum of a fragment's values in this lane: one row's, over its half of k.
template <int DT>
__device__ __forceinline__ float sum_of(u32x4 f) {
  if constexpr (DT == DDP_BF16)
    return ((bf16_lo(f[0]) + bf16_hi(f[0])) + (bf16_lo(f[1]) + bf16_hi(f[1]))) +
           ((bf16_lo(f[2]) + bf16_hi(f[2])) + (bf16_lo(f[3]) + bf16_hi(f[3])));
  else
    return (__uint_as_float(f[0]) + __uint_as_float(f[1])) + (__uint_as_float(f[2]) + __uint_as_float(f[3]));
}

// ---------------------------------------------------------------- loading a tile

constexpr uint32_t kFar = 0xfffffff0u;     // an offset outside every descriptor's range: reads as zeros
constexpr int32_t kMostRange = 0x0f000000; // of a descriptor, in 16-byte chunks

// Direct loads to LDS, for operands whose every chunk is 16-byte aligned and
// whole (`room` elements behind the last row make its last chunk whole). The
// descriptor ends with the operand, so a chunk past it reads as zeros; a row of C's side past the operand repeats the last one (its
// products are not stored).
template <class TL, bool ALONG, int THREADS, bool TURNED>
struct DirectLoader {
  const char* p;        // the tile at the current step
  int64_t advance;      // bytes per step
  int32_t left;         // chunks from p to the operand's end
  int32_t k_left;       // terms left
  int32_t until;        // TURNED: steps to the operand's last one
  int64_t back;         // and the way back from there
  uint32_t off[TL::N];  // of this lane's chunks, in bytes from p
  int32_t wave;
  u32x4 desc;

  // First term, within the step, of this lane's n-th chunk.
  __device__ __forceinline__ int k_of(int n) const {
    const int q = (n * (THREADS / 64) + wave) * 64 + (int(threadIdx.x) & 63);
    return ALONG ? TL::col_of(q) * TL::V : TL::row_of(q);
  }
  __device__ __forceinline__ void init(const void* base, int64_t ld, int64_t side, int64_t K, int64_t s0, int64_t k0, int64_t k1, int32_t room) {
    const int lane = int(threadIdx.x) & 63;
    wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t rows = ALONG ? side : K, cols = ALONG ? K : side;
    const int64_t start = ALONG ? s0 * ld + k0 : k0 * ld + s0;
    p = static_cast<const char*>(base) + start * TL::ES;
    left = int32_t(((rows - 1) * ld + cols + room - start) / TL::V);
    advance = ALONG ? TL::ROW : TL::STEP * ld * TL::ES;
    k_left = int32_t(k1 - k0);
#pragma unroll
    for (int n = 0; n < TL::N; ++n) {
      const int q = (n * (THREADS / 64) + wave) * 64 + lane;
      const int64_t row = TL::row_of(q);
      const int64_t r = ALONG && s0 + row >= side ? side - 1 - s0 : row;
      off[n] = uint32_t(r * ld * TL::ES + TL::col_of(q) * 16);
    }
    describe();
  }
  // The current step's loads into `lds`: load(n) for every n, then end().
  // Loads that the sum does not need read as zeros (FULL: it needs
  // all of them).
  __device__ __forceinline__ void describe() {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const int32_t range = left < 0 ? 0 : left < kMostRange ? left : kMostRange;
    desc = u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a))),
                 uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a >> 32))),
                 uint32_t(__builtin_amdgcn_readfirstlane(range)) << 4, 0x00020000u};
  }
  template <bool FULL, int SET = 0>
  __device__ __forceinline__ void load(const char* lds, int n) {
    const uint32_t to = uint32_t(reinterpret_cast<uintptr_t>((DDP_LDS const char*)lds));
    const uint32_t m = uint32_t(__builtin_amdgcn_readfirstlane(to + (n * (THREADS / 64) + wave) * 1024));
    uint32_t o = off[n];
    if (!FULL && k_left < TL::STEP) o = k_of(n) < k_left ? o : kFar;
    // No output register: the load ends in LDS, and every use of it stands
    // behind a wait for it and a barrier. (With the builtin, the
    // compiler waits for all direct loads before any read of LDS.) A direct
    // load needs one wait state after a write of M0, which nobody adds inside
    // assembly.
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(o), "s"(desc), "s"(m) : "m0");
  }
  template <int SET = 0>
  __device__ __forceinline__ void end() {
    p += advance;
    left -= int32_t(advance / 16);
    k_left -= TL::STEP;
    if (TURNED && --until == 0) {
      p -= back;
      left += int32_t(back / 16);
    }
    describe();
  }
  // Starts at step `first` of `steps` and comes back to the others at the end.
  __device__ __forceinline__ void turn_to(int32_t first, int32_t steps) {
    back = steps * advance;
    until = steps - first;
    p += first * advance;
    left -= int32_t(first * advance / 16);
    describe();
  }
  template <int SET = 0>
  __device__ __forceinline__ void commit(char*) {}
};

// Through registers, for operands of any alignment whose rows have a chunk's
// elements at least. Every chunk is one load at its element's alignment,
// without a branch that writes its registers (with one, each load is waited
// for before the next starts: twice as slow). A chunk that runs over the
// end of its row is loaded from as far back as it fits and shifted into place
// when it goes to LDS, zeros following; one past the sum's end is shifted out
// whole. PIPE: steps whose chunks are in registers or on their way there; with two, a
// step's loads have two steps' time.
template <int DT, class TL, bool ALONG, int THREADS, int PIPE>
struct AnyLoader {
  static constexpr int kWidth = TL::CPR * TL::V;  // "across": elements of a row in the tile
  const char* p;         // the tile at the current step
  int64_t row_bytes;
  int32_t k_left;        // terms left
  int32_t width;         // "across": elements of a row that exist
  int64_t off[TL::N];    // of this lane's chunks, in bytes from p
  int32_t back[TL::N];   // "across": elements that a chunk is loaded before its place
  bool shifted[PIPE];    // some chunk of the step is to be shifted
  int32_t shift[PIPE][TL::N];  // elements to shift out
  u32x4 x[PIPE][TL::N];

  static __device__ __forceinline__ int chunk(int n) { return n * THREADS + int(threadIdx.x); }
  __device__ __forceinline__ void init(const void* base, int64_t ld, int64_t side, int64_t, int64_t s0, int64_t k0, int64_t k1, int32_t) {
    row_bytes = ld * TL::ES;
    p = static_cast<const char*>(base) + (ALONG ? s0 * ld + k0 : k0 * ld + s0) * TL::ES;
    k_left = int32_t(k1 - k0);
    width = side - s0 < kWidth ? int32_t(side - s0) : kWidth;
#pragma unroll
    for (int n = 0; n < TL::N; ++n) {
      const int row = TL::row_of(chunk(n)), col = TL::col_of(chunk(n)) * TL::V;
      const int64_t r = ALONG && s0 + row >= side ? side - 1 - s0 : row;
      back[n] = !ALONG && col + TL::V > width ? col + TL::V - width : 0;
      off[n] = r * row_bytes + (col - back[n]) * TL::ES;  // from p, perhaps negative; never before the row
#pragma unroll
      for (int s = 0; s < PIPE; ++s) shift[s][n] = back[n];
    }
  }
  template <bool FULL, int SET = 0>
  __device__ __forceinline__ void load(const char*, int n) {
    int64_t o = off[n];
    if (!FULL && k_left < TL::STEP) {
      const int row = TL::row_of(chunk(n)), col = TL::col_of(chunk(n)) * TL::V;
      if (ALONG) {
        shift[SET][n] = col + TL::V > k_left ? col + TL::V - k_left : 0;
        o -= shift[SET][n] * TL::ES;
      } else if (row >= k_left) {
        o -= (row - (k_left - 1)) * row_bytes;
        shift[SET][n] = TL::V;
      }
    }
    if constexpr (DT == DDP_FP32)
      x[SET][n] = load_at<false, u32x4_at4>(p + o, 0);
    else
      x[SET][n] = load_at<false, u32x4_at2>(p + o, 0);
  }
  template <int SET = 0>
  __device__ __forceinline__ void end() {
    shifted[SET] = k_left < TL::STEP || (!ALONG && width < kWidth);
    p += ALONG ? TL::ROW : TL::STEP * row_bytes;
    k_left -= TL::STEP;
  }
  template <int SET = 0>
  __device__ __forceinline__ void commit(char* lds) {
    if (shifted[SET]) {
#pragma unroll
      for (int n = 0; n < TL::N; ++n) {
        const int bits = shift[SET][n] * TL::ES * 8;
        const unsigned __int128 v = __builtin_bit_cast(unsigned __int128, x[SET][n]);
        x[SET][n] = bits < 128 ? __builtin_bit_cast(u32x4, v >> bits) : u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int n = 0; n < TL::N; ++n) *reinterpret_cast<u32x4*>(lds + chunk(n) * 16) = x[SET][n];
  }
};

// Element by element, for rows shorter than a chunk.
template <int DT, class TL, bool ALONG, int THREADS>
struct ShortLoader {
  const void* base;
  int64_t ld, side, s0, k, k1;
  u32x4 x[TL::N];

  __device__ __forceinline__ void init(const void* b, int64_t ld_, int64_t side_, int64_t, int64_t s0_, int64_t k0, int64_t k1_, int32_t) {
    base = b, ld = ld_, side = side_, s0 = s0_, k = k0, k1 = k1_;
  }
  template <bool FULL, int SET = 0>
  __device__ __forceinline__ void load(const char*, int n) {
    const int q = n * THREADS + int(threadIdx.x);
    const int row = TL::row_of(q), col = TL::col_of(q) * TL::V;
    const int64_t r = ALONG ? (s0 + row < side ? s0 + row : side - 1) : k + row;
    const int64_t e = ALONG ? k + col : s0 + col, end = ALONG ? k1 : side;
    x[n] = u32x4{0u, 0u, 0u, 0u};
    for (int j = 0; j < TL::V; ++j) {
      if (e + j >= end || (!ALONG && r >= k1)) continue;
      if constexpr (DT == DDP_FP32)
        x[n][j] = static_cast<const uint32_t*>(base)[r * ld + e + j];
      else
        x[n][j >> 1] |= uint32_t(static_cast<const uint16_t*>(base)[r * ld + e + j]) << ((j & 1) * 16);
    }
  }
  template <int SET = 0>
  __device__ __forceinline__ void end() { k += TL::STEP; }
  template <int SET = 0>
  __device__ __forceinline__ void commit(char* lds) {
#pragma unroll
    for (int n = 0; n < TL::N; ++n) *reinterpret_cast<u32x4*>(lds + (n * THREADS + int(threadIdx.x)) * 16) = x[n];
  }
};

enum Loading { kDirect, kAny, kShort };
template <int LOAD, int DT, class TL, bool ALONG, int THREADS, bool TURNED, int PIPE>
using LoaderOf = std::conditional_t<LOAD == kDirect, DirectLoader<TL, ALONG, THREADS, TURNED>,
                                    std::conditional_t<LOAD == kAny, AnyLoader<DT, TL, ALONG, THREADS, PIPE>,
                                                       ShortLoader<DT, TL, ALONG, THREADS>>>;

// ---------------------------------------------------------------- groups of rows

// The bounds come from the device and are not trusted: each counts as the
// largest one up to it, within [0, rows]. So groups never overlap, and their
// tiles never outnumber a launch's blocks.
__device__ __forceinline__ int32_t bound_at(const LinearArgs& g, int32_t e) {
  const int64_t b = g.bounds[e];
  return b < 0 ? 0 : b < g.rows ? int32_t(b) : int32_t(g.rows);
}

// Sums, or the largest, of the values (none negative) of the lanes up to each
// one. Moves within rows of 16 lanes, then rows' last lanes to the rows
// behind: some 10 cycles each, a tenth of what a shuffle through LDS takes.
template <class F>
__device__ __forceinline__ int32_t scan_lanes(int32_t v, F&& join) {
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // from 1 lane before, 2, 4, 8 in the row
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // lane 15 to row 1, 47 to row 3
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // lane 31 to rows 2 and 3
  return v;
}
__device__ __forceinline__ int32_t larger(int32_t a, int32_t b) { return a > b ? a : b; }

// 64 groups from e0 on, one a lane.
struct GroupScan {
  int32_t begin, rows;     // of this lane's group
  int32_t tiles, until;    // its tiles of T rows; tiles up to and with it
};
template <int T>
__device__ __forceinline__ GroupScan scan_groups(const LinearArgs& g, int32_t e0, int32_t& bound, int32_t& tiles) {
  const int lane = int(threadIdx.x) & 63;
  const int32_t end = scan_lanes(larger(e0 + lane < g.groups ? bound_at(g, e0 + lane + 1) : 0, bound), larger);
  GroupScan s;
  s.begin = __builtin_amdgcn_update_dpp(bound, end, 0x138, 0xf, 0xf, false);  // the lane before's
  s.rows = e0 + lane < g.groups ? end - s.begin : 0;
  s.tiles = (s.rows + T - 1) / T;
  s.until = tiles + scan_lanes(s.tiles, [](int32_t a, int32_t b) { return a + b; });
  bound = __builtin_amdgcn_readlane(end, 63);
  tiles = __builtin_amdgcn_readlane(s.until, 63);
  return s;
}
// Tiles of T rows in all groups.
template <int T>
__device__ __forceinline__ int32_t tiles_of_groups(const LinearArgs& g, GroupScan& first) {
  int32_t bound = bound_at(g, 0), tiles = 0;
  first = scan_groups<T>(g, 0, bound, tiles);
  for (int32_t e0 = 64; e0 < g.groups; e0 += 64) scan_groups<T>(g, e0, bound, tiles);
  return tiles;
}
struct Group {
  int32_t index, begin, rows, tile;  // the group, its rows, and which of its tiles
};
// The group of tile number `tile` (below their number).
template <int T>
__device__ __forceinline__ Group group_of_tile(const LinearArgs& g, const GroupScan& first, int32_t tile) {
  int32_t bound = 0, tiles = 0, e0 = 0;
  GroupScan s = first;
  uint64_t hit = __ballot(tile < s.until);
  if (hit == 0) {
    bound = bound_at(g, 0);
    scan_groups<T>(g, 0, bound, tiles);
    do {
      e0 += 64;
      s = scan_groups<T>(g, e0, bound, tiles);
      hit = __ballot(tile < s.until);
    } while (hit == 0 && e0 + 64 < g.groups);
  }
  const int from = hit != 0 ? __builtin_ctzll(hit) : 0;
  return Group{e0 + from, __builtin_amdgcn_readlane(s.begin, from), __builtin_amdgcn_readlane(s.rows, from),
               tile - (__builtin_amdgcn_readlane(s.until, from) - __builtin_amdgcn_readlane(s.tiles, from))};
}
// Group number e.
__device__ __forceinline__ Group group_at(const LinearArgs& g, int32_t e) {
  int32_t bound = 0;
  for (int32_t f = int32_t(threadIdx.x) & 63; f <= e; f += 64) bound = larger(bound, bound_at(g, f));
  const int32_t begin = __builtin_amdgcn_readlane(scan_lanes(bound, larger), 63);
  return Group{e, begin, larger(bound_at(g, e + 1), begin) - begin, 0};
}

// ---------------------------------------------------------------- the losses' outputs

constexpr float kLog2E = 1.44269504f;

// From a tile of x w^T in registers (lane l: row l & 31, columns 8 q + 4 (l >> 5)
// + r of each 32 x 32 product), so a row's values lie in two lanes:
//
// row statistics: the maximum over the tile's columns and the sum of exp(z -
// maximum), which need no exchange but with the other half and, in LDS, with
// the waves beside this one; and z of the row's entries (its target, or the
// teacher's logits), found through LDS where a wave's columns hold any.
//
// row slopes: dz = slope dloss (exp(z - lse) - q), by rows through LDS, where q
// of the few entries is taken off. bf16: in one or two terms, the second what the
// first's rounding left, which together are off by 2^-16 of dz at most.
template <int DT, int DIR, int TI, int TJ, int WI, int WJ, int WK, int STAGES>
__device__ __forceinline__ void head_outputs(const LinearArgs& g, f32x16 (&acc)[TI / WI / 32][TJ / WJ / 32], char* lds, int64_t i0,
                                             int64_t j0, int wi, int wj, int wave, int wk, int lane, int tile_j) {
  constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32, THREADS = WI * WJ * WK * 64, PITCH = 32 * FJ + 4;
  static_assert((WI * WJ * 32 * PITCH + WJ * 2 * TI) * 4 <= STAGES * (TI + TJ) * 128 * WK, "the outputs' rows and statistics fit in LDS");
  const HeadArgs& h = g.head;
  const int half = lane >> 5, in = lane & 31;
  const int width = g.J - j0 - wj < 32 * FJ ? int(g.J - j0 - wj) : 32 * FJ;  // of the wave's columns inside, or less than 0
  float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  float* const stats = reinterpret_cast<float*>(lds) + WI * WJ * 32 * PITCH;  // [WJ][2][TI]
  const int64_t column = h.j_base + j0;                                       // of the vocabulary, the tile's first
#pragma unroll
  for (int a = 0; a < FI; ++a) {
    if (WK > 1 && wk > 0) break;  // the sums are the first waves'
    const int64_t i = i0 + wi + 32 * a + in;
    bool counts = i < g.I;
    int64_t row = counts ? i : 0;
    if (DIR == kRowStats && g.row_of == nullptr) {
      if (counts && h.targets == nullptr) counts = h.counted[row] != 0;
    } else if (counts) {
      row = g.row_of[i];
    }
    // The row's entries in this tile; of a target, `place` is known at once.
    int entry = 0, entries = 0, place = -1;
    if (h.targets != nullptr) {
      const int64_t t = counts ? h.targets[row] - column - wj : -1;
      if (t >= 0 && t < width) place = int(t), entries = 1;
    } else if (counts) {
      const int64_t at = row * (h.tiles + 1) + column / TJ;
      entry = h.starts[at];
      entries = h.starts[at + 1] - entry;
    }
    const auto place_of = [&](int k) __attribute__((always_inline)) {
      return h.targets != nullptr ? place : int(h.ids[row * h.top + k] - column - wj);
    };
    const auto to_lds = [&] __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < FJ; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4*>(mine + in * PITCH + 32 * b + 8 * q + 4 * half) =
              f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
      __builtin_amdgcn_wave_barrier();
    };
    // Values outside C become `outside`.
    const auto outside_is = [&](float outside) __attribute__((always_inline)) {
      if (width == 32 * FJ) return;
#pragma unroll
      for (int b = 0; b < FJ; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * b + 8 * (e >> 2) + 4 * half + (e & 3) >= width) acc[a][b][e] = outside;
    };
    // exp(scale v - x), with bf16 data as 2^(u v - y): one step less, and an error
    // of 2^-24 of the terms.
    const float u = DT == DDP_BF16 ? h.scale * kLog2E : h.scale;
    const auto power = [&](float v, float y) __attribute__((always_inline)) {
      return DT == DDP_BF16 ? __builtin_amdgcn_exp2f(fmaf(v, u, -y)) : expf(fmaf(v, u, -y));
    };
    if constexpr (DIR == kRowStats) {
      outside_is(-INFINITY);
      float most = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int b = 0; b < FJ; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) most = fmaxf(most, acc[a][b][e]);
      most = fmaxf(most, __shfl_xor(most, 32));
      const float base = most == -INFINITY ? 0.0f : most * u;
#pragma unroll
      for (int b = 0; b < FJ; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum += power(acc[a][b][e], base);
      sum += __shfl_xor(sum, 32);
      if (half == 0) {
        stats[(wj / (32 * FJ) * 2 + 0) * TI + wi + 32 * a + in] = most * h.scale;
        stats[(wj / (32 * FJ) * 2 + 1) * TI + wi + 32 * a + in] = sum;
      }
      if (__any(entries > 0)) {
        to_lds();
        for (int k = half; k < entries; k += 2) {
          const int at = place_of(entry + k);
          if (at >= 0 && at < width) h.picked[row * h.top + entry + k] = mine[in * PITCH + at] * h.scale;
        }
        __builtin_amdgcn_wave_barrier();
      }
    } else {
      float lse = 0.0f, slope = 0.0f;
      if (counts) {
        lse = h.lse[row];
        slope = h.slope * (h.dloss[row] / *g.factor);
        // A target or entry outside the vocabulary makes the row NaN.
        if (h.targets != nullptr ? h.targets[row] >= h.vocabulary : h.own_terms[row] != h.own_terms[row]) lse = NAN;
      }
      if (DT == DDP_BF16) lse *= kLog2E;
#pragma unroll
      for (int b = 0; b < FJ; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][b][e] = slope * power(acc[a][b][e], lse);
      outside_is(0.0f);
      to_lds();
      for (int k = 0; half == 0 && k < entries; ++k) {  // an id may come again: one lane a row, in order
        const int at = place_of(entry + k);
        if (at < 0 || at >= width) continue;
        const float q = h.targets != nullptr ? 1.0f : h.weights[row * h.top + entry + k];
        mine[in * PITCH + at] = fmaf(-q, slope, mine[in * PITCH + at]);
      }
      __builtin_amdgcn_wave_barrier();
      constexpr int LPR = 4 * FJ, RPP = 64 / LPR;  // lanes per row, rows per pass
      const int c = lane % LPR * 8;
#pragma unroll
      for (int p = 0; p < 32 / RPP; ++p) {
        const int r = p * RPP + lane / LPR;
        const float* src = mine + r * PITCH + c;
        const int64_t to = i0 + wi + 32 * a + r;
        float v[8], rest[8];
        for (int k = 0; k < 8; ++k) v[k] = src[k];
        if (to >= g.I || c >= width) continue;  // a row's last chunk is written whole, with zeros
        const int64_t at = to * g.ldc + j0 + wj + c;
        store_all8<DT, false>(g.c, at, v);
        if (DT == DDP_BF16 && g.terms > 1) {
          for (int k = 0; k < 8; ++k) rest[k] = v[k] - round_bf16(v[k]);
          store_all8<DT, false>(g.c, g.term + at, rest);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  if constexpr (DIR == kRowStats) {
    __syncthreads();
    for (int r = int(threadIdx.x); r < TI; r += THREADS) {
      if (i0 + r >= g.I) continue;
      float most = stats[r], sum = 0.0f;
      for (int w = 1; w < WJ; ++w) most = fmaxf(most, stats[w * 2 * TI + r]);
      const float base = most == -INFINITY ? 0.0f : most;
      for (int w = 0; w < WJ; ++w) {
        const float m = stats[w * 2 * TI + r];
        sum += stats[(w * 2 + 1) * TI + r] * exponential<DT>((m == -INFINITY ? base : m) - base);
      }
      h.stats[int64_t(tile_j) * 2 * g.rows + i0 + r] = most;
      h.stats[(int64_t(tile_j) * 2 + 1) * g.rows + i0 + r] = sum;
    }
  }
}

// ---------------------------------------------------------------- a weight gradient's outputs

// A whole tile's sums to C, of type GT, by rows through LDS, 32 rows at a time: a
// lane has 16 bytes of C, a row's lanes 128 or 256 together. Where they are added to
// what is there, the tile's old values are asked for up to two groups of 32 rows ahead of
// their use. NT: both pass the caches.
template <int GT, bool NT, int DIR, int FI, int FJ, int PITCH>
__device__ __forceinline__ void weight_outputs(const LinearArgs& g, f32x16 (&acc)[FI][FJ], float* mine, int64_t i, int64_t j, int lane) {
  constexpr int W = GT == DDP_FP32 ? 4 : 8, LPR = 32 * FJ / W, RPP = 64 / LPR, PASSES = 32 / RPP;
  constexpr int AHEAD = GT == DDP_FP32 && FI > 2 ? 1 : 2;  // more do not fit beside 128 sums a lane
  const float factor = DIR == kWeightTerms ? *g.factor : 1.0f;
  char* const c = static_cast<char*>(g.c) + ((i + lane / LPR) * g.ldc + j + lane % LPR * W) * (16 / W);
  const int64_t pass = RPP * g.ldc * (16 / W);  // bytes
  u32x4 old[AHEAD][PASSES];
  const auto load = [&](int a) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if constexpr (GT == DDP_FP32)
        old[a % AHEAD][p] = load_at<NT, u32x4_at4>(c + (a * PASSES + p) * pass, 0);
      else
        old[a % AHEAD][p] = load_at<NT, u32x4_at2>(c + (a * PASSES + p) * pass, 0);
    }
  };
  if (g.accumulate) {
    load(0);
    if (AHEAD > 1 && FI > 1) load(1);
  }
#pragma unroll
  for (int a = 0; a < FI; ++a) {
#pragma unroll
    for (int b = 0; b < FJ; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(mine + (lane & 31) * PITCH + 32 * b + 8 * q + 4 * (lane >> 5)) =
            f32x4{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
    float v[PASSES][W];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const float* src = mine + (p * RPP + lane / LPR) * PITCH + lane % LPR * W;
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(src + 4 * q);
        for (int k = 0; k < 4; ++k) v[p][4 * q + k] = x[k];
      }
      if constexpr (DIR == kWeightTerms)
        for (int k = 0; k < W; ++k) v[p][k] *= factor;
      if (g.accumulate) {
        const u32x4 o = old[a % AHEAD][p];
        if constexpr (GT == DDP_FP32) {
          for (int k = 0; k < 4; ++k) v[p][k] += __uint_as_float(o[k]);
        } else {
          for (int k = 0; k < 4; ++k) v[p][2 * k] += bf16_lo(o[k]), v[p][2 * k + 1] += bf16_hi(o[k]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (g.accumulate && a + AHEAD < FI) load(a + AHEAD);
    if (NT) asm volatile("; streamed");  // or the compiler may join these stores with those of the other variant
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      char* const to = c + (a * PASSES + p) * pass;
      if constexpr (GT == DDP_FP32)
        store4<DDP_FP32, NT>(to, 0, v[p]);
      else
        store_all8<DDP_BF16, NT>(to, 0, v[p]);
    }
    if (NT) asm volatile("; to here");
  }
}

// ---------------------------------------------------------------- the product

// Tile TI x TJ of C by WI x WJ waves. GROUPS: of the rows of one group. STAGES
// steps are in LDS or on their way there. WK: as many waves share each part of the
// tile and take 128 bytes of k each of a step that is as much longer.
template <int DT, int DIR, int TI, int TJ, int WI, int WJ, int LOAD, bool GROUPS = false, int STAGES = 2, int WK = 1>
__global__ __launch_bounds__(WI * WJ * WK * 64, 2) void k_linear(LinearArgs g) {
  constexpr int THREADS = WI * WJ * WK * 64;
  constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;  // 32 x 32 products per wave
  // Steps of 128 bytes of k, one on its way while one is multiplied. (Four
  // stages of 64 bytes, three of them on their way, ran 15 % slower: twice the
  // barriers. 4 waves with 128 x 128 products each read a third less from LDS
  // but have nobody to fill their waits: as fast without outputs to speak of,
  // 8192 x 8192 x 2048 input gradient through gelu_tanh 303 us against 269.)
  constexpr int SB = 128 * WK;
  static_assert(WK == 1 || (GROUPS && b_along(DIR)), "where waves share a part");
  using TA = Tile<DT, a_along(DIR), TI, SB, THREADS>;
  using TB = Tile<DT, b_along(DIR), TJ, SB, THREADS>;
  // Rows of a multiple of some KB: what all blocks read at a time, 128 bytes of
  // each row of B, lies in an eighth of the memory's channels or fewer, so blocks of
  // few rows, which read B from memory, begin at different steps. A probe that only reads
  // so, 256 MiB in rows of 4096 bytes: 4.5 TB/s as it was, 5.7 so, 5.9 in rows of 4224.
  constexpr bool TURNED = GROUPS && LOAD == kDirect && b_along(DIR);
  // Two steps of chunks in registers where they fit beside the sums: 1 row of 19208 columns of 2045 in fp32,
  // forward and backward, 252 us to 221.
  constexpr int PIPE = GROUPS && LOAD == kAny && WK == 1 && (TI < 128 || b_along(DIR)) ? 2 : 1;
  using LA = LoaderOf<LOAD, DT, TA, a_along(DIR), THREADS, TURNED, PIPE>;
  using LB = LoaderOf<LOAD, DT, TB, b_along(DIR), THREADS, TURNED, PIPE>;
  constexpr int STAGE = TA::BYTES + TB::BYTES;
  constexpr int PITCH = 32 * FJ + 4;  // floats; the outputs' way through LDS
  static_assert(WI * WJ * 32 * PITCH * 4 <= STAGES * STAGE, "the outputs' rows fit");
  static_assert((WK - 1) * TI * TJ * 4 <= STAGES * STAGE, "the sums that waves hand over fit");
  static_assert(STAGES == 2 || LOAD == kDirect, "loads through registers are one step ahead");
  __shared__ __attribute__((aligned(1024))) char lds[STAGES * STAGE];

  // Blocks go to the 8 XCDs in turn: XCD x takes the tiles of eighth x, in
  // groups of 4 tile rows, so that blocks that share operands share an L2
  // (8192 x 8192 x 2048 forward with z kept: 254 us; groups of 8, 258, of 1,
  // 283; tiles in the blocks' order, 299).
  // Of groups, the eighths are of the tiles that there are (rows grouped), or of
  // every group's tiles, as groups differ in length (sums grouped).
  int tiles_i = g.tiles_i;
  GroupScan scan;
  if constexpr (GROUPS && one_group(DIR)) {
    (is_weight(DIR) ? g.K : g.I) = DIR == kRowStats && g.bounds == nullptr ? g.rows : bound_at(g, 1);
    if (!is_weight(DIR)) tiles_i = int(g.I + TI - 1) / TI;
  } else if constexpr (GROUPS && !is_weight(DIR)) {
    tiles_i = tiles_of_groups<TI>(g, scan);
  }
  const int tiles = tiles_i * g.tiles_j;
  int at = g.begin + int(blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8);
  int group_index = 0;
  if constexpr (GROUPS) {
    const int eighth = (tiles * g.parts + 7) / 8, b = g.begin + int(blockIdx.x);
    if (eighth == 0) return;
    int n = b / 8;
    if constexpr (is_weight(DIR) && !one_group(DIR)) {
      group_index = n / eighth;
      n -= group_index * eighth;
      if (group_index >= g.groups) return;
    } else if (n >= eighth) {
      return;
    }
    at = b % 8 * eighth + n;
  }
  if (at >= tiles * g.parts) return;
  const int part = at / tiles, tile = at % tiles;
  // Experts have a tile row or two each: groups of 2 (4096 rows of 32, 4096 x 2048, input gradient
  // 227 us to 210; 8192 of 16 193 to 188, of 64 forward 310 to 297; 32768 of 64, 2048 x 1024, forward 234 and 237).
  constexpr int GROUP = GROUPS && !one_group(DIR) && !is_weight(DIR) ? 2 : 4;
  const int group = tile / (GROUP * g.tiles_j), in_group = tile % (GROUP * g.tiles_j);
  const int rows = tiles_i - GROUP * group < GROUP ? tiles_i - GROUP * group : GROUP;
  int64_t i0 = int64_t(GROUP * group + in_group % rows) * TI, j0 = int64_t(in_group / rows) * TJ;
  int32_t first_row = 0;
  if constexpr (GROUPS && one_group(DIR)) {
    if (is_weight(DIR)) g.part_k = ((g.K + TA::STEP - 1) / TA::STEP + g.parts - 1) / g.parts * TA::STEP;
  } else if constexpr (GROUPS) {
    // From here on the operands are the group's.
    Group e;
    if constexpr (is_weight(DIR)) {
      e = group_at(g, group_index);
      g.a = static_cast<const char*>(g.a) + e.begin * g.lda * TA::ES;
      g.b = static_cast<const char*>(g.b) + e.begin * g.ldb * TA::ES;
      g.c = static_cast<char*>(g.c) + group_index * g.I * g.ldc * (g.grad32 ? 4 : TA::ES);
      g.K = e.rows;
      const int32_t steps = (e.rows + TA::STEP - 1) / TA::STEP;
      g.part_k = int64_t((steps + g.parts - 1) / g.parts) * TA::STEP;
    } else {
      e = group_of_tile<TI>(g, scan, GROUP * group + in_group % rows);
      i0 = int64_t(e.tile) * TI;
      g.spread_from = e.index * 5;
      first_row = e.begin;
      g.a = static_cast<const char*>(g.a) + e.begin * g.lda * TA::ES;
      g.b = static_cast<const char*>(g.b) + e.index * g.b_group * TA::ES;
      if (DIR == DDP_LINEAR_FORWARD && g.bias != nullptr) g.bias = static_cast<const char*>(g.bias) + e.index * g.J * TA::ES;
      if constexpr (DIR == DDP_LINEAR_FORWARD || DIR == DDP_LINEAR_BACKWARD_INPUT) {
        g.c = static_cast<char*>(g.c) + e.begin * g.ldc * TA::ES;
        if (g.z != nullptr) g.z = static_cast<char*>(g.z) + e.begin * g.ldz * TA::ES;
      }
      g.I = e.rows;
    }
  }
  constexpr bool kMany = GROUPS && !one_group(DIR);
  // Rows of all groups' C, and this one's first.
  const int64_t all_i = !kMany ? g.I : is_weight(DIR) ? g.I * g.groups : g.rows;
  const int64_t first_i = !kMany ? 0 : is_weight(DIR) ? group_index * g.I : first_row;
  int64_t k0 = part * g.part_k, k1 = k0 + g.part_k < g.K ? k0 + g.part_k : g.K;
  if constexpr (GROUPS) {
    if (k0 > k1) k0 = k1;  // a part of a short group
  }
  const int steps = int((k1 - k0 + TA::STEP - 1) / TA::STEP);

  const int lane = int(threadIdx.x) & 63, all_wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int wave = WK > 1 ? all_wave % (WI * WJ) : all_wave, wk = WK > 1 ? all_wave / (WI * WJ) : 0;
  const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
  // A group's last tile is seldom full. A wave whose rows lie all behind the
  // group loads its share and multiplies nothing: the other wave of its SIMD has
  // the matrix unit to itself.
  const bool idle = i0 + wi >= g.I;
  f32x16 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b) acc[a][b] = f32x16{};
  // The bias gradient is the sum of A's rows, whose fragments pass through
  // the registers here anyway: every block of a tile row adds up its share of
  // the steps (the first column of waves does), on vector units that the
  // products leave idle. A pass of its own over dz took 12 us at 8192 x 2048.
  const int tile_j = in_group / rows;
  const bool sum_rows = DIR == DDP_LINEAR_BACKWARD_WEIGHT && g.row_sums != nullptr && wave % WJ == 0;
  float row_sum[FI] = {};

  const int terms = has_terms(DIR) ? g.terms : 1;
#pragma unroll 1
  for (int term = 0; term < (has_terms(DIR) ? terms : 1); ++term) {
    if (steps <= 0) break;
    if (has_terms(DIR) && term > 0) __syncthreads();  // every wave is done with the first term's operands
    LA la;
    LB lb;
    la.init(static_cast<const char*>(g.a) + (has_terms(DIR) ? term * g.term : 0), g.lda, g.I, g.K, i0, k0, k1, g.a_room);
    lb.init(g.b, g.ldb, g.J, g.K, j0, k0, k1, g.b_room);
    if constexpr (TURNED) {
      if (g.spread && (k1 - k0) % TA::STEP == 0) {
        const int32_t first = int32_t(uint32_t(g.spread_from + in_group / rows) * 11u % uint32_t(steps));
        la.turn_to(first, steps);
        lb.turn_to(first, steps);
      } else {
        la.until = lb.until = 0;
      }
    }
    u32x4 fa[2][FI], fb[2][FJ];
    // Fragment m of quarter s: B's first, then A's.
    const auto read_one = [&](const char* stage, int s, int to, int m) {
      if (m < FJ)
        fb[to][m] = TB::fragment(stage + TA::BYTES, wj, m, s + 4 * wk, lane);
      else
        fa[to][m - FJ] = TA::fragment(stage, wi, m - FJ, s + 4 * wk, lane);
    };
    // The products of the fragments in `from`, with step(m) after the m-th. The
    // order written is the schedule: left to itself, the compiler moves the
    // LDS reads down to the products that use them (8192 x 2048 x 8192 forward:
    // 212 us against 205).
    const auto products = [&](int from, auto&& step) {
#pragma unroll
      for (int m = 0; m < FI * FJ; ++m) {
        const int a = m / FJ, b = m % FJ;
        acc[a][b] = multiply<DT>(fb[from][b], fa[from][a], acc[a][b]);
        __builtin_amdgcn_sched_barrier(0);
        step(m);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Every wave is done with the stage read last, and every wave's loads of
    // the next one have landed.
    constexpr int P = FI * FJ, Q = SB / WK / 32, LOADS = TA::N + TB::N;
    const auto turn = [&](auto more_on_their_way) {
      if constexpr (PIPE > 1)  // what went to LDS had to be there
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      else if constexpr (STAGES > 2 && decltype(more_on_their_way)::value)  // loads of the steps behind the next one
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((STAGES - 2) * LOADS) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
    };
    const auto load_one = [&](char* stage, int n, auto full, auto set) __attribute__((always_inline)) {
      if (n < TA::N)
        la.template load<decltype(full)::value, decltype(set)::value>(stage, n);
      else
        lb.template load<decltype(full)::value, decltype(set)::value>(stage + TA::BYTES, n - TA::N);
    };
    const auto end_loads = [&](auto set) __attribute__((always_inline)) {
      la.template end<decltype(set)::value>();
      lb.template end<decltype(set)::value>();
    };
    const auto commit = [&](char* stage, auto set) __attribute__((always_inline)) {
      la.template commit<decltype(set)::value>(stage);
      lb.template commit<decltype(set)::value>(stage + TA::BYTES);
    };
    int until_rows = tile_j;  // steps until the next one whose rows this block adds up
    // One step: its products, with the loads of a later step into `to` under way
    // (LOADING; FULL: all of whose terms exist), and the next step's first reads from
    // `next` (MORE). With loads of two steps in registers, those of this call go to
    // `set`, and the other set's to LDS.
    const auto one_step = [&](const char* stage, const char* next, char* to, auto more, auto loading, auto full, auto set)
                              __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value, LOADING = decltype(loading)::value;
      constexpr std::integral_constant<int, PIPE == 2 ? 1 - decltype(set)::value : 0> ready{};
      if (GROUPS && !is_weight(DIR) && idle) {
        if (LOADING) {
#pragma unroll
          for (int n = 0; n < LOADS; ++n) load_one(to, n, full, set);
          end_loads(set);
          commit(to, ready);
        }
        if (MORE) turn(loading);
        return;
      }
      const bool sum_now = DIR == DDP_LINEAR_BACKWARD_WEIGHT && until_rows == 0;
      if (DIR == DDP_LINEAR_BACKWARD_WEIGHT) until_rows = sum_now ? g.tiles_j - 1 : until_rows - 1;
      const auto add_rows = [&](int from) {
        if (DIR == DDP_LINEAR_BACKWARD_WEIGHT && sum_now && sum_rows) {
#pragma unroll
          for (int a = 0; a < FI; ++a) row_sum[a] += sum_of<DT>(fa[from][a]);
        }
      };
      // All but the last 32 bytes of k: after each product a read of the next
      // 32 bytes, or one of the loads.
#pragma unroll
      for (int s = 0; s < Q - 1; ++s) {
        products(s & 1, [&](int m) __attribute__((always_inline)) {
#pragma unroll
          for (int r = 0; r < FI + FJ; ++r)
            if (r * P / (FI + FJ) == m) read_one(stage, s + 1, (s + 1) & 1, r);
          if (LOADING) {
#pragma unroll
            for (int n = 0; n < LOADS; ++n)
              if (n * P / LOADS == m && s == 0) load_one(to, n, full, set);
            if (s == 1 && m == P / 2) end_loads(set);
          }
        });
        add_rows(s & 1);
      }
      if (LOADING) commit(to, ready);
      if (MORE) turn(loading);
      products((Q - 1) & 1, [&](int m) __attribute__((always_inline)) {
        if (MORE) {
#pragma unroll
          for (int r = 0; r < FI + FJ; ++r)
            if (r * P / (FI + FJ) == m) read_one(next, 0, 0, r);
        }
      });
      add_rows((Q - 1) & 1);
      // The sums are there before anything else looks at them. The compiler's own
      // waits fell short where two last steps, on an even and an odd count, both end in
      // copies of the sums: it counted the instructions that a branch jumps over.
      if constexpr (PIPE == 2 && !MORE) {
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+v"(acc[0][0]));
#pragma unroll
        for (int m = 1; m < FI * FJ; ++m) asm volatile("" : "+v"(acc[m / FJ][m % FJ]));
      }
    };
    constexpr std::integral_constant<bool, true> yes{};
    constexpr std::integral_constant<bool, false> no{};
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, PIPE - 1> odd{};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {  // past the last step: zeros
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load_one(lds + s * STAGE, n, no, even);
      end_loads(even);
    }
    if constexpr (PIPE == 2) {
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load_one(lds, n, no, odd);
      end_loads(odd);
    }
    commit(lds, even);
    turn(yes);
#pragma unroll
    for (int m = 0; m < FI + FJ; ++m) read_one(lds, 0, 0, m);
    // Two steps at a time while the next ones are whole: the stages are fixed
    // then, and a wave's instructions between its products are few. (They
    // issue one by one, some 5 cycles each, while its products wait.)
    int t = 0;
    if constexpr (PIPE == 2) {
      // Loads run two steps ahead, past the last step too: they read as zeros.
      const int whole_steps = int((k1 - k0) / TA::STEP);
      for (; t + 3 < whole_steps; t += 2) {
        one_step(lds, lds + STAGE, lds + STAGE, yes, yes, yes, even);
        one_step(lds + STAGE, lds, lds, yes, yes, yes, odd);
      }
      for (; t + 2 < steps; t += 2) {
        one_step(lds, lds + STAGE, lds + STAGE, yes, yes, no, even);
        one_step(lds + STAGE, lds, lds, yes, yes, no, odd);
      }
      if (t + 1 < steps) {
        one_step(lds, lds + STAGE, lds + STAGE, yes, yes, no, even);
        one_step(lds + STAGE, nullptr, nullptr, no, no, no, odd);
      } else {
        one_step(lds, nullptr, nullptr, no, no, no, even);
      }
    } else if constexpr (STAGES == 2) {
      const int whole_steps = int((k1 - k0) / TA::STEP);
      for (; t + 2 < whole_steps; t += 2) {
        one_step(lds, lds + STAGE, lds + STAGE, yes, yes, yes, even);
        one_step(lds + STAGE, lds, lds, yes, yes, yes, even);
      }
      for (; t + 1 < steps; ++t) {
        char* const next = lds + ((t & 1) ^ 1) * STAGE;
        one_step(lds + (t & 1) * STAGE, next, next, yes, yes, no, even);
      }
      one_step(lds + (t & 1) * STAGE, nullptr, nullptr, no, no, no, even);
    } else {
      // The last steps' turns wait for all that is on its way, the first of them
      // longer than it has to.
      int at = 0;  // t % STAGES
      const auto after = [](int s) { return s + 1 == STAGES ? 0 : s + 1; };
      for (; t + STAGES - 1 < steps; ++t, at = after(at))
        one_step(lds + at * STAGE, lds + after(at) * STAGE, lds + (at == 0 ? STAGES - 1 : at - 1) * STAGE, yes, yes, no, even);
      for (; t + 1 < steps; ++t, at = after(at)) one_step(lds + at * STAGE, lds + after(at) * STAGE, nullptr, yes, no, no, even);
      one_step(lds + at * STAGE, nullptr, nullptr, no, no, no, even);
      if (steps < STAGES) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // zeros past the last step may still be on their way
    }
  }

  if (DIR == DDP_LINEAR_BACKWARD_WEIGHT && sum_rows) {
#pragma unroll
    for (int a = 0; a < FI; ++a) {
      const float r = row_sum[a] + __shfl_xor(row_sum[a], 32);  // both halves of k
      const int64_t i = i0 + wi + 32 * a + lane;
      if (lane < 32 && i < g.I) g.row_sums[(int64_t(part) * g.tiles_j + tile_j) * all_i + first_i + i] = r;
    }
  }

  if (kMany && is_weight(DIR) && g.K == 0 && g.accumulate && g.parts == 1) return;  // nothing is added

  if constexpr (WK > 1) {  // the first waves add up what the others have
    __syncthreads();
    f32x16* const sums = reinterpret_cast<f32x16*>(lds) + lane;
#pragma unroll
    for (int a = 0; a < FI; ++a)
#pragma unroll
      for (int b = 0; b < FJ; ++b)
        if (wk > 0) sums[(((wk - 1) * WI * WJ + wave) * FI * FJ + a * FJ + b) * 64] = acc[a][b];
    __syncthreads();
    if (wk == 0) {
      for (int o = 0; o < WK - 1; ++o)
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
          for (int b = 0; b < FJ; ++b) acc[a][b] += sums[((o * WI * WJ + wave) * FI * FJ + a * FJ + b) * 64];
    }
  }

  if constexpr (is_head(DIR)) {
    if (steps > 0) __syncthreads();  // every wave is done with the operands in LDS
    head_outputs<DT, DIR, TI, TJ, WI, WJ, WK, STAGES>(g, acc, lds, i0, j0, wi, wj, wave, wk, lane, tile_j);
    return;
  }

  // The outputs leave by rows: a wave writes 32 rows of its sums to LDS (a
  // lane holds four neighbouring columns of one row at a time) and reads them
  // back eight columns to a lane, so that loads and stores cover whole lines.
  // Each wave has its own part of LDS.
  if (steps > 0) __syncthreads();  // every wave is done with the operands there
  if (WK > 1 && wk > 0) return;
  float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  constexpr int LPR = 4 * FJ;        // lanes per row
  constexpr int RPP = 64 / LPR;      // rows per pass
  if constexpr (GROUPS && is_weight(DIR)) {
    if (g.parts == 1 && i0 + TI <= g.I && j0 + TJ <= g.J) {
      const auto outputs = [&](auto nt) __attribute__((always_inline)) {
        constexpr bool NT = decltype(nt)::value;
        if (DT == DDP_BF16 && !g.grad32)
          weight_outputs<DDP_BF16, NT, DIR, FI, FJ, PITCH>(g, acc, mine, i0 + wi, j0 + wj, lane);
        else
          weight_outputs<DDP_FP32, NT, DIR, FI, FJ, PITCH>(g, acc, mine, i0 + wi, j0 + wj, lane);
      };
      if (g.stream_c)
        outputs(std::integral_constant<bool, true>{});
      else
        outputs(std::integral_constant<bool, false>{});
      return;
    }
  }
  const int64_t i_lane = i0 + wi + lane / LPR;
  const int64_t j = j0 + wj + lane % LPR * 8;
  const int n = g.J - j >= 8 ? 8 : g.J - j > 0 ? int(g.J - j) : 0;
  float bias[8] = {};
  if (DIR == DDP_LINEAR_FORWARD && g.bias != nullptr && n > 0) load8<DT>(g.bias, j, n, bias);
  // Rows leave in batches of two passes, so that their values and what they
  // need besides stay in registers next to the sums. What a batch needs is
  // loaded before the stores of the batch before it: a later load would wait
  // for those, too. One copy of the code serves all batches.
  constexpr int BATCH = 2, ROWS = BATCH * RPP, PER = 32 / ROWS;
  const bool whole = i0 + TI <= g.I && j0 + TJ <= g.J;
  const int64_t jp = (g.J + 7) / 8 * 8;
  Extra x[BATCH];
  if (g.parts == 1 && whole) {
#pragma unroll
    for (int p = 0; p < BATCH; ++p) load_extra<DT, DIR>(g, i_lane + p * RPP, j, 8, x[p]);
  }
#pragma unroll 1
  for (int it = 0; it < FI * PER; ++it) {
    if (it % PER == 0) {
#pragma unroll
      for (int c = 0; c < FI; ++c) {
        if (c != it / PER) continue;
#pragma unroll
        for (int b = 0; b < FJ; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(mine + (lane & 31) * PITCH + 32 * b + 8 * q + 4 * (lane >> 5)) =
                f32x4{acc[c][b][4 * q], acc[c][b][4 * q + 1], acc[c][b][4 * q + 2], acc[c][b][4 * q + 3]};
      }
      __builtin_amdgcn_wave_barrier();
    }
    float v[BATCH][8];
#pragma unroll
    for (int p = 0; p < BATCH; ++p) {
      const float* src = mine + (it % PER * ROWS + lane / LPR + p * RPP) * PITCH + lane % LPR * 8;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(src), hi = *reinterpret_cast<const f32x4*>(src + 4);
      for (int k = 0; k < 4; ++k) v[p][k] = lo[k], v[p][4 + k] = hi[k];
    }
    __builtin_amdgcn_wave_barrier();
    const int64_t i = i_lane + it * ROWS;
    if (g.parts > 1) {
      if (kMany && DIR == DDP_LINEAR_FORWARD && part == 0) {  // the join does not know a row's group
#pragma unroll
        for (int p = 0; p < BATCH; ++p)
          for (int k = 0; k < 8; ++k) v[p][k] += bias[k];
      }
#pragma unroll
      for (int p = 0; p < BATCH; ++p)
        if (i + p * RPP < g.I && n > 0) store8<DDP_FP32>(g.partial, (part * all_i + first_i + i + p * RPP) * jp + j, 8, v[p]);
    } else if (whole) {
      const auto values = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < BATCH; ++p) before_store<DT, DIR, decltype(act)::value>(g, i + p * RPP, j, 8, v[p], x[p], bias);
      };
      switch (g.act) {
#define DDP_ACT_CASE(A)                           \
  case A:                                         \
    values(std::integral_constant<int, A>{});     \
    break;
        DDP_ACT_CASE(DDP_ACT_RELU)
        DDP_ACT_CASE(DDP_ACT_GELU)
        DDP_ACT_CASE(DDP_ACT_GELU_TANH)
        DDP_ACT_CASE(DDP_ACT_SILU)
#undef DDP_ACT_CASE
        default:
          values(std::integral_constant<int, DDP_ACT_NONE>{});
      }
      if (it + 1 < FI * PER) {
#pragma unroll
        for (int p = 0; p < BATCH; ++p) load_extra<DT, DIR>(g, i + ROWS + p * RPP, j, 8, x[p]);
      }
#pragma unroll
      for (int p = 0; p < BATCH; ++p) store_output<DT, DIR>(g, i + p * RPP, j, 8, v[p]);
    } else if (n > 0) {
#pragma unroll 1
      for (int p = 0; p < BATCH; ++p) {
        float w[8];
        for (int k = 0; k < 8; ++k) w[k] = p == 0 ? v[0][k] : v[1][k];
        if (i + p * RPP >= g.I) continue;
        Extra e;
        load_extra<DT, DIR>(g, i + p * RPP, j, n, e);
        finish<DT, DIR>(g, i + p * RPP, j, n, w, e, bias);
      }
    }
  }
}

// Joins the parts of every sum, in their order, and finishes the outputs. What
// the outputs need, and four parts at a time, are loaded before they are used: a
// launch has two blocks per CU or fewer, which hide little latency (257 x 640
// weight gradient: 4.0 us against 6.5 a part at a time; 1037 x 1023 forward in 7
// parts, 42 MB with residual and outputs: 9 either way).
template <int DT, int DIR, bool GROUPS = false>
__global__ __launch_bounds__(kThreads) void k_linear_join(LinearArgs g) {
  int64_t first = 0, end = g.I;   // the rows that are anybody's
  if constexpr (GROUPS && one_group(DIR)) {
    g.I = end = bound_at(g, 1);
  } else if constexpr (GROUPS) {
    __shared__ int32_t most[kThreads / 64];
    int32_t bound = 0;
    for (int32_t e = int32_t(threadIdx.x); e <= g.groups; e += kThreads) bound = larger(bound, bound_at(g, e));
    bound = scan_lanes(bound, larger);
    if ((threadIdx.x & 63) == 63) most[threadIdx.x >> 6] = bound;
    __syncthreads();
    first = bound_at(g, 0);
    end = larger(larger(most[0], most[1]), larger(most[2], most[3]));
  }
  const int64_t jv = (g.J + 7) / 8;
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= g.I * jv) return;
  const int64_t i = at / jv, j = at % jv * 8;
  if (GROUPS && (i < first || i >= end)) return;
  const int n = g.J - j >= 8 ? 8 : int(g.J - j);
  float bias[8] = {};
  if (DIR == DDP_LINEAR_FORWARD && g.bias != nullptr) load8<DT>(g.bias, j, n, bias);
  Extra x;
  load_extra<DT, DIR>(g, i, j, n, x);
  float v[8] = {};
  for (int p = 0; p < g.parts; p += 4) {
    float w[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u)  // past the last part: the last again, unused
      load8<DDP_FP32>(g.partial, (int64_t(p + u < g.parts ? p + u : g.parts - 1) * g.I + i) * jv * 8 + j, 8, w[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      for (int k = 0; k < 8; ++k) v[k] += p + u < g.parts ? w[u][k] : 0.0f;
  }
  finish<DT, DIR>(g, i, j, n, v, x, bias);
}

// ---------------------------------------------------------------- the bias gradient

// db (+)= sums of the columns of `rows` rows at src: the partial sums that the
// weight gradient's blocks leave (or dz itself, where there are none of those
// because the layer has no inputs). Four threads share a column.
template <int SRC, int DST>
__global__ __launch_bounds__(kThreads) void k_column_sums(const void* src, int64_t ld, int64_t rows, int64_t N, void* db,
                                                          int accumulate, int64_t begin) {
  __shared__ float sums[4][64];
  const int c = int(threadIdx.x) & 63, group = int(threadIdx.x) >> 6;
  const int64_t col = begin + int64_t(blockIdx.x) * 64 + c;
  float s = 0.0f;
  if (col < N) {
#pragma unroll 4
    for (int64_t r = group; r < rows; r += 4) s += Ops<SRC>::load1(src, r * ld + col);
  }
  sums[group][c] = s;
  __syncthreads();
  if (group != 0 || col >= N) return;
  s = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
  if (accumulate) s += Ops<DST>::load1(db, col);
  Ops<DST>::store1(db, col, DST == DDP_BF16 ? round_bf16(s) : s);
}

}  // namespace
}  // namespace ddp
