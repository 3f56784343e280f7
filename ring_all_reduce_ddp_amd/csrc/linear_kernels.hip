// A linear layer's products on the matrix instructions, each with what
// follows it in the same pass (ddp_train.h):
//
//   forward          z = x w^T + bias,  y = act(z) + residual
//   input gradient   dx = (dz w) * act'(z) + add
//   weight gradient  dw (+)= dz^T x,  db (+)= sum of dz's rows
//
// All three are C[i][j] = sum_k A(i, k) B(j, k). What differs is how an
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
#include <algorithm>
#include <cmath>
#include <new>

#include "train_internal.h"

namespace ddp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
#define DDP_LDS __attribute__((address_space(3)))

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
};

constexpr bool a_along(int dir) { return dir != DDP_LINEAR_BACKWARD_WEIGHT; }
constexpr bool b_along(int dir) { return dir == DDP_LINEAR_FORWARD; }

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
  if constexpr (DIR == DDP_LINEAR_BACKWARD_WEIGHT) {
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
  if constexpr (DIR == DDP_LINEAR_BACKWARD_WEIGHT) {
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
  if (DIR == DDP_LINEAR_BACKWARD_WEIGHT && g.grad32)
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
    if (ALONG) return (row / (256 / SB)) & (CPR - 1);
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
// whole. The descriptor ends with the operand, so a chunk past it reads as
// zeros; a row of C's side past the operand repeats the last one (its
// products are not stored).
template <class TL, bool ALONG, int THREADS>
struct DirectLoader {
  const char* p;        // the tile at the current step
  int64_t advance;      // bytes per step
  int32_t left;         // chunks from p to the operand's end
  int32_t k_left;       // terms left
  uint32_t off[TL::N];  // of this lane's chunks, in bytes from p
  int32_t wave;
  u32x4 desc;

  // First term, within the step, of this lane's n-th chunk.
  __device__ __forceinline__ int k_of(int n) const {
    const int q = (n * (THREADS / 64) + wave) * 64 + (int(threadIdx.x) & 63);
    return ALONG ? TL::col_of(q) * TL::V : TL::row_of(q);
  }
  __device__ __forceinline__ void init(const void* base, int64_t ld, int64_t side, int64_t K, int64_t s0, int64_t k0, int64_t k1) {
    const int lane = int(threadIdx.x) & 63;
    wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t rows = ALONG ? side : K, cols = ALONG ? K : side;
    const int64_t start = ALONG ? s0 * ld + k0 : k0 * ld + s0;
    p = static_cast<const char*>(base) + start * TL::ES;
    left = int32_t(((rows - 1) * ld + cols - start) / TL::V);
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
  template <bool FULL>
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
  __device__ __forceinline__ void end() {
    p += advance;
    left -= int32_t(advance / 16);
    k_left -= TL::STEP;
    describe();
  }
  __device__ __forceinline__ void commit(char*) {}
};

// Through registers, for operands of any alignment whose rows have a chunk's
// elements at least. Every chunk is one load at its element's alignment,
// without a branch that writes its registers (with one, each load is waited
// for before the next starts: twice as slow). A chunk that runs over the
// end of its row is loaded from as far back as it fits and shifted into place
// when it goes to LDS, zeros following; one past the sum's end is shifted out
// whole.
template <int DT, class TL, bool ALONG, int THREADS>
struct AnyLoader {
  static constexpr int kWidth = TL::CPR * TL::V;  // "across": elements of a row in the tile
  const char* p;         // the tile at the current step
  int64_t row_bytes;
  int32_t k_left;        // terms left
  int32_t width;         // "across": elements of a row that exist
  bool shifted;          // some chunk of the step is to be shifted
  int64_t off[TL::N];    // of this lane's chunks, in bytes from p
  int32_t shift[TL::N];  // elements to shift out
  u32x4 x[TL::N];

  static __device__ __forceinline__ int chunk(int n) { return n * THREADS + int(threadIdx.x); }
  __device__ __forceinline__ void init(const void* base, int64_t ld, int64_t side, int64_t, int64_t s0, int64_t k0, int64_t k1) {
    row_bytes = ld * TL::ES;
    p = static_cast<const char*>(base) + (ALONG ? s0 * ld + k0 : k0 * ld + s0) * TL::ES;
    k_left = int32_t(k1 - k0);
    width = side - s0 < kWidth ? int32_t(side - s0) : kWidth;
#pragma unroll
    for (int n = 0; n < TL::N; ++n) {
      const int row = TL::row_of(chunk(n)), col = TL::col_of(chunk(n)) * TL::V;
      const int64_t r = ALONG && s0 + row >= side ? side - 1 - s0 : row;
      const int back = !ALONG && col + TL::V > width ? col + TL::V - width : 0;
      off[n] = r * row_bytes + (col - back) * TL::ES;  // from p, perhaps negative; never before the row
      shift[n] = back;
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void load(const char*, int n) {
    int64_t o = off[n];
    if (!FULL && k_left < TL::STEP) {
      const int row = TL::row_of(chunk(n)), col = TL::col_of(chunk(n)) * TL::V;
      if (ALONG) {
        shift[n] = col + TL::V > k_left ? col + TL::V - k_left : 0;
        o -= shift[n] * TL::ES;
      } else if (row >= k_left) {
        o -= (row - (k_left - 1)) * row_bytes;
        shift[n] = TL::V;
      }
    }
    if constexpr (DT == DDP_FP32)
      x[n] = load_at<false, u32x4_at4>(p + o, 0);
    else
      x[n] = load_at<false, u32x4_at2>(p + o, 0);
  }
  __device__ __forceinline__ void end() {
    shifted = k_left < TL::STEP || (!ALONG && width < kWidth);
    p += ALONG ? TL::ROW : TL::STEP * row_bytes;
    k_left -= TL::STEP;
  }
  __device__ __forceinline__ void commit(char* lds) {
    if (shifted) {
#pragma unroll
      for (int n = 0; n < TL::N; ++n) {
        const int bits = shift[n] * TL::ES * 8;
        const unsigned __int128 v = __builtin_bit_cast(unsigned __int128, x[n]);
        x[n] = bits < 128 ? __builtin_bit_cast(u32x4, v >> bits) : u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int n = 0; n < TL::N; ++n) *reinterpret_cast<u32x4*>(lds + chunk(n) * 16) = x[n];
  }
};

// Element by element, for rows shorter than a chunk.
template <int DT, class TL, bool ALONG, int THREADS>
struct ShortLoader {
  const void* base;
  int64_t ld, side, s0, k, k1;
  u32x4 x[TL::N];

  __device__ __forceinline__ void init(const void* b, int64_t ld_, int64_t side_, int64_t, int64_t s0_, int64_t k0, int64_t k1_) {
    base = b, ld = ld_, side = side_, s0 = s0_, k = k0, k1 = k1_;
  }
  template <bool FULL>
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
  __device__ __forceinline__ void end() { k += TL::STEP; }
  __device__ __forceinline__ void commit(char* lds) {
#pragma unroll
    for (int n = 0; n < TL::N; ++n) *reinterpret_cast<u32x4*>(lds + (n * THREADS + int(threadIdx.x)) * 16) = x[n];
  }
};

enum Loading { kDirect, kAny, kShort };
template <int LOAD, int DT, class TL, bool ALONG, int THREADS>
using LoaderOf = std::conditional_t<LOAD == kDirect, DirectLoader<TL, ALONG, THREADS>,
                                    std::conditional_t<LOAD == kAny, AnyLoader<DT, TL, ALONG, THREADS>,
                                                       ShortLoader<DT, TL, ALONG, THREADS>>>;

// ---------------------------------------------------------------- the product

// Tile TI x TJ of C by WI x WJ waves.
template <int DT, int DIR, int TI, int TJ, int WI, int WJ, int LOAD>
__global__ __launch_bounds__(WI * WJ * 64, 2) void k_linear(LinearArgs g) {
  constexpr int THREADS = WI * WJ * 64;
  constexpr int FI = TI / WI / 32, FJ = TJ / WJ / 32;  // 32 x 32 products per wave
  // Steps of 128 bytes of k, one on its way while one is multiplied. (Four
  // stages of 64 bytes, three of them on their way, ran 15 % slower: twice the
  // barriers. 4 waves with 128 x 128 products each read a third less from LDS
  // but have nobody to fill their waits: as fast without outputs to speak of,
  // 8192 x 8192 x 2048 input gradient through gelu_tanh 303 us against 269.)
  constexpr int SB = 128;
  using TA = Tile<DT, a_along(DIR), TI, SB, THREADS>;
  using TB = Tile<DT, b_along(DIR), TJ, SB, THREADS>;
  using LA = LoaderOf<LOAD, DT, TA, a_along(DIR), THREADS>;
  using LB = LoaderOf<LOAD, DT, TB, b_along(DIR), THREADS>;
  constexpr int STAGE = TA::BYTES + TB::BYTES;
  constexpr int PITCH = 32 * FJ + 4;  // floats; the outputs' way through LDS
  static_assert(WI * WJ * 32 * PITCH * 4 <= 2 * STAGE, "the outputs' rows fit");
  __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];

  // Blocks go to the 8 XCDs in turn: XCD x takes the tiles of eighth x, in
  // groups of 4 tile rows, so that blocks that share operands share an L2
  // (8192 x 8192 x 2048 forward with z kept: 254 us; groups of 8, 258, of 1,
  // 283; tiles in the blocks' order, 299).
  const int tiles = g.tiles_i * g.tiles_j;
  const int at = g.begin + int(blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8);
  if (at >= tiles * g.parts) return;
  const int part = at / tiles, tile = at % tiles;
  constexpr int GROUP = 4;
  const int group = tile / (GROUP * g.tiles_j), in_group = tile % (GROUP * g.tiles_j);
  const int rows = g.tiles_i - GROUP * group < GROUP ? g.tiles_i - GROUP * group : GROUP;
  const int64_t i0 = int64_t(GROUP * group + in_group % rows) * TI, j0 = int64_t(in_group / rows) * TJ;
  const int64_t k0 = part * g.part_k, k1 = k0 + g.part_k < g.K ? k0 + g.part_k : g.K;
  const int steps = int((k1 - k0 + TA::STEP - 1) / TA::STEP);

  const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
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

  if (steps > 0) {
    LA la;
    LB lb;
    la.init(g.a, g.lda, g.I, g.K, i0, k0, k1);
    lb.init(g.b, g.ldb, g.J, g.K, j0, k0, k1);
    u32x4 fa[2][FI], fb[2][FJ];
    // Fragment m of quarter s: B's first, then A's.
    const auto read_one = [&](const char* stage, int s, int to, int m) {
      if (m < FJ)
        fb[to][m] = TB::fragment(stage + TA::BYTES, wj, m, s, lane);
      else
        fa[to][m - FJ] = TA::fragment(stage, wi, m - FJ, s, lane);
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
    const auto turn = [&] {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
    };
    constexpr int P = FI * FJ, Q = SB / 32, LOADS = TA::N + TB::N;
    const auto load_one = [&](char* stage, int n, auto full) __attribute__((always_inline)) {
      if (n < TA::N)
        la.template load<decltype(full)::value>(stage, n);
      else
        lb.template load<decltype(full)::value>(stage + TA::BYTES, n - TA::N);
    };
    int until_rows = tile_j;  // steps until the next one whose rows this block adds up
    // One step: its products, with the next step's loads under way (MORE; FULL:
    // all of whose terms exist).
    const auto one_step = [&](const char* stage, char* next, auto more, auto full) __attribute__((always_inline)) {
      constexpr bool MORE = decltype(more)::value;
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
          if (MORE) {
#pragma unroll
            for (int n = 0; n < LOADS; ++n)
              if (n * P / LOADS == m && s == 0) load_one(next, n, full);
            if (s == 1 && m == P / 2) {
              la.end();
              lb.end();
            }
          }
        });
        add_rows(s & 1);
      }
      if (MORE) {
        la.commit(next);
        lb.commit(next + TA::BYTES);
        turn();
      }
      products((Q - 1) & 1, [&](int m) __attribute__((always_inline)) {
        if (MORE) {
#pragma unroll
          for (int r = 0; r < FI + FJ; ++r)
            if (r * P / (FI + FJ) == m) read_one(next, 0, 0, r);
        }
      });
      add_rows((Q - 1) & 1);
    };
    constexpr std::integral_constant<bool, true> yes{};
    constexpr std::integral_constant<bool, false> no{};
#pragma unroll
    for (int n = 0; n < LOADS; ++n) load_one(lds, n, no);
    la.end();
    lb.end();
    la.commit(lds);
    lb.commit(lds + TA::BYTES);
    turn();
#pragma unroll
    for (int m = 0; m < FI + FJ; ++m) read_one(lds, 0, 0, m);
    // Two steps at a time while the next ones are whole: the stages are fixed
    // then, and a wave's instructions between its products are few. (They
    // issue one by one, some 5 cycles each, while its products wait.)
    const int whole_steps = int((k1 - k0) / TA::STEP);
    int t = 0;
    for (; t + 2 < whole_steps; t += 2) {
      one_step(lds, lds + STAGE, yes, yes);
      one_step(lds + STAGE, lds, yes, yes);
    }
    for (; t + 1 < steps; ++t) one_step(lds + (t & 1) * STAGE, lds + ((t & 1) ^ 1) * STAGE, yes, no);
    one_step(lds + (t & 1) * STAGE, nullptr, no, no);
  }

  if (DIR == DDP_LINEAR_BACKWARD_WEIGHT && sum_rows) {
#pragma unroll
    for (int a = 0; a < FI; ++a) {
      const float r = row_sum[a] + __shfl_xor(row_sum[a], 32);  // both halves of k
      const int64_t i = i0 + wi + 32 * a + lane;
      if (lane < 32 && i < g.I) g.row_sums[(int64_t(part) * g.tiles_j + tile_j) * g.I + i] = r;
    }
  }

  // The outputs leave by rows: a wave writes 32 rows of its sums to LDS (a
  // lane holds four neighbouring columns of one row at a time) and reads them
  // back eight columns to a lane, so that loads and stores cover whole lines.
  // Each wave has its own part of LDS.
  if (steps > 0) __syncthreads();  // every wave is done with the operands there
  float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  constexpr int LPR = 4 * FJ;        // lanes per row
  constexpr int RPP = 64 / LPR;      // rows per pass
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
#pragma unroll
      for (int p = 0; p < BATCH; ++p)
        if (i + p * RPP < g.I && n > 0) store8<DDP_FP32>(g.partial, (part * g.I + i + p * RPP) * jp + j, 8, v[p]);
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
template <int DT, int DIR>
__global__ __launch_bounds__(kThreads) void k_linear_join(LinearArgs g) {
  const int64_t jv = (g.J + 7) / 8;
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= g.I * jv) return;
  const int64_t i = at / jv, j = at % jv * 8;
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

// ---------------------------------------------------------------- few rows

// The forward product for up to kFewRows rows of x (tokens of an answer): w
// is read once and each value meets every row's, so the bound is w's bytes. A
// block takes 4 rows of w, its waves every fourth kilobyte of each; x stays in
// the caches. (1 row, 8192 x 2048 bf16: 6 us, 5.6 TB/s with w in the Infinity
// Cache. The whole call, without and with tiles: 1 and 2 rows 7.0 us and 10.4
// there, 7.0 and 10.8 at 4096 x 4096, fp32 12 and 26. 4 rows gain where outputs are
// few, 9.9 and 14.0 at 2048 x 8192, fp32 16 and 26 at 4096 x 4096, and lose where
// they are many, 16.5 and 10.5 at 8192 x 2048, 50 and 12.5 at 32000 x 1024.)
constexpr int kFewRows = 4, kFewOuts = 4;

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

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `blocks` blocks in launches of kMaxGrid at most: launch(first block, grid).
template <class F>
void launch_blocks(int64_t blocks, F&& launch) {
  for (int64_t b = 0; b < blocks; b += kMaxGrid) launch(b, dim3(unsigned(std::min(blocks - b, kMaxGrid))));
}

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

// How a product is cut: the tile's side (256 needs direct loads), and in how
// many parts the sum. Up to kFewRows rows of a forward product go without
// tiles.
struct Cut {
  bool few = false;
  int tile = 128;
  int32_t parts = 1;
  int64_t part_k = 0;
};

// The cut with the least time by a rough model in cycles. Its constants were
// fitted to the times of 250 products of 5 to 8192 rows, 64 to 8192 columns
// and terms, odd and even, on MI355X, each cut in up to 27 ways: the cut it
// picks takes 1.9 % longer than the best of them in the mean, 31 % at worst.
// A tile's step (128 bytes of k) takes `step` cycles of a CU that its blocks
// fill and `alone` of a block by itself, its outputs `ends`; parts cost a
// launch, a round each, and their bytes.
Cut cut_by_model(int dir, int32_t I, int32_t J, int32_t K, int dtype, bool direct) {
  Cut best;
  if (dir == DDP_LINEAR_FORWARD && I <= kFewRows) {
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
  const int32_t step = 128 / elem_bytes(dtype), steps = std::max(1, up(K, step));
  float least = INFINITY;
  for (int k = 0; k < n_shapes; ++k) {
    const Shape& sh = shapes[dtype == DDP_BF16][direct][k];
    const int64_t tiles = int64_t(up(I, sh.tile)) * up(J, sh.tile);
    for (int32_t want : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32}) {
      if (want > 1 && (want > steps / 2 || tiles * want > 4 * kCus * sh.fit)) break;
      const int32_t per = up(steps, want), parts = up(steps, per), on_cu = up(tiles * parts, kCus);
      float t = std::max(float(up(on_cu, sh.fit)) * (kStart + float(per) * sh.alone),
                         kStart + float(on_cu) * (float(per) * sh.step + sh.ends));
      if (parts > 1) t += kJoin + float(parts) * kPart + float(parts + 2) * float(I) * float(J) * (4 / kBytesPerCycle);
      if (t >= least) continue;
      least = t;
      best.tile = sh.tile;
      best.parts = parts;
      best.part_k = int64_t(per) * step;
    }
  }
  return best;
}

// The same, remembered per thread for the sizes seen last: the model takes a
// microsecond or two, and a call asks it three times.
Cut cut_of(int dir, int64_t I, int64_t J, int64_t K, int dtype, bool direct) {
  struct Seen {
    int64_t key[4] = {-1, -1, -1, -1};
    Cut cut;
  };
  static thread_local Seen seen[64];
  const int64_t key[4] = {I, J, K, dir * 4 + dtype * 2 + int(direct)};
  const uint64_t h = (uint64_t(I) * 31 + uint64_t(J) * 7 + uint64_t(K)) * 8 + uint64_t(key[3]);
  Seen& s = seen[(h ^ (h >> 7)) % 64];
  if (!std::equal(key, key + 4, s.key)) {
    s.cut = cut_by_model(dir, int32_t(I), int32_t(J), int32_t(K), dtype, direct);
    std::copy(key, key + 4, s.key);
  }
  return s.cut;
}

int64_t partial_bytes(const Cut& c, int64_t I, int64_t J) {
  return c.parts > 1 ? round_up(int64_t(c.parts) * I * round_up(J, 8) * 4, 256) : 0;
}
// The bias gradient's partial rows, one per part and tile column.
int64_t bias_bytes(const Cut& c, int64_t I, int64_t J) { return round_up(c.parts * div_up(J, c.tile) * I * 4, 256); }

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
  // Direct loads need whole, aligned chunks: the contiguous index of each
  // operand a multiple of a chunk, offsets within a tile below 2^32 bytes and
  // the whole operand below 2^31 chunks.
  const auto aligned = [&](const void* p, int64_t ld, int64_t rows, int64_t contiguous) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % V == 0 && contiguous % V == 0 && ld <= (int64_t(1) << 21) &&
           rows * (ld / V) < (int64_t(1) << 31);
  };
  const bool direct = aligned(g.a, g.lda, a_along(DIR) ? g.I : g.K, a_along(DIR) ? g.K : g.I) &&
                      aligned(g.b, g.ldb, b_along(DIR) ? g.J : g.K, b_along(DIR) ? g.K : g.J);
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
  const bool from16 = K == 0 && dtype == DDP_BF16;
  launch_blocks(div_up(N, 64), [&](int64_t begin, dim3 grid) {
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, sums, sums_ld, sums_rows, N, db, accumulate, begin * 64);
    };
    if (grad_dtype == DDP_BF16)
      from16 ? launch(k_column_sums<DDP_BF16, DDP_BF16>) : launch(k_column_sums<DDP_FP32, DDP_BF16>);
    else
      from16 ? launch(k_column_sums<DDP_BF16, DDP_FP32>) : launch(k_column_sums<DDP_FP32, DDP_FP32>);
  });
  DDP_HIP_TRY(hipGetLastError(), "ddp_linear_backward_weight: bias launch");
  return DDP_OK;
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
