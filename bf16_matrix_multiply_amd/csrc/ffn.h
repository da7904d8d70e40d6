// Internal launchers and device helpers of the feed-forward operators (the
// gated block, its backward pass and the 4-bit forms). Arguments are already
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bmm.h"
#include "common.h"

namespace bmm {

// Operand element of a product: kF16 and kBF16 of common.h, or 4-bit floats
// with a scale for every 32 K values.
enum : int { kMX4 = 2 };

// How a product is made: by tiles of so many rows x columns (gated: columns of
// both weights), or by the kernel for few rows (ffn_skinny.h).
enum TileSize : int {
  kTile128 = BMM_TILE_128X128,
  kTile256x128 = BMM_TILE_256X128,
  kTile256x192 = BMM_TILE_256X192,
  kTile256 = BMM_TILE_256X256,
  kSkinny = BMM_TILE_FEW_ROWS
};

// One product D = A * B^T on MFMA tiles. Which fields count depends on how
// the operands lie in memory and on the epilogue (ffn_tile.h).
struct TileArgs {
  const void* a;
  const void* b0;
  const void* b1;
  const uint8_t* as;   // 4-bit operands: scales of a, b0 and b1
  const uint8_t* bs0;
  const uint8_t* bs1;
  void* d;             // output; gated: H
  void* d1;            // gated: G (may be null); store: second block of rows
  void* d2;            // gated: U
  int64_t batch, M, N, K;   // rows, output columns, summed values
  int64_t lda, ldb, ldd;    // elements between rows (row-major operands)
  int64_t a_bs, b_bs;       // elements between batches (4-bit codes: bytes)
  int64_t as_bs, bs_bs;     // bytes between batches of scales
  int64_t b_sum;            // transposed packed B: summed values of each of its two sources
                            // (a multiple of 32) ...
  int64_t b_rows;           // ... and how many of them exist (the rest count as zero)
  // store: rows r < rows0 go to d, rows row1 <= r < row1 + rows0 to d1, others nowhere
  int64_t rows0, row1;
  int tile;                 // a TileSize
  int act;
  int out_type;             // bmm_elem_type: F32, F16 or BF16
  // split sum (store only): split s of `splits` takes slabs [s n / S, (s + 1) n / S) of the
  // n slabs and writes float32 to part + s * part_floats + (b * M + row) * N + column
  int splits;
  float* part;
  int64_t part_floats;
  const float* rescale;     // f16 store: the sums are multiplied by this power of two (null: 1)
};

// ---- launchers ----
hipError_t launch_gated(const TileArgs& a, int dtype, hipStream_t s);
// dG = dH U act'(G), dU = dH act(G), rounded to the operands' type, as (rows, 2 Fp) row-major
// [dG | dU], Fp = F rounded up to 32 with zeros in between. f16: multiplied by a power of
// two that suits its range; *rescale receives the one that undoes it, and peaks (so many
// words, gated_peaks) is scratch memory.
int64_t gated_peaks(int64_t rows, int64_t F);
hipError_t launch_gated_slopes(uint16_t* dgu, const uint16_t* dh, const uint16_t* g,
                               const uint16_t* u, int64_t rows, int64_t F, int64_t ld, int dtype,
                               int act, uint32_t* peaks, float* rescale, hipStream_t s);
hipError_t launch_gated_dx(const TileArgs& a, int dtype, hipStream_t s);
hipError_t launch_gated_dw(const TileArgs& a, int dtype, hipStream_t s);
hipError_t launch_mx4_quantize(uint8_t* codes, uint8_t* scales, const void* src, int64_t batch,
                               int64_t rows, int64_t K, int64_t ld, int elem_type, hipStream_t s);
hipError_t launch_mx4_dequantize(void* dst, const uint8_t* codes, const uint8_t* scales,
                                 int64_t batch, int64_t rows, int64_t K, int64_t ld,
                                 int elem_type, hipStream_t s);
hipError_t launch_mx4_mma(const TileArgs& a, hipStream_t s);
hipError_t launch_mx4_gated(const TileArgs& a, hipStream_t s);

// How a product of M rows, N columns (gated: of both weights) and so many slabs is cut.
struct TilePlan {
  int tile, splits;
  double ns;   // what the model expects
};
TilePlan plan_tiles(int64_t batch, int64_t M, int64_t N, int64_t slabs, bool may_split);
// The same for a product that has the kernel for few rows and no splits.
int plan_forward(int64_t batch, int64_t M, int64_t N, int64_t slabs);

// ---- activations ----
// exp is the hardware's 2^x (1 ulp) of x log2(e); the product's rounding makes
// the result good to about |x| 2^-24, well inside a half step of the 16-bit
// outputs (2^-8 and 2^-11). 1 / x is the hardware's (1 ulp). The hardware's 2^x
// gives 0 below 2^-126, so small values are made as the square of 2^(x/2):
// bf16 holds float32's subnormals.
__device__ __forceinline__ float exp_half(float x) {   // exp(x / 2)
  return __builtin_amdgcn_exp2f(x * 0.72134752044448170368f);
}
// exp(x) / (1 + exp(x)); exp is held below 2^60, where the quotient is 1.
__device__ __forceinline__ float sigmoid(float x) {
  const float r = __builtin_amdgcn_exp2f(__builtin_fminf(x * 0.72134752044448170368f, 30.f));
  const float e = r * r;
  return e * __builtin_amdgcn_rcpf(1.f + e);
}

// Phi(x) = erfc(-x / sqrt 2) / 2. erfc(z), z >= 0, as t exp(-z^2 + P(t)) with
// t = 1 / (1 + z / 2): the Chebyshev fit of Press et al., Numerical Recipes,
// "erfcc", whose error is below 1.2e-7 of the value everywhere, so the far
// negative tail of gelu keeps its relative accuracy.
__device__ __forceinline__ float normal_cdf(float x) {
  const float z = __builtin_fabsf(x) * 0.70710678118654752440f;
  const float t = __builtin_amdgcn_rcpf(1.f + 0.5f * z);
  float q = 0.17087277f;
  q = __builtin_fmaf(q, t, -0.82215223f);
  q = __builtin_fmaf(q, t, 1.48851587f);
  q = __builtin_fmaf(q, t, -1.13520398f);
  q = __builtin_fmaf(q, t, 0.27886807f);
  q = __builtin_fmaf(q, t, -0.18628806f);
  q = __builtin_fmaf(q, t, 0.09678418f);
  q = __builtin_fmaf(q, t, 0.37409196f);
  q = __builtin_fmaf(q, t, 1.00002368f);
  q = __builtin_fmaf(q, t, -1.26551223f);
  const float r = exp_half(q - z * z);
  const float half = 0.5f * t * r * r;
  return x < 0.f ? half : 1.f - half;
}

// 2 sqrt(2 / pi) (x + 0.044715 x^3): 0.5 (1 + tanh z) is sigmoid(2 z).
__device__ __forceinline__ float gelu_tanh_arg(float x) {
  return 1.59576912160573071f * (x + 0.044715f * x * x * x);
}

template <int ACT>
__device__ __forceinline__ float act(float x) {
  if constexpr (ACT == BMM_ACT_SILU) return x * sigmoid(x);
  if constexpr (ACT == BMM_ACT_GELU) return x * normal_cdf(x);
  if constexpr (ACT == BMM_ACT_GELU_TANH) return x * sigmoid(gelu_tanh_arg(x));
  return x <= 0.f ? 0.f : x;   // relu; a NaN stays
}

// act(x) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_and_slope(float x, float& a, float& slope) {
  if constexpr (ACT == BMM_ACT_SILU) {
    const float s = sigmoid(x);
    a = x * s;
    slope = __builtin_fmaf(a, 1.f - s, s);
  } else if constexpr (ACT == BMM_ACT_GELU) {
    const float p = normal_cdf(x);
    a = x * p;
    const float r = exp_half(-0.5f * x * x);
    slope = __builtin_fmaf(x, 0.39894228040143267794f * r * r, p);
  } else if constexpr (ACT == BMM_ACT_GELU_TANH) {
    const float s = sigmoid(gelu_tanh_arg(x));
    a = x * s;
    // beyond |x| = 64 s (1 - s) is 0; the square is held there so that 0 is not
    // multiplied by an infinity
    const float c = __builtin_fminf(__builtin_fabsf(x), 64.f);
    slope = __builtin_fmaf(a * (1.f - s), 1.59576912160573071f + 0.21406445f * (c * c), s);
  } else {
    a = x <= 0.f ? 0.f : x;
    slope = x > 0.f ? 1.f : 0.f;
  }
}

// ---- rounding to 16 bits (nearest even), two values a word ----
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == kBF16) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    const v2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    const v2 v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int DT>
__device__ __forceinline__ float half_bits_to_f32(uint32_t bits16) {
  if constexpr (DT == kBF16) {
    return __builtin_bit_cast(float, bits16 << 16);
  } else {
    return float(__builtin_bit_cast(_Float16, uint16_t(bits16)));
  }
}

// The power of two a scale byte stands for (0: 2^-127, below the normal floats).
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

}  // namespace bmm
