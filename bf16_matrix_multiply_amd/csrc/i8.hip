// Rows to 8-bit integers with a scale each: code = 127 x / max |x| rounded to
// nearest, ties to even, and scale = max |x| / 127 in float32.
//
// The quotient decides a code, and with 16-bit inputs it often is a half exactly
// (x half of the row's largest value gives 63.5), so it is rounded from the real
// quotient a / b, a = 127 x, b = max |x|, and not from a product with a rounded
// reciprocal: t = a r with r = 1 / b rounded, then t + r (a - t b), the residual
// exact by one fused multiply-add, is the correctly rounded quotient (Markstein).
// 16-bit inputs make a exact, and a quotient that is no half is further from one
// than float32's steps there; for float32 inputs a is held as two floats, and the
// sign of what remains after the quotient breaks what looks like a tie.
//
// Both a and b are multiplied by the same power of two before, so that the
// reciprocal is a normal number for every finite row.
//
// Bound by memory and, in between, by the arithmetic of the codes: 8192 x 8192 bf16 38-43
// us = 4.7-5.3 TB/s, 4095 x 4096 f16 14.7 us = 3.4 TB/s, one row of 16384 4.8 us.
#include "ffn.h"

namespace bmm {
namespace {

constexpr int kKept = 8;   // pieces of 8 values that a thread keeps between the two passes

template <int ET>
__device__ __forceinline__ int code_of(float x, float b, float r, float power) {
  const float xs = x * power, a = 127.f * xs;
  const float t = a * r;
  float q = __builtin_fmaf(__builtin_fmaf(-t, b, a), r, t);
  if constexpr (ET != BMM_ELEM_F32) return int(__builtin_rintf(q));
  const float low = __builtin_fmaf(127.f, xs, -a);   // 127 x = a + low
  q = __builtin_fmaf(__builtin_fmaf(-q, b, a) + low, r, q);
  const float past = __builtin_fmaf(-q, b, a) + low;   // the real quotient is q + past / b
  float k = __builtin_rintf(q);
  const float d = q - k;   // a half, and rounded to the even side of it?
  if (d == 0.5f && past > 0.f) k += 1.f;
  if (d == -0.5f && past < 0.f) k -= 1.f;
  return int(k);
}

// P threads a row: 64 (a wave, four rows a workgroup), 256 or 1024, so that a row is
// read once, in pieces that its threads keep; longer rows are read twice.
template <int ET, int P>
__global__ __launch_bounds__(P < 256 ? 256 : P) void quantize_kernel(int8_t* __restrict__ codes,
                                                                     float* __restrict__ scales,
                                                                     const void* __restrict__ src,
                                                                     int64_t rows, int64_t K,
                                                                     int64_t ld) {
  constexpr int kRowsHere = P < 256 ? 256 / P : 1;
  const int64_t row = int64_t(blockIdx.x) * kRowsHere + threadIdx.x / P;
  const int t = threadIdx.x % P;
  const int64_t pieces = row < rows ? K / 8 : 0, rounds = (K / 8 + kKept * P - 1) / (kKept * P);
  Eight<ET> x[kKept];
  auto load = [&](int64_t round) {
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int64_t c = (round * kKept + i) * P + t;
      if (c < pieces) x[i].load(src, row * ld + 8 * c);
      else x[i].zero();
    }
  };
  uint32_t top = 0;   // largest magnitude, as bits: ordered like the values, NaN above all
  for (int64_t round = 0; round < rounds; ++round) {
    load(round);
#pragma unroll
    for (int i = 0; i < kKept; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = umax(top, __builtin_bit_cast(uint32_t, x[i][e]) & 0x7fffffffu);
  }
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) top = umax(top, uint32_t(__shfl_xor(int(top), d, kWave)));
  if constexpr (P > kWave) {
    __shared__ uint32_t of_wave[P / kWave];
    if (t % kWave == 0) of_wave[t / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < P / kWave; ++w) top = umax(top, of_wave[w]);
  }
  if (row >= rows) return;
  const bool finite = top < 0x7f800000u;
  if (t == 0)
    scales[row] = finite ? __builtin_bit_cast(float, top) / 127.f : __builtin_nanf("");
  const int expo = 127 - int(top >> 23);
  const int held = expo < -100 ? -100 : expo > 100 ? 100 : expo;
  const float power = __builtin_bit_cast(float, uint32_t(127 + held) << 23);
  const float b = __builtin_bit_cast(float, top) * power;
  const float r = finite && top ? 1.f / b : 0.f;
  for (int64_t round = 0; round < rounds; ++round) {
    if (rounds > 1) load(round);
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int64_t c = (round * kKept + i) * P + t;
      if (c >= pieces) continue;
      uint32_t o[2] = {0, 0};
      if (finite && top) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e / 4] |= (uint32_t(code_of<ET>(x[i][e], b, r, power)) & 255u) << (8 * (e % 4));
      }
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2*>(codes + row * K + 8 * c) = u32x2{o[0], o[1]};
    }
  }
}

template <int ET>
hipError_t quantize(int8_t* codes, float* scales, const void* src, int64_t rows, int64_t K,
                    int64_t ld, hipStream_t s) {
  auto launch = [&](auto kern, int64_t threads) {
    const int64_t each = threads < 256 ? 256 / threads : 1;
    const int64_t most = each << 21;   // rows of one launch: 2^31 threads (2^32 are refused)
    for (int64_t first = 0; first < rows; first += most) {
      const int64_t n = rows - first < most ? rows - first : most;
      hipLaunchKernelGGL(kern, dim3(unsigned((n + each - 1) / each)),
                         dim3(unsigned(threads < 256 ? 256 : threads)), 0, s, codes + first * K,
                         scales + first,
                         static_cast<const char*>(src) + first * ld * (ET == BMM_ELEM_F32 ? 4 : 2),
                         n, K, ld);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (K <= 64 * 8 * kKept) return launch(quantize_kernel<ET, 64>, 64);
  if (K <= 256 * 8 * kKept) return launch(quantize_kernel<ET, 256>, 256);
  return launch(quantize_kernel<ET, 1024>, 1024);
}

}  // namespace

hipError_t launch_i8_quantize(int8_t* codes, float* scales, const void* src, int64_t rows, int64_t K,
                              int64_t ld, int elem_type, hipStream_t s) {
  switch (elem_type) {
    case BMM_ELEM_F32: return quantize<BMM_ELEM_F32>(codes, scales, src, rows, K, ld, s);
    case BMM_ELEM_F16: return quantize<BMM_ELEM_F16>(codes, scales, src, rows, K, ld, s);
    default: return quantize<BMM_ELEM_BF16>(codes, scales, src, rows, K, ld, s);
  }
}

}  // namespace bmm
