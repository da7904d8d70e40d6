// Microscaled 4-bit floats (OCP Microscaling Formats v1.0, MXFP4): to 4 bits
// and back.
//
// A block is 32 neighbouring K values of a row. Its scale is 2^e with
// e = floor(log2 of its largest magnitude) - 2 (2 = the exponent of the 4-bit
// format's largest value 6 = 1.5 * 2^2), held as the byte e + 127, at least 0;
// each value becomes x / 2^e rounded to nearest (ties to the even code) among
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, at most 6 in magnitude. A
// block that holds a NaN or an infinity gets the scale byte 255 (NaN).
//
// Layout: 16 rows x 128 K values are 1 KB in the order in which the 16x16x128
// MFMA's lanes take them (lane 16 g + i: row i, the block of K values 32 g ..),
// and the scales of 16 rows x 512 K values are 64 words, one a lane, whose four
// bytes are the lane's blocks of four 128-value steps. Rows up to the next
// multiple of 16 and K up to the next multiple of 512 are padded with zeros.
#include <type_traits>

#include "ffn.h"

namespace bmm {
namespace {

constexpr int kThreads = 256;

// The 32 values of a block as float32.
template <int ET>
__device__ __forceinline__ void load_block(const void* src, int64_t at, float (&v)[32]) {
  if constexpr (ET == BMM_ELEM_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4 x = load16f(static_cast<const float*>(src) + at + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = x[e];
    }
  } else {
    constexpr int DT = ET == BMM_ELEM_BF16 ? kBF16 : kF16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(src) + at + 8 * i);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[8 * i + 2 * w] = half_bits_to_f32<DT>(x[w] & 0xffffu);
        v[8 * i + 2 * w + 1] = half_bits_to_f32<DT>(x[w] >> 16);
      }
    }
  }
}

// One wave: 16 rows x 512 K values, a lane four blocks of its row.
template <int ET>
__global__ __launch_bounds__(kThreads) void quantize_kernel(uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            const void* __restrict__ src,
                                                            int64_t rows, int64_t K, int64_t ld,
                                                            int64_t r16, int64_t n) {
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kWave;
  if (w >= n) return;
  const int lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
  const int64_t s128 = (K + 127) / 128, s512 = (K + 511) / 512;
  const int64_t q = w % s512, r = w / s512;   // r: 16-row group, batches one after another
  const int64_t b = r / r16, row = 16 * (r % r16) + i;
  uint32_t word = 0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t step = 4 * q + t, k = 128 * step + 32 * g;
    if (step >= s128) break;
    u32x4 out = {0, 0, 0, 0};
    if (row < rows && k < K) {
      float v[32];
      load_block<ET>(src, (b * rows + row) * ld + k, v);
      uint32_t top = 0;   // largest magnitude, as bits: ordered like the values, NaN above all
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint32_t m = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
      const int expo = int(top >> 23) - 2;
      const uint32_t byte = top >= 0x7f800000u ? 255u : uint32_t(expo > 0 ? expo : 0);
      word |= byte << (8 * t);
      if (byte != 255u) {
        const float scale = mx4_scale(byte);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t o = 0;
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * d], v[8 * d + 1], scale, 0);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * d + 2], v[8 * d + 3], scale, 1);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * d + 4], v[8 * d + 5], scale, 2);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * d + 6], v[8 * d + 7], scale, 3);
          out[d] = o;
        }
      }
    }
    *reinterpret_cast<u32x4*>(codes + (r * s128 + step) * 1024 + 16 * lane) = out;
  }
  reinterpret_cast<uint32_t*>(scales)[w * 64 + lane] = word;
}

template <int ET>
__device__ __forceinline__ void store_block(void* dst, int64_t at, const float (&v)[32]) {
  if constexpr (ET == BMM_ELEM_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      store16f(static_cast<float*>(dst) + at + 4 * i,
               f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]});
  } else {
    constexpr int DT = ET == BMM_ELEM_BF16 ? kBF16 : kF16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + at + 8 * i) =
          u32x4{pack2<DT>(v[8 * i], v[8 * i + 1]), pack2<DT>(v[8 * i + 2], v[8 * i + 3]),
                pack2<DT>(v[8 * i + 4], v[8 * i + 5]), pack2<DT>(v[8 * i + 6], v[8 * i + 7])};
  }
}

template <int ET>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(void* __restrict__ dst,
                                                              const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              int64_t rows, int64_t K, int64_t ld,
                                                              int64_t r16, int64_t n) {
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kWave;
  if (w >= n) return;
  const int lane = threadIdx.x & (kWave - 1), i = lane & 15, g = lane >> 4;
  const int64_t s128 = (K + 127) / 128, s512 = (K + 511) / 512;
  const int64_t q = w % s512, r = w / s512;
  const int64_t b = r / r16, row = 16 * (r % r16) + i;
  if (row >= rows) return;
  const uint32_t word = reinterpret_cast<const uint32_t*>(scales)[w * 64 + lane];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t step = 4 * q + t, k = 128 * step + 32 * g;
    if (k >= K) break;
    const u32x4 c = *reinterpret_cast<const u32x4*>(codes + (r * s128 + step) * 1024 + 16 * lane);
    const uint32_t byte = (word >> (8 * t)) & 255u;
    const float scale = byte == 255u ? __builtin_nanf("") : mx4_scale(byte);
    float v[32];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[d], 1.f, 0);
      const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[d], 1.f, 1);
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[d], 1.f, 2);
      const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[d], 1.f, 3);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[8 * d + e] = p0[e] * scale;
        v[8 * d + 2 + e] = p1[e] * scale;
        v[8 * d + 4 + e] = p2[e] * scale;
        v[8 * d + 6 + e] = p3[e] * scale;
      }
    }
    store_block<ET>(dst, (b * rows + row) * ld + k, v);
  }
}

}  // namespace

hipError_t launch_mx4_quantize(uint8_t* codes, uint8_t* scales, const void* src, int64_t batch,
                               int64_t rows, int64_t K, int64_t ld, int elem_type, hipStream_t s) {
  const int64_t r16 = (rows + 15) / 16, n = batch * r16 * ((K + 511) / 512);
  const int64_t blocks = (n + kThreads / kWave - 1) / (kThreads / kWave);
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  auto kern = elem_type == BMM_ELEM_F32   ? quantize_kernel<BMM_ELEM_F32>
              : elem_type == BMM_ELEM_F16 ? quantize_kernel<BMM_ELEM_F16>
                                          : quantize_kernel<BMM_ELEM_BF16>;
  hipLaunchKernelGGL(kern, dim3(unsigned(blocks)), dim3(kThreads), 0, s, codes, scales, src, rows,
                     K, ld, r16, n);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(void* dst, const uint8_t* codes, const uint8_t* scales,
                                 int64_t batch, int64_t rows, int64_t K, int64_t ld,
                                 int elem_type, hipStream_t s) {
  const int64_t r16 = (rows + 15) / 16, n = batch * r16 * ((K + 511) / 512);
  const int64_t blocks = (n + kThreads / kWave - 1) / (kThreads / kWave);
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  auto kern = elem_type == BMM_ELEM_F32   ? dequantize_kernel<BMM_ELEM_F32>
              : elem_type == BMM_ELEM_F16 ? dequantize_kernel<BMM_ELEM_F16>
                                          : dequantize_kernel<BMM_ELEM_BF16>;
  hipLaunchKernelGGL(kern, dim3(unsigned(blocks)), dim3(kThreads), 0, s, dst, codes, scales, rows,
                     K, ld, r16, n);
  return hipGetLastError();
}

}  // namespace bmm
