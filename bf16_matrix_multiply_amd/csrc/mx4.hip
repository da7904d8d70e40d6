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
#include "ffn.h"

namespace bmm {
namespace {

constexpr int kThreads = 256;

// One wave: 16 rows x 512 K values. Four lanes share a block, 8 values each, and
// eight lanes read or write 128 neighbouring bytes of a row (16-bit values). Bound
// by memory: 8192 x 8192 bf16 to 4 bits and back 59 us = 5.8 TB/s (a copy: 5.1); with
// a block a lane, 64 lanes met 64 lines and it took 83 us.
struct Lane {
  int part, g0, row;   // 8 values of the block; first block of a pair; row of eight
  __device__ __forceinline__ Lane() {
    const int lane = threadIdx.x & (kWave - 1);
    part = lane & 3;
    g0 = (lane >> 2) & 1;
    row = lane >> 3;
  }
};

// The largest of four neighbouring lanes' values.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = umax(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xb1, 0xf, 0xf, true)));   // lanes 1 0 3 2
  return umax(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4e, 0xf, 0xf, true)));  // 2 3 0 1
}

template <int ET>
__global__ __launch_bounds__(kThreads) void quantize_kernel(uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            const void* __restrict__ src,
                                                            int64_t rows, int64_t K, int64_t ld,
                                                            int64_t r16, int64_t n) {
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kWave;
  if (w >= n) return;
  const Lane lane;
  const int64_t s128 = (K + 127) / 128, s512 = (K + 511) / 512;
  const int64_t q = w % s512, r = w / s512;   // r: 16-row group, batches one after another
  const int64_t b = r / r16;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = 8 * half + lane.row;
    const int64_t row = 16 * (r % r16) + i;
    Eight<ET> x[2][4];
#pragma unroll
    for (int pair = 0; pair < 2; ++pair)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t k = 128 * (4 * q + t) + 32 * (2 * pair + lane.g0);
        if (row < rows && k < K) x[pair][t].load(src, (b * rows + row) * ld + k + 8 * lane.part);
        else x[pair][t].zero();
      }
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      const int g = 2 * pair + lane.g0;
      uint32_t word = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const Eight<ET>& v = x[pair][t];
        uint32_t top = 0;   // largest magnitude, as bits: ordered like the values, NaN above all
#pragma unroll
        for (int e = 0; e < 8; ++e)
          top = umax(top, __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu);
        top = quad_max(top);
        const int expo = int(top >> 23) - 2;
        const uint32_t byte = top >= 0x7f800000u ? 255u : uint32_t(expo > 0 ? expo : 0);
        word |= byte << (8 * t);
        uint32_t o = 0;
        if (byte != 255u) {
          const float scale = mx4_scale(byte);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0], v[1], scale, 0);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2], v[3], scale, 1);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4], v[5], scale, 2);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6], v[7], scale, 3);
        }
        const int64_t step = 4 * q + t;
        if (step < s128)
          *reinterpret_cast<uint32_t*>(codes + (r * s128 + step) * 1024 + 256 * g + 16 * i +
                                       4 * lane.part) = o;
      }
      if (lane.part == 0) reinterpret_cast<uint32_t*>(scales)[w * 64 + 16 * g + i] = word;
    }
  }
}

template <int ET>
__device__ __forceinline__ void store_eight(void* dst, int64_t at, const float (&v)[8]) {
  if constexpr (ET == BMM_ELEM_F32) {
    float* p = static_cast<float*>(dst) + at;
    store16f_nt(p, f32x4{v[0], v[1], v[2], v[3]});
    store16f_nt(p + 4, f32x4{v[4], v[5], v[6], v[7]});
  } else {
    constexpr int DT = ET == BMM_ELEM_BF16 ? kBF16 : kF16;
    __builtin_nontemporal_store(u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]),
                                      pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])},
                                reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + at));
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
  const Lane lane;
  const int64_t s128 = (K + 127) / 128, s512 = (K + 511) / 512;
  const int64_t q = w % s512, r = w / s512;
  const int64_t b = r / r16;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = 8 * half + lane.row;
    const int64_t row = 16 * (r % r16) + i;
    if (row >= rows) continue;
    uint32_t c[2][4], word[2];
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      const int g = 2 * pair + lane.g0;
      word[pair] = reinterpret_cast<const uint32_t*>(scales)[w * 64 + 16 * g + i];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t step = 4 * q + t;
        if (step < s128)
          c[pair][t] = *reinterpret_cast<const uint32_t*>(codes + (r * s128 + step) * 1024 +
                                                          256 * g + 16 * i + 4 * lane.part);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int pair = 0; pair < 2; ++pair) {
        const int64_t k = 128 * (4 * q + t) + 32 * (2 * pair + lane.g0);
        if (k >= K) continue;
        const uint32_t byte = (word[pair] >> (8 * t)) & 255u;
        const float scale = byte == 255u ? __builtin_nanf("") : mx4_scale(byte);
        float v[8];
        const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[pair][t], 1.f, 0);
        const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[pair][t], 1.f, 1);
        const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[pair][t], 1.f, 2);
        const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[pair][t], 1.f, 3);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[e] = p0[e] * scale;
          v[2 + e] = p1[e] * scale;
          v[4 + e] = p2[e] * scale;
          v[6 + e] = p3[e] * scale;
        }
        store_eight<ET>(dst, (b * rows + row) * ld + k + 8 * lane.part, v);
      }
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
