// Host-side argument checks for every entry point. Pure C++ (no HIP calls),
// so each rejection path runs without a GPU.
#pragma once

#include <stdint.h>
#include <string>

#include "../../include/bmm.h"

namespace bmm {

struct Status {
  int code = BMM_OK;
  std::string msg;
  bool ok() const { return code == BMM_OK; }
};

// Sets the message bmm_last_error returns on this thread (defined with the
// entry points).
void set_last_error(const std::string& msg);

Status check_pack(const uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                  int64_t K, int64_t ld_src, int32_t atom_rows, int32_t atom_k);

Status check_pack_kmajor(const uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                         int64_t K, int64_t ld_src, int32_t atom_rows,
                         int32_t atom_k);

Status check_box(const void* dst, const void* src, const bmm_box_desc* d);

// Store (elem_type 0) or add reduction (a bmm_elem_type) into a global box;
// `what` prefixes the messages.
Status check_box_store(const void* dst, const void* img, const bmm_box_desc* d,
                       int32_t elem_type, const char* what);

Status check_mma(const float* D, const uint32_t* A, const uint32_t* B, const float* C,
                 int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep, int32_t dtype,
                 int32_t kernel, int32_t atom_k);

// Split count actually used: min(splits, number of 32-value K steps).
int64_t splitk_effective(int64_t K_rep, int32_t atom_k, int32_t splits);

Status check_splitk(const float* D, const uint32_t* A, const uint32_t* B, const float* C,
                    int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep, int32_t dtype,
                    int32_t atom_k, int32_t splits, const void* workspace,
                    int64_t workspace_bytes);

// Feed-forward operators (validate_ffn.cpp).
Status check_gated(const uint16_t* H, const uint16_t* G, const uint16_t* U, const uint16_t* X,
                   const uint32_t* Wg, const uint32_t* Wu, const bmm_gated_desc* d);
// Extents alone; `what` prefixes the messages.
Status check_gated_desc(const bmm_gated_desc* d, const char* what);
Status check_gated_backward(const uint16_t* dX, const uint16_t* dWg, const uint16_t* dWu,
                            const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                            const uint16_t* X, const uint32_t* Wg, const uint32_t* Wu,
                            const bmm_gated_desc* d, const void* workspace,
                            int64_t workspace_bytes, int64_t need);
// Bytes of a 4-bit operand's codes and scales, or -1 for invalid extents.
int64_t mx4_codes_bytes(int64_t batch, int64_t rows, int64_t K);
int64_t mx4_scales_bytes(int64_t batch, int64_t rows, int64_t K);
// A product of bmm_ffn_plan (4 bits: F columns).
Status check_ffn_plan(int32_t product, const bmm_gated_desc& d);
// Quantise (`mat` is read) or dequantise (`mat` is written).
Status check_mx4_convert(const void* mat, const uint8_t* codes, const uint8_t* scales,
                         int64_t batch, int64_t rows, int64_t K, int64_t ld, int32_t elem_type,
                         const char* what);
// Product (B1 null) or gated product (B0 = Wg, B1 = Wu).
Status check_mx4_product(const void* D, const uint8_t* A, const uint8_t* As, const uint8_t* B0,
                         const uint8_t* B0s, const uint8_t* B1, const uint8_t* B1s, bool gated,
                         int64_t batch, int64_t M, int64_t N, int64_t K, int64_t ld, int32_t act,
                         int32_t elem_type);

// Products by groups (validate_grouped.cpp). Extents alone; `what` prefixes the messages.
Status check_grouped_desc(const bmm_grouped_desc* d, bool gated, const char* what);
// Y = X W^T (W1, Y1 and Y2 null), or H, G and U from Wg and Wu.
Status check_grouped(const uint16_t* Y, const uint16_t* Y1, const uint16_t* Y2, const uint16_t* X,
                     const uint32_t* W, const uint32_t* W1, const int32_t* ends,
                     const bmm_grouped_desc* d, bool gated);
struct GroupedGrads {
  const uint16_t *dX, *dW, *dW1;      // dW1: gated only
  const uint16_t *dY, *G, *U, *X;     // gated: dY is dH
  const uint32_t *W, *W1;
};
Status check_grouped_backward(const GroupedGrads& g, const int32_t* ends, const bmm_grouped_desc* d,
                              bool gated, const void* workspace, int64_t workspace_bytes,
                              int64_t need);
Status check_i8_quantize(const void* src, const int8_t* codes, const float* scales, int64_t batch,
                         int64_t rows, int64_t K, int64_t ld, int32_t elem_type);
// Product (W1 null) or gated product.
Status check_i8_product(const void* D, const int8_t* A, const float* sa, const uint32_t* W,
                        const float* sw, const uint32_t* W1, const float* sw1, const int32_t* ends,
                        const bmm_i8_desc* d, bool gated);
Status check_group_plan(int32_t product, const bmm_grouped_desc& d);

// Largest image (bytes) one box repeat may stage through LDS.
constexpr int64_t kBoxImageLimit = 65536;

}  // namespace bmm
