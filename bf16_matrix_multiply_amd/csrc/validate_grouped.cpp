// Argument checks of the products by groups and of 8-bit integers.
#include "validate_ffn.h"

namespace bmm {
namespace {

constexpr int64_t kMaxGroups = 4096;   // every workgroup reads them all
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;      // ends are int32
constexpr int64_t kMaxI8K = int64_t(1) << 17;             // below it

Status check_ends(const int32_t* ends, const char* what) {
  if (!ends) return failw(what, BMM_EINVAL, "ends is null");
  if (reinterpret_cast<uintptr_t>(ends) & 3)
    return failw(what, BMM_EALIGN, "ends must be 4-byte aligned");
  return Status{};
}

Rows flat(const void* p, int64_t bytes, const char* name) { return {p, 1, bytes, 0, name}; }

}  // namespace

Status check_grouped_desc(const bmm_grouped_desc* d, bool gated, const char* what) {
  if (!d) return failw(what, BMM_EINVAL, "null descriptor");
  if (d->dtype != BMM_F16 && d->dtype != BMM_BF16)
    return failw(what, BMM_EINVAL, "dtype %lld is neither BMM_F16 nor BMM_BF16", d->dtype);
  if (gated && (d->act < BMM_ACT_SILU || d->act > BMM_ACT_RELU))
    return failw(what, BMM_EINVAL, "act %lld is not a bmm_act", d->act);
  if (!gated && d->act != 0) return failw(what, BMM_EINVAL, "act %lld without a gate", d->act);
  if (d->zero_tail != 0 && d->zero_tail != 1)
    return failw(what, BMM_EINVAL, "zero_tail %lld is neither 0 nor 1", d->zero_tail);
  if (d->groups < 0 || d->T < 0 || d->N < 0 || d->K < 0)
    return failw(what, BMM_EINVAL, "negative extent");
  if (d->groups < 1) return failw(what, BMM_EINVAL, "there must be a group");
  if (d->groups > kMaxGroups || d->T > kMaxRows || d->N > kMaxF || d->K > kMaxLd)
    return failw(what, BMM_EINVAL,
                 "extent too large (groups <= 4096, T < 2^31, width <= 2^20, K <= 2^21)");
  if (d->N % 8) return failw(what, BMM_EINVAL, "width (%lld) is not a multiple of 8", d->N);
  if (d->K % 16) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 16", d->K);
  if (d->ld_x < d->K) return failw(what, BMM_EINVAL, "ld_x (%lld) < K (%lld)", d->ld_x, d->K);
  if (d->ld_y < d->N) return failw(what, BMM_EINVAL, "ld_y (%lld) < width (%lld)", d->ld_y, d->N);
  if (d->ld_x > kMaxLd || d->ld_y > kMaxLd)
    return failw(what, BMM_EINVAL, "ld_x and ld_y are at most 2^21");
  if (d->ld_x % 8 || d->ld_y % 8)
    return failw(what, BMM_EALIGN, "ld_x (%lld) and ld_y (%lld) must be multiples of 8 elements",
                 d->ld_x, d->ld_y);
  if (mul_capped({d->T, d->ld_x, 2}) < 0 || mul_capped({d->T, d->ld_y, 2}) < 0 ||
      mul_capped({d->groups, d->N, d->K, 4}) < 0 || mul_capped({d->T, d->N + 32, 4}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  return Status{};
}

Status check_grouped(const uint16_t* Y, const uint16_t* Y1, const uint16_t* Y2, const uint16_t* X,
                     const uint32_t* W, const uint32_t* W1, const int32_t* ends,
                     const bmm_grouped_desc* d, bool gated) {
  const char* what = gated ? "grouped_gated" : "grouped_mma";
  Status st = check_grouped_desc(d, gated, what);
  if (!st.ok()) return st;
  if (!Y1 != !Y2) return failw(what, BMM_EINVAL, "G and U are given both or neither");
  if (d->T == 0 || d->N == 0) return Status{};
  const int64_t w = d->groups * d->N * d->K * 2;
  const Rows y{Y, d->T, d->N * 2, d->ld_y * 2, gated ? "H" : "Y"},
      y1{Y1, d->T, d->N * 2, d->ld_y * 2, "G"}, y2{Y2, d->T, d->N * 2, d->ld_y * 2, "U"},
      x{X, d->T, d->K * 2, d->ld_x * 2, "X"}, w0 = flat(W, w, gated ? "Wg" : "W"),
      w1 = flat(W1, gated ? w : 0, "Wu"), e = flat(ends, d->groups * 4, "ends");
  if (!(st = check_ends(ends, what)).ok()) return st;
  if (!(st = all_given(what, {y, x, w0, w1})).ok()) return st;
  if (!(st = all_aligned(what, {y, y1, y2, x, w0, w1})).ok()) return st;
  return disjoint(what, {y, y1, y2}, {x, w0, w1, e});
}

Status check_grouped_backward(const GroupedGrads& g, const int32_t* ends, const bmm_grouped_desc* d,
                              bool gated, const void* workspace, int64_t workspace_bytes,
                              int64_t need) {
  const char* what = gated ? "grouped_gated_backward" : "grouped_mma_backward";
  Status st = check_grouped_desc(d, gated, what);
  if (!st.ok()) return st;
  const int64_t w = d->groups * d->N * d->K * 2;
  if (gated && !g.dW != !g.dW1 && w > 0)
    return failw(what, BMM_EINVAL, "dWg and dWu are given both or neither");
  // (an empty gradient has no address: where either is empty, it may be the wanted one)
  if (!g.dX && !g.dW && w > 0 && d->T * d->K > 0)
    return failw(what, BMM_EINVAL, "no gradient is wanted");
  if (d->K == 0 || (d->T == 0 && w == 0)) return Status{};
  const int64_t y_bytes = d->N * 2, y_ld = d->ld_y * 2;
  const Rows dx = flat(g.dX, d->T * d->K * 2, "dX"), dw = flat(g.dW, w, gated ? "dWg" : "dW"),
             dw1 = flat(g.dW1, gated ? w : 0, "dWu"),
             dy{g.dY, d->T, y_bytes, y_ld, gated ? "dH" : "dY"}, gg{g.G, d->T, y_bytes, y_ld, "G"},
             u{g.U, d->T, y_bytes, y_ld, "U"}, x{g.X, d->T, d->K * 2, d->ld_x * 2, "X"},
             w0 = flat(g.W, w, gated ? "Wg" : "W"), w1 = flat(g.W1, gated ? w : 0, "Wu"),
             ws = flat(workspace, need, "workspace"), e = flat(ends, d->groups * 4, "ends");
  if (!(st = check_ends(ends, what)).ok()) return st;
  if (!(st = all_given(what, {dy})).ok()) return st;
  if (gated && !(st = all_given(what, {gg, u})).ok()) return st;
  if (g.dX && !(st = all_given(what, {w0, w1})).ok()) return st;
  if (g.dW && !(st = all_given(what, {x})).ok()) return st;
  if (workspace_bytes < need)
    return failw(what, BMM_EINVAL, "workspace_bytes %lld < %lld needed", workspace_bytes, need);
  if (!(st = all_given(what, {ws})).ok()) return st;
  if (!(st = all_aligned(what, {dx, dw, dw1, dy, gg, u, x, w0, w1, ws})).ok()) return st;
  return disjoint(what, {dx, dw, dw1, ws}, {dy, gg, u, x, w0, w1, e});
}

Status check_i8_quantize(const void* src, const int8_t* codes, const float* scales, int64_t batch,
                         int64_t rows, int64_t K, int64_t ld, int32_t elem_type) {
  const char* what = "i8_quantize";
  const int64_t size = elem_size(elem_type);
  if (!size)
    return failw(what, BMM_EINVAL, "elem_type %lld is not BMM_ELEM_F32, _F16 or _BF16", elem_type);
  if (batch < 0 || rows < 0 || K < 0) return failw(what, BMM_EINVAL, "negative extent");
  if (K % 32) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32", K);
  if (batch > kMaxExtent || rows > kMaxExtent || K >= kMaxK)
    return failw(what, BMM_EINVAL, "extent too large (K < 2^22)");
  if (ld < K) return failw(what, BMM_EINVAL, "ld (%lld) < K (%lld)", ld, K);
  if (ld > kMaxExtent || mul_capped({batch, rows, ld, size}) < 0 || mul_capped({batch, rows, 4}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  if (ld % 8) return failw(what, BMM_EALIGN, "ld (%lld) must be a multiple of 8 elements", ld);
  if (batch == 0 || rows == 0) return Status{};
  const Rows m{src, batch * rows, K * size, ld * size, "the matrix"},
      c = flat(codes, batch * rows * K, "codes"), s = flat(scales, batch * rows * 4, "scales");
  Status st = all_given(what, {m, c, s});
  if (!st.ok()) return st;
  if (!(st = all_aligned(what, {m, c})).ok()) return st;
  if (reinterpret_cast<uintptr_t>(scales) & 3)
    return failw(what, BMM_EALIGN, "scales must be 4-byte aligned");
  return disjoint(what, {c, s}, {m});
}

Status check_i8_product(const void* D, const int8_t* A, const float* sa, const uint32_t* W,
                        const float* sw, const uint32_t* W1, const float* sw1, const int32_t* ends,
                        const bmm_i8_desc* d, bool gated) {
  const char* what = gated ? "i8_gated" : "i8_mma";
  if (!d) return failw(what, BMM_EINVAL, "null descriptor");
  const int64_t size = elem_size(d->elem_type);
  if (!size || (gated && d->elem_type == BMM_ELEM_F32))
    return failw(what, BMM_EINVAL, gated ? "elem_type %lld is neither BMM_ELEM_F16 nor _BF16"
                                         : "elem_type %lld is not BMM_ELEM_F32, _F16 or _BF16",
                 d->elem_type);
  if (gated && (d->act < BMM_ACT_SILU || d->act > BMM_ACT_RELU))
    return failw(what, BMM_EINVAL, "act %lld is not a bmm_act", d->act);
  if (!gated && d->act != 0) return failw(what, BMM_EINVAL, "act %lld without a gate", d->act);
  if (d->zero_tail != 0 && d->zero_tail != 1)
    return failw(what, BMM_EINVAL, "zero_tail %lld is neither 0 nor 1", d->zero_tail);
  if (d->batch < 0 || d->M < 0 || d->N < 0 || d->K < 0)
    return failw(what, BMM_EINVAL, "negative extent");
  if (d->N % 8) return failw(what, BMM_EINVAL, "%lld columns are not a multiple of 8", d->N);
  if (d->K % 32) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32", d->K);
  if (ends && d->batch < 1) return failw(what, BMM_EINVAL, "there must be a group");
  if (d->batch > (ends ? kMaxGroups : kMaxExtent) || d->M > (ends ? kMaxRows : kMaxExtent) ||
      d->N > kMaxF || d->K >= kMaxI8K)
    return failw(what, BMM_EINVAL, "extent too large (columns <= 2^20, K < 2^17; with ends "
                                   "batch <= 4096, M < 2^31)");
  if (d->ld_a < d->K) return failw(what, BMM_EINVAL, "ld_a (%lld) < K (%lld)", d->ld_a, d->K);
  if (d->ld_d < d->N) return failw(what, BMM_EINVAL, "ld_d (%lld) < %lld columns", d->ld_d, d->N);
  if (d->ld_a > 2 * kMaxLd || d->ld_d > kMaxLd)
    return failw(what, BMM_EINVAL, "ld_a is at most 2^22, ld_d 2^21");
  if (d->ld_a % 16 || d->ld_d % 8)
    return failw(what, BMM_EALIGN, "ld_a (%lld) must be a multiple of 16, ld_d (%lld) of 8", d->ld_a,
                 d->ld_d);
  const int64_t copies = ends ? 1 : d->batch;
  if (mul_capped({copies, d->M, d->ld_a}) < 0 || mul_capped({copies, d->M, d->ld_d, size}) < 0 ||
      mul_capped({d->batch, d->N, d->K}) < 0 || mul_capped({d->batch, d->N, 4}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  if (copies == 0 || d->M == 0 || d->N == 0) return Status{};
  const int64_t w = d->batch * d->N * d->K, ws = d->batch * d->N * 4;
  const Rows out{D, copies * d->M, d->N * size, d->ld_d * size, gated ? "H" : "D"},
      a{A, copies * d->M, d->K, d->ld_a, gated ? "X" : "A"},
      as = flat(sa, copies * d->M * 4, gated ? "X_scales" : "A_scales"),
      w0 = flat(W, w, gated ? "Wg" : "B"), s0 = flat(sw, ws, gated ? "Wg_scales" : "B_scales"),
      w1 = flat(W1, gated ? w : 0, "Wu"), s1 = flat(sw1, gated ? ws : 0, "Wu_scales"),
      e = flat(ends, ends ? d->batch * 4 : 0, "ends");
  Status st = ends ? check_ends(ends, what) : Status{};
  if (!st.ok()) return st;
  if (!(st = all_given(what, {out, a, as, w0, s0, w1, s1})).ok()) return st;
  if (!(st = all_aligned(what, {out, a, w0, s0, w1, s1})).ok()) return st;
  if (reinterpret_cast<uintptr_t>(sa) & 3) {
    st = failw(what, BMM_EALIGN, "");
    st.msg += std::string(as.name) + " must be 4-byte aligned";
    return st;
  }
  return disjoint(what, {out}, {a, as, w0, s0, w1, s1, e});
}

Status check_group_plan(int32_t product, const bmm_grouped_desc& d) {
  const char* what = "group_plan";
  if (product < BMM_GROUPED_MMA || product > BMM_I8_GATED)
    return failw(what, BMM_EINVAL, "product %lld is not a bmm_group_product", product);
  if (product >= BMM_I8_MMA && (d.K % 32 || d.K >= kMaxI8K))
    return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32 below 2^17", d.K);
  bmm_grouped_desc one = d;
  if (product >= BMM_I8_MMA && one.groups == 0) one.groups = 1;   // one weight
  return check_grouped_desc(&one, true, what);
}

}  // namespace bmm
