// extern "C" entry points of the products by groups and of 8-bit integers
// (include/bmm.h): validate on the host, then enqueue the kernels on the caller's
// stream.
#include "abi_util.h"

namespace {

using bmm::guarded;
using bmm::hip_status;
using bmm::report;

// Layout of the backward passes' workspace: for the gated block as bmm_gated_backward's
// ([dG | dU], the factor that undoes their scaling, the peaks), then from slopes_bytes
// on the partial sums of one product at a time, or where both products are made in one
// launch of dX and from dw_parts on of dW.
struct GradPlan {
  int64_t dgu_bytes = 0, slopes_bytes = 0, dw_parts = 0, need = 0;
  bool both = false;  // in one launch
  int64_t sum = 0;    // values that dX sums: N, or both halves of [dG | dU]
  bmm::TilePlan dx, dw;
};

constexpr double kLaunchNs = 4000;

GradPlan plan_grads(const bmm_grouped_desc& d, bool gated) {
  GradPlan p;
  p.sum = d.N;
  if (gated) {
    p.sum = 2 * bmm::padded_width(d.N);
    p.dgu_bytes = d.T * p.sum * 2;
    const int64_t peaks = bmm::gated_peaks(d.T, d.N);
    p.slopes_bytes = (p.dgu_bytes + (peaks > 0 ? 4 * (1 + peaks) : 0) + 255) / 256 * 256;
  }
  p.dx = bmm::plan_group_rows(d.groups, d.T, d.K, (p.sum + 31) / 32, true);
  p.dw = bmm::plan_group_sums(d.groups, d.T, p.sum, d.K, false);
  if (p.dx.tile == bmm::kTile128) {
    // one launch, if dW's tiles do not cost more than it saves
    const bmm::TilePlan small = bmm::plan_group_sums(d.groups, d.T, p.sum, d.K, true);
    p.both = small.ns <= p.dw.ns + kLaunchNs;
    if (p.both) p.dw = small;
  }
  const int64_t dx = p.dx.splits > 1 ? p.dx.splits * d.T * d.K * 4 : 0;
  const int64_t dw = p.dw.splits > 1 ? p.dw.splits * d.groups * p.sum * d.K * 4 : 0;
  p.dw_parts = p.slopes_bytes + (p.both ? (dx + 255) / 256 * 256 : 0);
  p.need = p.slopes_bytes + dx;
  if (p.dw_parts + dw > p.need) p.need = p.dw_parts + dw;
  return p;
}

// A product by groups, dense in what the host knows of it.
bmm::TileArgs group_args(const bmm_grouped_desc& d, const int32_t* ends) {
  bmm::TileArgs a{};
  a.batch = d.groups;
  a.ends = ends;
  a.zero_tail = d.zero_tail;
  a.act = d.act;
  a.out_type = d.dtype == BMM_BF16 ? BMM_ELEM_BF16 : BMM_ELEM_F16;
  a.splits = 1;
  a.row1 = bmm::kNoRow;
  return a;
}

int forward_tile(const bmm_grouped_desc& d, bool gated) {
  return bmm::plan_group_forward(d.groups, d.T, gated ? 2 * d.N : d.N, d.K / 32);
}

int grouped(uint16_t* Y, uint16_t* Y1, uint16_t* Y2, const uint16_t* X, const uint32_t* W,
            const uint32_t* W1, const int32_t* ends, const bmm_grouped_desc* desc, bool gated,
            void* stream) {
  const bmm::Status st = bmm::check_grouped(Y, Y1, Y2, X, W, W1, ends, desc, gated);
  if (!st.ok()) return report(st);
  const bmm_grouped_desc& d = *desc;
  if (d.T == 0 || d.N == 0) return report(st);
  bmm::TileArgs a = group_args(d, ends);
  a.a = X;
  a.b0 = W;
  a.b1 = W1;
  a.d = Y;
  a.d1 = Y1;
  a.d2 = Y2;
  a.M = a.rows0 = d.T;
  a.N = d.N;
  a.K = d.K;
  a.lda = d.ld_x;
  a.ldd = d.ld_y;
  a.b_bs = d.N * d.K;
  a.tile = forward_tile(d, gated);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (gated) return hip_status(bmm::launch_grouped_gated(a, d.dtype, s), "grouped_gated launch");
  return hip_status(bmm::launch_grouped_mma(a, d.dtype, s), "grouped_mma launch");
}

int64_t grads_workspace(const bmm_grouped_desc* desc, bool gated, const char* what) {
  const bmm::Status st = bmm::check_grouped_desc(desc, gated, what);
  if (!st.ok()) return report(st);
  return plan_grads(*desc, gated).need;
}

int grouped_backward(const bmm::GroupedGrads& g, const int32_t* ends, const bmm_grouped_desc* desc,
                     bool gated, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* const what = gated ? "grouped_gated_backward" : "grouped_mma_backward";
  bmm::Status st = bmm::check_grouped_desc(desc, gated, what);
  if (!st.ok()) return report(st);
  const bmm_grouped_desc& d = *desc;
  const GradPlan plan = plan_grads(d, gated);
  st = bmm::check_grouped_backward(g, ends, desc, gated, workspace, workspace_bytes, plan.need);
  if (!st.ok()) return report(st);
  if (d.K == 0 || (d.T == 0 && d.N == 0)) return report(st);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* const parts = static_cast<char*>(workspace);
  // what the products take: dY, or [dG | dU] in the workspace
  const uint16_t* dy = g.dY;
  int64_t ld = d.ld_y;
  float* rescale = nullptr;
  if (gated) {
    uint16_t* const dgu = static_cast<uint16_t*>(workspace);
    uint32_t* peaks = nullptr;
    if (plan.dgu_bytes > 0) {
      rescale = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.dgu_bytes);
      peaks = reinterpret_cast<uint32_t*>(rescale + 1);
    }
    const int rc = hip_status(
        bmm::launch_gated_slopes(dgu, g.dY, g.G, g.U, d.T, d.N, d.ld_y, d.dtype, d.act,
                                 {ends, int(d.groups), int(d.T)}, peaks, rescale, s),
        "grouped_gated_backward slopes launch");
    if (rc != BMM_OK) return rc;
    dy = dgu;
    ld = plan.sum;
  }
  bmm::TileArgs dx = group_args(d, ends), dw = dx;
  const bool want_dx = g.dX && d.T > 0, want_dw = g.dW && d.N > 0;
  dx.a = dy;
  dx.b0 = g.W;
  dx.b1 = gated ? g.W1 : g.W;
  dx.d = const_cast<uint16_t*>(g.dX);
  dx.M = dx.rows0 = d.T;
  dx.N = dx.ldd = d.K;
  dx.K = plan.sum;
  dx.lda = ld;
  dx.b_bs = d.N * d.K;
  dx.b_sum = bmm::padded_width(d.N);
  dx.b_rows = d.N;
  dx.tile = plan.dx.tile;
  dx.splits = plan.dx.splits;
  dx.part = reinterpret_cast<float*>(parts + plan.slopes_bytes);
  dx.part_floats = d.T * d.K;
  dx.rescale = rescale;
  dw.a = dy;
  dw.b0 = g.X;
  dw.d = const_cast<uint16_t*>(g.dW);
  dw.d1 = const_cast<uint16_t*>(g.dW1);
  dw.M = plan.sum;
  dw.lda = ld;
  dw.rows0 = d.N;
  if (gated) dw.row1 = bmm::padded_width(d.N);
  dw.N = dw.ldd = d.K;
  dw.K = d.T;
  dw.ldb = d.ld_x;
  dw.tile = plan.dw.tile;
  dw.splits = plan.dw.splits;
  dw.part = reinterpret_cast<float*>(parts + plan.dw_parts);
  dw.part_floats = d.groups * plan.sum * d.K;
  dw.rescale = rescale;
  if (plan.both && want_dx && want_dw)
    return hip_status(bmm::launch_grouped_both(dx, dw, d.dtype, s), "grouped gradients launch");
  if (want_dx) {
    const int rc = hip_status(bmm::launch_grouped_dx(dx, d.dtype, s), "grouped dX launch");
    if (rc != BMM_OK) return rc;
  }
  if (want_dw) return hip_status(bmm::launch_grouped_dw(dw, d.dtype, s), "grouped dW launch");
  return report(st);
}

// groups 0: one weight for every batch.
int i8_tile(int64_t groups, int64_t batch, int64_t M, int64_t N, int64_t K) {
  return groups ? bmm::plan_group_forward(groups, M, N, K / 64)
                : bmm::plan_forward(batch, M, N, K / 64);
}

int i8_product(void* D, const int8_t* A, const float* sa, const uint32_t* W, const float* sw,
               const uint32_t* W1, const float* sw1, const int32_t* ends, const bmm_i8_desc* desc,
               bool gated, void* stream) {
  const bmm::Status st = bmm::check_i8_product(D, A, sa, W, sw, W1, sw1, ends, desc, gated);
  if (!st.ok()) return report(st);
  const bmm_i8_desc& d = *desc;
  if (d.batch == 0 || d.M == 0 || d.N == 0) return report(st);
  bmm::TileArgs a{};
  a.a = A;
  a.b0 = W;
  a.b1 = W1;
  a.sa = sa;
  a.sb0 = sw;
  a.sb1 = sw1;
  a.ends = ends;
  a.zero_tail = d.zero_tail;
  a.d = D;
  a.batch = d.batch;
  a.M = a.rows0 = d.M;
  a.row1 = bmm::kNoRow;
  a.N = d.N;
  a.K = d.K / 2;   // in 16-bit values, like the distances below
  a.lda = d.ld_a / 2;
  a.ldd = d.ld_d;
  a.a_bs = d.M * a.lda;
  a.b_bs = d.N * a.K;
  a.act = d.act;
  a.out_type = d.elem_type;
  a.splits = 1;
  a.tile = i8_tile(ends ? d.batch : 0, d.batch, d.M, gated ? 2 * d.N : d.N, d.K);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (gated) return hip_status(bmm::launch_i8_gated(a, s), "i8_gated launch");
  return hip_status(bmm::launch_i8_mma(a, s), "i8_mma launch");
}

}  // namespace

extern "C" {

int bmm_grouped_mma(uint16_t* Y, const uint16_t* X, const uint32_t* W, const int32_t* ends,
                    const bmm_grouped_desc* desc, void* stream) {
  return guarded(
      [&] { return grouped(Y, nullptr, nullptr, X, W, nullptr, ends, desc, false, stream); });
}

int bmm_grouped_gated(uint16_t* H, uint16_t* G, uint16_t* U, const uint16_t* X, const uint32_t* Wg,
                      const uint32_t* Wu, const int32_t* ends, const bmm_grouped_desc* desc,
                      void* stream) {
  return guarded([&] { return grouped(H, G, U, X, Wg, Wu, ends, desc, true, stream); });
}

int64_t bmm_grouped_mma_backward_workspace_bytes(const bmm_grouped_desc* desc) {
  return guarded([&] { return grads_workspace(desc, false, "grouped_mma_backward"); });
}

int64_t bmm_grouped_gated_backward_workspace_bytes(const bmm_grouped_desc* desc) {
  return guarded([&] { return grads_workspace(desc, true, "grouped_gated_backward"); });
}

int bmm_grouped_mma_backward(uint16_t* dX, uint16_t* dW, const uint16_t* dY, const uint16_t* X,
                             const uint32_t* W, const int32_t* ends, const bmm_grouped_desc* desc,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    const bmm::GroupedGrads g{dX, dW, nullptr, dY, nullptr, nullptr, X, W, nullptr};
    return grouped_backward(g, ends, desc, false, workspace, workspace_bytes, stream);
  });
}

int bmm_grouped_gated_backward(uint16_t* dX, uint16_t* dWg, uint16_t* dWu, const uint16_t* dH,
                               const uint16_t* G, const uint16_t* U, const uint16_t* X,
                               const uint32_t* Wg, const uint32_t* Wu, const int32_t* ends,
                               const bmm_grouped_desc* desc, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    const bmm::GroupedGrads g{dX, dWg, dWu, dH, G, U, X, Wg, Wu};
    return grouped_backward(g, ends, desc, true, workspace, workspace_bytes, stream);
  });
}

int bmm_i8_quantize(int8_t* codes, float* scales, const void* src, int64_t batch, int64_t rows,
                    int64_t K, int64_t ld_src, int32_t elem_type, void* stream) {
  return guarded([&] {
    const bmm::Status st =
        bmm::check_i8_quantize(src, codes, scales, batch, rows, K, ld_src, elem_type);
    if (!st.ok()) return report(st);
    if (batch == 0 || rows == 0) return report(st);
    return hip_status(bmm::launch_i8_quantize(codes, scales, src, batch * rows, K, ld_src, elem_type,
                                              static_cast<hipStream_t>(stream)),
                      "i8_quantize launch");
  });
}

int bmm_i8_mma(void* D, const int8_t* A, const float* A_scales, const uint32_t* B,
               const float* B_scales, const int32_t* ends, const bmm_i8_desc* desc, void* stream) {
  return guarded([&] {
    return i8_product(D, A, A_scales, B, B_scales, nullptr, nullptr, ends, desc, false, stream);
  });
}

int bmm_i8_gated(void* H, const int8_t* X, const float* X_scales, const uint32_t* Wg,
                 const float* Wg_scales, const uint32_t* Wu, const float* Wu_scales,
                 const int32_t* ends, const bmm_i8_desc* desc, void* stream) {
  return guarded([&] {
    return i8_product(H, X, X_scales, Wg, Wg_scales, Wu, Wu_scales, ends, desc, true, stream);
  });
}

int bmm_group_plan(int32_t product, int64_t groups, int64_t T, int64_t N, int64_t K,
                   int32_t* splits) {
  return guarded([&] {
    const bmm_grouped_desc d{groups, T, N, K, K, N, BMM_BF16, BMM_ACT_SILU, 0};
    const bmm::Status st = bmm::check_group_plan(product, d);
    if (!st.ok()) return report(st);
    const bool gated = product == BMM_GROUPED_GATED || product == BMM_GROUPED_GATED_DX ||
                       product == BMM_GROUPED_GATED_DW || product == BMM_I8_GATED;
    const bool dx = product == BMM_GROUPED_MMA_DX || product == BMM_GROUPED_GATED_DX;
    const bool dw = product == BMM_GROUPED_MMA_DW || product == BMM_GROUPED_GATED_DW;
    bmm::TilePlan plan{BMM_TILE_NONE, 1, 0};
    if (dx ? T == 0 || K == 0 : dw ? N == 0 || K == 0 : T == 0 || N == 0)
      ;   // nothing to make
    else if (dx)
      plan = plan_grads(d, gated).dx;
    else if (dw)
      plan = plan_grads(d, gated).dw;
    else if (product >= BMM_I8_MMA)
      plan.tile = i8_tile(groups, 1, T, gated ? 2 * N : N, K);
    else
      plan.tile = forward_tile(d, gated);
    if (splits) *splits = plan.splits;
    report(st);
    return plan.tile;
  });
}

}  // extern "C"
