// extern "C" entry points of the feed-forward operators (include/bmm.h):
// validate on the host, then enqueue the kernels on the caller's stream.
#include "abi_util.h"

namespace {

// Layout of the backward pass's workspace: [dG | dU], the factor that undoes their
// scaling and the peaks that it comes from (f16; kept for both types, so that a
// workspace serves either), then from slopes_bytes on the partial sums of one product
// at a time. dX's rows are made in two launches where a first part
// fills the chip in whole rounds of large tiles and the few rows left would cost
// another round: 32773 x 512, summed over 2048 values, 76 us against 90 (128 x 128
// tiles) and 98 (256 x 256) in one.
struct BackwardPlan {
  int64_t dgu_bytes, slopes_bytes, need;
  int64_t dx_rows;              // rows of the first launch
  bmm::TilePlan dx, dx_rest, dw;
};

constexpr double kLaunchNs = 4000;

BackwardPlan plan_backward(const bmm_gated_desc& d) {
  BackwardPlan p;
  const int64_t Fp2 = 2 * bmm::padded_width(d.F);
  p.dgu_bytes = d.batch * d.M * Fp2 * 2;
  const int64_t peaks = bmm::gated_peaks(d.batch * d.M, d.F);
  p.slopes_bytes = (p.dgu_bytes + (peaks > 0 ? 4 * (1 + peaks) : 0) + 255) / 256 * 256;
  p.dx = p.dx_rest = bmm::plan_tiles(d.batch, d.M, d.K, Fp2 / 32, true);
  p.dx_rows = d.M;
  const int64_t across = (d.K + 255) / 256, down = across > 0 ? 256 / across : 0;
  const int64_t body = down > 0 ? d.M / (256 * down) * (256 * down) : 0;
  if (d.batch == 1 && body > 0 && body < d.M) {
    const bmm::TilePlan first = bmm::plan_tiles(1, body, d.K, Fp2 / 32, true);
    const bmm::TilePlan rest = bmm::plan_tiles(1, d.M - body, d.K, Fp2 / 32, true);
    if (first.ns + rest.ns + kLaunchNs < p.dx.ns) {
      p.dx = first;
      p.dx_rest = rest;
      p.dx_rows = body;
    }
  }
  p.dw = bmm::plan_tiles(d.batch, Fp2, d.K, (d.M + 31) / 32, true);
  auto parts = [&](const bmm::TilePlan& plan, int64_t rows) {
    return plan.splits > 1 ? plan.splits * d.batch * rows * d.K * 4 : 0;
  };
  const int64_t sizes[] = {parts(p.dx, p.dx_rows), parts(p.dx_rest, d.M - p.dx_rows),
                           parts(p.dw, Fp2)};
  p.need = p.slopes_bytes;
  for (int64_t s : sizes)
    if (p.slopes_bytes + s > p.need) p.need = p.slopes_bytes + s;
  return p;
}

// The tile of a forward product: 16-bit gated, and the 4-bit product of N columns
// (gated: of both weights together).
int gated_tile(const bmm_gated_desc& d) {
  return bmm::plan_forward(d.batch, d.M, 2 * d.F, d.K / 32);
}
int mx4_tile(int64_t batch, int64_t M, int64_t N, int64_t K) {
  return bmm::plan_forward(batch, M, N, K / 128);
}

bmm::TileArgs gated_args(const bmm_gated_desc& d) {
  bmm::TileArgs a{};
  a.batch = d.batch;
  a.act = d.act;
  a.out_type = d.dtype == BMM_BF16 ? BMM_ELEM_BF16 : BMM_ELEM_F16;
  a.splits = 1;
  return a;
}

}  // namespace

extern "C" {

int bmm_gated(uint16_t* H, uint16_t* G, uint16_t* U, const uint16_t* X, const uint32_t* Wg,
              const uint32_t* Wu, const bmm_gated_desc* desc, void* stream) {
  return bmm::guarded([&] {
    const bmm::Status st = bmm::check_gated(H, G, U, X, Wg, Wu, desc);
    if (!st.ok()) return bmm::report(st);
    const bmm_gated_desc& d = *desc;
    if (d.batch == 0 || d.M == 0 || d.F == 0) return bmm::report(st);
    bmm::TileArgs a = gated_args(d);
    a.a = X;
    a.b0 = Wg;
    a.b1 = Wu;
    a.d = H;
    a.d1 = G;
    a.d2 = U;
    a.M = d.M;
    a.N = d.F;
    a.K = d.K;
    a.lda = d.ld_x;
    a.ldd = d.ld_h;
    a.a_bs = d.M * d.ld_x;
    a.b_bs = d.F * d.K;
    a.tile = gated_tile(d);
    return bmm::hip_status(bmm::launch_gated(a, d.dtype, static_cast<hipStream_t>(stream)),
                      "gated launch");
  });
}

int64_t bmm_gated_backward_workspace_bytes(const bmm_gated_desc* desc) {
  return bmm::guarded([&]() -> int64_t {
    const bmm::Status st = bmm::check_gated_desc(desc, "gated_backward");
    if (!st.ok()) return bmm::report(st);
    return plan_backward(*desc).need;
  });
}

int bmm_gated_backward(uint16_t* dX, uint16_t* dWg, uint16_t* dWu, const uint16_t* dH,
                       const uint16_t* G, const uint16_t* U, const uint16_t* X,
                       const uint32_t* Wg, const uint32_t* Wu, const bmm_gated_desc* desc,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  return bmm::guarded([&] {
    bmm::Status st = bmm::check_gated_desc(desc, "gated_backward");
    if (!st.ok()) return bmm::report(st);
    const bmm_gated_desc& d = *desc;
    const BackwardPlan plan = plan_backward(d);
    st = bmm::check_gated_backward(dX, dWg, dWu, dH, G, U, X, Wg, Wu, desc, workspace,
                                   workspace_bytes, plan.need);
    if (!st.ok()) return bmm::report(st);
    if (d.batch == 0 || d.K == 0 || (d.M == 0 && d.F == 0)) return bmm::report(st);
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t* const dgu = static_cast<uint16_t*>(workspace);
    float* const part =
        reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.slopes_bytes);
    const int64_t Fp = bmm::padded_width(d.F);
    float* rescale = nullptr;   // (no [dG | dU]: no factor either)
    uint32_t* peaks = nullptr;
    if (plan.dgu_bytes > 0) {
      rescale = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.dgu_bytes);
      peaks = reinterpret_cast<uint32_t*>(rescale + 1);
    }
    int rc = bmm::hip_status(bmm::launch_gated_slopes(dgu, dH, G, U, d.batch * d.M, d.F, d.ld_h,
                                                 d.dtype, d.act, {}, peaks, rescale, s),
                        "gated_backward slopes launch");
    if (rc != BMM_OK) return rc;
    auto rows_of_dx = [&](int64_t row, int64_t rows, const bmm::TilePlan& tiles) {
      bmm::TileArgs a = gated_args(d);
      a.a = dgu + row * 2 * Fp;
      a.b0 = Wg;
      a.b1 = Wu;
      a.d = dX + row * d.K;
      a.M = a.rows0 = rows;
      a.row1 = bmm::kNoRow;
      a.N = a.ldd = d.K;
      a.K = a.lda = 2 * Fp;
      a.a_bs = d.M * 2 * Fp;
      a.b_bs = d.F * d.K;
      a.b_sum = Fp;
      a.b_rows = d.F;
      a.tile = tiles.tile;
      a.splits = tiles.splits;
      a.part = part;
      a.part_floats = d.batch * rows * d.K;
      a.rescale = rescale;
      return bmm::hip_status(bmm::launch_gated_dx(a, d.dtype, s), "gated_backward dX launch");
    };
    if (dX && d.M > 0) {
      rc = rows_of_dx(0, plan.dx_rows, plan.dx);
      if (rc == BMM_OK && plan.dx_rows < d.M)
        rc = rows_of_dx(plan.dx_rows, d.M - plan.dx_rows, plan.dx_rest);
      if (rc != BMM_OK) return rc;
    }
    if (dWg && d.F > 0) {
      bmm::TileArgs a = gated_args(d);
      a.a = dgu;
      a.b0 = X;
      a.d = dWg;
      a.d1 = dWu;
      a.M = a.lda = 2 * Fp;
      a.rows0 = d.F;
      a.row1 = Fp;
      a.N = a.ldd = d.K;
      a.K = d.M;
      a.ldb = d.ld_x;
      a.a_bs = d.M * 2 * Fp;
      a.b_bs = d.M * d.ld_x;
      a.tile = plan.dw.tile;
      a.splits = plan.dw.splits;
      a.part = part;
      a.part_floats = d.batch * 2 * Fp * d.K;
      a.rescale = rescale;
      rc = bmm::hip_status(bmm::launch_gated_dw(a, d.dtype, s), "gated_backward dW launch");
    }
    return rc;
  });
}

int bmm_ffn_plan(int32_t product, int64_t batch, int64_t M, int64_t F, int64_t K,
                 int32_t* splits) {
  return bmm::guarded([&] {
    const bool four = product == BMM_FFN_MX4_MMA || product == BMM_FFN_MX4_GATED;
    const bmm_gated_desc d{batch, M, F, K, K, F, BMM_BF16, BMM_ACT_SILU};
    const bmm::Status st = bmm::check_ffn_plan(product, d);
    if (!st.ok()) return bmm::report(st);
    bmm::TilePlan plan{BMM_TILE_NONE, 1, 0};
    // (the backward pass writes the zeros of an empty sum: dX for F = 0, dWg and dWu for M = 0)
    const bool forward = four || product == BMM_FFN_GATED, dw = product == BMM_FFN_GATED_DW;
    if (batch == 0 || (forward ? M == 0 || F == 0 : K == 0 || (dw ? F : M) == 0))
      ;   // nothing to make
    else if (product == BMM_FFN_GATED)
      plan.tile = gated_tile(d);
    else if (four)
      plan.tile = mx4_tile(batch, M, product == BMM_FFN_MX4_GATED ? 2 * F : F, K);
    else {
      const BackwardPlan b = plan_backward(d);
      if (product == BMM_FFN_GATED_DX) plan = b.dx;
      else if (dw) plan = b.dw;
      else if (b.dx_rows < M) plan = b.dx_rest;
    }
    if (splits) *splits = plan.splits;
    bmm::report(st);
    return plan.tile;
  });
}

int64_t bmm_mx4_codes_bytes(int64_t batch, int64_t rows, int64_t K) {
  const int64_t n = bmm::mx4_codes_bytes(batch, rows, K);
  return n < 0 ? BMM_EINVAL : n;
}

int64_t bmm_mx4_scales_bytes(int64_t batch, int64_t rows, int64_t K) {
  const int64_t n = bmm::mx4_scales_bytes(batch, rows, K);
  return n < 0 ? BMM_EINVAL : n;
}

int bmm_mx4_quantize(uint8_t* codes, uint8_t* scales, const void* src, int64_t batch, int64_t rows,
                     int64_t K, int64_t ld_src, int32_t elem_type, void* stream) {
  return bmm::guarded([&] {
    const bmm::Status st = bmm::check_mx4_convert(src, codes, scales, batch, rows, K, ld_src,
                                                  elem_type, "mx4_quantize");
    if (!st.ok()) return bmm::report(st);
    if (batch == 0 || rows == 0 || K == 0) return bmm::report(st);
    return bmm::hip_status(bmm::launch_mx4_quantize(codes, scales, src, batch, rows, K, ld_src,
                                               elem_type, static_cast<hipStream_t>(stream)),
                      "mx4_quantize launch");
  });
}

int bmm_mx4_dequantize(void* dst, const uint8_t* codes, const uint8_t* scales, int64_t batch,
                       int64_t rows, int64_t K, int64_t ld_dst, int32_t elem_type, void* stream) {
  return bmm::guarded([&] {
    const bmm::Status st = bmm::check_mx4_convert(dst, codes, scales, batch, rows, K, ld_dst,
                                                  elem_type, "mx4_dequantize");
    if (!st.ok()) return bmm::report(st);
    if (batch == 0 || rows == 0 || K == 0) return bmm::report(st);
    return bmm::hip_status(bmm::launch_mx4_dequantize(dst, codes, scales, batch, rows, K, ld_dst,
                                                 elem_type, static_cast<hipStream_t>(stream)),
                      "mx4_dequantize launch");
  });
}

int bmm_mx4_mma(void* D, const uint8_t* A_codes, const uint8_t* A_scales, const uint8_t* B_codes,
                const uint8_t* B_scales, int64_t batch, int64_t M, int64_t N, int64_t K,
                int64_t ld_d, int32_t elem_type, void* stream) {
  return bmm::guarded([&] {
    const bmm::Status st =
        bmm::check_mx4_product(D, A_codes, A_scales, B_codes, B_scales, nullptr, nullptr, false,
                               batch, M, N, K, ld_d, 0, elem_type);
    if (!st.ok()) return bmm::report(st);
    if (batch == 0 || M == 0 || N == 0) return bmm::report(st);
    bmm::TileArgs a{};
    a.a = A_codes;
    a.as = A_scales;
    a.b0 = B_codes;
    a.bs0 = B_scales;
    a.d = D;
    a.batch = batch;
    a.M = a.rows0 = M;
    a.row1 = bmm::kNoRow;
    a.N = N;
    a.K = K;
    a.ldd = ld_d;
    a.a_bs = bmm::mx4_codes_bytes(1, M, K);
    a.as_bs = bmm::mx4_scales_bytes(1, M, K);
    a.b_bs = bmm::mx4_codes_bytes(1, N, K);
    a.bs_bs = bmm::mx4_scales_bytes(1, N, K);
    a.out_type = elem_type;
    a.splits = 1;
    a.tile = mx4_tile(batch, M, N, K);
    return bmm::hip_status(bmm::launch_mx4_mma(a, static_cast<hipStream_t>(stream)), "mx4_mma launch");
  });
}

int bmm_mx4_gated(void* H, const uint8_t* X_codes, const uint8_t* X_scales,
                  const uint8_t* Wg_codes, const uint8_t* Wg_scales, const uint8_t* Wu_codes,
                  const uint8_t* Wu_scales, int64_t batch, int64_t M, int64_t F, int64_t K,
                  int64_t ld_h, int32_t act, int32_t elem_type, void* stream) {
  return bmm::guarded([&] {
    const bmm::Status st =
        bmm::check_mx4_product(H, X_codes, X_scales, Wg_codes, Wg_scales, Wu_codes, Wu_scales,
                               true, batch, M, F, K, ld_h, act, elem_type);
    if (!st.ok()) return bmm::report(st);
    if (batch == 0 || M == 0 || F == 0) return bmm::report(st);
    bmm::TileArgs a{};
    a.a = X_codes;
    a.as = X_scales;
    a.b0 = Wg_codes;
    a.bs0 = Wg_scales;
    a.b1 = Wu_codes;
    a.bs1 = Wu_scales;
    a.d = H;
    a.batch = batch;
    a.M = M;
    a.N = F;
    a.K = K;
    a.ldd = ld_h;
    a.a_bs = bmm::mx4_codes_bytes(1, M, K);
    a.as_bs = bmm::mx4_scales_bytes(1, M, K);
    a.b_bs = bmm::mx4_codes_bytes(1, F, K);
    a.bs_bs = bmm::mx4_scales_bytes(1, F, K);
    a.act = act;
    a.out_type = elem_type;
    a.splits = 1;
    a.tile = mx4_tile(batch, M, 2 * F, K);
    return bmm::hip_status(bmm::launch_mx4_gated(a, static_cast<hipStream_t>(stream)),
                      "mx4_gated launch");
  });
}

}  // extern "C"
