// Argument checks of the feed-forward operators.
#include "validate_util.h"

namespace bmm {
namespace {

Status failw(const char* what, int code, const char* fmt, long long a = 0, long long b = 0) {
  Status s = fail(code, fmt, a, b);
  s.msg = std::string(what) + ": " + s.msg;
  return s;
}

// A row-major matrix: `rows` rows of `cols` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, cols, ld;
  const char* name;
  int64_t span() const { return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0; }
};

// Whether two matrices share a byte. Rows of one buffer that lie side by side
// (equal ld, columns apart) do not.
bool overlaps(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !bmm::overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.ld != b.ld || a.ld <= 0) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  // columns from a's to b's first one, in [0, ld)
  const int64_t d = y >= x ? int64_t((y - x) % uintptr_t(a.ld))
                           : (a.ld - int64_t((x - y) % uintptr_t(a.ld))) % a.ld;
  return !(d >= a.cols && a.ld - d >= b.cols);
}

// Every output against every input and every other output.
Status disjoint(const char* what, std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto q = o + 1; q != outs.end(); ++q)
      if (overlaps(*o, *q)) {
        Status s = failw(what, BMM_EOVERLAP, "");
        s.msg += std::string(o->name) + " overlaps " + q->name;
        return s;
      }
    for (const Rows& i : ins)
      if (overlaps(*o, i)) {
        Status s = failw(what, BMM_EOVERLAP, "");
        s.msg += std::string(o->name) + " overlaps " + i.name;
        return s;
      }
  }
  return Status{};
}

Status all_aligned(const char* what, std::initializer_list<Rows> ps) {
  for (const Rows& r : ps)
    if (!aligned16(r.p)) {
      Status s = failw(what, BMM_EALIGN, "");
      s.msg += std::string(r.name) + " must be 16-byte aligned";
      return s;
    }
  return Status{};
}

Status all_given(const char* what, std::initializer_list<Rows> ps) {
  for (const Rows& r : ps)
    if (!r.p && r.span() > 0) {
      Status s = failw(what, BMM_EINVAL, "");
      s.msg += std::string(r.name) + " is null";
      return s;
    }
  return Status{};
}

constexpr int64_t kMaxK = int64_t(1) << 22;    // below it (4-bit operands)
constexpr int64_t kMaxLd = int64_t(1) << 21;   // 32-bit offsets inside a tile's rows; the gated
                                               // block's K is such a distance too (dX, dWg, dWu)
constexpr int64_t kMaxF = int64_t(1) << 20;

int elem_size(int32_t t) {
  return t == BMM_ELEM_F32 ? 4 : t == BMM_ELEM_F16 || t == BMM_ELEM_BF16 ? 2 : 0;
}

}  // namespace

Status check_gated_desc(const bmm_gated_desc* d, const char* what) {
  if (!d) return failw(what, BMM_EINVAL, "null descriptor");
  if (d->dtype != BMM_F16 && d->dtype != BMM_BF16)
    return failw(what, BMM_EINVAL, "dtype %lld is neither BMM_F16 nor BMM_BF16", d->dtype);
  if (d->act < BMM_ACT_SILU || d->act > BMM_ACT_RELU)
    return failw(what, BMM_EINVAL, "act %lld is not a bmm_act", d->act);
  if (d->batch < 0 || d->M < 0 || d->F < 0 || d->K < 0)
    return failw(what, BMM_EINVAL, "negative extent");
  if (d->batch > kMaxExtent || d->M > kMaxExtent || d->F > kMaxF || d->K > kMaxLd)
    return failw(what, BMM_EINVAL, "extent too large (F <= 2^20, K <= 2^21)");
  if (d->F % 8) return failw(what, BMM_EINVAL, "F (%lld) is not a multiple of 8", d->F);
  if (d->K % 16) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 16", d->K);
  if (d->ld_x < d->K) return failw(what, BMM_EINVAL, "ld_x (%lld) < K (%lld)", d->ld_x, d->K);
  if (d->ld_h < d->F) return failw(what, BMM_EINVAL, "ld_h (%lld) < F (%lld)", d->ld_h, d->F);
  if (d->ld_x > kMaxLd || d->ld_h > kMaxLd)
    return failw(what, BMM_EINVAL, "ld_x and ld_h are at most 2^21");
  if (d->ld_x % 8 || d->ld_h % 8)
    return failw(what, BMM_EALIGN, "ld_x (%lld) and ld_h (%lld) must be multiples of 8 elements",
                 d->ld_x, d->ld_h);
  if (mul_capped({d->batch, d->M, d->ld_x, 2}) < 0 || mul_capped({d->batch, d->M, d->ld_h, 2}) < 0 ||
      mul_capped({d->batch, d->F, d->K, 4}) < 0 || mul_capped({d->batch, d->M, d->F + 32, 4}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  return Status{};
}

Status check_gated(const uint16_t* H, const uint16_t* G, const uint16_t* U, const uint16_t* X,
                   const uint32_t* Wg, const uint32_t* Wu, const bmm_gated_desc* d) {
  const char* what = "gated";
  Status st = check_gated_desc(d, what);
  if (!st.ok()) return st;
  if (!G != !U) return failw(what, BMM_EINVAL, "G and U are given both or neither");
  const int64_t rows = d->batch * d->M, w = d->batch * d->F * d->K * 2;
  if (rows == 0 || d->F == 0) return Status{};
  const Rows h{H, rows, d->F * 2, d->ld_h * 2, "H"}, g{G, rows, d->F * 2, d->ld_h * 2, "G"},
      u{U, rows, d->F * 2, d->ld_h * 2, "U"}, x{X, rows, d->K * 2, d->ld_x * 2, "X"},
      wg{Wg, 1, w, 0, "Wg"}, wu{Wu, 1, w, 0, "Wu"};
  if (!(st = all_given(what, {h, x, wg, wu})).ok()) return st;
  if (!(st = all_aligned(what, {h, g, u, x, wg, wu})).ok()) return st;
  return disjoint(what, {h, g, u}, {x, wg, wu});
}

Status check_gated_backward(const uint16_t* dX, const uint16_t* dWg, const uint16_t* dWu,
                            const uint16_t* dH, const uint16_t* G, const uint16_t* U,
                            const uint16_t* X, const uint32_t* Wg, const uint32_t* Wu,
                            const bmm_gated_desc* d, const void* workspace,
                            int64_t workspace_bytes, int64_t need) {
  const char* what = "gated_backward";
  Status st = check_gated_desc(d, what);
  if (!st.ok()) return st;
  if (!dWg != !dWu && d->batch * d->F * d->K > 0)
    return failw(what, BMM_EINVAL, "dWg and dWu are given both or neither");
  if (d->batch == 0 || d->K == 0 || (d->M == 0 && d->F == 0)) return Status{};
  if (!dX && !dWg && d->M > 0 && d->F > 0)
    return failw(what, BMM_EINVAL, "dX, dWg and dWu are all null");
  const int64_t rows = d->batch * d->M, w = d->batch * d->F * d->K * 2;
  const Rows dx{dX, 1, rows * d->K * 2, 0, "dX"}, dwg{dWg, 1, w, 0, "dWg"},
      dwu{dWu, 1, w, 0, "dWu"}, dh{dH, rows, d->F * 2, d->ld_h * 2, "dH"},
      g{G, rows, d->F * 2, d->ld_h * 2, "G"}, u{U, rows, d->F * 2, d->ld_h * 2, "U"},
      x{X, rows, d->K * 2, d->ld_x * 2, "X"}, wg{Wg, 1, w, 0, "Wg"}, wu{Wu, 1, w, 0, "Wu"},
      ws{workspace, 1, need, 0, "workspace"};
  if (!(st = all_given(what, {dh, g, u})).ok()) return st;
  if (dX && !(st = all_given(what, {wg, wu})).ok()) return st;
  if (dWg && !(st = all_given(what, {x})).ok()) return st;
  if (workspace_bytes < need)
    return failw(what, BMM_EINVAL, "workspace_bytes %lld < %lld needed", workspace_bytes, need);
  if (!(st = all_given(what, {ws})).ok()) return st;
  if (!(st = all_aligned(what, {dx, dwg, dwu, dh, g, u, x, wg, wu, ws})).ok()) return st;
  return disjoint(what, {dx, dwg, dwu, ws}, {dh, g, u, x, wg, wu});
}

int64_t mx4_codes_bytes(int64_t batch, int64_t rows, int64_t K) {
  if (batch < 0 || rows < 0 || K < 0 || K % 32 || K >= kMaxK || batch > kMaxExtent ||
      rows > kMaxExtent)
    return -1;
  return mul_capped({batch, (rows + 15) / 16, (K + 127) / 128, 1024});
}

int64_t mx4_scales_bytes(int64_t batch, int64_t rows, int64_t K) {
  if (mx4_codes_bytes(batch, rows, K) < 0) return -1;
  return mul_capped({batch, (rows + 15) / 16, (K + 511) / 512, 256});
}

Status check_ffn_plan(int32_t product, const bmm_gated_desc& d) {
  const char* what = "ffn_plan";
  if (product < BMM_FFN_GATED || product > BMM_FFN_MX4_GATED)
    return failw(what, BMM_EINVAL, "product %lld is not a bmm_ffn_product", product);
  if (product != BMM_FFN_MX4_MMA && product != BMM_FFN_MX4_GATED) return check_gated_desc(&d, what);
  if (d.F % 8) return failw(what, BMM_EINVAL, "%lld columns are not a multiple of 8", d.F);
  if (d.K % 32) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32", d.K);
  if (d.F > kMaxLd || mx4_codes_bytes(d.batch, d.M, d.K) < 0 ||
      mx4_codes_bytes(d.batch, d.F, d.K) < 0)
    return failw(what, BMM_EINVAL, "negative or too large (columns <= 2^21, K < 2^22)");
  return Status{};
}

Status check_mx4_convert(const void* mat, const uint8_t* codes, const uint8_t* scales,
                         int64_t batch, int64_t rows, int64_t K, int64_t ld, int32_t elem_type,
                         const char* what) {
  const int64_t size = elem_size(elem_type);
  if (!size)
    return failw(what, BMM_EINVAL, "elem_type %lld is not BMM_ELEM_F32, _F16 or _BF16", elem_type);
  if (batch < 0 || rows < 0 || K < 0) return failw(what, BMM_EINVAL, "negative extent");
  if (K % 32) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32", K);
  const int64_t cb = mx4_codes_bytes(batch, rows, K), sb = mx4_scales_bytes(batch, rows, K);
  if (cb < 0 || sb < 0) return failw(what, BMM_EINVAL, "extent too large (K < 2^22)");
  if (ld < K) return failw(what, BMM_EINVAL, "ld (%lld) < K (%lld)", ld, K);
  if (ld > kMaxExtent || mul_capped({batch, rows, ld, size}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  if (ld % 8) return failw(what, BMM_EALIGN, "ld (%lld) must be a multiple of 8 elements", ld);
  if (batch == 0 || rows == 0 || K == 0) return Status{};
  const Rows m{mat, batch * rows, K * size, ld * size, "the matrix"}, c{codes, 1, cb, 0, "codes"},
      s{scales, 1, sb, 0, "scales"};
  Status st = all_given(what, {m, c, s});
  if (!st.ok()) return st;
  if (!(st = all_aligned(what, {m, c, s})).ok()) return st;
  return disjoint(what, {m, c, s}, {});
}

Status check_mx4_product(const void* D, const uint8_t* A, const uint8_t* As, const uint8_t* B0,
                         const uint8_t* B0s, const uint8_t* B1, const uint8_t* B1s, bool gated,
                         int64_t batch, int64_t M, int64_t N, int64_t K, int64_t ld, int32_t act,
                         int32_t elem_type) {
  const char* what = gated ? "mx4_gated" : "mx4_mma";
  const int64_t size = elem_size(elem_type);
  if (!size || (gated && elem_type == BMM_ELEM_F32))
    return failw(what, BMM_EINVAL, gated ? "elem_type %lld is neither BMM_ELEM_F16 nor _BF16"
                                         : "elem_type %lld is not BMM_ELEM_F32, _F16 or _BF16",
                 elem_type);
  if (gated && (act < BMM_ACT_SILU || act > BMM_ACT_RELU))
    return failw(what, BMM_EINVAL, "act %lld is not a bmm_act", act);
  if (batch < 0 || M < 0 || N < 0 || K < 0) return failw(what, BMM_EINVAL, "negative extent");
  if (N % 8)
    return failw(what, BMM_EINVAL, "%lld columns are not a multiple of 8", N);
  if (K % 32) return failw(what, BMM_EINVAL, "K (%lld) is not a multiple of 32", K);
  const int64_t ab = mx4_codes_bytes(batch, M, K), asb = mx4_scales_bytes(batch, M, K);
  const int64_t bb = mx4_codes_bytes(batch, N, K), bsb = mx4_scales_bytes(batch, N, K);
  if (ab < 0 || asb < 0 || bb < 0 || bsb < 0)
    return failw(what, BMM_EINVAL, "extent too large (K < 2^22)");
  if (ld < N) return failw(what, BMM_EINVAL, "ld (%lld) < %lld columns", ld, N);
  if (ld > kMaxLd) return failw(what, BMM_EINVAL, "ld (%lld) is at most 2^21", ld);
  if (mul_capped({batch, M, ld, size}) < 0)
    return failw(what, BMM_EINVAL, "too large");
  if (ld % 8) return failw(what, BMM_EALIGN, "ld (%lld) must be a multiple of 8 elements", ld);
  if (batch == 0 || M == 0 || N == 0) return Status{};
  const Rows d{D, batch * M, N * size, ld * size, gated ? "H" : "D"},
      a{A, 1, ab, 0, gated ? "X_codes" : "A_codes"},
      as{As, 1, asb, 0, gated ? "X_scales" : "A_scales"},
      b0{B0, 1, bb, 0, gated ? "Wg_codes" : "B_codes"},
      b0s{B0s, 1, bsb, 0, gated ? "Wg_scales" : "B_scales"},
      b1{B1, 1, gated ? bb : 0, 0, "Wu_codes"}, b1s{B1s, 1, gated ? bsb : 0, 0, "Wu_scales"};
  Status st = all_given(what, {d, a, as, b0, b0s, b1, b1s});
  if (!st.ok()) return st;
  if (!(st = all_aligned(what, {d, a, as, b0, b0s, b1, b1s})).ok()) return st;
  return disjoint(what, {d}, {a, as, b0, b0s, b1, b1s});
}

}  // namespace bmm
