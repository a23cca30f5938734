// C ABI of the microscaled 4-bit (MX4) operators: argument checks and the choice of kernels.
#include "mx4.cuh"

#include <algorithm>

namespace monarch {

namespace {

// Limits that keep every launch grid and tensor-map extent in range: rows and columns of one
// block's matrix, and the blocks (a grid dimension).
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;
constexpr int kMaxCols = 1 << 20, kMaxBlocks = 65535;
constexpr int64_t kMaxWidth = int64_t(1) << 22;  // nblocks * cols

size_t al256(size_t b) { return (b + 255) & ~size_t(255); }
int64_t elem_bytes(int dtype) { return dtype == MONARCH_BF16 ? 2 : 4; }

int check_size(int64_t rows, int nb, int cols, int dtype) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  if (rows < 0 || nb <= 0 || cols <= 0) return MONARCH_ERR_DIMS;
  if (rows > kMaxRows || nb > kMaxBlocks || cols > kMaxCols || (int64_t)nb * cols > kMaxWidth)
    return MONARCH_ERR_UNSUPPORTED;
  return MONARCH_OK;
}
int check(const monarch_mx4_dims* d) {
  if (d == nullptr) return MONARCH_ERR_NULL;
  return check_size(d->rows, d->nblocks, d->cols, d->dtype);
}
Mx4Shape shape_of(const monarch_mx4_dims& d) { return Mx4Shape{d.rows, d.nblocks, d.cols}; }

int check(const monarch_mx4_linear_dims* d) {
  if (d == nullptr) return MONARCH_ERR_NULL;
  const int rc = check_size(d->rows, d->nblocks, d->in_blk, d->dtype);
  return rc != MONARCH_OK ? rc : check_size(d->rows, d->nblocks, d->out_blk, d->dtype);
}
Mx4Linear to_linear(const monarch_mx4_linear_dims& d) {
  return Mx4Linear{d.rows, d.nblocks, d.in_blk, d.out_blk, d.has_bias != 0, d.dtype};
}

int check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return MONARCH_ERR_NULL;
  for (const void* p : ps)
    if (!aligned16(p)) return MONARCH_ERR_ALIGN;
  return MONARCH_OK;
}

struct Range {
  uintptr_t p;
  uint64_t n;
  Range(const void* q, int64_t bytes) : p((uintptr_t)q), n(q != nullptr && bytes > 0 ? (uint64_t)bytes : 0) {}
};
// Outputs are disjoint from the inputs and from each other.
int check_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  auto hit = [](const Range& a, const Range& b) { return a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n; };
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (hit(*o, i)) return MONARCH_ERR_ALIAS;
    for (const Range* o2 = o + 1; o2 != outs.end(); ++o2)
      if (hit(*o, *o2)) return MONARCH_ERR_ALIAS;
  }
  return MONARCH_OK;
}
int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MONARCH_OK;
  if (ws == nullptr || have < need) return MONARCH_ERR_WORKSPACE;
  return ((uintptr_t)ws & 255u) != 0 ? MONARCH_ERR_ALIGN : MONARCH_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MONARCH_OK : MONARCH_ERR_CUDA; }

// Up to this many rows a plain X goes through the few-rows kernels (one launch, the weight read as it is);
// beyond them the weight is expanded for the bf16 products.  Both measured, 4096 -> 4096 and four 250 -> 1000 blocks:
// bf16 64 rows 21.4 and 8.2 us against 20.7 and 6.6 in two launches; fp32 32 rows 20.6 and 7.0, 64 rows 57.6 and 9.5
// against 30.5 and 9.4.
// So do more rows of a small weight, for which two launches are the greater cost: 300 rows of four 256 -> 256 blocks 6.2
// and 6.5, 1000 of 512 -> 128 5.0 and 7.4, 128 of sixty-four 64 -> 64 blocks 5.4 and 5.1; fp32 128 of four 256 -> 256 5.9
// and 9.8, 100 of sixty-four 64 -> 64 7.4 and 6.8.
bool few_rows(const Mx4Linear& d) {
  return d.rows <= (d.dtype == MONARCH_BF16 ? 64 : 32) || mx4_rows_little(d.w(), d.rows, d.dtype == MONARCH_BF16 ? 1 : 3);
}

size_t wfwd_workspace(const Mx4Linear& d) { return few_rows(d) ? 0 : mx4_gemm_fwd_bytes(d); }
size_t bwd_workspace(const Mx4Linear& d) { return d.rows == 0 ? 0 : mx4_gemm_bwd_bytes(d); }

Mx4Shape r_shape(const monarch_dims& d) { return Mx4Shape{d.out1, d.nb1, d.in1}; }
Mx4Shape l_shape(const monarch_dims& d) { return Mx4Shape{d.out2, d.nb2, d.in2}; }

int check_monarch(const monarch_dims* d) {
  int rc = monarch_validate(d);
  if (rc != MONARCH_OK) return rc;
  if ((rc = check_size(d->out1, d->nb1, d->in1, d->dtype)) != MONARCH_OK) return rc;
  return check_size(d->out2, d->nb2, d->in2, d->dtype);
}

// Whether the Monarch map is two products by the few-rows kernels, with the middle vector in fp32 in the workspace;
// else the factors are expanded there and the plain forward runs.  us, both ways: 200 rows of n = 4096 20.7 and 23.3,
// 400 36 and 25; 400 of n = 1024 11.1 and 17.0, 1000 23.0 and 17.6; four 256 -> 256 -> 1024 blocks, 100 rows 17 and 34,
// 400 56 and 36.  The plain forward's generic kernels are slower at any number (1000 rows of four 256 -> 256 -> 256
// blocks 47 and 460).
bool few_rows(const monarch_dims& d) {
  if (d.rows <= 64) return true;
  return mx4_rows_work(r_shape(d), d.rows) + mx4_rows_work(l_shape(d), d.rows) <= 13000 || monarch_fwd_path(&d) == 0;
}

// The few-rows kernels take a Monarch map this many rows at a time, with room for the middle vectors of so many.
constexpr int64_t kMonarchPass = 65536;
static_assert(kMonarchPass <= kRowsMost, "rows of one launch");

size_t monarch_workspace(const monarch_dims& d) {
  const Shape s = to_shape(d);
  if (few_rows(d)) return al256((size_t)(std::min(s.rows, kMonarchPass) * s.n_mid() * 4));
  const int64_t es = elem_bytes(d.dtype);
  return al256((size_t)(s.n_R() * es)) + al256((size_t)(s.n_L() * es));
}

}  // namespace
}  // namespace monarch

using namespace monarch;

extern "C" {

size_t monarch_mx4_code_bytes(const monarch_mx4_dims* d) {
  return check(d) != MONARCH_OK ? 0 : (size_t)shape_of(*d).code_bytes();
}
size_t monarch_mx4_scale_bytes(const monarch_mx4_dims* d) {
  return check(d) != MONARCH_OK ? 0 : (size_t)shape_of(*d).scale_bytes();
}

int monarch_mx4_quantise(const void* X, const monarch_mx4_dims* d, void* codes, void* scales, void* stream) {
  int rc = check(d);
  if (rc != MONARCH_OK) return rc;
  if (d->rows == 0) return MONARCH_OK;
  if ((rc = check_ptrs({X, codes, scales})) != MONARCH_OK) return rc;
  const Mx4Shape s = shape_of(*d);
  if ((rc = check_alias({Range(codes, s.code_bytes()), Range(scales, s.scale_bytes())},
                        {Range(X, s.rows * s.nblocks * s.cols * elem_bytes(d->dtype))})) != MONARCH_OK)
    return rc;
  return status_of(mx4_quantise(X, s, d->by_block != 0, d->dtype, (uint8_t*)codes, (uint8_t*)scales, (cudaStream_t)stream));
}

int monarch_mx4_dequantise(const void* codes, const void* scales, const monarch_mx4_dims* d, void* X, void* stream) {
  int rc = check(d);
  if (rc != MONARCH_OK) return rc;
  if (d->rows == 0) return MONARCH_OK;
  if ((rc = check_ptrs({codes, scales, X})) != MONARCH_OK) return rc;
  const Mx4Shape s = shape_of(*d);
  if ((rc = check_alias({Range(X, s.rows * s.nblocks * s.cols * elem_bytes(d->dtype))},
                        {Range(codes, s.code_bytes()), Range(scales, s.scale_bytes())})) != MONARCH_OK)
    return rc;
  const Mx4View q{(const uint8_t*)codes, (const uint8_t*)scales, s};
  return status_of(mx4_dequantise(q, d->by_block != 0, d->dtype, X, (cudaStream_t)stream));
}

size_t monarch_mx4_linear_wfwd_workspace_bytes(const monarch_mx4_linear_dims* d) {
  return check(d) != MONARCH_OK ? 0 : wfwd_workspace(to_linear(*d));
}
size_t monarch_mx4_linear_bwd_workspace_bytes(const monarch_mx4_linear_dims* d) {
  return check(d) != MONARCH_OK ? 0 : bwd_workspace(to_linear(*d));
}

int monarch_mx4_linear_path(const monarch_mx4_linear_dims* ld, int product) {
  if (check(ld) != MONARCH_OK) return -1;
  const Mx4Linear d = to_linear(*ld);
  switch (product) {
    case 0: return mx4_rows_quantised(d.w(), d.rows) ? kMx4Token : mx4_tc_path(d);
    case 1: return few_rows(d) ? mx4_rows_path(d.w(), d.rows, d.dtype == MONARCH_BF16 ? 1 : 3) : mx4_gemm_fwd_path(d);
    case 2: return mx4_gemm_dx_path(d);
    case 3: return mx4_gemm_dw_path(d);
    default: return -1;
  }
}
int monarch_mx4_fwd_path(const monarch_dims* d) {
  if (check_monarch(d) != MONARCH_OK) return -1;
  return few_rows(*d) ? 0 : monarch_fwd_path(d);
}

int monarch_mx4_linear_fwd(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                           const void* bias, const monarch_mx4_linear_dims* ld, void* Y, void* stream) {
  int rc = check(ld);
  if (rc != MONARCH_OK) return rc;
  if (ld->rows == 0) return MONARCH_OK;
  const Mx4Linear d = to_linear(*ld);
  if ((rc = check_ptrs({x_codes, x_scales, w_codes, w_scales, Y})) != MONARCH_OK) return rc;
  if (d.has_bias && (rc = check_ptrs({bias})) != MONARCH_OK) return rc;
  const int64_t es = elem_bytes(d.dtype), n_out = (int64_t)d.nb * d.out;
  const Mx4Shape xs = d.x(), ws = d.w();
  if ((rc = check_alias({Range(Y, d.rows * n_out * es)},
                        {Range(x_codes, xs.code_bytes()), Range(x_scales, xs.scale_bytes()), Range(w_codes, ws.code_bytes()),
                         Range(w_scales, ws.scale_bytes()), Range(d.has_bias ? bias : nullptr, n_out * es)})) != MONARCH_OK)
    return rc;
  const Mx4View x{(const uint8_t*)x_codes, (const uint8_t*)x_scales, xs}, w{(const uint8_t*)w_codes, (const uint8_t*)w_scales, ws};
  if (mx4_rows_quantised(ws, d.rows))
    return status_of(mx4_rows_fwd(x, w, d.has_bias ? bias : nullptr, Mx4Out::blocks(d.nb, d.out), Y, d.dtype, (cudaStream_t)stream));
  int* status = status_ptr();
  if (status == nullptr) return MONARCH_ERR_CUDA;
  return status_of(mx4_tc_fwd(x, w, d.has_bias ? bias : nullptr, d, Y, status, (cudaStream_t)stream));
}

int monarch_mx4_linear_wfwd(const void* X, const void* w_codes, const void* w_scales, const void* bias,
                            const monarch_mx4_linear_dims* ld, void* Y, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int rc = check(ld);
  if (rc != MONARCH_OK) return rc;
  if (ld->rows == 0) return MONARCH_OK;
  const Mx4Linear d = to_linear(*ld);
  if ((rc = check_ptrs({X, w_codes, w_scales, Y})) != MONARCH_OK) return rc;
  if (d.has_bias && (rc = check_ptrs({bias})) != MONARCH_OK) return rc;
  const size_t need = wfwd_workspace(d);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != MONARCH_OK) return rc;
  const int64_t es = elem_bytes(d.dtype), n_out = (int64_t)d.nb * d.out;
  const Mx4Shape ws = d.w();
  if ((rc = check_alias({Range(Y, d.rows * n_out * es), Range(workspace, (int64_t)need)},
                        {Range(X, d.rows * d.nb * d.in * es), Range(w_codes, ws.code_bytes()),
                         Range(w_scales, ws.scale_bytes()), Range(d.has_bias ? bias : nullptr, n_out * es)})) != MONARCH_OK)
    return rc;
  const Mx4View w{(const uint8_t*)w_codes, (const uint8_t*)w_scales, ws};
  const void* b = d.has_bias ? bias : nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  if (few_rows(d))
    return status_of(mx4_rows_fwd(X, d.dtype, w, b, d.rows, Mx4Out::blocks(d.nb, d.out), Y, d.dtype, false, st));
  int* status = status_ptr();
  if (status == nullptr) return MONARCH_ERR_CUDA;
  return status_of(mx4_gemm_fwd(X, w, b, d, Y, workspace, status, st));
}

int monarch_mx4_linear_bwd(const void* dY, const void* x_codes, const void* x_scales, const void* w_codes,
                           const void* w_scales, const monarch_mx4_linear_dims* ld, void* dX, void* dW, void* dbias,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check(ld);
  if (rc != MONARCH_OK) return rc;
  const Mx4Linear d = to_linear(*ld);
  // the operands that the wanted gradients read
  if (d.rows > 0 && (rc = check_ptrs({dY})) != MONARCH_OK) return rc;
  if (d.rows > 0 && dX != nullptr && (rc = check_ptrs({w_codes, w_scales, dX})) != MONARCH_OK) return rc;
  if (d.rows > 0 && dW != nullptr && (rc = check_ptrs({x_codes, x_scales, dW})) != MONARCH_OK) return rc;
  if (dW != nullptr && !aligned16(dW)) return MONARCH_ERR_ALIGN;
  if (d.has_bias && (rc = check_ptrs({dbias})) != MONARCH_OK) return rc;
  const size_t need = bwd_workspace(d);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != MONARCH_OK) return rc;
  const int64_t es = elem_bytes(d.dtype), n_out = (int64_t)d.nb * d.out;
  const Mx4Shape xs = d.x(), ws = d.w();
  if ((rc = check_alias({Range(dX, d.rows * d.nb * d.in * es), Range(dW, n_out * d.in * es),
                         Range(d.has_bias ? dbias : nullptr, n_out * es), Range(workspace, (int64_t)need)},
                        {Range(dY, d.rows * n_out * es), Range(x_codes, xs.code_bytes()), Range(x_scales, xs.scale_bytes()),
                         Range(w_codes, ws.code_bytes()), Range(w_scales, ws.scale_bytes())})) != MONARCH_OK)
    return rc;
  const Mx4View x{(const uint8_t*)x_codes, (const uint8_t*)x_scales, xs}, w{(const uint8_t*)w_codes, (const uint8_t*)w_scales, ws};
  cudaStream_t st = (cudaStream_t)stream;
  if (d.rows == 0) {  // nothing to sum
    if (dW != nullptr && cudaMemsetAsync(dW, 0, (size_t)(n_out * d.in * es), st) != cudaSuccess) return MONARCH_ERR_CUDA;
    return d.has_bias ? status_of(cudaMemsetAsync(dbias, 0, (size_t)(n_out * es), st)) : MONARCH_OK;
  }
  int* status = status_ptr();
  if (status == nullptr) return MONARCH_ERR_CUDA;
  return status_of(mx4_gemm_bwd(dY, x, w, d, dX, dW, d.has_bias ? dbias : nullptr, workspace, status, st));
}

size_t monarch_mx4_fwd_workspace_bytes(const monarch_dims* d) {
  return check_monarch(d) != MONARCH_OK ? 0 : monarch_workspace(*d);
}

int monarch_mx4_fwd(const void* X, const void* r_codes, const void* r_scales, const void* l_codes, const void* l_scales,
                    const monarch_dims* d, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_monarch(d);
  if (rc != MONARCH_OK) return rc;
  if (d->rows == 0) return MONARCH_OK;
  if ((rc = check_ptrs({X, r_codes, r_scales, l_codes, l_scales, Y})) != MONARCH_OK) return rc;
  const size_t need = monarch_workspace(*d);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != MONARCH_OK) return rc;
  const Shape s = to_shape(*d);
  const int64_t es = elem_bytes(d->dtype);
  const Mx4Shape rs = r_shape(*d), ls = l_shape(*d);
  if ((rc = check_alias({Range(Y, s.rows * s.n_out() * es), Range(workspace, (int64_t)need)},
                        {Range(X, s.rows * s.n_in() * es), Range(r_codes, rs.code_bytes()), Range(r_scales, rs.scale_bytes()),
                         Range(l_codes, ls.code_bytes()), Range(l_scales, ls.scale_bytes())})) != MONARCH_OK)
    return rc;
  const Mx4View r{(const uint8_t*)r_codes, (const uint8_t*)r_scales, rs}, l{(const uint8_t*)l_codes, (const uint8_t*)l_scales, ls};
  cudaStream_t st = (cudaStream_t)stream;
  if (few_rows(*d)) {
    // U = blockdiag(R) X, written through P, then blockdiag(L) of contiguous slices, through P_out.  The
    // second kernel may ask for L at once: whatever wrote it had ended when the first began.
    const Mx4Out out = s.out_transpose ? Mx4Out::transposed(s.nb2, s.out2) : Mx4Out::blocks(s.nb2, s.out2);
    for (int64_t r0 = 0; r0 < s.rows; r0 += kMonarchPass) {
      const int64_t rows = std::min(s.rows - r0, kMonarchPass);
      const char* x = (const char*)X + r0 * s.n_in() * es;
      char* y = (char*)Y + r0 * s.n_out() * es;
      if (mx4_rows_fwd(x, d->dtype, r, nullptr, rows, Mx4Out::transposed(s.nb1, s.out1), workspace, MONARCH_F32, false, st) != cudaSuccess ||
          mx4_rows_fwd(workspace, MONARCH_F32, l, nullptr, rows, out, y, d->dtype, true, st) != cudaSuccess)
        return MONARCH_ERR_CUDA;
    }
    return MONARCH_OK;
  }
  char* R = (char*)workspace;
  char* L = R + al256((size_t)(s.n_R() * es));
  if (mx4_dequantise(r, true, d->dtype, R, st) != cudaSuccess || mx4_dequantise(l, true, d->dtype, L, st) != cudaSuccess)
    return MONARCH_ERR_CUDA;
  return fwd_dispatch(X, R, L, Y, s, d->dtype, st);
}

}  // extern "C"
