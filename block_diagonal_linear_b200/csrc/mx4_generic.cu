// Tiled FMA products with MX4 operands, for every size and both types:
//   forward   Y[r][b*out + o]  = sum_i A[b][r][i] W[b][o][i] (+ bias)   A: MX4 or plain X
//   backward  dX[r][b*in + i]  = sum_o dY[r][b*out + o] W[b][o][i]
//             dW[b][o][i]      = sum_r dY[r][b*out + o] X[b][r][i]
// One kernel computes D[m][n] = sum_k A(m, k) B(n, k) in 64 x 64 tiles, 4 x 4 results a thread and
// 16 steps of k in shared memory at a time; where an operand lies and how it is decoded is its
// loader's business.  Sums are fp32 in the order of k, so results repeat bit for bit.  These kernels
// serve fp32 tensors and the block sizes that the tensor-core kernels do not take; they are bound by
// the FMA pipe.
#include "mx4.cuh"

namespace monarch {

namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

// A(m, k) = X[m][b*cols + k] of a plain (rows, nb*cols) tensor.
template <typename T>
struct PlainRows {
  const T* p;
  int64_t rows, pitch;
  int cols;
  static constexpr bool kFast = true;  // k is the contiguous index
  __device__ float operator()(int b, int64_t m, int64_t k) const {
    return m < rows && k < cols ? mx4::load(p + m * pitch + (int64_t)b * cols + k) : 0.f;
  }
};
// A(m, k) = X[k][b*cols + m]: the same tensor, rows as the inner index.
template <typename T>
struct PlainCols {
  const T* p;
  int64_t rows, pitch;
  int cols;
  static constexpr bool kFast = false;
  __device__ float operator()(int b, int64_t m, int64_t k) const {
    return m < cols && k < rows ? mx4::load(p + k * pitch + (int64_t)b * cols + m) : 0.f;
  }
};
__device__ __forceinline__ float mx4_at(const Mx4View& q, int b, int64_t r, int64_t c) {
  const uint8_t byte = q.codes[q.s.code_row(b, r) + (c >> 1)];
  const uint32_t code = (c & 1) ? byte >> 4 : byte & 15;
  return mx4::decode(code) * mx4::scale_value(q.scales[q.s.scale_at(b, r, (int)(c >> 5))]);
}
// (m, k) = element [b][m][k] of an MX4 tensor.
struct Mx4Rows {
  Mx4View q;
  static constexpr bool kFast = true;
  __device__ float operator()(int b, int64_t m, int64_t k) const {
    return m < q.s.rows && k < q.s.cols ? mx4_at(q, b, m, k) : 0.f;
  }
};
// (m, k) = element [b][k][m].
struct Mx4Cols {
  Mx4View q;
  static constexpr bool kFast = false;
  __device__ float operator()(int b, int64_t m, int64_t k) const {
    return m < q.s.cols && k < q.s.rows ? mx4_at(q, b, k, m) : 0.f;
  }
};

// One 64 x 16 operand tile: consecutive threads walk the operand's contiguous index.
template <class L>
__device__ __forceinline__ void fill(float (*s)[kTile + 1], const L& load, int b, int64_t m0, int64_t k0) {
#pragma unroll
  for (int i = 0; i < kTile * kStep / kThreads; ++i) {
    const int e = i * kThreads + threadIdx.x;
    const int m = L::kFast ? e / kStep : e % kTile, k = L::kFast ? e % kStep : e / kTile;
    s[k][m] = load(b, m0 + m, k0 + k);
  }
}

template <class LA, class LB, typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_fma_kernel(LA la, LB lb, int64_t M, int64_t N, int64_t K, int64_t mtiles, Mx4Out o,
                   const T* __restrict__ bias, T* __restrict__ D) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int b = blockIdx.z;
  const int64_t n0 = (int64_t)blockIdx.y * kTile;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  for (int64_t mt = blockIdx.x; mt < mtiles; mt += gridDim.x) {
    const int64_t m0 = mt * kTile;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kStep) {
      __syncthreads();
      fill(sa, la, b, m0, k0);
      fill(sb, lb, b, n0, k0);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = sa[k][tm + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = sb[k][tn + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + tm + 16 * i;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tn + 16 * j;
        if (n >= N) continue;
        const float v = bias != nullptr ? acc[i][j] + mx4::load(bias + (int64_t)b * N + n) : acc[i][j];
        st_from_f32(D + o.at(b, m, n), v);
      }
    }
  }
}

template <class LA, class LB, typename T>
cudaError_t launch_fma(const LA& la, const LB& lb, int64_t M, int64_t N, int64_t K, int nb, const Mx4Out& o,
                       const void* bias, void* D, cudaStream_t st) {
  const int64_t mt = (M + kTile - 1) / kTile, nt = (N + kTile - 1) / kTile;
  return launch_kernel(mx4_fma_kernel<LA, LB, T>, dim3((unsigned)(mt < (1 << 20) ? mt : (1 << 20)), (unsigned)nt, (unsigned)nb),
                       dim3(kThreads), 0, st, false, la, lb, M, N, K, mt, o, (const T*)bias, (T*)D);
}

// ---------------------------------------------------------------- bias gradient
// Column sums of dY in two steps: every CTA sums kBiasRows rows of 64 columns in fp32 (four row
// lanes, joined in a fixed order), then one thread per column adds the parts in order.
constexpr int kBiasRows = 256, kBiasCols = 64;

template <typename T>
__global__ void __launch_bounds__(256) mx4_dbias_part_kernel(const T* __restrict__ dY, int64_t rows, int64_t cols,
                                                             float* __restrict__ part) {
  __shared__ float s[4][kBiasCols];
  const int c = threadIdx.x % kBiasCols, lane = threadIdx.x / kBiasCols;
  const int64_t col = (int64_t)blockIdx.y * kBiasCols + c;
  const int64_t r0 = (int64_t)blockIdx.x * kBiasRows, r1 = r0 + kBiasRows < rows ? r0 + kBiasRows : rows;
  float acc = 0.f;
  if (col < cols)
    for (int64_t r = r0 + lane; r < r1; r += 4) acc += mx4::load(dY + r * cols + col);
  s[lane][c] = acc;
  __syncthreads();
  if (lane == 0 && col < cols) part[(int64_t)blockIdx.x * cols + col] = (s[0][c] + s[1][c]) + (s[2][c] + s[3][c]);
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dbias_sum_kernel(const float* __restrict__ part, int64_t nparts, int64_t cols,
                                                            T* __restrict__ dbias) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  float acc = 0.f;
  for (int64_t k = 0; k < nparts; ++k) acc += part[k * cols + c];
  st_from_f32(dbias + c, acc);
}

template <typename T>
cudaError_t dbias_t(const void* dY, int64_t rows, int64_t cols, float* part, void* dbias, cudaStream_t st) {
  const int64_t n = (rows + kBiasRows - 1) / kBiasRows;
  if (n > 0) {
    const cudaError_t e = launch_kernel(mx4_dbias_part_kernel<T>, dim3((unsigned)n, (unsigned)((cols + kBiasCols - 1) / kBiasCols)),
                                        dim3(256), 0, st, false, (const T*)dY, rows, cols, part);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(mx4_dbias_sum_kernel<T>, dim3((unsigned)((cols + 255) / 256)), dim3(256), 0, st, false,
                       (const float*)part, n, cols, (T*)dbias);
}

}  // namespace

template <typename TX, typename TY>
static cudaError_t generic_wfwd_t(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y,
                                  cudaStream_t st) {
  const PlainRows<TX> a{(const TX*)X, rows, (int64_t)w.s.nblocks * w.s.cols, w.s.cols};
  return launch_fma<PlainRows<TX>, Mx4Rows, TY>(a, {w}, rows, w.s.rows, w.s.cols, w.s.nblocks, o, bias, Y, st);
}
cudaError_t mx4_generic_wfwd(const void* X, int x_dtype, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o,
                             void* Y, int y_dtype, cudaStream_t st) {
  if (x_dtype == MONARCH_BF16)
    return y_dtype == MONARCH_BF16 ? generic_wfwd_t<__nv_bfloat16, __nv_bfloat16>(X, w, bias, rows, o, Y, st)
                                   : generic_wfwd_t<__nv_bfloat16, float>(X, w, bias, rows, o, Y, st);
  return y_dtype == MONARCH_BF16 ? generic_wfwd_t<float, __nv_bfloat16>(X, w, bias, rows, o, Y, st)
                                 : generic_wfwd_t<float, float>(X, w, bias, rows, o, Y, st);
}

template <typename T>
static cudaError_t generic_bwd_x_t(const void* dY, const Mx4View& w, const Mx4Linear& d, void* dX, cudaStream_t st) {
  const PlainRows<T> a{(const T*)dY, d.rows, (int64_t)d.nb * d.out, d.out};
  return launch_fma<PlainRows<T>, Mx4Cols, T>(a, {w}, d.rows, d.in, d.out, d.nb, Mx4Out::blocks(d.nb, d.in), nullptr, dX, st);
}
cudaError_t mx4_generic_bwd_x(const void* dY, const Mx4View& w, const Mx4Linear& d, void* dX, cudaStream_t st) {
  return d.dtype == MONARCH_BF16 ? generic_bwd_x_t<__nv_bfloat16>(dY, w, d, dX, st)
                                 : generic_bwd_x_t<float>(dY, w, d, dX, st);
}

template <typename T>
static cudaError_t generic_bwd_w_t(const void* dY, const Mx4View& x, const Mx4Linear& d, void* dW, cudaStream_t st) {
  const PlainCols<T> a{(const T*)dY, d.rows, (int64_t)d.nb * d.out, d.out};
  return launch_fma<PlainCols<T>, Mx4Cols, T>(a, {x}, d.out, d.in, d.rows, d.nb, Mx4Out{(int64_t)d.out * d.in, d.in, 1},
                                                        nullptr, dW, st);
}
cudaError_t mx4_generic_bwd_w(const void* dY, const Mx4View& x, const Mx4Linear& d, void* dW, cudaStream_t st) {
  return d.dtype == MONARCH_BF16 ? generic_bwd_w_t<__nv_bfloat16>(dY, x, d, dW, st)
                                 : generic_bwd_w_t<float>(dY, x, d, dW, st);
}

size_t mx4_dbias_bytes(int64_t rows, int64_t cols) {
  return (size_t)((rows + kBiasRows - 1) / kBiasRows) * (size_t)cols * 4;
}
cudaError_t mx4_dbias(const void* dY, int64_t rows, int64_t cols, int dtype, float* part, void* dbias,
                      cudaStream_t st) {
  return dtype == MONARCH_BF16 ? dbias_t<__nv_bfloat16>(dY, rows, cols, part, dbias, st)
                               : dbias_t<float>(dY, rows, cols, part, dbias, st);
}

}  // namespace monarch
