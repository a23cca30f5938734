// Rounding to MX4 and back.
//
// quantise: of every 32 values along a row, byte = exponent field of the largest magnitude - 2, each
// value times 2^(127 - byte) (exact) to the nearest E2M1 code.  One thread takes one scale block:
// its 32 values stay in registers between the maximum and the rounding, so X is read once.  Four
// neighbouring threads share a row's 4 scale blocks and a warp takes 8 rows: reads are 256
// (bf16) or 512 (fp32) contiguous bytes a row, the codes 64, and a scale tile's 4 bytes of a row
// leave as one store.  Threads behind the last row or scale block write the tile's zero bytes.
// Bound by memory: elem size + 17/32 bytes a value.
//
// dequantise: the same split, codes in and values out; code times scale is exact in both types.
#include "mx4.cuh"

namespace monarch {

namespace {

constexpr int kQThreads = 256, kQRows = kQThreads / 4;

// Address of element (b, r, c) of the plain tensor.
template <typename T>
__device__ __forceinline__ int64_t plain_at(const Mx4Shape& s, bool by_block, int b, int64_t r, int64_t c) {
  return by_block ? ((int64_t)b * s.rows + r) * s.cols + c : r * ((int64_t)s.nblocks * s.cols) + (int64_t)b * s.cols + c;
}

__device__ __forceinline__ void unpack16(const uint4& u, float* v, const __nv_bfloat16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4& u, float* v, const float*) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}

// VEC: rows and scale blocks of the plain tensor start on 16 bytes (cols * element size is a
// multiple of 16), so that every 16 bytes of a block lie wholly inside or outside the row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    mx4_quantise_kernel(const T* __restrict__ X, Mx4Shape s, bool by_block, uint8_t* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t rtiles) {
  constexpr int PER = 16 / sizeof(T);
  const int b = blockIdx.z, kb = blockIdx.y * 4 + (threadIdx.x & 3);
  for (int64_t rt = blockIdx.x; rt < rtiles; rt += gridDim.x) {
    const int64_t r = rt * kQRows + threadIdx.x / 4;
    const bool mine = r < s.rows && kb < s.kblocks();
    float v[32];
    if (mine) {
      const T* p = X + plain_at<T>(s, by_block, b, r, (int64_t)kb * 32);
      const int n = s.cols - kb * 32;
      if (VEC) {
        uint4 u[32 / PER];
#pragma unroll
        for (int i = 0; i < 32 / PER; ++i) u[i] = i * PER < n ? *(const uint4*)(p + i * PER) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 32 / PER; ++i) unpack16(u[i], v + i * PER, (const T*)nullptr);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < n ? mx4::load(p + i) : 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
    uint32_t top = 0;  // magnitudes order like their bits, NaN above infinity
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    const uint32_t byte = mx4::scale_byte(top);
    if (mine) {
      const float f = mx4::inv_scale(byte);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = byte == 255 ? 0.f : v[8 * i + e] * f;
        w[i] = mx4::encode8(t);
      }
      *(uint4*)(codes + s.code_row(b, r) + (int64_t)kb * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the four scale bytes of a row in one store; pad rows and blocks hold 0
    uint32_t word = byte << (8 * (threadIdx.x & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if ((threadIdx.x & 3) == 0) *(uint32_t*)(scales + s.scale_at(b, r, kb)) = word;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    mx4_dequantise_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, Mx4Shape s, bool by_block,
                          T* __restrict__ X, int64_t rtiles) {
  constexpr int PER = 16 / sizeof(T);
  const int b = blockIdx.z, kb = blockIdx.y * 4 + (threadIdx.x & 3);
  if (kb >= s.kblocks()) return;
  for (int64_t rt = blockIdx.x; rt < rtiles; rt += gridDim.x) {
    const int64_t r = rt * kQRows + threadIdx.x / 4;
    if (r >= s.rows) return;
    const uint4 u = __ldg((const uint4*)(codes + s.code_row(b, r) + (int64_t)kb * 16));
    const float f = mx4::scale_value(__ldg(scales + s.scale_at(b, r, kb)));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    T* p = X + plain_at<T>(s, by_block, b, r, (int64_t)kb * 32);
    const int n = s.cols - kb * 32;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = mx4::decode((w[i / 8] >> (4 * (i % 8))) & 15u) * f;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < 32 / PER; ++i) {
        if (i * PER >= n) break;
        uint4 o;
        if (sizeof(T) == 2)
          o = make_uint4(ptx::pack_bf16x2(v[i * PER], v[i * PER + 1]), ptx::pack_bf16x2(v[i * PER + 2], v[i * PER + 3]),
                         ptx::pack_bf16x2(v[i * PER + 4 % PER], v[i * PER + 5 % PER]),
                         ptx::pack_bf16x2(v[i * PER + 6 % PER], v[i * PER + 7 % PER]));
        else
          o = make_uint4(__float_as_uint(v[i * PER]), __float_as_uint(v[i * PER + 1]), __float_as_uint(v[i * PER + 2]),
                         __float_as_uint(v[i * PER + 3]));
        *(uint4*)(p + i * PER) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) st_from_f32(p + i, v[i]);
    }
  }
}

bool rows_of_16_bytes(const Mx4Shape& s, int dtype) { return (int64_t)s.cols * (dtype == MONARCH_BF16 ? 2 : 4) % 16 == 0; }

template <typename T, bool VEC>
cudaError_t quantise_t(const void* X, const Mx4Shape& s, bool by_block, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int64_t rt = s.ratoms() * (128 / kQRows);
  return launch_kernel(mx4_quantise_kernel<T, VEC>, dim3((unsigned)(rt < (1 << 20) ? rt : (1 << 20)), (unsigned)s.katoms(), (unsigned)s.nblocks),
                       dim3(kQThreads), 0, st, false, (const T*)X, s, by_block, codes, scales, rt);
}
template <typename T, bool VEC>
cudaError_t dequantise_t(const Mx4View& q, bool by_block, void* X, cudaStream_t st) {
  const int64_t rt = (q.s.rows + kQRows - 1) / kQRows;
  return launch_kernel(mx4_dequantise_kernel<T, VEC>, dim3((unsigned)(rt < (1 << 20) ? rt : (1 << 20)), (unsigned)q.s.katoms(), (unsigned)q.s.nblocks),
                       dim3(kQThreads), 0, st, false, q.codes, q.scales, q.s, by_block, (T*)X, rt);
}

}  // namespace

cudaError_t mx4_quantise(const void* X, const Mx4Shape& s, bool by_block, int dtype, uint8_t* codes, uint8_t* scales,
                         cudaStream_t st) {
  const bool vec = rows_of_16_bytes(s, dtype);
  if (dtype == MONARCH_BF16)
    return vec ? quantise_t<__nv_bfloat16, true>(X, s, by_block, codes, scales, st)
               : quantise_t<__nv_bfloat16, false>(X, s, by_block, codes, scales, st);
  return vec ? quantise_t<float, true>(X, s, by_block, codes, scales, st)
             : quantise_t<float, false>(X, s, by_block, codes, scales, st);
}

cudaError_t mx4_dequantise(const Mx4View& q, bool by_block, int dtype, void* X, cudaStream_t st) {
  const bool vec = rows_of_16_bytes(q.s, dtype);
  if (dtype == MONARCH_BF16)
    return vec ? dequantise_t<__nv_bfloat16, true>(q, by_block, X, st) : dequantise_t<__nv_bfloat16, false>(q, by_block, X, st);
  return vec ? dequantise_t<float, true>(q, by_block, X, st) : dequantise_t<float, false>(q, by_block, X, st);
}

}  // namespace monarch
