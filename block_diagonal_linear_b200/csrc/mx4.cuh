// Microscaled 4-bit (MX4) tensors: layout, element conversions and the launchers of mx4*.cu.
//
// A tensor of nblocks matrices of (rows, cols) is cut along cols into scale blocks of 32 (zeros
// behind the end of a row).  Every value is an E2M1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign
// bit) times its block's scale 2^(byte - 127) (E8M0; byte 255 stands for NaN).
//   codes   [nblocks][rows][ceil(cols / 32) * 16] bytes, element 2i in the low half of byte i
//   scales  [nblocks][ceil(rows / 128)][ceil(cols / 128)][512] bytes: the 128 rows x 4 scale blocks
//           of a tile at (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4, which is the order a
//           tcgen05.cp of 32 lanes x 128 bits wants; rows and blocks behind the end hold byte 0.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace monarch {

struct Mx4Shape {
  int64_t rows;
  int nblocks, cols;
  __host__ __device__ int kblocks() const { return (cols + 31) / 32; }         // scale blocks of a row
  __host__ __device__ int pitch() const { return kblocks() * 16; }             // bytes of a row's codes
  __host__ __device__ int katoms() const { return (cols + 127) / 128; }        // scale tiles along a row
  __host__ __device__ int64_t ratoms() const { return (rows + 127) / 128; }    // scale tiles along the rows
  __host__ __device__ int64_t code_bytes() const { return (int64_t)nblocks * rows * pitch(); }
  __host__ __device__ int64_t scale_bytes() const { return (int64_t)nblocks * ratoms() * katoms() * 512; }
  __host__ __device__ int64_t code_row(int b, int64_t r) const { return ((int64_t)b * rows + r) * pitch(); }
  // offset of the scale byte of (block b, row r, scale block kb)
  __host__ __device__ int64_t scale_at(int b, int64_t r, int kb) const {
    return ((((int64_t)b * ratoms() + (r >> 7)) * katoms() + (kb >> 2)) << 9) +
           ((r & 31) << 4) + (((r >> 5) & 3) << 2) + (kb & 3);
  }
};

struct Mx4View {  // codes and scales of one tensor
  const uint8_t* codes;
  const uint8_t* scales;
  Mx4Shape s;
};

namespace mx4 {

// One element in fp32.  A plain load: the header's __ldg of a bf16 is an assembly statement that the
// compiler takes to have no effects, and it may then be issued ahead of the bounds test before it.
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)*(const uint16_t*)p << 16);
}

// Scale byte of a block whose largest magnitude has these fp32 bits (sign cleared):
// floor(log2(amax)) - 2 + 127, not below 0; 255 for a block with an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? 255u : (uint32_t)(e > 2 ? e - 2 : 0);
}
// 2^(127 - byte): what a block's values are multiplied by before they are rounded.  Exact for
// byte 0 .. 252; the NaN byte gives 0 (its codes carry nothing).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return byte == 255 ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127), a subnormal for byte 0.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}
// Eight values to codes (v[0] in the lowest four bits): nearest, ties to the even code, cut at 6.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Eight codes to bf16 without their scale, divided by 2^126: the E2M1 exponent and mantissa bits land
// on the bf16 ones, so that one multiplication by a power of two finishes the job (a code of 0.5 is a
// bf16 subnormal here and becomes a normal number by it).  p[j] holds codes j (low half) and j + 4.
__device__ __forceinline__ void spread8(uint32_t w, uint32_t (&p)[4]) {
  p[0] = ((w << 12) & 0x80008000u) | ((w << 6) & 0x01c001c0u);
  p[1] = ((w << 8) & 0x80008000u) | ((w << 2) & 0x01c001c0u);
  p[2] = ((w << 4) & 0x80008000u) | ((w >> 2) & 0x01c001c0u);
  p[3] = (w & 0x80008000u) | ((w >> 6) & 0x01c001c0u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes and their scale byte to bf16 pairs (2i, 2i + 1); every product is exact, subnormals and all.
__device__ __forceinline__ void values8(uint32_t w, uint32_t byte, uint32_t (&v)[4]) {
  const uint32_t s = (byte == 0 ? 0x0040u : byte == 255 ? 0x7fc0u : byte << 7) * 0x00010001u;  // 2^(byte - 127)
  uint32_t p[4];
  spread8(w, p);
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = mul_bf16x2(mul_bf16x2(p[j], 0x7e807e80u), s);  // 2^126 first
  v[0] = __byte_perm(p[0], p[1], 0x5410);
  v[1] = __byte_perm(p[2], p[3], 0x5410);
  v[2] = __byte_perm(p[0], p[1], 0x7632);
  v[3] = __byte_perm(p[2], p[3], 0x7632);
}

// fp32 bits whose upper half is a NaN if they are one: a NaN's payload may lie in the lower half alone, and
// the upper half by itself would then be an infinity.
__device__ __forceinline__ uint32_t nan_in_top(uint32_t bits) {
  return (bits << 1) > 0xff000000u ? bits | 0x00400000u : bits;
}

// Words o .. o + 4 of eight (o in 0 .. 3).
__device__ __forceinline__ void pick5(const uint32_t (&w)[8], int o, uint32_t (&r)[5]) {
  uint32_t t[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = (o & 2) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) r[i] = (o & 1) ? t[i + 1] : t[i];
}
// Eight values from an address of any alignment, n of them (<= 0: none) inside the row, zeros behind it: the
// aligned 16-byte words that hold them, shifted into place.  end: the end of the tensor (a tensor begins
// on 16 bytes), behind which no word may reach.  x: bf16 pairs or fp32 bits.
__device__ __forceinline__ void load8_any(const __nv_bfloat16* p, int n, const __nv_bfloat16* end, uint32_t (&x)[8]) {
  uint32_t r[4] = {};
  if (n > 0) {
    const uintptr_t a = (uintptr_t)p & ~(uintptr_t)15;
    const int at = (int)((uintptr_t)p & 15), last = at + 2 * min(n, 8);  // bytes from a
    if (a + (last > 16 ? 32 : 16) <= (uintptr_t)end) {
      const uint4 u = *(const uint4*)a, v = last > 16 ? *(const uint4*)(a + 16) : make_uint4(0, 0, 0, 0);
      const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      uint32_t t[5];
      pick5(w, at >> 2, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = __byte_perm(t[i], t[i + 1], (at & 2) ? 0x5432u : 0x3210u);
      if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] &= (2 * i < n ? 0xffffu : 0u) | (2 * i + 1 < n ? 0xffff0000u : 0u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) r[i / 2] |= (uint32_t)*(const uint16_t*)(p + i) << (16 * (i & 1));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = r[i];
}
__device__ __forceinline__ void load8_any(const float* p, int n, const float* end, uint32_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0;
  if (n <= 0) return;
  const uintptr_t a = (uintptr_t)p & ~(uintptr_t)15;
  const int at = (int)((uintptr_t)p & 15) >> 2;
  if (n >= 8 && a + 48 <= (uintptr_t)end) {
    const uint4 u = *(const uint4*)a, v = *(const uint4*)(a + 16), q = at ? *(const uint4*)(a + 32) : make_uint4(0, 0, 0, 0);
    const uint32_t w0[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w}, w1[8] = {v.x, v.y, v.z, v.w, q.x, q.y, q.z, q.w};
    uint32_t t0[5], t1[5];
    pick5(w0, at, t0);
    pick5(w1, at, t1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = t0[i];
      x[4 + i] = t1[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) x[i] = __float_as_uint(p[i]);
  }
}

// A warp's 32 rows x 128 bytes of results: written to shared memory as 128-byte swizzled lines (one row a
// lane; the layout that a TMA store of 32 rows takes), and from there to rows of any alignment.
template <typename T, int CC>
__device__ __forceinline__ void slab_write(uint32_t slab, int lane, const uint32_t (&v)[CC]) {
  static_assert(CC * sizeof(T) == 128, "a row is 128 bytes");
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t at = slab + lane * 128 + (((uint32_t)q ^ (uint32_t)(lane & 7)) << 4);
    if (sizeof(T) == 2)
      ptx::st_shared_v4(at, ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 0) % CC]), __uint_as_float(v[(8 * q + 1) % CC])),
                        ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 2) % CC]), __uint_as_float(v[(8 * q + 3) % CC])),
                        ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 4) % CC]), __uint_as_float(v[(8 * q + 5) % CC])),
                        ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 6) % CC]), __uint_as_float(v[(8 * q + 7) % CC])));
    else
      ptx::st_shared_v4(at, v[(4 * q) % CC], v[(4 * q + 1) % CC], v[(4 * q + 2) % CC], v[(4 * q + 3) % CC]);
  }
}
// rows, cols: how many of the 32 and CC are stored; lanes along the columns, eight rows in flight (row by
// row the loads' latency bounded products of odd widths).
template <typename T, int CC>
__device__ __forceinline__ void slab_store(const uint8_t* slab, int lane, T* dst, int64_t pitch, int rows, int cols) {
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {
    T v[8][CC / 32];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < CC / 32; ++e) {
        const int byte = (e * 32 + lane) * (int)sizeof(T);
        v[i][e] = *(const T*)(slab + (r0 + i) * 128 + (((byte >> 4) ^ i) << 4) + (byte & 15));
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < CC / 32; ++e)
        if (r0 + i < rows && e * 32 + lane < cols) dst[(r0 + i) * pitch + e * 32 + lane] = v[i][e];
  }
}

}  // namespace mx4

// ---- launchers (cudaError_t; arguments already checked) ----
// by_block: X is (nblocks, rows, cols); otherwise (rows, nblocks * cols).
cudaError_t mx4_quantise(const void* X, const Mx4Shape& s, bool by_block, int dtype, uint8_t* codes, uint8_t* scales,
                         cudaStream_t st);
cudaError_t mx4_dequantise(const Mx4View& q, bool by_block, int dtype, void* X, cudaStream_t st);

// Where result (block b, row m, column n) of a product goes.
struct Mx4Out {
  int64_t b, m, n;  // strides in elements
  __host__ __device__ int64_t at(int64_t blk, int64_t row, int64_t col) const { return blk * b + row * m + col * n; }
  // (rows, nb * out)
  static Mx4Out blocks(int64_t nb, int64_t out) { return Mx4Out{out, nb * out, 1}; }
  // the same with a block's results nb apart: column n of block b at n * nb + b
  static Mx4Out transposed(int64_t nb, int64_t out) { return Mx4Out{1, nb * out, nb}; }
};

struct Mx4Linear {
  int64_t rows;
  int nb, in, out;
  bool has_bias;
  int dtype;
  Mx4Shape x() const { return Mx4Shape{rows, nb, in}; }
  Mx4Shape w() const { return Mx4Shape{out, nb, in}; }
};
// Kernels of the products, as monarch_mx4_linear_path names them.
enum Mx4Path {
  kMx4Token = 0, kMx4Batch = 1,                                                                        // mx4_rows.cu
  kMx4Tile64 = 2, kMx4Tile128 = 3, kMx4Tile256 = 4, kMx4Kept = 5, kMx4Pair = 6, kMx4Runs = 7,         // mx4_tc.cu
  kMx4Gemm = 8, kMx4GemmPair = 9, kMx4Split = 16,                                                      // mx4_gemm.cu; + if K is split
};

// Both operands in MX4 on the block-scaled tensor cores, every size and both types (mx4_tc.cu).
cudaError_t mx4_tc_fwd(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                       cudaStream_t st);
int mx4_tc_path(const Mx4Linear& d);
// What the direct few-rows kernel does, in products of 16 outputs, 128 inputs and 8 tokens, and whether that is little
// (6 us or so) where X comes in `parts` bf16 parts.
double mx4_rows_work(const Mx4Shape& w, int64_t rows);
bool mx4_rows_little(const Mx4Shape& w, int64_t rows, int parts);
constexpr int64_t kRowsMost = 8 * 65535;  // rows that the few-rows kernels take
// X as it is, few rows (mx4_rows.cu); X, Y fp32 or bf16.  w_early: no kernel of the stream that may still
// run writes the weight, so it may be read ahead of the grid-dependency wait.
cudaError_t mx4_rows_fwd(const void* X, int x_dtype, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y,
                         int y_dtype, bool w_early, cudaStream_t st);
int mx4_rows_path(const Mx4Shape& w, int64_t rows, int parts);
// The same with X in MX4, and whether that is quicker than the tensor-core kernel for both operands in MX4.
bool mx4_rows_quantised(const Mx4Shape& w, int64_t rows);
cudaError_t mx4_rows_fwd(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Out& o, void* Y, int y_dtype, cudaStream_t st);
// Products with a plain operand on the bf16 tensor cores, every size and both types (mx4_gemm.cu); ws: the
// bytes that the size query gives.  dX, dW and dbias may be NULL.
int mx4_gemm_fwd_path(const Mx4Linear& d);
int mx4_gemm_dx_path(const Mx4Linear& d);
int mx4_gemm_dw_path(const Mx4Linear& d);
size_t mx4_gemm_fwd_bytes(const Mx4Linear& d);
cudaError_t mx4_gemm_fwd(const void* X, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, void* ws, int* status,
                         cudaStream_t st);
size_t mx4_gemm_bwd_bytes(const Mx4Linear& d);
cudaError_t mx4_gemm_bwd(const void* dY, const Mx4View& x, const Mx4View& w, const Mx4Linear& d, void* dX, void* dW, void* dbias,
                         void* ws, int* status, cudaStream_t st);

}  // namespace monarch
