// Rounding to MX4 and back.
//
// quantise: of every 32 values along a row, byte = exponent field of the largest magnitude - 2, each
// value times 2^(127 - byte) (exact) to the nearest E2M1 code.  One thread takes one scale block, so
// that what a block costs beyond its values is paid once and X is read once; four neighbouring lanes
// take a row's four blocks of a scale tile and a warp 8 rows: 256 (bf16) or 512 (fp32) contiguous bytes
// a row.  Threads behind the last row or scale block write the tile's zero bytes.  Bound by memory,
// the element size + 17/32 bytes a value, and by the ALU not far behind: with 8 values a thread and
// shuffles for the maximum it took 41.9 us where this takes 29.0 us (16384 x 4096 bf16).
//
// dequantise, expand: the same split, codes in and values out; code times scale is exact in both types.
//
// A thread's own stretch of a row is read in 16-byte loads and written in 32-byte stores, whole sectors
// (28.6 us for 16384 x 4096 bf16; 59.7 for rows of 4 x 1000 with 16-byte stores).  Other rows go through a tile
// in shared memory: in, as the aligned 16-byte words that cover them (rows of 4 x 1001: 50.2 us, element by element 91.7); out, in
// 16-byte pieces (4 x 1000: 36.7) or elements (4 x 1001: 53.6), lanes along the columns.
#include "mx4.cuh"

namespace monarch {

namespace {

constexpr int kQThreads = 256, kQRows = kQThreads / 4;

// Offset of element (b, r, c) of the plain tensor, and of the next row.
__device__ __forceinline__ int64_t plain_row(const Mx4Shape& s, bool by_block) {
  return by_block ? s.cols : (int64_t)s.nblocks * s.cols;
}
__device__ __forceinline__ int64_t plain_at(const Mx4Shape& s, bool by_block, int b, int64_t r, int c) {
  return r * plain_row(s, by_block) + (by_block ? (int64_t)b * s.rows * s.cols : (int64_t)b * s.cols) + c;
}
// The 64 rows x 128 columns of a CTA in shared memory.
template <typename T>
struct Tile {
  static constexpr int PITCH = 128 * sizeof(T) + 16, WORDS = PITCH / 16;  // room for a row's misalignment
  uint8_t bytes[kQRows * PITCH];
  __device__ __forceinline__ T* at(int row, int col) { return (T*)(bytes + row * PITCH) + col; }
};
// Brings rows in as the aligned 16-byte words that cover them: element c of row r comes to stand at byte
// (address of the row) % 16 + c * sizeof(T) of its line.  p: the tile's first element in the plain tensor,
// end: that tensor's end, behind which no word may reach.
template <typename T>
__device__ __forceinline__ void tile_in(Tile<T>& t, const T* __restrict__ p, int64_t row, int rows, int cols, const T* end) {
  constexpr int U = 5, N = kQRows * Tile<T>::WORDS;
  const int len = min(cols, 128) * (int)sizeof(T);
  for (int e0 = threadIdx.x; e0 < N; e0 += U * kQThreads) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * kQThreads, r = e / Tile<T>::WORDS, j = e - r * Tile<T>::WORDS;
      const uintptr_t a = (uintptr_t)(p + r * row), w = (a & ~(uintptr_t)15) + 16 * j;
      v[u] = make_uint4(0, 0, 0, 0);
      if (e < N && r < rows && w < a + len) {
        if (w + 16 <= (uintptr_t)end) {
          v[u] = *(const uint4*)w;
        } else {  // the tensor's last elements
          uint32_t x[4] = {};
#pragma unroll
          for (int i = 0; i < 16 / (int)sizeof(T); ++i)
            if (w + (i + 1) * sizeof(T) <= (uintptr_t)end) {
              if (sizeof(T) == 2)
                x[i / 2] |= (uint32_t)*(const uint16_t*)(w + 2 * i) << (16 * (i & 1));
              else
                x[i % 4] = *(const uint32_t*)(w + 4 * i);
            }
          v[u] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * kQThreads;
      if (e < N) *(uint4*)(t.bytes + 16 * e) = v[u];
    }
  }
}
// Writes rows out from column 0 of their lines, lanes along the columns, in 16-byte pieces (rows are whole
// numbers of them) or in elements (whole aligned words with single elements at the ends measured slower).
template <typename T, int PIECE>
__device__ __forceinline__ void tile_out(Tile<T>& t, T* p, int64_t row, int rows, int cols) {
  constexpr int N = PIECE / sizeof(T), PER = 128 / N;
  for (int e = threadIdx.x; e < kQRows * PER; e += kQThreads) {
    const int r = e / PER, c = e % PER * N;
    if (r >= rows || c >= cols) continue;
    if (PIECE == 16)
      *(uint4*)(p + r * row + c) = *(const uint4*)t.at(r, c);
    else
      p[r * row + c] = *t.at(r, c);
  }
}

// The 32 values of a scale block, n of them (<= 0: none) inside the row, zeros behind it; p is 16-byte
// aligned and n a whole number of 16 bytes.
struct BlockBf16 {
  uint32_t w[16];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = 8 * i < n ? *(const uint4*)(p + 8 * i) : make_uint4(0, 0, 0, 0);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  }
  // the same from a line of a tile, at any 2-byte offset
  __device__ __forceinline__ void load_line(const uint8_t* line, int at, int n) {
    const uint32_t* src = (const uint32_t*)(line + (at & ~3));
    const uint32_t sel = (at & 2) ? 0x5432u : 0x3210u;
    uint32_t last = src[0];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t next = (i < 15 || (at & 2)) ? src[i + 1] : 0u;
      w[i] = __byte_perm(last, next, sel);
      last = next;
    }
    if (n < 32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] &= (2 * i < n ? 0xffffu : 0u) | (2 * i + 1 < n ? 0xffff0000u : 0u);
    }
  }
  // fp32 bits of the largest magnitude (magnitudes order like their bits, NaN above infinity)
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 16; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ uint32_t codes(int i, float f) const {  // of values 8i .. 8i + 7
    float t[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[2 * e] = __uint_as_float(w[4 * i + e] << 16) * f;
      t[2 * e + 1] = __uint_as_float(w[4 * i + e] & 0xffff0000u) * f;
    }
    return mx4::encode8(t);
  }
};
struct BlockF32 {
  float v[32];
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const float4 u = n > 4 * h ? *(const float4*)(p + 4 * h) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
    }
  }
  __device__ __forceinline__ void load_line(const uint8_t* line, int at, int n) {
    const float* src = (const float*)(line + at);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? src[i] : 0.f;
  }
  __device__ __forceinline__ uint32_t top() const {
    float m = fabsf(v[0]);  // max.NaN: a NaN wins
#pragma unroll
    for (int i = 1; i < 32; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
    return __float_as_uint(m);
  }
  __device__ __forceinline__ uint32_t codes(int i, float f) const {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = v[8 * i + e] * f;
    return mx4::encode8(t);
  }
};
template <typename T> struct BlockOf;
template <> struct BlockOf<__nv_bfloat16> { using type = BlockBf16; };
template <> struct BlockOf<float> { using type = BlockF32; };

// VEC: rows are whole numbers of 16 bytes.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads)
    mx4_quantise_kernel(const T* __restrict__ X, Mx4Shape s, bool by_block, uint8_t* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t rtiles) {
  __shared__ __align__(16) uint8_t mem[VEC ? 16 : sizeof(Tile<T>)];
  Tile<T>& tile = *(Tile<T>*)mem;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.z, kq = threadIdx.x & 3, kb = blockIdx.y * 4 + kq, rr = threadIdx.x >> 2;
  const bool kin = kb < s.kblocks();
  for (int64_t rt = blockIdx.x; rt < rtiles; rt += gridDim.x) {
    const int64_t r = rt * kQRows + rr;
    const bool mine = kin && r < s.rows;
    typename BlockOf<T>::type v;
    if (VEC) {
      v.load(X + plain_at(s, by_block, b, r, kb * 32), mine ? s.cols - kb * 32 : 0);
    } else {
      const int64_t r0 = rt * kQRows;
      const int c0 = blockIdx.y * 128;
      const T* p = X + plain_at(s, by_block, b, r0, c0);
      __syncthreads();  // the previous tile has been read
      tile_in(tile, p, plain_row(s, by_block), (int)min((int64_t)kQRows, s.rows - r0), s.cols - c0,
              X + s.rows * s.nblocks * s.cols);
      __syncthreads();
      v.load_line(tile.bytes + rr * Tile<T>::PITCH, (int)((uintptr_t)(p + rr * plain_row(s, by_block)) & 15) + kq * 32 * (int)sizeof(T),
                  mine ? s.cols - kb * 32 : 0);
    }
    const uint32_t byte = mx4::scale_byte(v.top());
    if (mine) {
      const float f = mx4::inv_scale(byte);
      uint4 u = make_uint4(v.codes(0, f), v.codes(1, f), v.codes(2, f), v.codes(3, f));
      if (byte == 255) u = make_uint4(0, 0, 0, 0);
      *(uint4*)(codes + s.code_row(b, r) + kb * 16) = u;
    }
    scales[s.scale_at(b, r, kb)] = (uint8_t)byte;  // rows and blocks behind the end hold 0
  }
}

// Writes a block's bf16 pairs as values at p, n of the 32, in pieces of 32 or 16 bytes.
template <int PIECE>
__device__ __forceinline__ void store_block(__nv_bfloat16* p, int n, const uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 64 / PIECE; ++i)
    if (i * PIECE / 2 < n) {
      if (PIECE == 32)
        ptx::st_global_v8(p + 16 * i, &v[(8 * i) % 16]);
      else
        *(uint4*)(p + 8 * i) = make_uint4(v[(4 * i) % 16], v[(4 * i + 1) % 16], v[(4 * i + 2) % 16], v[(4 * i + 3) % 16]);
    }
}
template <int PIECE>
__device__ __forceinline__ void store_block(float* p, int n, const uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[2 * e] = v[4 * i + e] << 16;
      u[2 * e + 1] = v[4 * i + e] & 0xffff0000u;
    }
    if (PIECE == 32) {
      if (8 * i < n) ptx::st_global_v8(p + 8 * i, u);
    } else {
      if (8 * i < n) *(uint4*)(p + 8 * i) = make_uint4(u[0], u[1], u[2], u[3]);
      if (8 * i + 4 < n) *(uint4*)(p + 8 * i + 4) = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }
}

// PIECE: bytes that rows of X are whole numbers of: 32, 16, or sizeof(T).
template <typename T, int PIECE>
__global__ void __launch_bounds__(kQThreads)
    mx4_dequantise_kernel(Mx4View q, bool by_block, T* __restrict__ X, int64_t rtiles) {
  __shared__ __align__(16) uint8_t mem[PIECE == 32 ? 16 : sizeof(Tile<T>)];
  Tile<T>& tile = *(Tile<T>*)mem;
  // No early start for the next kernel: a map whose factor these values are would only wait.
  ptx::griddep_wait();
  const Mx4Shape& s = q.s;
  const int b = blockIdx.z, kq = threadIdx.x & 3, kb = blockIdx.y * 4 + kq, rr = threadIdx.x >> 2;
  const bool kin = kb < s.kblocks();
  for (int64_t rt = blockIdx.x; rt < rtiles; rt += gridDim.x) {
    const int64_t r = rt * kQRows + rr;
    const bool mine = r < s.rows;
    const uint4 u = kin && mine ? *(const uint4*)(q.codes + s.code_row(b, r) + kb * 16) : make_uint4(0, 0, 0, 0);
    const uint32_t byte = kin && mine ? q.scales[s.scale_at(b, r, kb)] : 0u;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t t[4];
      mx4::values8(w[i], byte, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = t[e];
    }
    if (PIECE == 32) {
      if (mine) store_block<32>(X + plain_at(s, by_block, b, r, kb * 32), s.cols - kb * 32, v);
    } else {
      const int64_t r0 = rt * kQRows;
      const int c0 = blockIdx.y * 128;
      __syncthreads();  // the previous tile has been read
      store_block<16>(tile.at(rr, kq * 32), 32, v);
      __syncthreads();
      tile_out<T, PIECE == 32 ? 16 : PIECE>(tile, X + plain_at(s, by_block, b, r0, c0), plain_row(s, by_block),
                                            (int)min((int64_t)kQRows, s.rows - r0), s.cols - c0);
    }
  }
}

bool rows_of_16_bytes(const Mx4Shape& s, int dtype) { return (int64_t)s.cols * (dtype == MONARCH_BF16 ? 2 : 4) % 16 == 0; }
dim3 grid_for(const Mx4Shape& s, int64_t rtiles) {
  return dim3((unsigned)(rtiles < (1 << 20) ? rtiles : (1 << 20)), (unsigned)s.katoms(), (unsigned)s.nblocks);
}

template <typename T, bool VEC>
cudaError_t quantise_t(const void* X, const Mx4Shape& s, bool by_block, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int64_t rt = s.ratoms() * (128 / kQRows);  // whole scale tiles
  return launch_kernel(mx4_quantise_kernel<T, VEC>, grid_for(s, rt), dim3(kQThreads), 0, st, true, (const T*)X, s, by_block,
                       codes, scales, rt);
}
template <typename T, int PIECE>
cudaError_t dequantise_t(const Mx4View& q, bool by_block, void* X, cudaStream_t st) {
  const int64_t rt = (q.s.rows + kQRows - 1) / kQRows;
  return launch_kernel(mx4_dequantise_kernel<T, PIECE>, grid_for(q.s, rt), dim3(kQThreads), 0, st, true, q, by_block, (T*)X, rt);
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

template <typename T>
static cudaError_t dequantise_any(const Mx4View& q, bool by_block, void* X, cudaStream_t st) {
  const int64_t row = (int64_t)q.s.cols * sizeof(T);
  if (row % 32 == 0 && ((uintptr_t)X & 31u) == 0) return dequantise_t<T, 32>(q, by_block, X, st);
  return row % 16 == 0 ? dequantise_t<T, 16>(q, by_block, X, st) : dequantise_t<T, (int)sizeof(T)>(q, by_block, X, st);
}
cudaError_t mx4_dequantise(const Mx4View& q, bool by_block, int dtype, void* X, cudaStream_t st) {
  return dtype == MONARCH_BF16 ? dequantise_any<__nv_bfloat16>(q, by_block, X, st) : dequantise_any<float>(q, by_block, X, st);
}

}  // namespace monarch
