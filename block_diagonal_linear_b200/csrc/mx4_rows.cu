// Few tokens through an MX4 weight:  Y(r; b, o) = sum_i X[r][b*in + i] W^[b][o][i] (+ bias), X as it is.
//
// A decoding step reads the whole weight for a handful of tokens, so the kernel is bound by the
// latency and bandwidth of that one read (17/32 bytes a weight).  The product runs on mma.sync
// m16n8k16 with the weights as the 16-row operand and 8 tokens as the columns: codes become bf16
// values in registers (exact), X enters as one bf16 part, or, in fp32, as 2 or 3 parts that are cut
// off one after another (3 parts hold all 24 bits; 2 leave 2^-16, below a bf16 result's half step).
//
// A warp takes 16 outputs and walks scale tiles of 128 inputs: a lane holds one whole scale block of
// two outputs (16 bytes of codes each), so that one multiplier serves all of a lane's values; which
// input stands where inside an MMA does not matter as long as both operands agree.  The 16 outputs
// are 4 neighbours in each of the 4 column groups of a scale tile, whose scale words are contiguous.
// Warps of a CTA split the inputs (up to 8 ways) and then outputs; their sums join in shared memory
// in a fixed order.  Every lane asks for up to four scale tiles before it uses the first.
#include "mx4.cuh"
#include "tc_common.cuh"

namespace monarch {

namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 4;  // scale tiles in flight

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight neighbouring inputs of one token in fp32 bits or bf16 pairs; zero behind the end.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, uint32_t (&x)[8]) {
  if (VEC) {
    const uint4 u = n > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? *(const uint16_t*)(p + 2 * i) : 0u;
      const uint32_t hi = 2 * i + 1 < n ? *(const uint16_t*)(p + 2 * i + 1) : 0u;
      x[i] = lo | (hi << 16);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int n, uint32_t (&x)[8]) {
  if (VEC) {
    const uint4 u = n > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0), w = n > 4 ? *(const uint4*)(p + 4) : make_uint4(0, 0, 0, 0);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? *(const uint32_t*)(p + i) : 0u;
  }
}

// Pairs (j, j + 4), j = 0..3, of the eight inputs as bf16 operands of part 0 .. PARTS-1.
template <int PARTS>
__device__ __forceinline__ void split8(const uint32_t (&x)[8], uint32_t (&b)[PARTS][4], const __nv_bfloat16*) {
  b[0][0] = __byte_perm(x[0], x[2], 0x5410);
  b[0][1] = __byte_perm(x[0], x[2], 0x7632);
  b[0][2] = __byte_perm(x[1], x[3], 0x5410);
  b[0][3] = __byte_perm(x[1], x[3], 0x7632);
}
template <int PARTS>
__device__ __forceinline__ void split8(const uint32_t (&x)[8], uint32_t (&b)[PARTS][4], const float*) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = __uint_as_float(x[i]);
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) b[p][j] = __byte_perm(__float_as_uint(rest[j]), __float_as_uint(rest[j + 4]), 0x7632);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t top = __float_as_uint(rest[i]) & 0xffff0000u;  // exact difference; none for infinities and NaN
      rest[i] = (top & 0x7f800000u) == 0x7f800000u ? 0.f : rest[i] - __uint_as_float(top);
    }
  }
}

template <typename TX, int PARTS, typename TY, bool VEC, int NT>
__global__ void __launch_bounds__(kWarps * 32)
    mx4_rows_kernel(const TX* X, Mx4View w, int64_t rows, Mx4Out o, const TY* bias, TY* Y, int wk, bool w_early) {
  __shared__ float part[kWarps][16][8 * NT + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int kw = warp % wk, mw = warp / wk;  // this warp's share of the inputs, and its 16 outputs
  const int b = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.z * (8 * NT);
  const int64_t mt = (int64_t)blockIdx.x * (kWarps / wk) + mw;  // 8 of them in 128 outputs
  // MMA row m = 4i + j is output 128*(mt/8) + 4*(mt%8) + i + 32*j
  const int64_t o0 = (mt >> 3) * 128 + (mt & 7) * 4 + (g >> 2) + 32 * (g & 3), o1 = o0 + 2;
  const int katoms = w.s.katoms(), kblocks = w.s.kblocks();
  const int64_t ratom = mt >> 3;
  const bool in_range = ratom < w.s.ratoms();
  const uint8_t* c0 = w.codes + w.s.code_row(b, o0) + t * 16;
  const uint8_t* c1 = w.codes + w.s.code_row(b, o1) + t * 16;
  const uint8_t* sc = w.scales + ((((int64_t)b * w.s.ratoms() + ratom) * katoms) << 9) + (((mt & 7) * 4 + (g >> 2)) << 4) + ((g & 3) << 2);
  const int64_t pitch = (int64_t)w.s.nblocks * w.s.cols;

  float acc[NT][4] = {};
  uint4 q0[kAhead], q1[kAhead];
  uint32_t s0[kAhead], s1[kAhead];
  auto fetch = [&](int ka0) {  // this warp's next kAhead scale tiles: ka0, ka0 + wk, ...
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int ka = ka0 + i * wk;
      const bool ok = in_range && ka < katoms && ka * 4 + t < kblocks;
      q0[i] = ok && o0 < w.s.rows ? *(const uint4*)(c0 + (int64_t)ka * 64) : make_uint4(0, 0, 0, 0);
      q1[i] = ok && o1 < w.s.rows ? *(const uint4*)(c1 + (int64_t)ka * 64) : make_uint4(0, 0, 0, 0);
      s0[i] = ok ? *(const uint32_t*)(sc + (int64_t)ka * 512) : 0u;
      s1[i] = ok ? *(const uint32_t*)(sc + (int64_t)ka * 512 + 32) : 0u;
    }
  };
  // weights that no kernel of this stream is still writing may be asked for ahead of the wait
  if (w_early) {
    fetch(kw);
    ptx::griddep_wait();
  } else {
    ptx::griddep_wait();
    fetch(kw);
  }
  ptx::griddep_launch_dependents();

  for (int ka0 = kw; ka0 < katoms; ka0 += kAhead * wk) {
    if (ka0 != kw) fetch(ka0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int ka = ka0 + i * wk;
      if (ka >= katoms) break;
      // codes -> bf16: spread8 leaves value / 2^126; scales up to 2^1 fold into one multiplication
      const uint32_t e0 = (s0[i] >> (8 * t)) & 255u, e1 = (s1[i] >> (8 * t)) & 255u;
      const bool big = e0 > 128u || e1 > 128u;
      const uint32_t f0 = (e0 > 128u ? 253u : e0 + 126u) * 0x00800080u, f1 = (e1 > 128u ? 253u : e1 + 126u) * 0x00800080u;
      uint32_t a0[16], a1[16];  // word v's pair j at 4v + j
      const uint32_t w0[4] = {q0[i].x, q0[i].y, q0[i].z, q0[i].w}, w1[4] = {q1[i].x, q1[i].y, q1[i].z, q1[i].w};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t p0[4], p1[4];
        mx4::spread8(w0[v], p0);
        mx4::spread8(w1[v], p1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a0[4 * v + j] = mul_bf16x2(p0[j], f0);
          a1[4 * v + j] = mul_bf16x2(p1[j], f1);
        }
      }
      if (__any_sync(0xffffffffu, big)) {  // 2^(byte - 127) itself, and NaN
        const uint32_t h0 = e0 > 128u ? (e0 == 255u ? 0x7fc07fc0u : e0 * 0x00800080u) : 0x3f803f80u;
        const uint32_t h1 = e1 > 128u ? (e1 == 255u ? 0x7fc07fc0u : e1 * 0x00800080u) : 0x3f803f80u;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          a0[j] = mul_bf16x2(a0[j], h0);
          a1[j] = mul_bf16x2(a1[j], h1);
        }
      }
      const int k = ka * 128 + t * 32;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t r = r0 + n * 8 + g;
        const TX* p = X + r * pitch + (int64_t)b * w.s.cols + k;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t x[8], bp[PARTS][4];
          load8<VEC>(p + 8 * v, r < rows ? w.s.cols - k - 8 * v : 0, x);
          split8<PARTS>(x, bp, (const TX*)nullptr);
          // mma.sync cuts its sums off (2^-23 a step, always towards zero): an fp32 result takes them in
          // runs of 32 inputs and joins the runs with rounded additions (4096 inputs: 1.3e-6 off without)
          float run[4] = {};
          float(&sum)[4] = PARTS == 3 ? run : acc[n];
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q) {
            mma_16816(sum, a0[4 * v], a1[4 * v], a0[4 * v + 1], a1[4 * v + 1], bp[q][0], bp[q][1]);
            mma_16816(sum, a0[4 * v + 2], a1[4 * v + 2], a0[4 * v + 3], a1[4 * v + 3], bp[q][2], bp[q][3]);
          }
          if (PARTS == 3) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] += run[e];
          }
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][g + 8 * (e >> 1)][n * 8 + 2 * t + (e & 1)] = acc[n][e];
  __syncthreads();
  // join the input shares in order; consecutive threads take consecutive outputs of one token
  const int mtiles = kWarps / wk;
  for (int e = threadIdx.x; e < mtiles * 16 * 8 * NT; e += kWarps * 32) {
    const int m = e % 16, tile = (e / 16) % mtiles, n = e / (16 * mtiles);
    const int64_t tt = (int64_t)blockIdx.x * mtiles + tile;
    // row order that walks the outputs: four neighbours, then the next group of 32
    const int64_t out = (tt >> 3) * 128 + (tt & 7) * 4 + (m & 3) + 32 * (m >> 2);
    const int row = 4 * (m & 3) + (m >> 2);
    if (out >= w.s.rows || r0 + n >= rows) continue;
    float v = 0.f;
    for (int k = 0; k < wk; ++k) v += part[tile * wk + k][row][n];
    if (bias != nullptr) v += mx4::load(bias + (int64_t)b * w.s.rows + out);
    st_from_f32(Y + o.at(b, r0 + n, out), v);
  }
}

template <typename TX, int PARTS, typename TY, bool VEC, int NT>
cudaError_t launch(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                   cudaStream_t st) {
  int wk = 1;
  while (wk < kWarps && wk * 2 <= w.s.katoms()) wk *= 2;
  const int64_t mtiles = (w.s.rows + 127) / 128 * 8;
  const int per = kWarps / wk;
  return launch_kernel(mx4_rows_kernel<TX, PARTS, TY, VEC, NT>,
                       dim3((unsigned)((mtiles + per - 1) / per), (unsigned)w.s.nblocks, (unsigned)((rows + 8 * NT - 1) / (8 * NT))),
                       dim3(kWarps * 32), 0, st, true, (const TX*)X, w, rows, o, (const TY*)bias, (TY*)Y, wk, w_early);
}

template <typename TX, int PARTS, typename TY>
cudaError_t launch_rows(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                        cudaStream_t st) {
  const bool vec = w.s.cols * sizeof(TX) % 16 == 0;
  if (rows <= 8)
    return vec ? launch<TX, PARTS, TY, true, 1>(X, w, bias, rows, o, Y, w_early, st)
               : launch<TX, PARTS, TY, false, 1>(X, w, bias, rows, o, Y, w_early, st);
  if (rows <= 16)
    return vec ? launch<TX, PARTS, TY, true, 2>(X, w, bias, rows, o, Y, w_early, st)
               : launch<TX, PARTS, TY, false, 2>(X, w, bias, rows, o, Y, w_early, st);
  return vec ? launch<TX, PARTS, TY, true, 4>(X, w, bias, rows, o, Y, w_early, st)
             : launch<TX, PARTS, TY, false, 4>(X, w, bias, rows, o, Y, w_early, st);
}

}  // namespace

cudaError_t mx4_rows_fwd(const void* X, int x_dtype, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y,
                         int y_dtype, bool w_early, cudaStream_t st) {
  if (x_dtype == MONARCH_BF16)
    return y_dtype == MONARCH_BF16 ? launch_rows<__nv_bfloat16, 1, __nv_bfloat16>(X, w, bias, rows, o, Y, w_early, st)
                                   : launch_rows<__nv_bfloat16, 1, float>(X, w, bias, rows, o, Y, w_early, st);
  return y_dtype == MONARCH_BF16 ? launch_rows<float, 2, __nv_bfloat16>(X, w, bias, rows, o, Y, w_early, st)
                                 : launch_rows<float, 3, float>(X, w, bias, rows, o, Y, w_early, st);
}

}  // namespace monarch
