// Few tokens through an MX4 weight:  Y(r; b, o) = sum_i X[r][b*in + i] W^[b][o][i] (+ bias), X as it is or in MX4.
//
// A decoding step reads the whole weight for a handful of tokens, so the kernels are bound by the
// latency and bandwidth of that one read (17/32 bytes a weight).  The product runs on mma.sync
// m16n8k16 with the weights as the 16-row operand and 8 tokens as the columns: codes become bf16
// values in registers (exact), X enters as one bf16 part, or, in fp32 (a Monarch map's middle vector too,
// whatever the result's type), as 3 parts that are cut off one after another and hold all 24 bits; an MX4 X
// becomes bf16 values as the weight does.
//
// A warp takes 16 outputs and walks scale tiles of 128 inputs: a lane holds one whole scale block of
// two outputs (16 bytes of codes each), so that one multiplier serves all of a lane's values; which
// input stands where inside an MMA does not matter as long as both operands agree.  Every lane asks for
// up to four scale tiles of codes before it uses the first.  The inputs are split up to 8 ways, and the
// shares' sums join in a fixed order.
//
// Up to 8 bf16 tokens, and more where inputs are short or the weight small (mx4_token_kernel), the shares are warps
// of a CTA and a lane reads its inputs where they are.  Warps that are left take further tiles, or neighbouring blocks: of
// a transposed result (a Monarch stage) these lie next to each other (32 tokens through sixty-four 64 x 64 blocks
// twice: 6.0 us, 14 with a block a CTA).  With a large weight every warp would gather and cut its own inputs
// too often (4096 -> 4096: 16.5 us for 32 bf16 tokens against 12.2, 12.2 for one in fp32 against 8.1); there
// (mx4_batch_kernel, up to 64 tokens a pass) the shares are CTAs of a cluster, and a CTA's 8 warps take 128 outputs
// and share one copy of the inputs in shared memory, already cut into parts, in the order in which lanes read it.
#include <type_traits>

#include "mx4.cuh"
#include "tc_common.cuh"

namespace monarch {

namespace {

constexpr int kWarps = 8;

using mx4::mul_bf16x2;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight neighbouring inputs of one token in fp32 bits or bf16 pairs, n of them (<= 0: none) inside the row;
// zero behind its end.  VEC: rows are whole numbers of 16 bytes; end: of X.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, const __nv_bfloat16* end, uint32_t (&x)[8]) {
  if (VEC) {
    const uint4 u = n > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  } else {
    mx4::load8_any(p, n, end, x);
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int n, const float* end, uint32_t (&x)[8]) {
  if (VEC) {
    const uint4 u = n > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0), w = n > 4 ? *(const uint4*)(p + 4) : make_uint4(0, 0, 0, 0);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  } else {
    mx4::load8_any(p, n, end, x);
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
  for (int i = 0; i < 8; ++i) rest[i] = __uint_as_float(mx4::nan_in_top(x[i]));
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

// One scale tile's codes of a lane: 32 codes of two outputs and their scale words.
struct Codes {
  uint4 q0, q1;
  uint32_t s0, s1;
};
struct CodeRows {  // a lane's two outputs, g and g + 8 of the warp's sixteen
  const uint8_t *c0, *c1, *s0, *s1;
  bool in0, in1;
  int katoms, kblocks, t;
  __device__ CodeRows(const Mx4View& w, int b, int64_t o, int t_) : t(t_) {
    in0 = o < w.s.rows;
    in1 = o + 8 < w.s.rows;
    katoms = w.s.katoms();
    kblocks = w.s.kblocks();
    c0 = w.codes + w.s.code_row(b, o) + t * 16;
    c1 = w.codes + w.s.code_row(b, o + 8) + t * 16;
    s0 = w.scales + w.s.scale_at(b, o, 0);
    s1 = w.scales + w.s.scale_at(b, o + 8, 0);
  }
  __device__ __forceinline__ Codes at(int ka) const {
    const bool ok = ka < katoms && ka * 4 + t < kblocks;
    Codes c;
    c.q0 = ok && in0 ? *(const uint4*)(c0 + (int64_t)ka * 64) : make_uint4(0, 0, 0, 0);
    c.q1 = ok && in1 ? *(const uint4*)(c1 + (int64_t)ka * 64) : make_uint4(0, 0, 0, 0);
    c.s0 = ok && in0 ? *(const uint32_t*)(s0 + (int64_t)ka * 512) : 0u;
    c.s1 = ok && in1 ? *(const uint32_t*)(s1 + (int64_t)ka * 512) : 0u;
    return c;
  }
};
// Codes to bf16 values: word v's pair (j, j + 4) at 4v + j.  spread8 leaves value / 2^126; scales up to 2^1
// fold into one multiplication, larger ones and NaN take a second.
__device__ __forceinline__ void values(const Codes& c, int t, uint32_t (&a0)[16], uint32_t (&a1)[16]) {
  const uint32_t e0 = (c.s0 >> (8 * t)) & 255u, e1 = (c.s1 >> (8 * t)) & 255u;
  const bool big = e0 > 128u || e1 > 128u;
  const uint32_t f0 = (e0 > 128u ? 253u : e0 + 126u) * 0x00800080u, f1 = (e1 > 128u ? 253u : e1 + 126u) * 0x00800080u;
  const uint32_t w0[4] = {c.q0.x, c.q0.y, c.q0.z, c.q0.w}, w1[4] = {c.q1.x, c.q1.y, c.q1.z, c.q1.w};
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
}
// The same for the 32 codes of one token's scale block.
__device__ __forceinline__ void values(uint4 q, uint32_t e, uint32_t (&a)[16]) {
  const uint32_t f = (e > 128u ? 253u : e + 126u) * 0x00800080u;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t p[4];
    mx4::spread8(w[v], p);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[4 * v + j] = mul_bf16x2(p[j], f);
  }
  if (__any_sync(0xffffffffu, e > 128u)) {
    const uint32_t h = e > 128u ? (e == 255u ? 0x7fc07fc0u : e * 0x00800080u) : 0x3f803f80u;
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] = mul_bf16x2(a[j], h);
  }
}
// acc += the 32 inputs' products of word v.  mma.sync cuts its sums off (2^-23 a step, always towards
// zero): RUNS, for fp32 operands and fp32 results, takes them in runs of 32 inputs and joins the runs with rounded
// additions (4096 inputs: 1.3e-6 off without, 1e-7 with).
template <int PARTS, bool RUNS>
__device__ __forceinline__ void product(float (&acc)[4], const uint32_t (&a0)[16], const uint32_t (&a1)[16], int v,
                                        const uint32_t (&bp)[PARTS][4]) {
  float run[4] = {};
  float(&sum)[4] = RUNS ? run : acc;
#pragma unroll
  for (int q = PARTS - 1; q >= 0; --q) {
    mma_16816(sum, a0[4 * v], a1[4 * v], a0[4 * v + 1], a1[4 * v + 1], bp[q][0], bp[q][1]);
    mma_16816(sum, a0[4 * v + 2], a1[4 * v + 2], a0[4 * v + 3], a1[4 * v + 3], bp[q][2], bp[q][3]);
  }
  if (RUNS) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += run[e];
  }
}

constexpr int kAhead = 4;  // scale tiles of codes in flight

constexpr int kPlane = 16 * 9 + 4;  // a warp's sums, 16 outputs x 8 tokens: padded, 8 blocks x 4 outputs in 32 banks

struct QuantisedX {};  // in place of X's type: X is an Mx4 view

// Warps of a CTA: 2^lk shares of the inputs, 2^lb neighbouring blocks, `per` tiles of 16 outputs; 8 tokens.
template <typename TX, int PARTS, typename TY, bool VEC, int AHEAD>
__global__ void __launch_bounds__(kWarps * 32, 2)
    mx4_token_kernel(const TX* X, Mx4View xq, Mx4View w, int64_t rows, Mx4Out o, const TY* bias, TY* Y, int lk, int lb, int per,
                     bool w_early) {
  constexpr bool QX = std::is_same<TX, QuantisedX>::value, RUNS = PARTS == 3 || sizeof(TY) == 4;
  __shared__ float part[kWarps * kPlane];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int wk = 1 << lk, nbw = 1 << lb;
  const int kw = warp & (wk - 1), bw = (warp >> lk) & (nbw - 1), mw = warp >> (lk + lb);
  const int64_t tile0 = (int64_t)blockIdx.x * per, r0 = (int64_t)blockIdx.z * 8, r = r0 + g;
  const int b0 = blockIdx.y * nbw, b = min(b0 + bw, w.s.nblocks - 1);
  CodeRows cr(w, b, (tile0 + mw) * 16 + g, t);
  if (mw >= per) cr.katoms = 0;  // nothing to do but the join
  const int64_t pitch = (int64_t)w.s.nblocks * w.s.cols;
  const TX *p = QX ? nullptr : X + r * pitch + (int64_t)b * w.s.cols + t * 32, *end = QX ? nullptr : X + rows * pitch;
  const uint8_t* xc = QX ? xq.codes + xq.s.code_row(b, r) + t * 16 : nullptr;
  const uint8_t* xs = QX ? xq.scales + xq.s.scale_at(b, r, 0) + t : nullptr;

  float acc[4] = {};
  Codes c[AHEAD];
  // weights that no kernel of this stream is still writing may be asked for ahead of the wait
  if (!w_early) ptx::griddep_wait();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) c[i] = cr.at(kw + i * wk);
  if (w_early) ptx::griddep_wait();
  ptx::griddep_launch_dependents();

#pragma unroll 1
  for (int ka0 = kw; ka0 < cr.katoms; ka0 += AHEAD * wk) {
    if (AHEAD > 1 && ka0 != kw) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) c[i] = cr.at(ka0 + i * wk);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int ka = ka0 + i * wk;
      if (ka >= cr.katoms) break;
      uint32_t a0[16], a1[16];
      if constexpr (QX) {  // a lane's 32 inputs are one scale block of its token
        const bool live = r < rows && ka * 4 + t < cr.kblocks;
        const uint4 q = live ? *(const uint4*)(xc + (int64_t)ka * 64) : make_uint4(0, 0, 0, 0);
        const uint32_t byte = live ? xs[(int64_t)ka * 512] : 0u;
        uint32_t x[16];
        values(c[i], t, a0, a1);
        if (AHEAD == 1) c[0] = cr.at(ka + wk);
        values(q, byte, x);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint32_t bp[1][4] = {{x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]}};
          product<1, RUNS>(acc, a0, a1, v, bp);
        }
      } else {
        uint32_t x[4][8];
#pragma unroll
        for (int v = 0; v < 4; ++v)
          load8<VEC>(p + ka * 128 + 8 * v, r < rows ? w.s.cols - ka * 128 - t * 32 - 8 * v : 0, end, x[v]);
        values(c[i], t, a0, a1);
        if (AHEAD == 1) c[0] = cr.at(ka + wk);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t bp[PARTS][4];
          split8<PARTS>(x[v], bp, (const TX*)nullptr);
          product<PARTS, RUNS>(acc, a0, a1, v, bp);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[warp * kPlane + (g + 8 * (e >> 1)) * 9 + 2 * t + (e & 1)] = acc[e];
  __syncthreads();
  // join the shares in order; consecutive threads take neighbours in Y: outputs, or blocks where it is transposed.
  // A thread has one output of every so many tokens.
  const int m = threadIdx.x & ((128 >> lk) - 1);
  const int row = o.n == 1 ? m & 15 : (m >> lb) & 15, q = o.n == 1 ? m >> (7 - lk - lb) : m & (nbw - 1);
  const int tile = o.n == 1 ? (m >> 4) & ((kWarps >> (lk + lb)) - 1) : m >> (4 + lb);
  const int64_t out = (tile0 + tile) * 16 + row;
  if (tile >= per || out >= w.s.rows || b0 + q >= w.s.nblocks) return;
  const float add = bias != nullptr ? mx4::load(bias + (int64_t)(b0 + q) * w.s.rows + out) : 0.f;
  const float* sum = part + (((tile << lb) + q) << lk) * kPlane + row * 9;
  TY* y = Y + o.at(b0 + q, r0, out);
  const int tokens = (int)min((int64_t)8, rows - r0);
#pragma unroll 4
  for (int n = threadIdx.x >> (7 - lk); n < tokens; n += 2 << lk) {
    float v = 0.f;
    for (int k = 0; k < wk; ++k) v += sum[k * kPlane + n];
    st_from_f32(y + n * o.m, v + add);
  }
}

// Shared memory of mx4_batch_kernel: PARTS copies of 8 * NT tokens x kAhead scale tiles in bf16, 16-byte
// chunks of 8 inputs (pairs j, j + 4), chunk c of token r at c ^ swizzle(c, r) so that the lanes of a
// load find eight different bank groups; later the sums [per][8 * NT][kSumPitch].
__device__ __forceinline__ int chunk_at(int token, int c) {
  return token * (kAhead * 16) + (c ^ (((c >> 3) & 1) | ((token & 1) << 1)));
}

constexpr int kSumPitch = 20;  // 16 outputs of a token, padded: 16-byte reads, few bank conflicts

// All 8 warps bring the inputs in; the first `per` compute.
template <typename TX, int PARTS, typename TY, bool VEC, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2)
    mx4_batch_kernel(const TX* X, Mx4View w, int64_t rows, Mx4Out o, const TY* bias, TY* Y, int shares, int per, bool w_early) {
  constexpr bool RUNS = PARTS == 3 || sizeof(TY) == 4;
  constexpr int U = sizeof(TX) == 2 ? 8 : 4;  // chunks of 8 inputs a thread asks for before it stores the first
  extern __shared__ uint4 xs[];  // [PARTS][8 * NT][kAhead * 16]
  constexpr int PLANE = 8 * NT * kAhead * 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int rank = (int)ptx::cluster_ctarank();
  const bool works = warp < per;  // output tiles of the CTA, one a warp
  const int64_t tile0 = (int64_t)(blockIdx.x / shares) * per;
  const int b = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.z * (8 * NT);
  const int tokens = (int)min((int64_t)(8 * NT), rows - r0);
  const int64_t pitch = (int64_t)w.s.nblocks * w.s.cols;
  const TX* xb = X + r0 * pitch + (int64_t)b * w.s.cols;
  const CodeRows cr(w, b, (tile0 + warp) * 16 + g, t);
  // this CTA's scale tiles: consecutive ones, kAhead at a time
  const int each = (cr.katoms + shares - 1) / shares;
  const int lo = rank * each, hi = min(cr.katoms, lo + each);

  float acc[NT][4] = {};
  Codes c[kAhead];
  if (!w_early) ptx::griddep_wait();
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (works && lo + i < hi) c[i] = cr.at(lo + i);
  if (w_early) ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  for (int ka0 = lo; ka0 < hi; ka0 += kAhead) {
    const int n = min(kAhead, hi - ka0);
    if (ka0 != lo) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (works && i < n) c[i] = cr.at(ka0 + i);
      __syncthreads();  // the previous inputs have been read
    }
    for (int e0 = threadIdx.x; e0 < tokens * n * 16; e0 += U * kWarps * 32) {
      uint32_t x[U][8];
      int token[U], ch[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e = e0 + u * kWarps * 32;
        token[u] = e / (n * 16);
        ch[u] = e - token[u] * (n * 16);
        load8<VEC>(xb + token[u] * pitch + ka0 * 128 + ch[u] * 8, token[u] < tokens ? w.s.cols - ka0 * 128 - ch[u] * 8 : 0,
                   X + rows * pitch, x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t bp[PARTS][4];
        split8<PARTS>(x[u], bp, (const TX*)nullptr);
        if (token[u] < tokens) {
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            xs[q * PLANE + chunk_at(token[u], ch[u])] = make_uint4(bp[q][0], bp[q][1], bp[q][2], bp[q][3]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i >= n || !works) break;
      uint32_t a0[16], a1[16];
      values(c[i], t, a0, a1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= tokens) break;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t bp[PARTS][4];
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            // columns of tokens behind the last are never stored: any finite or other value may stand there
            const uint4 u = xs[q * PLANE + chunk_at(nt * 8 + g, i * 16 + t * 4 + v)];
            bp[q][0] = u.x; bp[q][1] = u.y; bp[q][2] = u.z; bp[q][3] = u.w;
          }
          product<PARTS, RUNS>(acc[nt], a0, a1, v, bp);
        }
      }
    }
  }
  __syncthreads();
  float* part = (float*)xs;
  if (works) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(warp * 8 * NT + nt * 8 + 2 * t + (e & 1)) * kSumPitch + g + 8 * (e >> 1)] = acc[nt][e];
  }
  ptx::cluster_sync_all();
  // join the shares in order; four neighbouring outputs of one token a thread, consecutive threads take
  // consecutive outputs, the cluster's CTAs take turns
  for (int e = rank * kWarps * 32 + threadIdx.x; e < per * 4 * tokens; e += shares * kWarps * 32) {
    const int q = e % 4, tile = (e / 4) % per, n = e / (4 * per);
    const int64_t out = (tile0 + tile) * 16 + q * 4;
    if (out >= w.s.rows) continue;
    const uint32_t at = ptx::smem_u32(&part[(tile * 8 * NT + n) * kSumPitch + q * 4]);
    float4 u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < shares) u[k] = ptx::ld_cluster_f32x4(ptx::mapa_shared(at, k));
    float v[4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < shares) {
        v[0] += u[k].x;
        v[1] += u[k].y;
        v[2] += u[k].z;
        v[3] += u[k].w;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (out + i >= w.s.rows) break;
      if (bias != nullptr) v[i] += mx4::load(bias + (int64_t)b * w.s.rows + out + i);
      st_from_f32(Y + o.at(b, r0 + n, out + i), v[i]);
    }
  }
  ptx::cluster_sync_all();  // the others may still read this CTA's sums
}

template <typename TX, int PARTS, typename TY, bool VEC>
cudaError_t launch_token(const void* X, const Mx4View& xq, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                         cudaStream_t st) {
  const int64_t mtiles = (w.s.rows + 15) / 16;
  int lk = 0, lb = 0;
  while (lk < 3 && 2 << lk <= w.s.katoms()) ++lk;
  // neighbouring blocks: in place of tiles where these are fewer or where the result is transposed
  while (lk + lb < 3 && 2 << lb <= w.s.nblocks && (o.n != 1 || mtiles << (lk + lb) < kWarps)) ++lb;
  const int room = kWarps >> (lk + lb), per = (int)(mtiles < room ? mtiles : room);
  const dim3 grid((unsigned)((mtiles + per - 1) / per), (unsigned)((w.s.nblocks + (1 << lb) - 1) >> lb), (unsigned)((rows + 7) / 8));
  const dim3 block(kWarps * 32);
  // shares of one or two scale tiles run quicker in less code (16 tokens of 1024 -> 1024: 2.1 us, 2.4 with four
  // tiles ahead), the longest want the loads (8 of 4096 -> 4096 in fp32: 15.2 us and 18.1 without)
  return w.s.katoms() <= 2 << lk
             ? launch_kernel(mx4_token_kernel<TX, PARTS, TY, VEC, 1>, grid, block, 0, st, true, (const TX*)X, xq, w, rows,
                             o, (const TY*)bias, (TY*)Y, lk, lb, per, w_early)
             : launch_kernel(mx4_token_kernel<TX, PARTS, TY, VEC, kAhead>, grid, block, 0, st, true, (const TX*)X, xq, w, rows,
                             o, (const TY*)bias, (TY*)Y, lk, lb, per, w_early);
}

template <typename TX, int PARTS, typename TY, bool VEC, int NT>
cudaError_t launch_batch(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                         cudaStream_t st) {
  const int64_t mtiles = (w.s.rows + 15) / 16;
  const int per = (int)(mtiles < kWarps ? mtiles : kWarps);
  // only as many shares as it takes to give every SM a CTA: each of them costs a start and a join
  const int64_t ctas = (mtiles + per - 1) / per * w.s.nblocks * ((rows + 8 * NT - 1) / (8 * NT));
  int shares = 1;
  while (shares < 8 && shares * 2 <= w.s.katoms() && ctas * shares < num_sms()) shares *= 2;
  const size_t inputs = (size_t)PARTS * 8 * NT * kAhead * 256, sums = (size_t)per * 8 * NT * kSumPitch * 4;
  const size_t smem = inputs > sums ? inputs : sums;
  cudaError_t e = ensure_smem_attr((const void*)mx4_batch_kernel<TX, PARTS, TY, VEC, NT>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((mtiles + per - 1) / per * shares), (unsigned)w.s.nblocks, (unsigned)((rows + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)shares, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, mx4_batch_kernel<TX, PARTS, TY, VEC, NT>, (const TX*)X, w, rows, o, (const TY*)bias, (TY*)Y, shares, per,
                         w_early);
  if (e == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return e;
}

template <typename TX, int PARTS, typename TY, bool VEC>
cudaError_t launch_vec(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                       cudaStream_t st) {
  // The direct kernel for short inputs, and as long as cutting inputs and expanding codes for every 16 outputs of every
  // 8 tokens is little work.  us, direct and batch: 32 bf16 tokens of sixty-four 64 -> 64 blocks 2.2 and 4.1, 64 of
  // 256 -> 4096 4.9 and 6.9, 32 of 1024 -> 1024 2.6 and 5.3, of 1024 -> 4096 7.9 and 7.2, of 4096 -> 4096 16.5 and 12.2; 16
  // fp32 tokens of 1024 -> 1024 3.8 and 5.2, of 1024 -> 4096 10.1 and 6.9
  if (mx4_rows_path(w.s, rows, PARTS) == kMx4Token)
    return launch_token<TX, PARTS, TY, VEC>(X, Mx4View{}, w, bias, rows, o, Y, w_early, st);
  if constexpr (PARTS > 1) {
    if (rows <= 8) return launch_batch<TX, PARTS, TY, VEC, 1>(X, w, bias, rows, o, Y, w_early, st);
  }
  if (rows <= 16) return launch_batch<TX, PARTS, TY, VEC, 2>(X, w, bias, rows, o, Y, w_early, st);
  if constexpr (PARTS == 1) {
    if (rows > 32) return launch_batch<TX, PARTS, TY, VEC, 8>(X, w, bias, rows, o, Y, w_early, st);
  }
  // several parts of 64 tokens would leave an SM one CTA: 32 tokens a pass
  return launch_batch<TX, PARTS, TY, VEC, 4>(X, w, bias, rows, o, Y, w_early, st);
}

template <typename TX, int PARTS, typename TY>
cudaError_t launch_rows(const void* X, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y, bool w_early,
                        cudaStream_t st) {
  return w.s.cols * sizeof(TX) % 16 == 0 ? launch_vec<TX, PARTS, TY, true>(X, w, bias, rows, o, Y, w_early, st)
                                         : launch_vec<TX, PARTS, TY, false>(X, w, bias, rows, o, Y, w_early, st);
}

}  // namespace

double mx4_rows_work(const Mx4Shape& w, int64_t rows) {
  return (double)w.nblocks * (double)((w.rows + 15) / 16) * w.katoms() * (double)((rows + 7) / 8);
}
bool mx4_rows_little(const Mx4Shape& w, int64_t rows, int parts) {
  return mx4_rows_work(w, rows) <= (parts == 1 ? 5120 : 3072);
}

int mx4_rows_path(const Mx4Shape& w, int64_t rows, int parts) {
  return (parts == 1 && rows <= 8) || w.katoms() <= 2 || mx4_rows_little(w, rows, parts) ? kMx4Token : kMx4Batch;
}

cudaError_t mx4_rows_fwd(const void* X, int x_dtype, const Mx4View& w, const void* bias, int64_t rows, const Mx4Out& o, void* Y,
                         int y_dtype, bool w_early, cudaStream_t st) {
  if (x_dtype == MONARCH_BF16)
    return y_dtype == MONARCH_BF16 ? launch_rows<__nv_bfloat16, 1, __nv_bfloat16>(X, w, bias, rows, o, Y, w_early, st)
                                   : launch_rows<__nv_bfloat16, 1, float>(X, w, bias, rows, o, Y, w_early, st);
  return y_dtype == MONARCH_BF16 ? launch_rows<float, 3, __nv_bfloat16>(X, w, bias, rows, o, Y, w_early, st)
                                 : launch_rows<float, 3, float>(X, w, bias, rows, o, Y, w_early, st);
}

// The tensor-core kernel takes 2.5 us and 0.37 for every 256 inputs, this one 1.7 and 0.6 for 1000 units of work.  us,
// this one and that: 1 row of 4096 -> 4096 6.0 and 8.6, 16 rows 10.9 and 8.7; 32 of 1024 -> 1024 2.8 and 4.0, 64 5.0 and
// 4.1; 16 of four 256 -> 1024 blocks 2.4 and 2.9, 32 3.1 and 2.9.
bool mx4_rows_quantised(const Mx4Shape& w, int64_t rows) {
  return mx4_rows_work(w, rows) <= 1000 + 550 * ((w.cols + 255) / 256);
}
cudaError_t mx4_rows_fwd(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Out& o, void* Y, int y_dtype, cudaStream_t st) {
  return y_dtype == MONARCH_BF16
             ? launch_token<QuantisedX, 1, __nv_bfloat16, true>(nullptr, x, w, bias, x.s.rows, o, Y, false, st)
             : launch_token<QuantisedX, 1, float, true>(nullptr, x, w, bias, x.s.rows, o, Y, false, st);
}

}  // namespace monarch
