// Products of a plain tensor with MX4 values on the bf16 tensor cores (tcgen05 kind::f16):
//
//   forward   Y[r][b*out + o]  = sum_i X[r][b*in + i] W^[b][o][i] (+ bias)     A = X,  B = W^
//   backward  dX[r][b*in + i]  = sum_o dY[r][b*out + o] W^[b][o][i]            A = dY, B = W^ (inner index N)
//             dW[b][o][i]      = sum_r dY[r][b*out + o] X^[b][r][i]            A = dY, B = X^ (rows as K)
//
// MX4 values are exact in bf16, so the MX4 operand is expanded once into the workspace (2 bytes a
// value against the product's 2 * rows operations on it) and the product is a bf16 GEMM with fp32
// sums.  A plain bf16 operand whose rows TMA can address (16-byte multiples) is read where it is;
// others are copied into padded rows first, and fp32 ones are cut into three bf16 parts there, which
// hold all 24 bits: the product then runs over K three times, once a part, smallest part first,
// against the same B.
//
// One kernel: D = A B^T per block in 256 x 256 tiles on CTA pairs (cta_group::2: each CTA loads half of
// A and half of B, so a stage of K = 64 costs an SM 32 KB for a 128 x 256 share), or in 128 x 128
// tiles on single CTAs where there are too few large tiles.  Either operand may have K as its inner
// index (rows of 128 swizzled bytes) or its M / N index (chunks of 64 x 64); all tensor maps are per
// block, so tiles that hang over a block's edge read zeros and write nothing there.  A long K with few
// tiles is split; the parts are written in fp32 and summed in order.
// The tensor cores cut their sums off towards zero, which over a long K moves them all the same way (8192 inputs of
// one sign, fp32: 5.4e-6 too small).  So sums leave TMEM in runs, of 512 inputs for fp32 and of 4096 for bf16 operands; the
// epilogue, idle under the MMAs of the next run, adds these up in registers with rounded additions (fp32 7e-8 off at any K).  fp32
// products take 2 to 6 % longer for it (8192 x 4096 -> 4096 549 and 567 us, odd widths up to 10 %), bf16 ones the same time.
// Roles: warp 0 TMA producer, warp 1 MMA issuer (of the pair's first CTA), warps 2..9 epilogue (two warps a
// TMEM lane quadrant, alternate 128-byte chunks of columns, each staging and storing its own 32 rows).
#include <algorithm>

#include "mx4.cuh"
#include "tc_common.cuh"

namespace monarch {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kSlab = 32 * 128;  // a warp's 32 rows x 128 bytes of results

struct GJob {
  int nb, mtiles, ntiles, nsplit;
  int64_t units;
  int64_t m;           // rows of D, for the epilogue without TMA
  int n;               // columns of D per block
  int64_t d_b, d_m, d_s;  // D strides (elements) of a block, a row and a split, for the epilogue without TMA
  int nk, parts;       // K stages of one part; parts of A
  int stages_per_split;
  int run;             // K stages that TMEM sums before the epilogue takes them over
  int beside;          // run beside the kernel that was launched just before (see the kernel)
  int a_chunks, b_chunks;  // inner index M / N: copies a stage takes (see load_operand)
  int a_bytes, b_bytes;    // of a CTA's stage
};

template <bool PAIR_, bool A_MN_, bool B_MN_, typename T_, bool TMA_OUT_>
struct GCfg {
  static constexpr bool PAIR = PAIR_, A_MN = A_MN_, B_MN = B_MN_, TMA_OUT = TMA_OUT_;
  using T = T_;
  static constexpr int BN = PAIR ? 256 : 128;
  static constexpr int BM = PAIR ? 256 : 128;              // rows of a unit; 128 per CTA
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;  // this CTA's 128 rows of each, K = 64
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NSTAGE = 5;
  static constexpr int TAIL = 5120;
  static constexpr int SMEM_BYTES = kEpiWarps * kSlab + NSTAGE * STAGE + TAIL + 1024;
  static constexpr int TMEM_COLS = 2 * BN;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct GBars {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float bias[kEpiWarps][128];  // of a warp's chunks of the current tile
};
static_assert(sizeof(GBars) <= 5120, "bars");

struct GUnit {
  int b, mt, nt, split;
};
// n tile fastest, then block, m tile, split
__device__ __forceinline__ GUnit unit_at(const GJob& j, int64_t unit) {
  GUnit c;
  uint32_t u = (uint32_t)unit;  // checked on the host
  c.nt = (int)(u % (uint32_t)j.ntiles);
  u /= (uint32_t)j.ntiles;
  c.b = (int)(u % (uint32_t)j.nb);
  u /= (uint32_t)j.nb;
  c.mt = (int)(u % (uint32_t)j.mtiles);
  c.split = (int)(u / (uint32_t)j.mtiles);
  return c;
}
__device__ __forceinline__ void stage_range(const GJob& j, int split, int* lo, int* hi) {
  *lo = split * j.stages_per_split;
  *hi = min(j.nk * j.parts, *lo + j.stages_per_split);
}

template <bool PAIR>
__device__ __forceinline__ void load3(void* dst, const CUtensorMap* m, uint64_t* bar, uint32_t bar0, int x, int y, int z,
                                      uint64_t pol) {
  if (PAIR)
    ptx::tma_load_3d_pair(dst, m, bar0, x, y, z, pol);
  else
    ptx::tma_load_3d(dst, m, bar, x, y, z, pol);
}
// 128 rows (M or N index r0 ..) x 64 of K (index k0 ..) of one operand.  MN: the inner index of the map is
// the operand's row, and `chunks` says how its two 64-wide halves come: 0: in one box of a 4-D map, 1: the first
// alone, 2: one after the other.  b_k: the batch coordinate, which for an MN operand may also hold the part.
template <bool PAIR, bool MN>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* m, int chunks, uint64_t* bar, uint32_t bar0,
                                             int r0, int k0, int b_k, uint64_t pol) {
  if (!MN) {
    load3<PAIR>(dst, m, bar, bar0, k0, r0, b_k, pol);
  } else if (chunks == 0) {
    if (PAIR)
      ptx::tma_load_4d_pair(dst, m, bar0, 0, k0, r0 / 64, b_k, pol);
    else
      ptx::tma_load_4d(dst, m, bar, 0, k0, r0 / 64, b_k, pol);
  } else {
    load3<PAIR>(dst, m, bar, bar0, r0, k0, b_k, pol);
    if (chunks == 2) load3<PAIR>(dst + 8192, m, bar, bar0, r0 + 64, k0, b_k, pol);
  }
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const __grid_constant__ GJob job, const typename C::T* bias,
                    typename C::T* D, int* status) {
  using T = typename C::T;
  constexpr bool PAIR = C::PAIR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* stg = smem;
  uint8_t* ring = smem + kEpiWarps * kSlab;
  GBars* bars = (GBars*)(ring + C::NSTAGE * C::STAGE);
  int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
  const bool first = rank == 0;
  const int64_t cl = PAIR ? blockIdx.x / 2 : blockIdx.x, ncl = PAIR ? gridDim.x / 2 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSTAGE; ++i) {
      ptx::mbar_init(&bars->full[i], 1);
      ptx::mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->acc_full[i], 1);
      ptx::mbar_init(&bars->acc_empty[i], (PAIR ? 2 : 1) * kEpiWarps);
    }
    ptx::mbar_init(&bars->mma_done, 1);
    bars->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(&bars->tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync_all();  // both CTAs' barriers exist and TMEM is allocated
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // beside: the kernel just before neither writes what this one reads nor touches what it writes, and had
  // itself waited for all before it when it let this one start; so this one takes the SMs that it leaves
  // free, and waits for it at the end (for the kernels after this one, which see both as done)
  if (!job.beside) ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    // ================================================================ TMA producer (both CTAs of a pair)
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmA);
      ptx::tma_prefetch_desc(&tmB);
      if (C::TMA_OUT) ptx::tma_prefetch_desc(&tmD);
      const uint64_t pol = ptx::policy_evict_normal();
      const uint32_t full0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(&bars->full[0]), 0) : 0u;
      uint32_t it = 0;
      bool ok = true;
      for (int64_t u = cl; u < job.units && ok; u += ncl) {
        const GUnit c = unit_at(job, u);
        int lo, hi;
        stage_range(job, c.split, &lo, &hi);
        const int m0 = c.mt * C::BM + (int)rank * 128, n0 = c.nt * C::BN + (int)rank * 128;
        for (int kb = lo; kb < hi; ++kb, ++it) {
          const int st = it % C::NSTAGE;
          if (!wait_or_abort(&bars->empty[st], ((it / C::NSTAGE) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
          uint8_t* sa = ring + st * C::STAGE;
          if (first) ptx::mbar_arrive_expect_tx(&bars->full[st], (PAIR ? 2 : 1) * (job.a_bytes + job.b_bytes));
          const uint32_t fb = full0 + (uint32_t)(st * sizeof(uint64_t));
          const int part = kb / job.nk, k0 = (kb - part * job.nk) * 64;
          if (C::A_MN)
            load_operand<PAIR, true>(sa, &tmA, job.a_chunks, &bars->full[st], fb, m0, k0, c.b * job.parts + part, pol);
          else
            load_operand<PAIR, false>(sa, &tmA, 0, &bars->full[st], fb, m0, kb * 64, c.b, pol);
          load_operand<PAIR, C::B_MN>(sa + C::A_BYTES, &tmB, job.b_chunks, &bars->full[st], fb, n0, k0, c.b, pol);
        }
      }
      if (!PAIR) {  // no copy may still be in flight when the CTA leaves (a pair's MMAs wait for theirs)
        const uint32_t issued = it;
        for (uint32_t k = (issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0); k < issued; ++k)
          ptx::mbar_wait_bounded(&bars->full[k % C::NSTAGE], (k / C::NSTAGE) & 1, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer (the pair's first CTA)
    if (first) {
      constexpr uint32_t idesc = make_idesc(C::BM, C::BN) | (C::A_MN ? 1u << 15 : 0u) | (C::B_MN ? 1u << 16 : 0u);
      const uint32_t ra = ptx::smem_u32(ring), rb = ra + C::A_BYTES;
      const uint64_t dA = C::A_MN ? make_sdesc_lbo(ra, 8192, 1024, 2) : make_sdesc(ra, 1024, 2);
      const uint64_t dB = C::B_MN ? make_sdesc_lbo(rb, 8192, 1024, 2) : make_sdesc(rb, 1024, 2);
      constexpr uint64_t ka = (C::A_MN ? 2048 : 32) >> 4, kb_ = (C::B_MN ? 2048 : 32) >> 4;
      uint32_t it = 0, n = 0;  // stages and runs
      bool ok = true;
      for (int64_t u = cl; u < job.units && ok; u += ncl) {
        const GUnit c = unit_at(job, u);
        int lo, hi;
        stage_range(job, c.split, &lo, &hi);
        for (int r0 = lo; r0 < hi && ok; r0 += job.run, ++n) {
          const int slot = n & 1, r1 = min(hi, r0 + job.run);
          if (!all_wait_or_abort(&bars->acc_empty[slot], ((n >> 1) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t d = tmem + slot * C::BN;
          for (int kb = r0; kb < r1; ++kb, ++it) {
            const int st = it % C::NSTAGE;
            if (!all_wait_or_abort(&bars->full[st], (it / C::NSTAGE) & 1, abort_flag, status)) { ok = false; break; }
            ptx::tc_fence_after();
            const uint64_t soff = (uint64_t)((st * C::STAGE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t acc = (kb > r0 || kk > 0) ? 1u : 0u;
              if (PAIR)
                ptx::mma_bf16_ss_pair_elect(d, dA + soff + kk * ka, dB + soff + kk * kb_, idesc, acc);
              else
                ptx::mma_bf16_ss_elect(d, dA + soff + kk * ka, dB + soff + kk * kb_, idesc, acc);
            }
            if (PAIR)
              ptx::mma_commit_pair_elect(&bars->empty[st], 0x3);
            else
              ptx::mma_commit_elect(&bars->empty[st]);
          }
          if (!ok) break;
          if (PAIR)
            ptx::mma_commit_pair_elect(&bars->acc_full[slot], 0x3);
          else
            ptx::mma_commit_elect(&bars->acc_full[slot]);
        }
      }
      if (PAIR)
        ptx::mma_commit_pair_elect(&bars->mma_done, 0x3);
      else
        ptx::mma_commit_elect(&bars->mma_done);
    }
    if (lane == 0) wait_mma_done(&bars->mma_done, abort_flag, status);
    __syncwarp();
  } else {
    // ================================================================ epilogue (8 warps a CTA)
    constexpr int CC = 128 / (int)sizeof(T);  // columns of a 128-byte chunk
    constexpr int NCH = C::BN / CC, MINE = NCH / 2, NB = MINE * CC / 32;
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2;  // warps 2..5: even chunks, 6..9: odd ones
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    uint8_t* slab = stg + ew * kSlab;
    const uint32_t slab_s = ptx::smem_u32(slab);
    float* bias_s = bars->bias[ew];
    const uint32_t acc_empty0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(&bars->acc_empty[0]), 0) : 0u;
    float next_bias[NB];
    auto fetch_bias = [&](int64_t u) {
      const GUnit c = unit_at(job, u);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int col = c.nt * C::BN + ((32 * i / CC) * 2 + half) * CC + (32 * i) % CC + lane;
        next_bias[i] = u < job.units && col < job.n ? mx4::load(bias + (int64_t)c.b * job.n + col) : 0.f;
      }
    };
    if (bias != nullptr) fetch_bias(cl);
    uint32_t n = 0;  // runs
    bool ok = true;
    auto release = [&](int slot) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (first)
          ptx::mbar_arrive(&bars->acc_empty[slot]);
        else
          ptx::mbar_arrive_cluster(acc_empty0 + (uint32_t)(slot * sizeof(uint64_t)));
      }
    };
    for (int64_t u = cl; u < job.units; u += ncl) {
      const GUnit c = unit_at(job, u);
      const int n0 = c.nt * C::BN;
      const int64_t m0 = (int64_t)c.mt * C::BM + (int64_t)rank * 128 + quad * 32;  // this warp's rows
      if (bias != nullptr) {
        __syncwarp();  // the previous tile's has been read
#pragma unroll
        for (int i = 0; i < NB; ++i) bias_s[32 * i + lane] = next_bias[i];
        __syncwarp();
        fetch_bias(u + ncl);  // asked for a tile ahead
      }
      int lo, hi;
      stage_range(job, c.split, &lo, &hi);
      if (hi - lo > job.run) {
        // the runs' sums in registers; with the last one they go back to its columns, so that they need not stay
        // in registers beside the stores
        constexpr int KEPT = MINE * CC;
        float kept[KEPT];
#pragma unroll
        for (int e = 0; e < KEPT; ++e) kept[e] = 0.f;
        for (;; lo += job.run, ++n) {
          if (!(ok = all_wait_or_abort(&bars->acc_full[n & 1], (n >> 1) & 1, abort_flag, status))) break;
          ptx::tc_fence_after();
          const bool last = hi - lo <= job.run;
          const uint32_t at = tmem + lane_off + (n & 1) * C::BN + half * CC;
#pragma unroll
          for (int e = 0; e < KEPT; e += 16) {
            uint32_t t16[16];
            ptx::tmem_ld16(at + 2 * (e / CC) * CC + e % CC, t16);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) kept[e + k] += __uint_as_float(t16[k]);
          }
          if (last) {
#pragma unroll
            for (int e = 0; e < KEPT; e += 16) {
              uint32_t t16[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) t16[k] = __float_as_uint(kept[e + k]);
              ptx::tmem_st16(at + 2 * (e / CC) * CC + e % CC, t16);
            }
            ptx::tmem_wait_st();
            break;
          }
          release(n & 1);
        }
      } else {
        ok = all_wait_or_abort(&bars->acc_full[n & 1], (n >> 1) & 1, abort_flag, status);
        ptx::tc_fence_after();
      }
      if (!ok) break;
      const uint32_t tb = tmem + lane_off + (n & 1) * C::BN;
#pragma unroll 1
      for (int i = 0; i < MINE; ++i) {
        const int ch = 2 * i + half;
        if (n0 + ch * CC >= job.n || m0 >= job.m) break;  // behind the block's last column or row
        uint32_t v[CC];
#pragma unroll
        for (int q = 0; q < CC / 16; ++q) {
          uint32_t t16[16];
          ptx::tmem_ld16(tb + ch * CC + q * 16, t16);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[q * 16 + e] = t16[e];
        }
        ptx::tmem_wait_ld();
        if (bias != nullptr) {
#pragma unroll
          for (int e = 0; e < CC; e += 4) {
            const float4 f = *(const float4*)(bias_s + i * CC + e);
            v[e] = __float_as_uint(__uint_as_float(v[e]) + f.x);
            v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) + f.y);
            v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) + f.z);
            v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) + f.w);
          }
        }
        if (C::TMA_OUT && lane == 0) ptx::bulk_wait_read_all();  // what last left the slab has been read
        __syncwarp();
        mx4::slab_write<T, CC>(slab_s, lane, v);
        if (C::TMA_OUT) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_4d(&tmD, slab, n0 + ch * CC, c.b, (int)m0, c.split);
            ptx::bulk_commit_group();
          }
        } else {  // a row pitch that is no multiple of 16 bytes
          __syncwarp();
          mx4::slab_store<T, CC>(slab, lane, D + c.split * job.d_s + m0 * job.d_m + c.b * job.d_b + n0 + ch * CC, job.d_m,
                                 (int)min((int64_t)32, job.m - m0), job.n - n0 - ch * CC);
        }
      }
      release(n++ & 1);
    }
    if (C::TMA_OUT && lane == 0) ptx::bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync_all();  // neither CTA leaves while the pair's MMAs or its peer may use it
  ptx::tc_fence_after();
  if (warp == 1) {
    if (PAIR)
      ptx::tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (job.beside) ptx::griddep_wait();
}

// ---------------------------------------------------------------- operand preparation
// What the products need first, in one launch of up to four jobs: MX4 operands in bf16, a plain operand in
// rows that TMA can address, and the bias gradient's partial sums (which read dY, so that the products
// find it in L2).  A job takes a range of the blocks.

// out[b][r][c] = value of element (b, r, c), zero for cols <= c < pitch (a multiple of 64): one thread a scale
// block, 64 rows x 128 columns a CTA; bound by the write of 2 bytes a value.
struct ExpandJob {
  Mx4View q;
  __nv_bfloat16* out;
  int pitch, ktiles;
  int64_t rtiles, blocks;  // 0 blocks: no job
};
__device__ __forceinline__ void expand_tile(const ExpandJob& j, int64_t blk) {
  const Mx4Shape& s = j.q.s;
  const int kt = (int)(blk % j.ktiles);
  blk /= j.ktiles;
  const int b = (int)(blk / j.rtiles);
  const int64_t r = (blk - b * j.rtiles) * 64 + (threadIdx.x >> 2);
  const int kb = kt * 4 + (threadIdx.x & 3);
  if (r >= s.rows || kb * 32 >= j.pitch) return;
  uint4 u = make_uint4(0, 0, 0, 0);
  uint32_t byte = 0;
  if (kb < s.kblocks()) {
    u = *(const uint4*)(j.q.codes + s.code_row(b, r) + kb * 16);
    byte = j.q.scales[s.scale_at(b, r, kb)];
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t[4];
    mx4::values8(w[i], byte, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * i + e] = t[e];
  }
  __nv_bfloat16* p = j.out + ((int64_t)b * s.rows + r) * j.pitch + kb * 32;
  ptx::st_global_v8(p, v);
  ptx::st_global_v8(p + 16, v + 8);
}

// out[r][b][p][c] = part p of X[r][b*cols + c], zero behind cols: bf16 is copied, fp32 cut into three bf16
// parts, the smallest first (see above; infinities and NaN stay in the largest).
struct StageJob {
  const void* X;
  __nv_bfloat16* out;
  int64_t nrb;  // rows * blocks
  int cols, pitch;
  int64_t blocks;
};
// times 8 values a thread: bf16 45.5 us with 4 and 47.0 with 2 (1316 rows of ten 66 <- 1703 blocks backward), fp32, whose
// three parts fill the registers, 110.4 and 107.8 (3010 rows of five 200 <- 1331)
constexpr int stage_per(int parts) { return parts == 1 ? 4 : 2; }
template <typename T>
__device__ __forceinline__ void stage_rows(const StageJob& j, int64_t blk) {
  constexpr int PARTS = sizeof(T) == 2 ? 1 : 3, kStagePer = stage_per(PARTS);
  const uint32_t words = j.pitch / 8;  // 16-byte words of a row
  const int64_t first = blk * (256 * kStagePer), total = j.nrb * words;
  const T* X = (const T*)j.X;
  uint32_t x[kStagePer][8];
  int64_t to[kStagePer];
#pragma unroll
  for (int u = 0; u < kStagePer; ++u) {
    const int64_t e = first + u * 256 + threadIdx.x, row = e / words;
    const int c = (int)(e - row * words) * 8;
    to[u] = row * PARTS * j.pitch + c;
    mx4::load8_any(X + row * j.cols + c, e < total ? j.cols - c : 0, X + j.nrb * j.cols, x[u]);
  }
#pragma unroll
  for (int u = 0; u < kStagePer; ++u) {
    if (first + u * 256 + threadIdx.x >= total) break;
    uint4* dst = (uint4*)(j.out + to[u]);
    if (PARTS == 1) {
      *dst = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = mx4::nan_in_top(x[u][i]);
#pragma unroll
      for (int p = PARTS - 1; p >= 0; --p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(x[u][2 * i], x[u][2 * i + 1], 0x7632);
        dst[p * words] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t top = x[u][i] & 0xffff0000u;
          x[u][i] = (top & 0x7f800000u) == 0x7f800000u ? 0u : __float_as_uint(__uint_as_float(x[u][i]) - __uint_as_float(top));
        }
      }
    }
  }
}

// part[k][c] = sum of rows [k * kBiasRows, + kBiasRows) of dY's column c, in a fixed order: a warp takes
// every NW-th row, a lane 16 bytes of it, or, where rows are no multiple of 16 bytes, 8 columns out of the
// aligned words that cover them (2683 rows of 20646 in bf16: 18 us beside their staging, 48 element by element), or
// one column where that would leave most SMs without work (301 rows of 1665 in fp32: 14 us for the whole backward
// pass, 24 with 8 columns).  With one part the sums are dbias.
constexpr int kBiasRows = 256;
struct BiasJob {
  const void* dY;
  float* part;
  void* dbias;
  int64_t rows, cols;
  int lane, cgroups;  // columns of a lane; groups of 32 lanes
  int64_t nparts, blocks;
};
template <typename T, int W, bool VEC, int NW>
__device__ __forceinline__ void bias_part(const BiasJob& j, int64_t blk, float (*sums)[32 * 8]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t k = blk / j.cgroups;
  const int64_t c0 = (blk - k * j.cgroups) * (32 * W), c = c0 + lane * W;
  const int64_t r0 = k * kBiasRows, r1 = min(j.rows, r0 + kBiasRows);
  const T* p = (const T*)j.dY + c;
  float acc[W] = {};
  if (c < j.cols) {
    constexpr int U = VEC || W == 1 ? 8 : sizeof(T) == 2 ? 4 : 2, N = (W * sizeof(T) + 3) / 4;  // rows in flight, words of a lane's columns
    const T* end = (const T*)j.dY + j.rows * j.cols;
    for (int64_t r = r0 + warp; r < r1; r += NW * U) {
      uint32_t v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool live = r + NW * u < r1;
        if (VEC) {
          const uint4 q = live ? *(const uint4*)(p + (r + NW * u) * j.cols) : make_uint4(0, 0, 0, 0);
          v[u][0] = q.x, v[u][1] = q.y, v[u][2] = q.z, v[u][3] = q.w;
        } else if (W == 1) {
          v[u][0] = live ? __float_as_uint(mx4::load(p + (r + NW * u) * j.cols)) : 0u;
        } else {
          mx4::load8_any(p + (r + NW * u) * j.cols, live ? (int)min((int64_t)8, j.cols - c) : 0, end, v[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (sizeof(T) == 2 && W > 1) {
            acc[(2 * i) % W] += __uint_as_float(v[u][i] << 16);
            acc[(2 * i + 1) % W] += __uint_as_float(v[u][i] & 0xffff0000u);
          } else {
            acc[i % W] += __uint_as_float(v[u][i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) sums[warp][lane * W + i] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * W; e += 32 * NW) {
    if (c0 + e >= j.cols) break;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += sums[w][e];
    if (j.nparts == 1)
      st_from_f32((T*)j.dbias + c0 + e, v);
    else
      j.part[k * j.cols + c0 + e] = v;
  }
}

template <typename T, int NW>
__device__ __forceinline__ void bias_block(const BiasJob& j, int64_t blk, float (*sums)[32 * 8]) {
  if (j.cols * sizeof(T) % 16 == 0)
    bias_part<T, 16 / sizeof(T), true, NW>(j, blk, sums);
  else if (j.lane == 8)
    bias_part<T, 8, false, NW>(j, blk, sums);
  else
    bias_part<T, 1, false, NW>(j, blk, sums);
}
// The same in the room that dX's product leaves on its SMs (11776 registers, 24 KB), which it begins beside:
// dY was ready before that did.  Its last CTA waits for that product, so that whoever waits for this kernel has
// waited for both.
constexpr int kBesideWarps = 4;
template <typename T>
__global__ void __launch_bounds__(kBesideWarps * 32, 7) mx4_bias_kernel(const __grid_constant__ BiasJob bias) {
  __shared__ float sums[kBesideWarps][32 * 8];
  ptx::griddep_launch_dependents();
  bias_block<T, kBesideWarps>(bias, blockIdx.x, sums);
  if (blockIdx.x == gridDim.x - 1) ptx::griddep_wait();
}

template <typename T>
__global__ void __launch_bounds__(256, 4)  // the most demanding job must not cost the others their occupancy
    mx4_prepare_kernel(const __grid_constant__ BiasJob bias, const __grid_constant__ ExpandJob e0, const __grid_constant__ ExpandJob e1,
                       const __grid_constant__ StageJob stage) {
  __shared__ float sums[8][32 * 8];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int64_t blk = blockIdx.x;
  if (blk < bias.blocks) {
    bias_block<T, 8>(bias, blk, sums);
    return;
  }
  blk -= bias.blocks;
  if (blk < stage.blocks) {
    stage_rows<T>(stage, blk);
    return;
  }
  blk -= stage.blocks;
  if (blk < e0.blocks)
    expand_tile(e0, blk);
  else
    expand_tile(e1, blk - e0.blocks);
}

// What is left to add at the end, parts in order: out[e] over nsplit parts of n values (+ bias[e % width]).
struct SumJob {
  const float* part;
  void* out;
  int64_t n, nsplit;
  const void* bias;
  int64_t width;
};
template <typename T>
__global__ void __launch_bounds__(256)
    mx4_sum_kernel(const __grid_constant__ SumJob j0, const __grid_constant__ SumJob j1, const __grid_constant__ SumJob j2) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t total = j0.n + j1.n + j2.n;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const bool second = e >= j0.n, third = e >= j0.n + j1.n;
    const SumJob& j = third ? j2 : second ? j1 : j0;
    const int64_t i = e - (third ? j0.n + j1.n : second ? j0.n : 0);
    float acc = 0.f;
#pragma unroll 8
    for (int64_t s = 0; s < j.nsplit; ++s) acc += j.part[s * j.n + i];
    if (j.bias != nullptr) acc += mx4::load((const T*)j.bias + i % j.width);
    st_from_f32((T*)j.out + i, acc);
  }
}

unsigned blocks_for(int64_t threads) {
  const int64_t n = (threads + 255) / 256, most = (int64_t)num_sms() * 16;
  return (unsigned)(n < 1 ? 1 : n < most ? n : most);
}

int up(int v, int to) { return (v + to - 1) / to * to; }
int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }
size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

// ---------------------------------------------------------------- tensor maps
bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  EncodeTiledFn enc = get_encode();
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc != nullptr && enc(m, type, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A bf16 operand: (inner, outer, batch) with strides in elements.
struct Operand {
  const void* p;
  int64_t inner, outer, batch;
  int64_t s_outer, s_batch;
};
// M (or N) index outside.  A box is no longer than the `extent` rows of the operand, if it is alone (rows behind the
// last are dear to TMA: 2000 rows of two 2048 -> 16 blocks forward 10.4 us and 9.4 so, dW 23.4 and 13.7 with half of
// its tile); what stands behind belongs to results that are not stored.
bool kmajor_map(CUtensorMap* m, const Operand& o, int64_t extent, bool alone, int* bytes) {
  const int rows = alone && extent < 128 ? (int)((extent + 7) / 8 * 8) : 128;
  *bytes = rows * 128;
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)o.batch};
  const cuuint64_t st[2] = {(cuuint64_t)o.s_outer * 2, (cuuint64_t)o.s_batch * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o.p, dims, st, box);
}
bool mnmajor_map(CUtensorMap* m, const Operand& o, int64_t extent, bool alone, int* bytes, int* chunks) {
  const bool half = alone && extent <= 64;
  *bytes = half ? 8192 : 16384;
  *chunks = half ? 1 : o.inner % 64 == 0 ? 0 : 2;
  if (*chunks == 0) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)o.outer, (cuuint64_t)o.inner / 64, (cuuint64_t)o.batch};
    const cuuint64_t st[3] = {(cuuint64_t)o.s_outer * 2, 128, (cuuint64_t)o.s_batch * 2};
    const cuuint32_t box[4] = {64, 64, 2, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, o.p, dims, st, box);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)o.batch};
  const cuuint64_t st[2] = {(cuuint64_t)o.s_outer * 2, (cuuint64_t)o.s_batch * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o.p, dims, st, box);
}

// D: columns n, rows m of nb blocks; strides in elements of a row, a block and a split.
struct Result {
  void* p;
  int64_t m;
  int n, nb;
  int64_t d_m, d_b, d_s;
};

struct Plan {
  bool pair;
  int nsplit, per_split;
};
// 256 x 256 tiles on pairs or 128 x 128 on single CTAs, and how many parts of K: whichever takes the least
// time by this count of microseconds: rounds over the SMs, 0.40 (pair) or 0.33 a stage of 64 inputs (8192 x 1024 ->
// 4096: 52.4 us on pairs, 81 on single CTAs), a tile's start and epilogue, and, when K is split, the partial
// sums' way out and back.
Plan plan_for(int64_t m, int n, int nb, int nk) {
  Plan best{};
  double least = 1e30;
  for (int pair = 0; pair < 2; ++pair) {
    const int bm = pair ? 256 : 128;
    const int64_t tiles = (m + bm - 1) / bm * ((n + bm - 1) / bm) * nb, slots = pair ? num_sms() / 2 : num_sms();
    for (int want = 1; want <= 64 && want * 4 <= std::max(nk, 4); want *= 2) {
      const int per = (nk + want - 1) / want, ns = (nk + per - 1) / per;
      const int64_t rounds = (tiles * ns + slots - 1) / slots;
      double t = (double)rounds * (per * (pair ? 0.40 : 0.33) + (pair ? 2.0 : 1.2));
      if (ns > 1) t += 4.0 + (double)m * n * nb * 4 * (ns + 1) / 4e6;
      if (t < least) {
        least = t;
        best = Plan{pair != 0, ns, per};
      }
    }
  }
  return best;
}
size_t part_bytes(const Plan& p, int64_t results) { return p.nsplit > 1 ? (size_t)p.nsplit * (size_t)results * 4 : 0; }

template <class C>
cudaError_t launch(const Operand& a, const Operand& b, const Result& d, const void* bias, GJob j, int* status, cudaStream_t st) {
  using T = typename C::T;
  CUtensorMap mA, mB, mD;
  constexpr bool alone = !C::PAIR;  // a pair's two CTAs hold different rows
  if (!(C::A_MN ? mnmajor_map(&mA, a, d.m, alone, &j.a_bytes, &j.a_chunks) : kmajor_map(&mA, a, d.m, alone, &j.a_bytes)) ||
      !(C::B_MN ? mnmajor_map(&mB, b, d.n, alone, &j.b_bytes, &j.b_chunks) : kmajor_map(&mB, b, d.n, alone, &j.b_bytes)))
    return cudaErrorInvalidValue;
  if (C::TMA_OUT) {
    const cuuint64_t dims[4] = {(cuuint64_t)d.n, (cuuint64_t)d.nb, (cuuint64_t)d.m, (cuuint64_t)j.nsplit};
    const cuuint64_t strides[3] = {(cuuint64_t)d.d_b * sizeof(T), (cuuint64_t)d.d_m * sizeof(T), (cuuint64_t)d.d_s * sizeof(T)};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / sizeof(T)), 1, 32, 1};
    if (!encode(&mD, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, d.p, dims, strides, box))
      return cudaErrorInvalidValue;
  } else {
    mD = mA;  // unused
  }
  j.mtiles = (int)((d.m + C::BM - 1) / C::BM);
  j.ntiles = (d.n + C::BN - 1) / C::BN;
  j.units = (int64_t)j.nb * j.mtiles * j.ntiles * j.nsplit;
  if (j.units > (int64_t(1) << 31)) return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_attr((const void*)mx4_gemm_kernel<C>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t slots = C::PAIR ? num_sms() / 2 : num_sms();
  const int64_t n = j.units < slots ? j.units : slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(C::PAIR ? 2 * n : n));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = C::PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<C>, mA, mB, mD, j, (const T*)bias, (T*)d.p, status);
  if (e == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return e;
}

template <bool A_MN, bool B_MN, typename T>
cudaError_t gemm(const Operand& a, const Operand& b, const Result& d, const void* bias, int nb, int64_t k, int parts, const Plan& p,
                 bool beside, int* status, cudaStream_t st) {
  GJob j = {};
  j.beside = beside;
  j.nb = nb;
  j.nsplit = p.nsplit;
  j.m = d.m;
  j.n = d.n;
  j.d_b = d.d_b;
  j.d_m = d.d_m;
  j.d_s = d.d_s;
  j.nk = (int)((k + 63) / 64);
  j.parts = parts;
  j.stages_per_split = p.per_split;
  j.run = parts == 1 ? 64 : p.nsplit == 1 && j.nk <= 8 ? 24 : 8;  // 24: one run, in which 8 stages are the leading part's
  const bool tma = d.d_m * sizeof(T) % 16 == 0 && d.d_b * sizeof(T) % 16 == 0 && d.d_s * sizeof(T) % 16 == 0;
  if (p.pair)
    return tma ? launch<GCfg<true, A_MN, B_MN, T, true>>(a, b, d, bias, j, status, st)
               : launch<GCfg<true, A_MN, B_MN, T, false>>(a, b, d, bias, j, status, st);
  return tma ? launch<GCfg<false, A_MN, B_MN, T, true>>(a, b, d, bias, j, status, st)
             : launch<GCfg<false, A_MN, B_MN, T, false>>(a, b, d, bias, j, status, st);
}

int parts_of(int dtype) { return dtype == MONARCH_BF16 ? 1 : 3; }
// A plain (rows, nb * blk) operand is read where it is if it is bf16 and TMA can address its blocks.
bool direct(int dtype, int blk) { return dtype == MONARCH_BF16 && blk % 8 == 0; }
size_t staged_bytes(const Mx4Linear& d, int blk) {
  return direct(d.dtype, blk) ? 0 : al256((size_t)d.rows * d.nb * parts_of(d.dtype) * up(blk, 64) * 2);
}
size_t expanded_bytes(const Mx4Shape& s) { return al256((size_t)s.nblocks * s.rows * up(s.cols, 64) * 2); }
int stages(int64_t k, int dtype) { return (int)((k + 63) / 64) * parts_of(dtype); }
Plan fwd_plan(const Mx4Linear& d) { return plan_for(d.rows, d.out, d.nb, stages(d.in, d.dtype)); }
Plan dx_plan(const Mx4Linear& d) { return plan_for(d.rows, d.in, d.nb, stages(d.out, d.dtype)); }
Plan dw_plan(const Mx4Linear& d) { return plan_for(d.out, d.in, d.nb, stages(d.rows, d.dtype)); }
size_t fwd_part_bytes(const Mx4Linear& d) { return al256(part_bytes(fwd_plan(d), d.rows * d.nb * d.out)); }
size_t dx_part_bytes(const Mx4Linear& d) { return al256(part_bytes(dx_plan(d), d.rows * d.nb * d.in)); }
size_t dw_part_bytes(const Mx4Linear& d) { return al256(part_bytes(dw_plan(d), (int64_t)d.nb * d.out * d.in)); }

ExpandJob expand_job(const Mx4View& q, void* out) {
  ExpandJob j;
  j.q = q;
  j.out = (__nv_bfloat16*)out;
  j.pitch = up(q.s.cols, 64);
  j.ktiles = (j.pitch + 127) / 128;
  j.rtiles = (q.s.rows + 63) / 64;
  j.blocks = j.rtiles * j.ktiles * q.s.nblocks;
  return j;
}
// The K-major view of a plain operand, and the job that stages it into `ws` if that is needed.
Operand staged(const void* X, const Mx4Linear& d, int blk, void* ws, StageJob* job) {
  *job = StageJob{};
  const int parts = parts_of(d.dtype);
  if (direct(d.dtype, blk)) return Operand{X, blk, d.rows, d.nb, (int64_t)d.nb * blk, blk};
  const int pitch = up(blk, 64);
  *job = StageJob{X, (__nv_bfloat16*)ws, d.rows * d.nb, blk, pitch, 0};
  job->blocks = (job->nrb * (pitch / 8) + 256 * stage_per(parts) - 1) / (256 * stage_per(parts));
  return Operand{ws, (int64_t)parts * pitch, d.rows, d.nb, (int64_t)d.nb * parts * pitch, (int64_t)parts * pitch};
}
int64_t bias_parts(const Mx4Linear& d) { return (d.rows + kBiasRows - 1) / kBiasRows; }
size_t bias_part_bytes(const Mx4Linear& d) {
  return d.has_bias && bias_parts(d) > 1 ? al256((size_t)bias_parts(d) * d.nb * d.out * 4) : 0;
}
cudaError_t prepare(const Mx4Linear& d, const BiasJob& b, const ExpandJob& e0, const ExpandJob& e1, const StageJob& s, cudaStream_t st) {
  const int64_t blocks = b.blocks + e0.blocks + e1.blocks + s.blocks;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return d.dtype == MONARCH_BF16
             ? launch_kernel(mx4_prepare_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(256), 0, st, true, b, e0, e1, s)
             : launch_kernel(mx4_prepare_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, st, true, b, e0, e1, s);
}
// A K-major operand with its rows as K: one batch entry per (block, part).
Operand rows_as_k(const Operand& o, const Mx4Linear& d, int blk) {
  if (direct(d.dtype, blk)) return o;
  const int parts = parts_of(d.dtype), pitch = up(blk, 64);
  return Operand{o.p, pitch, o.outer, (int64_t)d.nb * parts, o.s_outer, pitch};
}
Operand expanded(const void* p, const Mx4Shape& s) {
  const int pitch = up(s.cols, 64);
  return Operand{p, pitch, s.rows, s.nblocks, pitch, (int64_t)pitch * s.rows};
}

// One product into `out` (results in the order of `r`), or into fp32 parts when K is split.
template <bool A_MN, bool B_MN>
cudaError_t product(const Operand& a, const Operand& b, Result r, const void* bias, const Mx4Linear& d, int64_t k, const Plan& p,
                    float* part, int64_t results, bool beside, int* status, cudaStream_t st) {
  const int parts = parts_of(d.dtype);
  r.d_s = results;
  if (p.nsplit > 1) {
    r.p = part;
    return gemm<A_MN, B_MN, float>(a, b, r, nullptr, d.nb, k, parts, p, beside, status, st);
  }
  r.d_s = up64(results);  // one part: any stride that a tensor map takes
  return d.dtype == MONARCH_BF16 ? gemm<A_MN, B_MN, __nv_bfloat16>(a, b, r, bias, d.nb, k, parts, p, beside, status, st)
                                 : gemm<A_MN, B_MN, float>(a, b, r, bias, d.nb, k, parts, p, beside, status, st);
}
cudaError_t sum(int dtype, const SumJob& j0, const SumJob& j1, const SumJob& j2, cudaStream_t st) {
  const int64_t n = j0.n + j1.n + j2.n;
  if (n == 0) return cudaSuccess;
  return dtype == MONARCH_BF16 ? launch_kernel(mx4_sum_kernel<__nv_bfloat16>, dim3(blocks_for(n)), dim3(256), 0, st, true, j0, j1, j2)
                               : launch_kernel(mx4_sum_kernel<float>, dim3(blocks_for(n)), dim3(256), 0, st, true, j0, j1, j2);
}

// Scratch: the operands in bf16, split sums of dX and of dW, parts of dbias.
struct BwdWs {
  size_t w, x, dy, part_x, part_w, bias, total;
};
BwdWs bwd_layout(const Mx4Linear& d) {
  BwdWs l;
  l.w = 0;
  l.x = l.w + expanded_bytes(d.w());
  l.dy = l.x + expanded_bytes(d.x());
  l.part_x = l.dy + staged_bytes(d, d.out);
  l.part_w = l.part_x + dx_part_bytes(d);
  l.bias = l.part_w + dw_part_bytes(d);
  l.total = l.bias + bias_part_bytes(d);
  return l;
}

}  // namespace

static int path_of(const Plan& p) { return (p.pair ? kMx4GemmPair : kMx4Gemm) + (p.nsplit > 1 ? kMx4Split : 0); }
int mx4_gemm_fwd_path(const Mx4Linear& d) { return path_of(fwd_plan(d)); }
int mx4_gemm_dx_path(const Mx4Linear& d) { return path_of(dx_plan(d)); }
int mx4_gemm_dw_path(const Mx4Linear& d) { return path_of(dw_plan(d)); }

size_t mx4_gemm_fwd_bytes(const Mx4Linear& d) { return expanded_bytes(d.w()) + staged_bytes(d, d.in) + fwd_part_bytes(d); }

cudaError_t mx4_gemm_fwd(const void* X, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, void* ws, int* status,
                         cudaStream_t st) {
  char* wd = (char*)ws;
  char* xs = wd + expanded_bytes(d.w());
  float* part = (float*)(xs + staged_bytes(d, d.in));
  StageJob sj;
  const Operand a = staged(X, d, d.in, xs, &sj);
  cudaError_t e = prepare(d, BiasJob{}, expand_job(w, wd), ExpandJob{}, sj, st);
  if (e != cudaSuccess) return e;
  const int64_t width = (int64_t)d.nb * d.out, results = d.rows * width;
  const Plan p = fwd_plan(d);
  e = product<false, false>(a, expanded(wd, d.w()), Result{Y, d.rows, d.out, d.nb, width, d.out, 0}, bias, d, d.in, p, part, results,
                            false, status, st);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return sum(d.dtype, SumJob{part, Y, results, p.nsplit, bias, width}, SumJob{}, SumJob{}, st);
}

size_t mx4_gemm_bwd_bytes(const Mx4Linear& d) { return bwd_layout(d).total; }

cudaError_t mx4_gemm_bwd(const void* dY, const Mx4View& x, const Mx4View& w, const Mx4Linear& d, void* dX, void* dW, void* dbias,
                         void* ws, int* status, cudaStream_t st) {
  const BwdWs l = bwd_layout(d);
  char* base = (char*)ws;
  float *part_x = (float*)(base + l.part_x), *part_w = (float*)(base + l.part_w);
  const int64_t n_in = (int64_t)d.nb * d.in, n_out = (int64_t)d.nb * d.out;
  StageJob sj;
  const Operand a = staged(dY, d, d.out, base + l.dy, &sj);
  if (dX == nullptr && dW == nullptr) sj.blocks = 0;
  const int es = d.dtype == MONARCH_BF16 ? 2 : 4;
  BiasJob bj = {};
  if (dbias != nullptr) {
    const int lane = n_out * es % 16 == 0 ? 16 / es : bias_parts(d) * ((n_out + 255) / 256) >= 2 * num_sms() ? 8 : 1;
    bj = BiasJob{dY, (float*)(base + l.bias), dbias, d.rows, n_out, lane, (int)((n_out + 32 * lane - 1) / (32 * lane)), bias_parts(d), 0};
    bj.blocks = bj.nparts * bj.cgroups;
  }
  // dbias beside dX's product, if that lasts as long as a pass over dY in the room it leaves: by the operations on
  // a byte of dY.  us with dbias in the first launch and beside: 8192 x 1024 -> 4096 118.5 and 112.2, 2048 rows of
  // eight 384 -> 512 blocks 35.8 and 33.2, of four 256 -> 1024 65.9 and 68.5 (8192 rows; in fp32, 1500: 53.2 and 50.9).
  const bool apart = dbias != nullptr && dX != nullptr && dW != nullptr && d.rows * n_out * es >= 1 << 20 &&
                     d.in * parts_of(d.dtype) >= 192 * es;
  cudaError_t e = prepare(d, apart ? BiasJob{} : bj, dX != nullptr ? expand_job(w, base + l.w) : ExpandJob{}, dW != nullptr ? expand_job(x, base + l.x) : ExpandJob{},
                          sj, st);
  if (e != cudaSuccess) return e;
  SumJob sum_x = {}, sum_w = {}, sum_b = {};
  if (dX != nullptr) {
    const Plan p = dx_plan(d);
    e = product<false, true>(a, expanded(base + l.w, d.w()), Result{dX, d.rows, d.in, d.nb, n_in, d.in, 0}, nullptr, d, d.out, p, part_x,
                             d.rows * n_in, false, status, st);
    if (e != cudaSuccess) return e;
    if (p.nsplit > 1) sum_x = SumJob{part_x, dX, d.rows * n_in, p.nsplit, nullptr, 1};
  }
  if (apart) {
    const dim3 grid((unsigned)bj.blocks), block(kBesideWarps * 32);
    e = d.dtype == MONARCH_BF16 ? launch_kernel(mx4_bias_kernel<__nv_bfloat16>, grid, block, 0, st, true, bj)
                                : launch_kernel(mx4_bias_kernel<float>, grid, block, 0, st, true, bj);
    if (e != cudaSuccess) return e;
  }
  if (dW != nullptr) {
    const Plan p = dw_plan(d);
    // beside dX's product, if that went before (and dbias): its operands were ready when that began
    e = product<true, true>(rows_as_k(a, d, d.out), expanded(base + l.x, d.x()), Result{dW, d.out, d.in, d.nb, d.in, (int64_t)d.out * d.in, 0},
                            nullptr, d, d.rows, p, part_w, n_out * d.in, dX != nullptr, status, st);
    if (e != cudaSuccess) return e;
    if (p.nsplit > 1) sum_w = SumJob{part_w, dW, n_out * d.in, p.nsplit, nullptr, 1};
  }
  if (dbias != nullptr && bj.nparts > 1) sum_b = SumJob{bj.part, dbias, n_out, bj.nparts, nullptr, 1};
  return sum(d.dtype, sum_x, sum_w, sum_b, st);
}

}  // namespace monarch
