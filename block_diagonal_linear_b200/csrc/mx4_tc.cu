// Block-diagonal product with both operands in MX4 on the block-scaled tensor cores (tcgen05
// kind::mxf4, E2M1 operands, one E8M0 scale per 32 values):
//
//   Y[r][b*out + o] = sum_i X^[b][r][i] W^[b][o][i] (+ bias)     fp32 sums in TMEM.
//
// Products of two codes are exact and the hardware applies both scales to them before they join the
// fp32 sum, so the result is rounded once, in the epilogue.
//
// Tiles are 256 x 256 on CTA pairs (cta_group::2: each CTA loads 128 rows of X and 128 of W, 35 KB a stage
// for its 128 x 256 share; alone it would load 51 KB), or 128 x 64..256 on single CTAs where there are too few
// large ones or K is short; a CTA may then keep the one tile of W it works on.  A long product (8192 x 4096 ->
// 4096: 62.9 us) is bound by the MMAs, 46 us with everything else left out; waiting for loads adds 7, the scale
// copies, which take turns with the MMAs, 5, the epilogue 5.  Short ones are bound by Y's writes (10000 rows of
// four 256 -> 1024 blocks: 17.0 us, a library's fill of Y alone 22).  A stage of the
// ring holds 256 values of K as 128-byte swizzled rows, with the scale tiles (512 bytes for 128 rows x 128
// values; a quantised tensor keeps them in the order that tcgen05.cp wants).  The MMA warp copies a
// stage's scale tiles to TMEM and issues four MMAs of K = 64.  K beyond the tensor is filled with zero
// codes and zero scale bytes (2^-127) by TMA, and steps of K that lie wholly behind the end are not issued.
//
// TMEM (512 columns): two accumulators, so that the epilogue of one tile runs under the MMAs of the
// next.  With BN = 256 they overlap in 40 columns, [0, 256) and [216, 472): the epilogue reads the
// chunks with the shared columns first and then lets the next tile begin.  Scales take [472, 508), three
// buffers for 128 values of K each, so that the copy for the next 128 does not wait for the MMAs that
// read the last ones (8192 x 4096 -> 4096: 81.5 us with one buffer a stage, 72.9 with the copies between the MMAs).
// Roles: warp 0 TMA producer, warp 1 MMA issuer (of the pair's first CTA) and TMEM owner, warps 2..9
// epilogue: two warps a TMEM lane quadrant, one row a thread, alternate 128-byte chunks of columns.  Each
// warp stages and stores its own 32 rows, so that no warp waits for another (with four warps that met at
// barriers around a common staging buffer the epilogue bounded short K: 10000 rows of four 256 -> 1024
// blocks took 28.4 us, with these 20.4, and with the steps after them 17.0).
#include "mx4.cuh"
#include "tc_common.cuh"

namespace monarch {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kSfCol = 472;  // first TMEM column of the scales
constexpr int kSlab = 32 * 128;  // a warp's 32 rows x 128 bytes of output
// The tensor cores cut their sums off towards zero.  Steps of 64 exact products are few: fp32 results of 16384 inputs are
// 2.3e-7 off at most, but those of 65536 inputs of one sign 4.2e-6 and of 262144 4.7e-5 (1.3e-7 so).  So from here on fp32 results join
// runs of 4096 inputs with rounded additions, in the 128 x 128 tile.
constexpr int kRunFrom = 16384;

struct Job {
  int nb, mtiles, ntiles;
  int64_t units;
  int64_t rows;
  int out;
  int ksteps;  // MMA steps of 64 values
  int x_bytes, w_bytes;  // of X's and W's codes in a stage
  int64_t x_ratoms, w_ratoms;
};

// KEEP: a CTA has one tile of W, whose up to four stages stay in shared memory, and every so many row tiles of
// X; only X's stages come with every tile.
// RUNS: sums leave TMEM every RUN stages and join with rounded additions (see below).
template <int BN_, bool PAIR_, bool KEEP_ = false, bool RUNS_ = false>
struct Cfg {
  static constexpr bool PAIR = PAIR_, KEEP = KEEP_, RUNS = RUNS_;
  static constexpr int RUN = 16;  // 4096 values
  static_assert(!RUNS || (!KEEP && 2 * BN_ <= (int)kSfCol), "accumulators without common columns");
  static_assert(!(PAIR && KEEP), "pairs share W's tiles already");
  static constexpr int BN = BN_, BM = PAIR ? 256 : 128;  // of a unit; a CTA holds 128 rows
  static constexpr int BROWS = PAIR ? BN / 2 : BN;       // rows of W that a CTA loads
  static constexpr int NT = BN >= 128 ? BN / 128 : 1;    // scale tiles of W per 128 values of K
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BROWS * 128;
  static constexpr int SFA_BYTES = 1024, SFB_BYTES = 1024 * NT;
  // X's part of a stage, and W's: behind it, or (KEEP) in a ring of its own behind X's
  static constexpr int XSTAGE = A_BYTES + SFA_BYTES, WSTAGE = B_BYTES + SFB_BYTES;
  static constexpr int STAGE = KEEP ? XSTAGE : XSTAGE + WSTAGE;
  static constexpr int WPITCH = KEEP ? WSTAGE : STAGE, WKEPT = KEEP ? 4 : 0;
  static constexpr int SLOT1 = BN == 256 ? 216 : BN;     // first column of the second accumulator
  // output slabs of a warp; long products want a further stage more than a second slab (pairs, 8192 x 2048 -> 4096:
  // 40.8 us with two, 38.1 with one), short ones the slab (singles, 128 inputs: 17.2 and 18.0)
  static constexpr int SLABS = PAIR || KEEP ? 1 : 2;
  static constexpr int STG_BYTES = SLABS * kEpiWarps * kSlab;
  static constexpr int TAIL = 5120;
  static constexpr int NSTAGE_RAW = (kSmemBudget - STG_BYTES - TAIL - WKEPT * WSTAGE) / STAGE;
  static constexpr int NSTAGE = NSTAGE_RAW > 8 ? 8 : NSTAGE_RAW;
  static constexpr int SMEM_BYTES = STG_BYTES + NSTAGE * STAGE + WKEPT * WSTAGE + TAIL + 1024;
  static_assert(STAGE % 1024 == 0 && NSTAGE >= 2 && SLOT1 + BN <= (int)kSfCol && SMEM_BYTES <= 227 * 1024, "layout");
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t wfull[4];  // KEEP: of W's stages
  uint64_t acc_full[2];
  uint64_t acc_next;  // the next tile's accumulator may be written
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float bias[kEpiWarps][128];  // of a warp's chunks of the current tile
};
static_assert(sizeof(Bars) <= 5120, "bars");

// Instruction descriptor of kind::mxf4: A, B E2M1, scales E8M0, byte pair `pair` of the scale words.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int pair) {
  return ((uint32_t)(pair * 2) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)(pair * 2) << 29);
}
// Unswizzled 32 x 16-byte scale tile: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

struct Unit {
  int b, mt, nt;
};
template <bool KEEP>
__device__ __forceinline__ Unit unit_at(const Job& j, int64_t unit) {
  Unit c;
  if (KEEP) {  // a row tile of this CTA's tile of W
    const uint32_t w = blockIdx.x % (uint32_t)(j.nb * j.ntiles);
    c.nt = (int)(w % (uint32_t)j.ntiles);
    c.b = (int)(w / (uint32_t)j.ntiles);
    c.mt = (int)unit;
    return c;
  }
  uint32_t u = (uint32_t)unit;  // Y would be larger than any memory before this overflows; checked on the host
  c.nt = (int)(u % (uint32_t)j.ntiles);
  u /= (uint32_t)j.ntiles;
  c.b = (int)(u % (uint32_t)j.nb);
  c.mt = (int)(u / (uint32_t)j.nb);
  return c;
}

template <bool PAIR>
__device__ __forceinline__ void load3(void* dst, const CUtensorMap* m, uint64_t* bar, uint32_t bar0, int x, int y, int z,
                                      uint64_t pol) {
  if (PAIR)
    ptx::tma_load_3d_pair(dst, m, bar0, x, y, z, pol);
  else
    ptx::tma_load_3d(dst, m, bar, x, y, z, pol);
}

template <class C, typename T, bool TMA_OUT>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmSX, const __grid_constant__ CUtensorMap tmSW,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Job job, const T* bias, T* Y, int* status) {
  constexpr bool PAIR = C::PAIR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* stg = smem;
  uint8_t* ring = smem + C::STG_BYTES;
  uint8_t* wring = ring + (C::KEEP ? C::NSTAGE * C::STAGE : C::XSTAGE);
  Bars* bars = (Bars*)(ring + C::NSTAGE * C::STAGE + C::WKEPT * C::WSTAGE);
  int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
  const bool first = rank == 0;
  const int64_t cl = PAIR ? blockIdx.x / 2 : blockIdx.x, ncl = PAIR ? gridDim.x / 2 : gridDim.x;
  const int nkb = (job.ksteps + 3) / 4;  // stages of a unit
  // this CTA's units: every ncl-th; KEEP: row tiles, shared out among the CTAs with the same tile of W
  const int64_t nw = C::KEEP ? (int64_t)job.nb * job.ntiles : 1;
  const int64_t u0 = cl / nw, u1 = C::KEEP ? job.mtiles : job.units, ustep = C::KEEP ? (ncl - 1 - cl % nw) / nw + 1 : ncl;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSTAGE; ++i) {
      ptx::mbar_init(&bars->full[i], 1);
      ptx::mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < C::WKEPT; ++i) ptx::mbar_init(&bars->wfull[i], 1);
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&bars->acc_full[i], 1);
    ptx::mbar_init(&bars->acc_next, (PAIR ? 2 : 1) * kEpiWarps);
    ptx::mbar_init(&bars->mma_done, 1);
    bars->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(&bars->tmem_base, 512);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&bars->tmem_base, 512);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync_all();  // both CTAs' barriers exist and TMEM is allocated
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  ptx::griddep_wait();  // the operands may come from the previous kernel of the stream
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    // ================================================================ TMA producer (both CTAs of a pair)
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmX);
      ptx::tma_prefetch_desc(&tmW);
      ptx::tma_prefetch_desc(&tmSX);
      ptx::tma_prefetch_desc(&tmSW);
      if (TMA_OUT) ptx::tma_prefetch_desc(&tmY);
      const uint64_t pol = ptx::policy_evict_normal();
      const uint32_t full0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(&bars->full[0]), 0) : 0u;
      uint32_t it = 0;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok; u += ustep) {
        const Unit c = unit_at<C::KEEP>(job, u);
        const int xt = c.mt * (C::BM / 128) + (int)rank;  // this CTA's scale tile of X rows
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int st = it % C::NSTAGE;
          uint8_t* sa = ring + st * C::STAGE;
          uint8_t* sb = wring + st * C::WPITCH;
          uint64_t* fl = &bars->full[st];
          const uint32_t fb = full0 + (uint32_t)(st * sizeof(uint64_t));
          // two scale tiles of 128 values each: 128 words a tile; all of W's rows in both CTAs.  Tiles behind
          // the tensor are zeros, those behind a block belong to columns that are not stored.
          if (C::KEEP && u == u0) {
            uint8_t* sw = wring + kb * C::WPITCH;
            ptx::mbar_arrive_expect_tx(&bars->wfull[kb], C::WSTAGE - C::B_BYTES + job.w_bytes);
            load3<PAIR>(sw, &tmW, &bars->wfull[kb], 0, kb * 128, c.nt * C::BN, c.b, pol);
            load3<PAIR>(sw + C::B_BYTES, &tmSW, &bars->wfull[kb], 0, 0, 2 * kb, (int)(c.b * job.w_ratoms) + c.nt * C::BN / 128, pol);
          }
          if (!wait_or_abort(&bars->empty[st], ((it / C::NSTAGE) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
          if (first) ptx::mbar_arrive_expect_tx(fl, (PAIR ? 2 : 1) * (C::STAGE - C::A_BYTES + job.x_bytes - (C::KEEP ? 0 : C::B_BYTES - job.w_bytes)));
          load3<PAIR>(sa, &tmX, fl, fb, kb * 128, xt * 128, c.b, pol);
          if (!C::KEEP) load3<PAIR>(sb, &tmW, fl, fb, kb * 128, c.nt * C::BN + (int)rank * C::BROWS, c.b, pol);
          load3<PAIR>(sa + C::A_BYTES, &tmSX, fl, fb, 0, 2 * kb, (int)(c.b * job.x_ratoms) + xt, pol);
          if (!C::KEEP)
            load3<PAIR>(sb + C::B_BYTES, &tmSW, fl, fb, 0, 2 * kb, (int)(c.b * job.w_ratoms) + c.nt * C::BN / 128, pol);
        }
      }
      if (!PAIR) {  // no copy may still be in flight when the CTA leaves (a pair's MMAs wait for theirs)
        const uint32_t issued = it;
        for (uint32_t k = (issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0); k < issued; ++k)
          ptx::mbar_wait_bounded(&bars->full[k % C::NSTAGE], (k / C::NSTAGE) & 1, kWaitLimitNs);
        if (C::KEEP)  // as many of W's as of X's first tile, at least
          for (uint32_t k = 0; k < (uint32_t)nkb && k < issued + (ok ? 0 : 1); ++k)
            ptx::mbar_wait_bounded(&bars->wfull[k], 0, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer (the pair's first CTA)
    if (first) {
      const uint32_t ring_s = ptx::smem_u32(ring);
      const uint32_t wring_s = ptx::smem_u32(wring);
      const uint64_t dA = make_sdesc(ring_s, 1024, 2), dB = make_sdesc(wring_s, 1024, 2);
      const uint64_t dSA = scale_desc(ring_s + C::A_BYTES), dSB = scale_desc(wring_s + C::B_BYTES);
      const int run = C::RUNS ? C::RUN : nkb;
      uint32_t it = 0, n = 0, sf = 0;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok; u += ustep) {
        for (int k0 = 0; k0 < nkb && ok; k0 += run, ++n) {
          const int slot = n & 1;
          // the epilogue has begun the tile before this one (and so finished the one before that, whose
          // columns this tile takes) and has read the columns that the two share
          if (n > 0 && !all_wait_or_abort(&bars->acc_next, (n - 1) & 1, abort_flag, status)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t d = tmem + slot * C::SLOT1;
          // BN = 64: every second tile takes the upper half of its scale tile's four columns
          const uint32_t sfb_off = C::BN == 64 ? 2 * (uint32_t)(unit_at<C::KEEP>(job, u).nt & 1) : 0u;
          for (int kb = k0; kb < min(nkb, k0 + run); ++kb, ++it) {
            const int st = it % C::NSTAGE;
            if (!all_wait_or_abort(&bars->full[st], (it / C::NSTAGE) & 1, abort_flag, status)) { ok = false; break; }
            const int ws = C::KEEP ? kb : st;
            if (C::KEEP && n == 0 && !all_wait_or_abort(&bars->wfull[ws], 0, abort_flag, status)) { ok = false; break; }
            ptx::tc_fence_after();
            const uint64_t soff = (uint64_t)((st * C::STAGE) >> 4), woff = (uint64_t)((ws * C::WPITCH) >> 4);
            const int steps = job.ksteps - 4 * kb < 4 ? job.ksteps - 4 * kb : 4;
#pragma unroll
            for (int a = 0; a < 2; ++a) {  // 128 values of K: scale tiles, then two MMAs
              if (2 * a >= steps) break;
              const uint32_t sfa = tmem + kSfCol + sf * (4 + 4 * C::NT), sfb = sfa + 4;
              sf = sf == 2 ? 0 : sf + 1;
              if (PAIR)
                ptx::tmem_cp_32x128b_pair_elect(sfa, dSA + soff + a * (512 >> 4));
              else
                ptx::tmem_cp_32x128b_elect(sfa, dSA + soff + a * (512 >> 4));
#pragma unroll
              for (int j = 0; j < C::NT; ++j) {
                const uint64_t from = dSB + woff + ((j * 1024 + a * 512) >> 4);
                if (PAIR)
                  ptx::tmem_cp_32x128b_pair_elect(sfb + j * 4, from);
                else
                  ptx::tmem_cp_32x128b_elect(sfb + j * 4, from);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int kk = 2 * a + k;
                if (kk >= steps) break;
                const uint32_t acc = (kb > k0 || kk > 0) ? 1u : 0u;
                if (PAIR)
                  ptx::mma_mxf4_ss_pair_elect(d, dA + soff + kk * 2, dB + woff + kk * 2, idesc_mxf4(C::BM, C::BN, k), sfa, sfb, acc);
                else
                  ptx::mma_mxf4_ss_elect(d, dA + soff + kk * 2, dB + woff + kk * 2, idesc_mxf4(C::BM, C::BN, k), sfa, sfb + sfb_off, acc);
              }
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
    constexpr int NCH = C::BN / CC;
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2;  // warps 2..5: even chunks, 6..9: odd ones
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    uint8_t* slab = stg + ew * C::SLABS * kSlab;
    const uint32_t slab_s = ptx::smem_u32(slab);
    float* bias_s = bars->bias[ew];
    const uint32_t next0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(&bars->acc_next), 0) : 0u;
    const int64_t pitch = (int64_t)job.nb * job.out;
    constexpr int MINE = (NCH + 1) / 2;  // chunks of a warp
    constexpr int NB = MINE * CC / 32;
    float next_bias[NB];
    auto fetch_bias = [&](int64_t u) {
      const Unit c = unit_at<C::KEEP>(job, u);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int ch = (32 * i / CC) * 2 + half, col = c.nt * C::BN + ch * CC + (32 * i) % CC + lane;
        next_bias[i] = u < u1 && ch < NCH && col < job.out ? mx4::load(bias + (int64_t)c.b * job.out + col) : 0.f;
      }
    };
    if (bias != nullptr) fetch_bias(u0);
    auto next = [&] {  // the MMAs may begin the next accumulator
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (first)
          ptx::mbar_arrive(&bars->acc_next);
        else
          ptx::mbar_arrive_cluster(next0);
      }
    };
    uint32_t n = 0, stored = 0;
    for (int64_t u = u0; u < u1; u += ustep, ++n) {
      const Unit c = unit_at<C::KEEP>(job, u);
      const int n0 = c.nt * C::BN;
      const int64_t m0 = (int64_t)c.mt * C::BM + (int64_t)rank * 128 + quad * 32;  // this warp's rows
      if (bias != nullptr) {
        __syncwarp();  // the previous tile's has been read
#pragma unroll
        for (int i = 0; i < NB; ++i) bias_s[32 * i + lane] = next_bias[i];
        __syncwarp();
        fetch_bias(u + ustep);  // asked for a tile ahead: the epilogue has no time to wait for it
      }
      if constexpr (C::RUNS) {
        constexpr int KEPT = MINE * CC;
        float kept[KEPT];
        bool ok = true;
#pragma unroll
        for (int e = 0; e < KEPT; ++e) kept[e] = 0.f;
        for (int left = nkb;; left -= C::RUN, ++n) {
          if (!(ok = all_wait_or_abort(&bars->acc_full[n & 1], (n >> 1) & 1, abort_flag, status))) break;
          ptx::tc_fence_after();
          const uint32_t at = tmem + lane_off + (n & 1) * C::SLOT1 + half * CC;
#pragma unroll
          for (int e = 0; e < KEPT; e += 16) {
            uint32_t t16[16];
            ptx::tmem_ld16(at + 2 * (e / CC) * CC + e % CC, t16);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              kept[e + k] += __uint_as_float(t16[k]);
              t16[k] = __float_as_uint(kept[e + k]);
            }
            if (left <= C::RUN) ptx::tmem_st16(at + 2 * (e / CC) * CC + e % CC, t16);  // for the stores below
          }
          if (left <= C::RUN) break;
          next();
        }
        if (!ok) break;
        ptx::tmem_wait_st();
      } else {
        if (!all_wait_or_abort(&bars->acc_full[n & 1], (n >> 1) & 1, abort_flag, status)) break;
        ptx::tc_fence_after();
      }
      const int slot = n & 1;
      const uint32_t tb = tmem + lane_off + slot * C::SLOT1;
#pragma unroll 1
      for (int i = 0; i < MINE; ++i) {
        // the first accumulator's shared columns are its last
        const int ch = (slot == 0 ? MINE - 1 - i : i) * 2 + half;
        const bool live = ch < NCH && n0 + ch * CC < job.out && m0 < job.rows;
        uint32_t v[CC];
        if (live) {
#pragma unroll
          for (int q = 0; q < CC / 16; ++q) {
            uint32_t t16[16];
            ptx::tmem_ld16(tb + ch * CC + q * 16, t16);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[q * 16 + e] = t16[e];
          }
          ptx::tmem_wait_ld();
        }
        if (i == 0) next();
        if (!live) continue;
        if (bias != nullptr) {
          const float* bs = bias_s + (ch >> 1) * CC;
#pragma unroll
          for (int e = 0; e < CC; e += 4) {
            const float4 f = *(const float4*)(bs + e);
            v[e] = __float_as_uint(__uint_as_float(v[e]) + f.x);
            v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) + f.y);
            v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) + f.z);
            v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) + f.w);
          }
        }
        const int sbuf = stored++ % C::SLABS;
        if (TMA_OUT && lane == 0) {  // what last left this slab has been read
          if (C::SLABS == 2)
            ptx::bulk_wait_read_allbut1();
          else
            ptx::bulk_wait_read_all();
        }
        __syncwarp();
        mx4::slab_write<T, CC>(slab_s + sbuf * kSlab, lane, v);
        if (TMA_OUT) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_3d(&tmY, slab + sbuf * kSlab, n0 + ch * CC, c.b, (int)m0);
            ptx::bulk_commit_group();
          }
        } else {
          // rows whose pitch is no multiple of 16 bytes
          __syncwarp();
          mx4::slab_store<T, CC>(slab + sbuf * kSlab, lane, Y + m0 * pitch + (int64_t)c.b * job.out + n0 + ch * CC, pitch,
                                 (int)min((int64_t)32, job.rows - m0), job.out - n0 - ch * CC);
        }
      }
    }
    if (TMA_OUT && lane == 0) ptx::bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync_all();  // neither CTA leaves while the pair's MMAs or its peer may use it
  ptx::tc_fence_after();
  if (warp == 1) {
    if (PAIR)
      ptx::tmem_dealloc_pair(tmem, 512);
    else
      ptx::tmem_dealloc(tmem, 512);
  }
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
            const cuuint32_t (&box)[3], CUtensorMapSwizzle swz, CUtensorMapL2promotion prom) {
  EncodeTiledFn enc = get_encode();
  cuuint32_t estr[3] = {1, 1, 1};
  return enc != nullptr && enc(m, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, prom,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// (bytes of a row, rows, blocks) of a code buffer, boxes of 128 bytes x box_rows.
bool code_map(CUtensorMap* m, const Mx4View& q, int box_rows) {
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, {(cuuint64_t)q.s.pitch(), (cuuint64_t)q.s.rows, (cuuint64_t)q.s.nblocks},
                {(cuuint64_t)q.s.pitch(), (cuuint64_t)q.s.pitch() * (cuuint64_t)q.s.rows}, {128, (cuuint32_t)box_rows, 1},
                CU_TENSOR_MAP_SWIZZLE_128B,
                q.s.pitch() % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE);
}
// (words of a scale tile, tiles along K, tiles along the rows of all blocks), boxes of 2 x n tiles.
bool scale_map(CUtensorMap* m, const Mx4View& q, int n) {
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, q.scales, {128, (cuuint64_t)q.s.katoms(), (cuuint64_t)(q.s.ratoms() * q.s.nblocks)},
                {512, (cuuint64_t)q.s.katoms() * 512}, {128, 2, (cuuint32_t)n}, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// (columns of a block, blocks, rows) of Y, boxes of 128 bytes x 32 rows, clipped to their block.
template <typename T>
bool out_map(CUtensorMap* m, void* Y, const Mx4Linear& d) {
  return encode(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, Y,
                {(cuuint64_t)d.out, (cuuint64_t)d.nb, (cuuint64_t)d.rows},
                {(cuuint64_t)d.out * sizeof(T), (cuuint64_t)d.out * d.nb * sizeof(T)}, {(cuuint32_t)(128 / sizeof(T)), 1, 32},
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

template <class C, typename T, bool TMA_OUT>
cudaError_t launch(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                   cudaStream_t st) {
  CUtensorMap mX, mW, mSX, mSW, mY;
  // Rows behind the last are dear to TMA (one row of 4096 -> 4096: 19.3 us with boxes of 128 rows, 8.6 with 8), and
  // what stands in their place may be anything: its results are not stored.  So a box ends with the tensor.
  const int x_rows = !C::PAIR && d.rows < 128 ? (int)((d.rows + 7) / 8 * 8) : 128;
  const int w_rows = !C::PAIR && d.out < C::BROWS ? (d.out + 7) / 8 * 8 : C::BROWS;
  if (!code_map(&mX, x, x_rows) || !code_map(&mW, w, w_rows) || !scale_map(&mSX, x, 1) || !scale_map(&mSW, w, C::NT))
    return cudaErrorInvalidValue;
  if (!TMA_OUT)
    mY = mX;  // unused
  else if (!out_map<T>(&mY, Y, d))
    return cudaErrorInvalidValue;
  Job j;
  j.nb = d.nb;
  j.mtiles = (int)((d.rows + C::BM - 1) / C::BM);
  j.ntiles = (d.out + C::BN - 1) / C::BN;
  j.units = (int64_t)j.nb * j.mtiles * j.ntiles;
  if (j.units > (int64_t(1) << 31)) return cudaErrorInvalidValue;
  j.rows = d.rows;
  j.out = d.out;
  j.ksteps = (x.s.kblocks() + 1) / 2;
  j.x_bytes = x_rows * 128;
  j.w_bytes = w_rows * 128;
  j.x_ratoms = x.s.ratoms();
  j.w_ratoms = w.s.ratoms();
  cudaError_t e = ensure_smem_attr((const void*)mx4_tc_kernel<C, T, TMA_OUT>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t slots = C::PAIR ? num_sms() / 2 : num_sms(), n = j.units < slots ? j.units : slots;
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
  e = cudaLaunchKernelEx(&cfg, mx4_tc_kernel<C, T, TMA_OUT>, mX, mW, mSX, mSW, mY, j, (const T*)bias, (T*)Y, status);
  if (e == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return e;
}

template <class C, typename T>
cudaError_t launch_out(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                       cudaStream_t st) {
  return (int64_t)d.out * sizeof(T) % 16 == 0 ? launch<C, T, true>(x, w, bias, d, Y, status, st)
                                              : launch<C, T, false>(x, w, bias, d, Y, status, st);
}

// Which kernel a product takes (a Mx4Path).
int choose(const Mx4Linear& d) {
  if (d.dtype == MONARCH_F32 && d.in > kRunFrom) return kMx4Runs;
  const int pitch = d.x().pitch();
  // The tile whose rounds over the SMs take the least time: a tile costs a stage's share of the way from
  // L2 for every 256 inputs, and its epilogue.  Microseconds from 8192 rows -> 4096 (256 x 256 pairs, 128 x 256
  // single, 128 x 256 with W kept): 19.8, 14.0 and 15.0 with 256 inputs, 22.5, 17.5 and 17.2 with 512, 26.9, 27.4 and
  // 24.9 with 1024; 62.7 and 66.7 with 4096, where W does not fit.  A pair's two CTAs wait for each other once a
  // tile, which only a long K hides; with W kept there is one tile of W a CTA, which costs rounds.  TMA takes rows
  // of codes whose pitch is no multiple of 32 bytes in smaller pieces (single and kept with 96 inputs 22.0 and 16.6).
  struct Tile {
    int bm, bn;
    double stage, fixed;
  };
  const Tile tiles[4] = {{256, 256, 0.46, 2.3}, {128, 256, 0.62, 1.3}, {128, 128, 0.42, 1.0}, {128, 64, 0.30, 0.8}};
  const double part = pitch % 32 != 0 ? 1.2 : pitch % 128 != 0 ? 0.33 : 0.0;  // for a short last stage
  const int stages = (d.in + 255) / 256;
  int best = 0;
  double least = 1e30;
  for (int i = 0; i < 4; ++i) {
    if (i < 3 && d.out <= tiles[i].bn / 2) continue;  // half of it or more would be empty
    const int64_t units = (d.rows + tiles[i].bm - 1) / tiles[i].bm * d.nb * ((d.out + tiles[i].bn - 1) / tiles[i].bn);
    const int64_t slots = i == 0 ? num_sms() / 2 : num_sms();
    const double t = (double)((units + slots - 1) / slots) * (stages * tiles[i].stage + tiles[i].fixed + part * tiles[i].bn / 256);
    if (t < least) {
      least = t;
      best = i;
    }
  }
  // W kept: where its tiles are full ones, so that no CTA has a lighter one than the others, and every 32-byte
  // sector of Y has one writer (the CTAs of a row are at different rows: sixteen 90 -> 250 blocks 82 us, 64 without)
  const int64_t wtiles = (int64_t)d.nb * ((d.out + 255) / 256), share = num_sms() / wtiles;
  if (stages <= 4 && share > 0 && d.out >= (d.out + 255) / 256 * 230 && (int64_t)d.out * (d.dtype == MONARCH_BF16 ? 2 : 4) % 32 == 0) {
    const int64_t mtiles = (d.rows + 127) / 128, rounds = (mtiles + share - 1) / share;
    if ((double)rounds * (stages * 0.33 + 1.6) + stages * 0.35 < least) return kMx4Kept;
  }
  const int path[4] = {kMx4Pair, kMx4Tile256, kMx4Tile128, kMx4Tile64};
  return path[best];
}

template <typename T>
cudaError_t launch_type(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                        cudaStream_t st) {
  switch (choose(d)) {
    case kMx4Pair: return launch_out<Cfg<256, true>, T>(x, w, bias, d, Y, status, st);
    case kMx4Tile256: return launch_out<Cfg<256, false>, T>(x, w, bias, d, Y, status, st);
    case kMx4Tile128: return launch_out<Cfg<128, false>, T>(x, w, bias, d, Y, status, st);
    case kMx4Kept: return launch<Cfg<256, false, true>, T, true>(x, w, bias, d, Y, status, st);
    case kMx4Runs:
      if constexpr (sizeof(T) == 4) return launch_out<Cfg<128, false, false, true>, T>(x, w, bias, d, Y, status, st);
    default: return launch_out<Cfg<64, false>, T>(x, w, bias, d, Y, status, st);
  }
}

}  // namespace

int mx4_tc_path(const Mx4Linear& d) { return choose(d); }

cudaError_t mx4_tc_fwd(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                       cudaStream_t st) {
  return d.dtype == MONARCH_BF16 ? launch_type<__nv_bfloat16>(x, w, bias, d, Y, status, st)
                                 : launch_type<float>(x, w, bias, d, Y, status, st);
}

}  // namespace monarch
