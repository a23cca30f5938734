// Block-diagonal product with both operands in MX4 on the block-scaled tensor cores (tcgen05
// kind::mxf4, E2M1 operands, one E8M0 scale per 32 values):
//
//   Y[r][b*out + o] = sum_i X^[b][r][i] W^[b][o][i] (+ bias)     128 x BN tiles, fp32 in TMEM.
//
// Products of two codes are exact and the hardware applies both scales to them before they join the
// fp32 sum, so the result is rounded once, in the epilogue.
//
// A stage of the ring holds 256 values of K: 128 rows of X codes and BN rows of W codes as 128-byte
// swizzled rows (one TMA box each) and their scale tiles (512 bytes for 128 rows x 128 values, one bulk
// copy per 128 rows: a quantised tensor keeps them in the order that tcgen05.cp wants).  The MMA warp
// copies a stage's scale tiles to TMEM and issues four MMAs of K = 64.  K beyond the tensor is filled
// with zero codes by TMA, the scale bytes behind the end are 0 (2^-127), and steps of K that lie wholly
// behind the end are not issued.
//
// TMEM (512 columns): two accumulators, so that the epilogue of one tile runs under the MMAs of the
// next.  With BN = 256 they overlap in 32 columns, [0, 256) and [224, 480): the epilogue reads the
// chunk with the shared columns first and then lets the next tile begin.  Scales take [480, 504).
// Roles: warp 0 TMA producer, warp 1 MMA issuer and TMEM owner, warps 2..5 epilogue (one TMEM lane
// quadrant each, one row per thread).
#include "mx4.cuh"
#include "tc_common.cuh"

namespace monarch {

namespace {

constexpr int kThreads = 192;
constexpr int kEpiWarps = 4;
constexpr uint32_t kSfCol = 480;
constexpr int kStagingChunk = 128 * 128;  // 128 rows x 128 bytes

struct Job {
  int nb, mtiles, ntiles;
  int64_t units;
  int64_t rows;
  int out;
  int ksteps;  // MMA steps of 64 values
  int katoms;  // scale tiles along K
  int64_t x_ratoms, w_ratoms;
};

template <int BN_>
struct Cfg {
  static constexpr int BN = BN_, BM = 128;
  static constexpr int NT = BN >= 128 ? BN / 128 : 1;  // scale tiles of W per 128 values of K
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SFA_BYTES = 1024, SFB_BYTES = 1024 * NT;
  static constexpr int STAGE = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int SLOT1 = BN == 256 ? 224 : BN;   // first column of the second accumulator
  static constexpr int NSTAGE_RAW = (kSmemBudget - 2 * kStagingChunk - 2048 - 1024) / STAGE;
  static constexpr int NSTAGE = NSTAGE_RAW > 8 ? 8 : NSTAGE_RAW;
  static constexpr int SMEM_BYTES = 2 * kStagingChunk + NSTAGE * STAGE + 2048 + 1024;
  static_assert(STAGE % 1024 == 0 && NSTAGE >= 2 && SLOT1 + BN <= 480, "layout");
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2];
  uint64_t acc_next;  // the next tile's accumulator may be written
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  float bias[256];
};
static_assert(sizeof(Bars) <= 2048, "bars");

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
__device__ __forceinline__ Unit unit_at(const Job& j, int64_t u) {
  Unit c;
  c.nt = (int)(u % j.ntiles);
  u /= j.ntiles;
  c.b = (int)(u % j.nb);
  c.mt = (int)(u / j.nb);
  return c;
}

template <class C, typename T, bool TMA_OUT>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Job job,
                  const uint8_t* __restrict__ x_scales, const uint8_t* __restrict__ w_scales, const T* bias, T* Y,
                  int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* stg = smem;
  uint8_t* ring = smem + 2 * kStagingChunk;
  Bars* bars = (Bars*)(ring + C::NSTAGE * C::STAGE);
  int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int nkb = (job.ksteps + 3) / 4;  // stages of a unit

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSTAGE; ++i) {
      ptx::mbar_init(&bars->full[i], 1);
      ptx::mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) ptx::mbar_init(&bars->acc_full[i], 1);
    ptx::mbar_init(&bars->acc_next, kEpiWarps);
    ptx::mbar_init(&bars->mma_done, 1);
    bars->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bars->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  ptx::griddep_wait();  // the operands may come from the previous kernel of the stream
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    // ================================================================ TMA producer
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmX);
      ptx::tma_prefetch_desc(&tmW);
      if (TMA_OUT) ptx::tma_prefetch_desc(&tmY);
      const uint64_t pol = ptx::policy_evict_normal();
      uint32_t it = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; u < job.units && ok; u += gridDim.x) {
        const Unit c = unit_at(job, u);
        const uint8_t* sx = x_scales + ((((int64_t)c.b * job.x_ratoms + c.mt) * job.katoms) << 9);
        const int64_t wt = (int64_t)c.nt * C::BN / 128;
        const uint8_t* sw = w_scales + ((((int64_t)c.b * job.w_ratoms + wt) * job.katoms) << 9);
        const int nw = (int)(job.w_ratoms - wt < C::NT ? job.w_ratoms - wt : C::NT);  // scale tiles in range
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int st = it % C::NSTAGE;
          if (!wait_or_abort(&bars->empty[st], ((it / C::NSTAGE) & 1) ^ 1, abort_flag, status)) { ok = false; break; }
          uint8_t* sa = ring + st * C::STAGE;
          uint8_t* sb = sa + C::A_BYTES;
          uint8_t* sfa = sb + C::B_BYTES;
          uint8_t* sfb = sfa + C::SFA_BYTES;
          const uint32_t sf = (uint32_t)(job.katoms - 2 * kb >= 2 ? 1024 : 512);
          ptx::mbar_arrive_expect_tx(&bars->full[st], C::A_BYTES + C::B_BYTES + sf * (1 + nw));
          ptx::tma_load_3d(sa, &tmX, &bars->full[st], kb * 128, c.mt * C::BM, c.b, pol);
          ptx::tma_load_3d(sb, &tmW, &bars->full[st], kb * 128, c.nt * C::BN, c.b, pol);
          ptx::bulk_load(sfa, sx + kb * 1024, sf, &bars->full[st]);
          for (int j = 0; j < nw; ++j)
            ptx::bulk_load(sfb + j * 1024, sw + (((int64_t)j * job.katoms) << 9) + kb * 1024, sf, &bars->full[st]);
        }
      }
      const uint32_t issued = it;
      for (uint32_t k = (issued > (uint32_t)C::NSTAGE ? issued - C::NSTAGE : 0); k < issued; ++k)
        ptx::mbar_wait_bounded(&bars->full[k % C::NSTAGE], (k / C::NSTAGE) & 1, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    const uint32_t ring_s = ptx::smem_u32(ring);
    const uint64_t dA = make_sdesc(ring_s, 1024, 2), dB = make_sdesc(ring_s + C::A_BYTES, 1024, 2);
    const uint64_t dSA = scale_desc(ring_s + C::A_BYTES + C::B_BYTES);
    const uint64_t dSB = scale_desc(ring_s + C::A_BYTES + C::B_BYTES + C::SFA_BYTES);
    const uint32_t sfa = tmem + kSfCol, sfb = sfa + 8;
    uint32_t it = 0, n = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < job.units && ok; u += gridDim.x, ++n) {
      const int slot = n & 1;
      // the epilogue has begun the tile before this one (and so finished the one before that, whose
      // columns this tile takes) and has read the columns that the two share
      if (n > 0 && !warp_wait_or_abort(lane, &bars->acc_next, (n - 1) & 1, abort_flag, status)) { ok = false; break; }
      ptx::tc_fence_after();
      const uint32_t d = tmem + slot * C::SLOT1;
      // BN = 64: every second tile takes the upper half of its scale tile's four columns
      const uint32_t sfb_u = C::BN == 64 ? sfb + 2 * (uint32_t)(unit_at(job, u).nt & 1) : sfb;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int st = it % C::NSTAGE;
        if (!warp_wait_or_abort(lane, &bars->full[st], (it / C::NSTAGE) & 1, abort_flag, status)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint64_t soff = (uint64_t)((st * C::STAGE) >> 4);
        const int steps = job.ksteps - 4 * kb < 4 ? job.ksteps - 4 * kb : 4;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          if (2 * a < steps) {
            ptx::tmem_cp_32x128b_elect(sfa + a * 4, dSA + soff + a * (512 >> 4));
#pragma unroll
            for (int j = 0; j < C::NT; ++j)
              ptx::tmem_cp_32x128b_elect(sfb + a * 4 * C::NT + j * 4, dSB + soff + (j * 1024 + a * 512 >> 4));
          }
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < steps)
            ptx::mma_mxf4_ss_elect(d, dA + soff + kk * 2, dB + soff + kk * 2, idesc_mxf4(C::BM, C::BN, kk & 1),
                                   sfa + (kk / 2) * 4, sfb_u + (kk / 2) * 4 * C::NT, (kb > 0 || kk > 0) ? 1u : 0u);
        ptx::mma_commit_elect(&bars->empty[st]);
      }
      if (!ok) break;
      ptx::mma_commit_elect(&bars->acc_full[slot]);
    }
    ptx::mma_commit_elect(&bars->mma_done);
    if (lane == 0) wait_mma_done(&bars->mma_done, abort_flag, status);
    __syncwarp();
  } else {
    // ================================================================ epilogue (4 warps)
    constexpr int CC = 128 / (int)sizeof(T);  // columns of a 128-byte chunk
    constexpr int NCH = C::BN / CC;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int et = threadIdx.x - 64;  // 0 .. 127
    const bool leader = et == 0;
    const uint32_t stg_s = ptx::smem_u32(stg);
    const int64_t pitch = (int64_t)job.nb * job.out;
    uint32_t n = 0, chunk_n = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < job.units && ok; u += gridDim.x, ++n) {
      const Unit c = unit_at(job, u);
      const int slot = n & 1;
      const int n0 = c.nt * C::BN;
      if (bias != nullptr) {
        ptx::named_bar_sync(1, kEpiWarps * 32);  // the previous tile's bias has been read
#pragma unroll
        for (int i = et; i < C::BN; i += kEpiWarps * 32)
          bars->bias[i] = n0 + i < job.out ? mx4::load(bias + (int64_t)c.b * job.out + n0 + i) : 0.f;
      }
      // one verdict for the four warps: none may leave while another waits for it at a barrier
      ok = ptx::named_bar_all(1, kEpiWarps * 32, wait_or_abort(&bars->acc_full[slot], (n >> 1) & 1, abort_flag, status));
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t tb = tmem + lane_off + slot * C::SLOT1;
      for (int i = 0; i < NCH; ++i) {
        // the first accumulator's shared columns are its last
        const int ch = (C::BN == 256 && slot == 0) ? NCH - 1 - i : i;
        uint32_t v[CC];
#pragma unroll
        for (int q = 0; q < CC / 16; ++q) {
          uint32_t t16[16];
          ptx::tmem_ld16(tb + ch * CC + q * 16, t16);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[q * 16 + e] = t16[e];
        }
        ptx::tmem_wait_ld();
        if (i == 0) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->acc_next);
        }
        if (n0 + ch * CC >= job.out) continue;  // behind the block's last output
        if (bias != nullptr) {
#pragma unroll
          for (int e = 0; e < CC; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + bars->bias[ch * CC + e]);
        }
        const int sbuf = chunk_n++ & 1;
        // what last left this staging buffer must have been read
        if (TMA_OUT && leader) ptx::bulk_wait_read_allbut1();
        ptx::named_bar_sync(2, kEpiWarps * 32);
        const uint32_t base = stg_s + sbuf * kStagingChunk + r * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t at = base + (((uint32_t)q ^ (uint32_t)(r & 7)) << 4);
          if (sizeof(T) == 2)
            ptx::st_shared_v4(at, ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 0) % CC]), __uint_as_float(v[(8 * q + 1) % CC])),
                              ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 2) % CC]), __uint_as_float(v[(8 * q + 3) % CC])),
                              ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 4) % CC]), __uint_as_float(v[(8 * q + 5) % CC])),
                              ptx::pack_bf16x2(__uint_as_float(v[(8 * q + 6) % CC]), __uint_as_float(v[(8 * q + 7) % CC])));
          else
            ptx::st_shared_v4(at, v[(4 * q) % CC], v[(4 * q + 1) % CC], v[(4 * q + 2) % CC], v[(4 * q + 3) % CC]);
        }
        if (TMA_OUT) {
          ptx::fence_proxy_async_smem();
          ptx::named_bar_sync(2, kEpiWarps * 32);
          if (leader) {
            ptx::tma_store_3d(&tmY, stg + sbuf * kStagingChunk, n0 + ch * CC, c.b, c.mt * C::BM);
            ptx::bulk_commit_group();
          }
        } else {
          // rows whose pitch is no multiple of 16 bytes: the warp writes its own 32 rows, lanes along
          // the columns
          __syncwarp();
          const int cols = job.out - n0 - ch * CC;
          for (int rr = 0; rr < 32; ++rr) {
            const int64_t row = (int64_t)c.mt * C::BM + quad * 32 + rr;
            if (row >= job.rows) break;
            const uint8_t* src = stg + sbuf * kStagingChunk + (quad * 32 + rr) * 128;
            T* dst = Y + row * pitch + (int64_t)c.b * job.out + n0 + ch * CC;
#pragma unroll
            for (int e = 0; e < CC / 32; ++e) {
              const int col = e * 32 + lane, byte = col * (int)sizeof(T);
              if (col < cols) dst[col] = *(const T*)(src + (((byte >> 4) ^ (rr & 7)) << 4) + (byte & 15));
            }
          }
        }
      }
    }
    if (TMA_OUT && leader) ptx::bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// (bytes of a row, rows, blocks) of a code buffer, boxes of 128 bytes x box_rows.
bool code_map(CUtensorMap* m, const Mx4View& q, int box_rows) {
  EncodeTiledFn enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)q.s.pitch(), (cuuint64_t)q.s.rows, (cuuint64_t)q.s.nblocks};
  cuuint64_t strides[2] = {(cuuint64_t)q.s.pitch(), (cuuint64_t)q.s.pitch() * (cuuint64_t)q.s.rows};
  cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(q.codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (columns of a block, blocks, rows) of Y, boxes of 128 bytes x 128 rows, clipped to their block.
template <typename T>
bool out_map(CUtensorMap* m, void* Y, const Mx4Linear& d) {
  EncodeTiledFn enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d.out, (cuuint64_t)d.nb, (cuuint64_t)d.rows};
  cuuint64_t strides[2] = {(cuuint64_t)d.out * sizeof(T), (cuuint64_t)d.out * d.nb * sizeof(T)};
  cuuint32_t box[3] = {(cuuint32_t)(128 / sizeof(T)), 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, Y, dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename T, bool TMA_OUT>
cudaError_t launch(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                   cudaStream_t st) {
  using C = Cfg<BN>;
  CUtensorMap mX, mW, mY;
  if (!code_map(&mX, x, C::BM) || !code_map(&mW, w, BN)) return cudaErrorInvalidValue;
  if (!TMA_OUT)
    mY = mX;  // unused
  else if (!out_map<T>(&mY, Y, d))
    return cudaErrorInvalidValue;
  Job j;
  j.nb = d.nb;
  j.mtiles = (int)x.s.ratoms();
  j.ntiles = (d.out + BN - 1) / BN;
  j.units = (int64_t)j.nb * j.mtiles * j.ntiles;
  j.rows = d.rows;
  j.out = d.out;
  j.ksteps = (x.s.kblocks() + 1) / 2;
  j.katoms = x.s.katoms();
  j.x_ratoms = x.s.ratoms();
  j.w_ratoms = w.s.ratoms();
  cudaError_t e = ensure_smem_attr((const void*)mx4_tc_kernel<C, T, TMA_OUT>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t grid = j.units < num_sms() ? j.units : num_sms();
  return launch_kernel(mx4_tc_kernel<C, T, TMA_OUT>, dim3((unsigned)grid), dim3(kThreads), C::SMEM_BYTES, st, true, mX, mW, mY,
                       j, x.scales, w.scales, (const T*)bias, (T*)Y, status);
}

template <int BN, typename T>
cudaError_t launch_out(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                       cudaStream_t st) {
  return (int64_t)d.out * sizeof(T) % 16 == 0 ? launch<BN, T, true>(x, w, bias, d, Y, status, st)
                                              : launch<BN, T, false>(x, w, bias, d, Y, status, st);
}

template <typename T>
cudaError_t launch_type(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                        cudaStream_t st) {
  // the widest tile that the outputs fill, halved while there are fewer tiles than SMs
  int bn = d.out > 128 ? 256 : d.out > 64 ? 128 : 64;
  while (bn > 64 && x.s.ratoms() * d.nb * ((d.out + bn - 1) / bn) < num_sms()) bn /= 2;
  switch (bn) {
    case 64: return launch_out<64, T>(x, w, bias, d, Y, status, st);
    case 128: return launch_out<128, T>(x, w, bias, d, Y, status, st);
    default: return launch_out<256, T>(x, w, bias, d, Y, status, st);
  }
}

}  // namespace

cudaError_t mx4_tc_fwd(const Mx4View& x, const Mx4View& w, const void* bias, const Mx4Linear& d, void* Y, int* status,
                       cudaStream_t st) {
  return d.dtype == MONARCH_BF16 ? launch_type<__nv_bfloat16>(x, w, bias, d, Y, status, st)
                                 : launch_type<float>(x, w, bias, d, Y, status, st);
}

}  // namespace monarch
