// fp4_gemm.cu -- products of microscaled 4-bit matrices on the block-scaled tensor cores.
//
//   out[m, n] = ga[m] gb[n] sum_k a[m, k] b[n, k]  (+ sum_j ext_b[j, n] ext_a[m, j])
//
// a: tokens, b: weight rows, both E2M1 codes with block scales along k; tcgen05.mma
// kind::mxf4nvf4 multiplies codes and scales and adds in fp32. The weight is the 128-lane
// operand, tokens are the columns of the accumulator.
#include <algorithm>

#include "fp4_device.cuh"

namespace qlora {
namespace {

constexpr int kStepCols = 256;   // K per pipeline step: one 128-byte swizzled row of codes
constexpr int kPRows = 128;      // weight rows per tile = TMEM lanes
constexpr uint32_t kPBytes = kPRows * 128;
constexpr uint32_t kSfTile = 512;

struct Fp4Args {
  const uint8_t* sp;   // scales of the weight side, tiled
  const uint8_t* sq;   // scales of the token side, tiled
  const float* gp;     // gscale of the weight side or NULL, one or per row
  const float* gq;
  int gp_rows, gq_rows;  // per-row gscale
  int64_t P, Q;          // weight rows, tokens
  int64_t K;
  int ktiles;            // scale tiles along a row
  int steps;             // pipeline steps over K
  int p_tiles;           // tiles along the weight rows
  int ext_mmas;          // 16-wide MMAs per extension step (0: none)
  bool ext_mn;           // the extension's weight-side operand is MN-major
  void* out;             // [Q, ld]
  int64_t ld;
  bool out_f32;
  int* err;
};

// ------------------------------------------------------------------ split kernel
// One tile of 128 weight rows x NT tokens per CTA; the `cs` CTAs of a cluster take parts of K
// and add their accumulators through distributed shared memory in rank order.
// Warp 0: TMA, warp 1: MMA and TMEM, warps 2-5: epilogue.
constexpr int kSplitThreads = 192;
constexpr int split_nq(int nt) { return (nt + 127) / 128; }  // scale row tiles of the tokens
constexpr int split_stages(int nt) { return nt <= 64 ? 4 : nt <= 128 ? 5 : 4; }
constexpr uint32_t split_stage_bytes(int nt) { return kPBytes + nt * 128; }
constexpr uint32_t split_sf_bytes(int nt) { return 4 * kSfTile * (1 + split_nq(nt)); }
constexpr uint32_t split_smem(int nt) {
  return 1024 + split_stages(nt) * (split_stage_bytes(nt) + split_sf_bytes(nt)) + 256;
}
constexpr uint32_t split_set_cols(int nt) { return 16 + 16 * split_nq(nt); }
constexpr uint32_t split_tmem(int nt) {
  return nt + 2 * split_set_cols(nt) <= 128 ? 128 : nt + 2 * split_set_cols(nt) <= 256 ? 256 : 512;
}

template <Fp4 F, int NT>
__global__ void __launch_bounds__(kSplitThreads, 1)
    k_fp4_gemm_split(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_ext_p,
                     const __grid_constant__ CUtensorMap tm_ext_q, const Fp4Args args, const int cs) {
  constexpr int S = split_stages(NT);
  constexpr int NQ = split_nq(NT);
  constexpr uint32_t kQBytes = NT * 128;
  constexpr int kTileStep = kStepCols / kFp4TileCols<F>;  // scale tiles per step: 2 or 4
  constexpr int kMmaTile = 4 / kTileStep;                 // MMAs per scale tile: 2 or 1
  constexpr uint32_t kSet = split_set_cols(NT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* p_s = smem;                         // [S][kPBytes]
  uint8_t* q_s = p_s + S * kPBytes;            // [S][kQBytes]
  uint8_t* sfp_s = q_s + S * kQBytes;          // [S][4][512]
  uint8_t* sfq_s = sfp_s + S * 4 * kSfTile;    // [S][NQ][4][512]
  uint64_t* full = reinterpret_cast<uint64_t*>(sfq_s + S * NQ * 4 * kSfTile);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / cs;
  const int64_t p0 = static_cast<int64_t>(tile % args.p_tiles) * kPRows;
  const int64_t q0 = static_cast<int64_t>(tile / args.p_tiles) * NT;
  const int s_begin = static_cast<int>(static_cast<int64_t>(args.steps) * rank / cs);
  const int s_end = static_cast<int>(static_cast<int64_t>(args.steps) * (rank + 1) / cs);
  const int nmain = s_end - s_begin;
  const int nsteps = nmain + (rank == 0 && args.ext_mmas > 0 ? 2 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, split_tmem(NT));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  griddep_wait_and_release();

  if (warp == 0) {
    if (elect_one()) {
      int issued = 0;
      const int64_t prow_tile = p0 / 128, qrow_tile = q0 / 128;
      const int nq = (NQ == 2 && args.Q - q0 > 128) ? 2 : 1;  // token scale tiles that exist
      for (int i = 0; i < nsteps; ++i) {
        const int s = i % S;
        if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1u, abort_flag)) {
          record_error(args.err, abort_flag, kErrTimeoutProducer);
          break;
        }
        if (i < nmain) {
          const int step = s_begin + i;
          const int t0 = step * kTileStep;
          const uint32_t sf = static_cast<uint32_t>(min(kTileStep, args.ktiles - t0)) * kSfTile;
          mbar_arrive_expect_tx(&full[s], kPBytes + kQBytes + sf * (1 + nq));
          tma_load_2d(p_s + s * kPBytes, &tm_p, &full[s], step * 128, static_cast<int>(p0));
          tma_load_2d(q_s + s * kQBytes, &tm_q, &full[s], step * 128, static_cast<int>(q0));
          bulk_load(sfp_s + s * 4 * kSfTile, args.sp + (prow_tile * args.ktiles + t0) * kSfTile, sf,
                    &full[s]);
          for (int h = 0; h < nq; ++h)
            bulk_load(sfq_s + (s * NQ + h) * 4 * kSfTile,
                      args.sq + ((qrow_tile + h) * args.ktiles + t0) * kSfTile, sf, &full[s]);
        } else {
          // bf16 extension: hi part, then lo part of the token operand; columns past r are 0
          mbar_arrive_expect_tx(&full[s], kPBytes + kQBytes);
          if (args.ext_mn) {
            tma_load_2d(p_s + s * kPBytes, &tm_ext_p, &full[s], static_cast<int>(p0), 0);
            tma_load_2d(p_s + s * kPBytes + 8192, &tm_ext_p, &full[s], static_cast<int>(p0) + 64, 0);
          } else {
            tma_load_2d(p_s + s * kPBytes, &tm_ext_p, &full[s], 0, static_cast<int>(p0));
          }
          tma_load_2d(q_s + s * kQBytes, &tm_ext_q, &full[s], (i - nmain) * 64, static_cast<int>(q0));
        }
        ++issued;
      }
      if (*abort_flag)
        for (int i = max(0, issued - S); i < issued; ++i)
          mbar_wait_drain(&full[i % S], (i / S) & 1u);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc_ext = idesc_bf16_f32(kPRows, NT, args.ext_mn, false);
      bool ok = true;
      int done = 0;
      for (int i = 0; i < nsteps && ok; ++i) {
        const int s = i % S;
        ok = mbar_wait(&full[s], (i / S) & 1u, abort_flag);
        // The scale columns of step i were last read by the MMAs of step i - 2 (two sets, used
        // in turn), and MMAs of different kinds are not ordered with each other: wait for the
        // completion of step i - 2, and for step i - 1 where the kind changes.
        if (ok && i < nmain && i >= 2)
          ok = mbar_wait(&empty[(i - 2) % S], ((i - 2) / S) & 1u, abort_flag);
        if (ok && i == nmain && i >= 1)
          ok = mbar_wait(&empty[(i - 1) % S], ((i - 1) / S) & 1u, abort_flag);
        if (!ok) {
          record_error(args.err, abort_flag, kErrTimeoutMma);
          break;
        }
        tc_fence_after();
        const uint32_t pa = smem_u32(p_s + s * kPBytes), qa = smem_u32(q_s + s * kQBytes);
        const uint64_t dq = smem_desc_sw128(qa, 16, 1024);
        if (i < nmain) {
          const uint64_t dp = smem_desc_sw128(pa, 16, 1024);
          const uint32_t sfp = tmem_d + NT + (i & 1) * kSet, sfq = sfp + 16;
          const int64_t left = args.K - static_cast<int64_t>(s_begin + i) * kStepCols;
          const int mmas = left >= kStepCols ? 4 : static_cast<int>((left + 63) / 64);
          for (int kk = 0; kk < mmas; ++kk) {
            const int t = kk / kMmaTile, sub = kk % kMmaTile;
            if (sub == 0) {
              tmem_cp_scales(sfp + t * 4, smem_desc_scales(smem_u32(sfp_s + (s * 4 + t) * kSfTile)));
              for (int h = 0; h < NQ; ++h)
                tmem_cp_scales(sfq + (t * NQ + h) * 4,
                               smem_desc_scales(smem_u32(sfq_s + ((s * NQ + h) * 4 + t) * kSfTile)));
            }
            umma_fp4<F == Fp4::kMx ? 2 : 4>(
                tmem_d, dp + kk * 2u, dq + kk * 2u,
                idesc_fp4(kPRows, NT, F == Fp4::kMx, F == Fp4::kMx ? 2 * sub : 0), sfp + t * 4,
                sfq + t * NQ * 4, (i | kk) != 0);
          }
        } else {
          const uint64_t dp = args.ext_mn ? smem_desc_sw128(pa, 8192, 1024) : smem_desc_sw128(pa, 16, 1024);
          const uint32_t adv = args.ext_mn ? 128u : 2u;
          for (int kk = 0; kk < args.ext_mmas; ++kk)
            umma_bf16(tmem_d, dp + kk * adv, dq + kk * 2u, idesc_ext, (i | kk) != 0);
        }
        umma_commit(&empty[s]);
        ++done;
      }
      umma_commit(acc_full);
      mbar_wait_drain(acc_full, 0);
      uint32_t par;
      for (int s = 0; s < S; ++s)
        if (last_use(done, S, s, par)) mbar_wait_drain(&empty[s], par);
    }
  } else {
    const bool got = mbar_wait(acc_full, 0, abort_flag) && !*abort_flag;
    if (!got && !*abort_flag) record_error(args.err, abort_flag, kErrTimeoutEpilogue);
    tc_fence_after();
    const int quarter = warp & 3;
    const int64_t p = p0 + quarter * 32 + lane;
    const uint32_t taddr = tmem_d + (static_cast<uint32_t>(quarter * 32) << 16);
    float* part = reinterpret_cast<float*>(smem);  // [NT][128], over the consumed stages
    const float gp = args.gp ? args.gp[args.gp_rows ? min(p, args.P - 1) : 0] : 1.f;
    // value of (p, token q) -> output
    auto store_pair = [&](int64_t q, float v0, float v1) {  // tokens q and q + 1
      v0 *= gp;
      v1 *= gp;
      if (args.gq) {
        v0 *= args.gq[args.gq_rows ? min(q, args.Q - 1) : 0];
        v1 *= args.gq[args.gq_rows ? min(q + 1, args.Q - 1) : 0];
      }
      if (args.out_f32) {
        float* o = static_cast<float*>(args.out) + q * args.ld + p;
        if (p < args.P && q < args.Q) o[0] = v0;
        if (p < args.P && q + 1 < args.Q) o[args.ld] = v1;
      } else {
        // even lanes write rows p, p + 1 of token q, odd lanes rows p - 1, p of token q + 1
        const float got = __shfl_xor_sync(~0u, (lane & 1) ? v0 : v1, 1);
        const int64_t tq = q + (lane & 1), tp = p & ~int64_t{1};
        const uint32_t w = (lane & 1) ? pack_bf16x2_rn(got, v1) : pack_bf16x2_rn(v0, got);
        if (tp < args.P && tq < args.Q)
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.out) + tq * args.ld + tp) = w;
      }
    };
    if (got) {
#pragma unroll 1
      for (int c = 0; c < NT / 32; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_ld_wait();
        if (cs > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) part[(c * 32 + j) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]);
        } else if (q0 + c * 32 < args.Q) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            store_pair(q0 + c * 32 + j, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        }
      }
    }
    if (cs > 1) {
      cluster_sync_all();
      // rank r sums and writes tokens [r, r + 1) NT / cs of the tile
      const int span = NT / cs;
      const int t0 = rank * span;
      for (int t = t0; t < t0 + span; t += 2) {
        if (q0 + t >= args.Q) break;
        float v0 = 0.f, v1 = 0.f;
        for (int r = 0; r < cs; ++r) {
          v0 += ld_cluster_f32(part + t * 128 + quarter * 32 + lane, r);
          v1 += ld_cluster_f32(part + (t + 1) * 128 + quarter * 32 + lane, r);
        }
        if (!*abort_flag) store_pair(q0 + t, v0, v1);
      }
    }
  }
  if (cs > 1) {
    __syncwarp();
    if (warp < 2) cluster_sync_all();  // the epilogue warps' first barrier
    cluster_sync_all();                // no CTA leaves while its sums are being read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_d, split_tmem(NT));
  }
}

// ------------------------------------------------------------------ pair kernel
// A persistent CTA pair per two SMs; a tile is 256 weight rows x 256 tokens. Each CTA holds 128
// weight rows of the operand, 128 tokens of the other, its rows' scales and all 256 tokens'
// scales, and accumulates its 128 rows x 256 tokens in its own tensor memory.
//
// Tensor memory: two 256-column accumulators used in turn and two sets of scale columns. They
// do not fit side by side (2 * 256 + 2 * 48 > 512), so the accumulators share the columns
// [160, 256): the epilogue reads those first and then lets the next tile's MMAs start, while
// it goes on with the other 160 columns.
//
// Warp 0: TMA, warp 1: MMA (in the leader) and tensor memory, warps 2-9: epilogue, two warps
// for each quarter of the lanes.
constexpr int kPairThreads = 320;
constexpr int kPairStages = 5;
constexpr int kPairTile = 256;                // weight rows and tokens of a tile
constexpr uint32_t kPairQBytes = 128 * 128;
constexpr uint32_t kPairSf = 4 * kSfTile;     // scales of 128 rows and one step (NVFP4)
constexpr uint32_t kPairStage = kPBytes + kPairQBytes + 3 * kPairSf;
constexpr uint32_t kPairEpi = 8 * 2 * 32 * 32 * 2;
constexpr uint32_t kPairSmem = 1024 + kPairStages * kPairStage + kPairEpi + 256;
static_assert(kPairSmem <= 227 * 1024, "shared memory per CTA");
constexpr uint32_t kAcc1 = 160;               // first column of the second accumulator
constexpr uint32_t kSfCol = 416;              // first scale column; sets of 48
constexpr int kEpiWarps = 8;

struct PairTile {
  int64_t p0, q0;
};
// Tiles in groups of eight token tiles, so that the tiles in flight at one time form a block
// that shares operands in L2.
__device__ __forceinline__ PairTile pair_tile(int t, int p_tiles, int q_tiles) {
  constexpr int kGroup = 8;
  const int per = kGroup * p_tiles;
  const int g = t / per, in = t - g * per;
  const int width = min(kGroup, q_tiles - g * kGroup);
  return {static_cast<int64_t>(in / width) * kPairTile,
          static_cast<int64_t>(g * kGroup + in % width) * kPairTile};
}

template <Fp4 F, bool OUT_F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_fp4_gemm_pair(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_sp, const __grid_constant__ CUtensorMap tm_sq,
                    const __grid_constant__ CUtensorMap tm_ext_p,
                    const __grid_constant__ CUtensorMap tm_ext_q,
                    const __grid_constant__ CUtensorMap tm_out, const Fp4Args args) {
  constexpr int S = kPairStages;
  constexpr int kTileStep = kStepCols / kFp4TileCols<F>;  // scale tiles per step: 2 or 4
  constexpr int kMmaTile = 4 / kTileStep;                 // MMAs per scale tile: 2 or 1
  constexpr uint32_t kSfBytes = kTileStep * kSfTile;      // of 128 rows and one step
  constexpr uint32_t kStepTx = 2 * (kPBytes + kPairQBytes + 3 * kSfBytes);  // both CTAs
  constexpr uint32_t kExtTx = 2 * (kPBytes + kPairQBytes);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* p_s = smem;                          // [S][kPBytes]
  uint8_t* q_s = p_s + S * kPBytes;             // [S][kPairQBytes]
  uint8_t* epi_s = q_s + S * kPairQBytes;       // [8 warps][2][32][32] bf16
  uint8_t* sfp_s = epi_s + kPairEpi;            // [S][kPairSf]
  uint8_t* sfq_s = sfp_s + S * kPairSf;         // [S][2 kPairSf]: two row tiles, kSfBytes each
  uint64_t* full = reinterpret_cast<uint64_t*>(sfq_s + S * 2 * kPairSf);  // the leader's counts
  uint64_t* empty = full + S;                   // [S] MMAs reading the slot done (both CTAs)
  uint64_t* acc_full = empty + S;               // accumulator complete (both CTAs)
  uint64_t* acc_part = acc_full + 1;            // shared columns read out (the leader's counts)
  uint64_t* mma_drain = acc_part + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int q_tiles = static_cast<int>((args.Q + kPairTile - 1) / kPairTile);
  const int tiles = args.p_tiles * q_tiles;
  const int clusters = gridDim.x / 2, first = blockIdx.x / 2;
  const int my_tiles = first < tiles ? (tiles - 1 - first) / clusters + 1 : 0;
  const int ext = args.ext_mmas > 0 ? 2 : 0;  // extension steps, ahead of a tile's others
  const int total = args.steps + ext;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_part, 2 * kEpiWarps);
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait_and_release();

  if (warp == 0) {
    // ------------------------------------------------ TMA: this CTA's share of every step
    if (elect_one()) {
      int n = 0;  // steps issued
      bool ok = true;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const PairTile t = pair_tile(first + i * clusters, args.p_tiles, q_tiles);
        const int p0 = static_cast<int>(t.p0) + 128 * rank, q0 = static_cast<int>(t.q0) + 128 * rank;
        for (int k = 0; k < total; ++k, ++n) {
          const int s = n % S;
          if (n >= S && !mbar_wait(&empty[s], ((n / S) - 1) & 1u, abort_flag)) {
            record_error(args.err, abort_flag, kErrTimeoutProducer);
            ok = false;
            break;
          }
          const uint32_t bar = cluster_addr(&full[s], 0);
          uint8_t *ps = p_s + s * kPBytes, *qs = q_s + s * kPairQBytes;
          if (k < ext) {  // bf16: hi part, then lo part of the token operand
            if (rank == 0) mbar_arrive_expect_tx(&full[s], kExtTx);
            if (args.ext_mn) {
              tma_load_2d_pair(ps, &tm_ext_p, bar, p0, 0);
              tma_load_2d_pair(ps + 8192, &tm_ext_p, bar, p0 + 64, 0);
            } else {
              tma_load_2d_pair(ps, &tm_ext_p, bar, 0, p0);
            }
            tma_load_2d_pair(qs, &tm_ext_q, bar, k * 64, q0);
          } else {
            const int step = k - ext;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], kStepTx);
            tma_load_2d_pair(ps, &tm_p, bar, step * 128, p0);
            tma_load_2d_pair(qs, &tm_q, bar, step * 128, q0);
            const int x = step * kTileStep * 64;  // in 8-byte elements
            tma_load_2d_pair(sfp_s + s * kPairSf, &tm_sp, bar, x, p0 / 128);
            tma_load_2d_pair(sfq_s + s * 2 * kPairSf, &tm_sq, bar, x, static_cast<int>(t.q0 / 128));
          }
        }
      }
      // after an abort, the leader lets the copies in flight (both CTAs') land
      if (*abort_flag && rank == 0)
        for (int j = max(0, n - S); j < n; ++j) mbar_wait_drain(&full[j % S], (j / S) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one()) {
      const uint32_t idesc_ext = idesc_bf16_f32(kPairTile, kPairTile, args.ext_mn, false);
      const uint32_t ext_adv = args.ext_mn ? 128u : 2u;
      int n = 0;
      bool ok = true;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const uint32_t d = tmem + (i & 1) * kAcc1;
        // The epilogue has the shared columns of tile i - 1 in registers (and, having begun
        // that tile, all of tile i - 2, which used this accumulator).
        if (i >= 1) ok = mbar_wait_cluster(acc_part, (i - 1) & 1u, abort_flag);
        tc_fence_after();
        for (int k = 0; k < total && ok; ++k) {
          const int s = n % S;
          ok = mbar_wait(&full[s], (n / S) & 1u, abort_flag);
          // The scale columns of this step were last read by the MMAs two steps ago (two sets,
          // used in turn), and MMAs of different kinds are not ordered with each other: wait
          // for the completion of step n - 2, or of n - 1 where the kind changes. (At the
          // start of a tile everything before it is complete: its epilogue has begun.)
          if (ok && k == ext && ext)
            ok = mbar_wait(&empty[(n - 1) % S], ((n - 1) / S) & 1u, abort_flag);
          else if (ok && k >= ext + 2)
            ok = mbar_wait(&empty[(n - 2) % S], ((n - 2) / S) & 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t pa = smem_u32(p_s + s * kPBytes);
          const uint64_t dq = smem_desc_sw128(smem_u32(q_s + s * kPairQBytes), 16, 1024);
          if (k < ext) {
            const uint64_t dp = args.ext_mn ? smem_desc_sw128(pa, 8192, 1024) : smem_desc_sw128(pa, 16, 1024);
            for (int kk = 0; kk < args.ext_mmas; ++kk)
              umma_bf16_pair(d, dp + kk * ext_adv, dq + kk * 2u, idesc_ext, (k | kk) != 0);
          } else {
            const uint64_t dp = smem_desc_sw128(pa, 16, 1024);
            const uint32_t sfp = tmem + kSfCol + (n & 1) * 48, sfq = sfp + 16;
            const uint32_t sp = smem_u32(sfp_s + s * kPairSf), sq = smem_u32(sfq_s + s * 2 * kPairSf);
            const int64_t left = args.K - static_cast<int64_t>(k - ext) * kStepCols;
            const int mmas = left >= kStepCols ? 4 : static_cast<int>((left + 63) / 64);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk >= mmas) break;
              const int tl = kk / kMmaTile, sub = kk % kMmaTile;
              if (sub == 0) {
                tmem_cp_scales_pair(sfp + tl * 4, smem_desc_scales(sp + tl * kSfTile));
                tmem_cp_scales_pair(sfq + tl * 8, smem_desc_scales(sq + tl * kSfTile));
                tmem_cp_scales_pair(sfq + tl * 8 + 4, smem_desc_scales(sq + kSfBytes + tl * kSfTile));
              }
              umma_fp4_pair<F == Fp4::kMx ? 2 : 4>(
                  d, dp + kk * 2u, dq + kk * 2u,
                  idesc_fp4(kPairTile, kPairTile, F == Fp4::kMx, F == Fp4::kMx ? 2 * sub : 0),
                  sfp + tl * 4, sfq + tl * 8, (k | kk) != 0);
            }
          }
          umma_commit_pair(&empty[s]);
          if (k == total - 1) umma_commit_pair(acc_full);
          ++n;
        }
      }
      if (!ok) record_error(args.err, abort_flag, kErrTimeoutMma);
      umma_commit_pair(mma_drain);
    }
  } else {
    // ------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stage2 = epi_s + (warp - 2) * (2 * 32 * 32 * 2);
    const uint32_t part_bar = cluster_addr(acc_part, 0);
    if (lane == 0) tma_prefetch_desc(&tm_out);
    int chunks = 0;  // stage buffers used
    for (int i = 0; i < my_tiles; ++i) {
      const PairTile t = pair_tile(first + i * clusters, args.p_tiles, q_tiles);
      const int64_t p0 = t.p0 + 128 * rank + quarter * 32;
      // this warp's four 32-token chunks: the shared columns first. Accumulator 0 shares its
      // chunks 5-7, accumulator 1 its chunks 0-2.
      const int shared0 = (i & 1) ? 0 : 5, own0 = (i & 1) ? 3 : 0;
      const int c0 = shared0 + 2 * half, c1 = half ? own0 + 2 : shared0 + 1;
      const int c2 = own0 + (half ? 3 : 0), c3 = own0 + (half ? 4 : 1);
      const int cs[4] = {c0, c1, c2, c3};
      float gq[4], gp[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gq[j] = 1.f;
        gp[j] = 1.f;
        if (args.gq) gq[j] = __ldg(args.gq + (args.gq_rows ? min(t.q0 + cs[j] * 32 + lane, args.Q - 1) : 0));
        // rows lane / 4 + 8 j of the quarter (bf16 output), row lane (fp32 output, j = 0)
        const int64_t row = p0 + (OUT_F32 ? lane : (lane >> 2) + 8 * j);
        if (args.gp) gp[j] = __ldg(args.gp + (args.gp_rows ? min(row, args.P - 1) : 0));
      }
      if (!mbar_wait(acc_full, i & 1u, abort_flag)) {
        if (!*abort_flag) record_error(args.err, abort_flag, kErrTimeoutEpilogue);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + (i & 1) * kAcc1 + (static_cast<uint32_t>(quarter * 32) << 16);
      // tensor memory -> registers: 32 rows x 32 tokens
      auto fetch = [&](int c, uint32_t (&v)[32]) {
        if constexpr (OUT_F32) {
          tmem_ld_32x32b_x32(taddr + c * 32, v);
        } else {
          uint32_t lo[16], hi[16];
          tmem_ld_16x256b_x4(taddr + c * 32, lo);
          tmem_ld_16x256b_x4(taddr + (16u << 16) + c * 32, hi);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = lo[j], v[16 + j] = hi[j];
        }
      };
      auto emit = [&](int j, const uint32_t (&v)[32]) {
        const int64_t q = t.q0 + cs[j] * 32;
        if (q >= args.Q) return;
        if constexpr (OUT_F32) {
          // the chunk fills both stage buffers: stage[token][row]
          const uint32_t st = smem_u32(stage2);
          if (chunks >= 1 && elect_one()) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float x = __uint_as_float(v[k]) * gp[0];
            if (args.gq) x *= __shfl_sync(~0u, gq[j], k);
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + k * 128 + lane * 4), "f"(x) : "memory");
          }
        } else {
          // bf16 pairs of adjacent tokens, transposed by stmatrix into stage[token][row]: a
          // token's 64 bytes are four 16-byte groups, group g at slot g ^ ((token >> 1) & 3),
          // the 64-byte swizzle of the tile store
          const uint32_t st = smem_u32(stage2) + (chunks & 1) * 2048;
          if (chunks >= 2 && elect_one()) bulk_wait_group_read<1>();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // tokens 8k..8k+7 of the chunk
            float g0 = 1.f, g1 = 1.f;
            if (args.gq) {
              g0 = __shfl_sync(~0u, gq[j], 8 * k + 2 * (lane & 3));
              g1 = __shfl_sync(~0u, gq[j], 8 * k + 2 * (lane & 3) + 1);
            }
            uint32_t w[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {  // rows lane / 4 + 8m
              const int at = (m >> 1) * 16 + 4 * k + (m & 1) * 2;
              w[m] = pack_bf16x2_rn(__uint_as_float(v[at]) * gp[m] * g0,
                                    __uint_as_float(v[at + 1]) * gp[m] * g1);
            }
            const int tok = 8 * k + (lane & 7);
            stmatrix_x4_trans(st + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (p0 < args.P && elect_one()) {
          tma_store_2d(&tm_out, OUT_F32 ? stage2 : stage2 + (chunks & 1) * 2048, static_cast<int>(p0),
                       static_cast<int>(q));
          bulk_commit_group();
        }
        ++chunks;
      };
      uint32_t v0[32], v1[32];
      fetch(c0, v0);
      if (half == 0) fetch(c1, v1);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(part_bar);
      emit(0, v0);
      if (half != 0) {
        fetch(c1, v1);
        tmem_ld_wait();
      }
      emit(1, v1);
      fetch(c2, v0);
      tmem_ld_wait();
      emit(2, v0);
      fetch(c3, v1);
      tmem_ld_wait();
      emit(3, v1);
    }
    if (elect_one()) bulk_wait_group_all();  // tile stores done before the CTA exits
  }
  // The MMAs are complete and the arrivals of the last commits have landed, in each CTA, before
  // tensor memory and the barriers go.
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_wait_drain(mma_drain, 0);
    uint32_t par;
    for (int s = 0; s < S && !*abort_flag; ++s)
      if (last_use(my_tiles * total, S, s, par)) mbar_wait_drain(&empty[s], par);
  }
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  cluster_sync_all();
}

// ------------------------------------------------------------------ host side
constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapDataType kBf16Map = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;

// The extension's operand maps (boxes of 128 weight rows, q_box tokens); tp and tq stand in
// when there is none.
qlora_status ext_maps(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                      uint32_t q_box, CUtensorMap* xp, CUtensorMap* xq) {
  if (!ext) return QLORA_OK;
  if (ext->mn_major) QL_MAP(xp, kBf16Map, ext->p, b.rows, ext->r, b.rows * 2, 64, 64, kSw128);
  else QL_MAP(xp, kBf16Map, ext->p, ext->r, b.rows, ext->r * 2, 64, kPRows, kSw128);
  QL_MAP(xq, kBf16Map, ext->q, 128, a.rows, 256, 64, q_box, kSw128);
  return QLORA_OK;
}

template <Fp4 F, int NT>
qlora_status run_split(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                       Fp4Args args, int cs, cudaStream_t st) {
  CUtensorMap tp, tq, xp, xq;
  QL_MAP(&tp, kU8, b.codes, b.cols / 2, b.rows, b.cols / 2, 128, kPRows, kSw128);
  QL_MAP(&tq, kU8, a.codes, a.cols / 2, a.rows, a.cols / 2, 128, NT, kSw128);
  xp = tp;
  xq = tq;
  qlora_status q = ext_maps(a, b, ext, NT, &xp, &xq);
  if (q != QLORA_OK) return q;
  auto kern = k_fp4_gemm_split<F, NT>;
  constexpr uint32_t smem = split_smem(NT);
  QL_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * ((a.rows + NT - 1) / NT);
  if (tiles * cs > (int64_t{1} << 30)) {
    set_last_error("the product has too many tiles");
    return QLORA_ERR_SHAPE;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cs));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  note_launches(1);
  QL_TRY(cudaLaunchKernelEx(&cfg, kern, tp, tq, xp, xq, args, cs));
  return QLORA_OK;
}

template <Fp4 F>
qlora_status run_pair(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                      Fp4Args args, cudaStream_t st) {
  CUtensorMap tp, tq, sp, sq, xp, xq, to;
  QL_MAP(&tp, kU8, b.codes, b.cols / 2, b.rows, b.cols / 2, 128, kPRows, kSw128);
  QL_MAP(&tq, kU8, a.codes, a.cols / 2, a.rows, a.cols / 2, 128, 128, kSw128);
  // scale tiles as rows of 8-byte elements: 64 per tile
  constexpr uint32_t box = kStepCols / kFp4TileCols<F> * 64;
  constexpr CUtensorMapDataType kU64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
  const uint64_t srow = static_cast<uint64_t>(args.ktiles) * 512;
  QL_MAP(&sp, kU64, b.scales, srow / 8, (b.rows + 127) / 128, srow, box, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  QL_MAP(&sq, kU64, a.scales, srow / 8, (a.rows + 127) / 128, srow, box, 2, CU_TENSOR_MAP_SWIZZLE_NONE);
  xp = tp;
  xq = tq;
  qlora_status q = ext_maps(a, b, ext, 128, &xp, &xq);
  if (q != QLORA_OK) return q;
  if (args.out_f32)
    QL_MAP(&to, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, args.out, b.rows, a.rows, b.rows * 4, 32, 32,
           CU_TENSOR_MAP_SWIZZLE_NONE);
  else
    QL_MAP(&to, kBf16Map, args.out, b.rows, a.rows, b.rows * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  args.p_tiles = static_cast<int>((b.rows + kPairTile - 1) / kPairTile);
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * ((a.rows + kPairTile - 1) / kPairTile);
  if (tiles > (int64_t{1} << 30)) {
    set_last_error("the product has too many tiles");
    return QLORA_ERR_SHAPE;
  }
  auto kern = args.out_f32 ? k_fp4_gemm_pair<F, true> : k_fp4_gemm_pair<F, false>;
  QL_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem));
  const int grid = 2 * static_cast<int>(std::min<int64_t>(tiles, num_sms() / 2));
  QL_TRY(launch_pdl(kern, dim3(grid), dim3(kPairThreads), kPairSmem, st, tp, tq, sp, sq, xp, xq, to, args));
  return QLORA_OK;
}

template <Fp4 F>
qlora_status run_product(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                         const Fp4Args& args, cudaStream_t st) {
  const int64_t M = a.rows;
  if (M > 128) return run_pair<F>(a, b, ext, args, st);
  const int nt = M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * ((M + nt - 1) / nt);
  int cs = 1;
  while (cs < 8 && cs * 2 <= args.steps && tiles * cs * 2 <= 2 * num_sms()) cs *= 2;
  switch (nt) {
    case 32: return run_split<F, 32>(a, b, ext, args, cs, st);
    case 64: return run_split<F, 64>(a, b, ext, args, cs, st);
    case 128: return run_split<F, 128>(a, b, ext, args, cs, st);
    default: return run_split<F, 256>(a, b, ext, args, cs, st);
  }
}

}  // namespace

qlora_status fp4_product(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                         void* out, bool out_f32, cudaStream_t st) {
  Fp4Args args;
  args.sp = b.scales;
  args.sq = a.scales;
  args.gp = b.gscale;
  args.gq = a.gscale;
  args.gp_rows = b.gscale_rows > 1;
  args.gq_rows = a.gscale_rows > 1;
  args.P = b.rows;
  args.Q = a.rows;
  args.K = a.cols;
  args.ktiles = static_cast<int>(fp4_ktiles(a.cols, a.format));
  args.steps = static_cast<int>((a.cols + kStepCols - 1) / kStepCols);
  args.p_tiles = static_cast<int>((b.rows + kPRows - 1) / kPRows);
  args.ext_mmas = ext ? (ext->r + 15) / 16 : 0;
  args.ext_mn = ext && ext->mn_major;
  args.out = out;
  args.ld = b.rows;
  args.out_f32 = out_f32;
  args.err = device_error_word();
  return a.format == QLORA_FP4_MX ? run_product<Fp4::kMx>(a, b, ext, args, st)
                                  : run_product<Fp4::kNv>(a, b, ext, args, st);
}

}  // namespace qlora
