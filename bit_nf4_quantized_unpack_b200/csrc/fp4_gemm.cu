// fp4_gemm.cu -- products of microscaled 4-bit matrices on the block-scaled tensor cores.
//
//   out[m, n] = ga[m] gb[n] sum_k a[m, k] b[n, k]  (+ sum_j ext_b[j, n] ext_a[m, j])
//
// a: tokens, b: weight rows, both E2M1 codes with block scales along k; tcgen05.mma
// kind::mxf4nvf4 multiplies codes and scales and adds in fp32. The weight is the 128-lane
// operand, tokens are the columns of the accumulator.
//
// gscales and T may have been written by a kernel that was still running when this one began:
// plain loads behind griddep_wait, never the read-only path (__ldg).
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
// Few tokens (Q <= NT): reading the weight once bounds the time. A CTA takes 128 weight rows and
// all tokens; the `cs` CTAs of a cluster share the steps over K, put their accumulators in
// shared memory and each add up a part of the tokens through distributed shared memory, in
// rank order.
//
// With the rank-r term, `t` holds the fp32 [Q, r] values in parts; rank 0's epilogue warps add
// them and turn them into the bf16 hi and lo operands in shared memory.
//
// Launched behind a kernel that itself waited for everything before it (`early`), the CTAs
// fetch their first weight tiles before they wait for the tokens.
//
// Warp 0: TMA, warp 1: MMA and tensor memory, warps 2-5: epilogue. Tensor memory: an
// accumulator of NT columns, then 32 scale columns for each slot of the ring.
constexpr int kSplitThreads = 192;
constexpr uint32_t split_slot_bytes(int nt) { return kPBytes + nt * 128 + 8 * kSfTile; }
constexpr uint32_t split_smem(int nt, int slots) {
  return 1024 + slots * split_slot_bytes(nt) + 2 * nt * 128 + 512;
}
constexpr int kSplitMaxSlots = 8;

struct SplitArgs {
  int cs;           // CTAs of a cluster
  int slots;        // of the ring, at most kSplitMaxSlots
  uint32_t tmem;    // columns to allocate
  const float* t;   // [t_parts][Q, r] fp32 or NULL
  int t_parts;
  float* t_out;     // [Q, r] or NULL: their sum
  int r;
  float scale;
  bool early;
};

template <Fp4 F, int NT>
__global__ void __launch_bounds__(kSplitThreads)
    k_fp4_gemm_split(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_ext_p, const Fp4Args args,
                     const SplitArgs sa) {
  constexpr uint32_t kQBytes = NT * 128;
  constexpr int kTileStep = kStepCols / kFp4TileCols<F>;  // scale tiles per step: 2 or 4
  constexpr int kMmaTile = 4 / kTileStep;                 // MMAs per scale tile: 2 or 1
  const int S = sa.slots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* p_s = smem;                         // [S][kPBytes]
  uint8_t* q_s = p_s + S * kPBytes;            // [S][kQBytes]
  uint8_t* ext_s = q_s + S * kQBytes;          // [2][kQBytes] rank-r token operand, hi | lo
  uint8_t* sfp_s = ext_s + 2 * kQBytes;        // [S][4][512]
  uint8_t* sfq_s = sfp_s + S * 4 * kSfTile;    // [S][4][512]
  uint64_t* full = reinterpret_cast<uint64_t*>(sfq_s + S * 4 * kSfTile);
  uint64_t* empty = full + kSplitMaxSlots;
  uint64_t* acc_full = empty + kSplitMaxSlots;
  uint64_t* ext_ready = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ext_ready + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = sa.cs;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / cs;
  const int s_begin = static_cast<int>(static_cast<int64_t>(args.steps) * rank / cs);
  const int nmain = static_cast<int>(static_cast<int64_t>(args.steps) * (rank + 1) / cs) - s_begin;
  const bool ext = rank == 0 && args.ext_mmas > 0;  // one more step, after the others
  const int nsteps = nmain + ext;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(ext_ready, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, sa.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (elect_one()) {
      const int p0 = tile * kPRows;
      auto load_weight = [&](int i, int s) {
        uint8_t* dst = p_s + s * kPBytes;
        if (i < nmain) {
          const int step = s_begin + i, t0 = step * kTileStep;
          const uint32_t sf = static_cast<uint32_t>(min(kTileStep, args.ktiles - t0)) * kSfTile;
          mbar_arrive_expect_tx(&full[s], kPBytes + kQBytes + 2 * sf);
          tma_load_2d(dst, &tm_p, &full[s], step * 128, p0);
          bulk_load(sfp_s + s * 4 * kSfTile, args.sp + (static_cast<int64_t>(tile) * args.ktiles + t0) * kSfTile,
                    sf, &full[s]);
        } else {
          mbar_arrive_expect_tx(&full[s], kPBytes);
          if (args.ext_mn) {
            tma_load_2d(dst, &tm_ext_p, &full[s], p0, 0);
            tma_load_2d(dst + 8192, &tm_ext_p, &full[s], p0 + 64, 0);
          } else {
            tma_load_2d(dst, &tm_ext_p, &full[s], 0, p0);
          }
        }
      };
      const int ahead = sa.early ? min(S, nsteps) : 0;
      for (int i = 0; i < ahead; ++i) load_weight(i, i);
      griddep_wait_and_release();
      int issued = 0, s = 0;
      uint32_t phase = 1;  // of empty[s] before its latest use
      for (int i = 0; i < nsteps; ++i) {
        if (i >= S && !mbar_wait(&empty[s], phase, abort_flag)) {
          record_error(args.err, abort_flag, kErrTimeoutProducer);
          break;
        }
        if (i >= ahead) load_weight(i, s);
        if (i < nmain) {
          const int step = s_begin + i, t0 = step * kTileStep;
          tma_load_2d(q_s + s * kQBytes, &tm_q, &full[s], step * 128, 0);
          bulk_load(sfq_s + s * 4 * kSfTile, args.sq + static_cast<int64_t>(t0) * kSfTile,
                    static_cast<uint32_t>(min(kTileStep, args.ktiles - t0)) * kSfTile, &full[s]);
        }
        ++issued;
        if (++s == S) s = 0, phase ^= 1;
      }
      if (*abort_flag)
        for (int i = max(0, issued - S); i < issued; ++i) mbar_wait_drain(&full[i % S], (i / S) & 1u);
    }
  } else if (warp == 1) {
    griddep_wait_and_release();
    if (elect_one()) {
      const uint32_t idesc_ext = idesc_bf16_f32(kPRows, NT, args.ext_mn, false);
      int done = 0, s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; i < nsteps; ++i) {
        ok = mbar_wait(&full[s], phase, abort_flag);
        // MMAs of different kinds are not ordered with each other: before the rank-r step, wait
        // for the completion of the one before. (Every ring slot has its own scale columns, so
        // a slot that is full again has had its columns read.)
        if (ok && i == nmain) {
          ok = mbar_wait(ext_ready, 0, abort_flag);
          if (ok && i >= 1) ok = mbar_wait(&empty[(i - 1) % S], ((i - 1) / S) & 1u, abort_flag);
        }
        if (!ok) {
          record_error(args.err, abort_flag, kErrTimeoutMma);
          break;
        }
        tc_fence_after();
        const uint32_t pa = smem_u32(p_s + s * kPBytes);
        if (i < nmain) {
          const uint64_t dp = smem_desc_sw128(pa, 16, 1024);
          const uint64_t dq = smem_desc_sw128(smem_u32(q_s + s * kQBytes), 16, 1024);
          const uint32_t sfp = tmem + NT + s * 32, sfq = sfp + 16;
          const uint32_t sp = smem_u32(sfp_s + s * 4 * kSfTile), sq = smem_u32(sfq_s + s * 4 * kSfTile);
          const int64_t left = args.K - static_cast<int64_t>(s_begin + i) * kStepCols;
          const int mmas = left >= kStepCols ? 4 : static_cast<int>((left + 63) / 64);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= mmas) break;
            const int t = kk / kMmaTile, sub = kk % kMmaTile;
            if (sub == 0) {
              tmem_cp_scales(sfp + t * 4, smem_desc_scales(sp + t * kSfTile));
              tmem_cp_scales(sfq + t * 4, smem_desc_scales(sq + t * kSfTile));
            }
            umma_fp4<F == Fp4::kMx ? 2 : 4>(
                tmem, dp + kk * 2u, dq + kk * 2u,
                idesc_fp4(kPRows, NT, F == Fp4::kMx, F == Fp4::kMx ? 2 * sub : 0), sfp + t * 4,
                sfq + t * 4, (i | kk) != 0);
          }
        } else {
          const uint64_t dp = args.ext_mn ? smem_desc_sw128(pa, 8192, 1024) : smem_desc_sw128(pa, 16, 1024);
          const uint32_t adv = args.ext_mn ? 128u : 2u;
          for (int part = 0; part < 2; ++part) {
            const uint64_t dq = smem_desc_sw128(smem_u32(ext_s + part * kQBytes), 16, 1024);
            for (int kk = 0; kk < args.ext_mmas; ++kk)
              umma_bf16(tmem, dp + kk * adv, dq + kk * 2u, idesc_ext, (i | part | kk) != 0);
          }
        }
        umma_commit(&empty[s]);
        ++done;
        if (++s == S) s = 0, phase ^= 1;
      }
      umma_commit(acc_full);
      mbar_wait_drain(acc_full, 0);
      uint32_t par;
      for (int j = 0; j < S; ++j)
        if (last_use(done, S, j, par)) mbar_wait_drain(&empty[j], par);
    }
  } else {
    griddep_wait_and_release();
    const int quarter = warp & 3, tid = threadIdx.x - 64;
    const int Q = static_cast<int>(args.Q);
    if (ext) {
      // scale t / (ga gb) as bf16 hi and lo parts in the K-major swizzled operand layout
      const float ib = args.gp ? 1.f / *args.gp : 1.f;
#pragma unroll 4
      for (int i = tid; i < NT * 8; i += 128) {  // eight values of a token: one 16-byte group
        const int q = i >> 3, j = (i & 7) * 8;
        float v[8] = {};
        if (q < Q && j < sa.r) {
          const float ia = args.gq ? 1.f / args.gq[args.gq_rows ? q : 0] : 1.f;
#pragma unroll 4
          for (int part = 0; part < sa.t_parts; ++part) {
            const float4* src =
                reinterpret_cast<const float4*>(sa.t + (static_cast<int64_t>(part) * Q + q) * sa.r + j);
            const float4 x = src[0], y = src[1];
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
            v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
          }
          if (sa.t_out && tile == 0) {
            float4* dst = reinterpret_cast<float4*>(sa.t_out + static_cast<int64_t>(q) * sa.r + j);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[k] * sa.scale * ia * ib;
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[k] = pack_bf16x2_rn(v[2 * k], v[2 * k + 1]);
          lo[k] = bf16x2_rest_rn(v[2 * k], v[2 * k + 1], hi[k]);
        }
        const uint32_t off = sw128_kmajor_offset(q, i & 7);
        *reinterpret_cast<uint4*>(ext_s + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(ext_s + kQBytes + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(ext_ready);
    }
    // this CTA's tokens (a share of the cluster's), and this lane's four rows of every fourth
    const int span = (Q + cs - 1) / cs, t0 = min(Q, rank * span), t1 = min(Q, t0 + span);
    const int r4 = quarter * 32 + (lane & 7) * 4;
    const int64_t p4 = static_cast<int64_t>(tile) * kPRows + r4;
    float g4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      g4[j] = args.gp ? args.gp[args.gp_rows ? min(p4 + j, args.P - 1) : 0] : 1.f;
    const bool got = mbar_wait(acc_full, 0, abort_flag) && !*abort_flag;
    if (!got && !*abort_flag) record_error(args.err, abort_flag, kErrTimeoutEpilogue);
    tc_fence_after();
    // every step has been multiplied, so the ring is free: sums as [token][128 rows]
    float* part = reinterpret_cast<float*>(smem);
    if (got) {
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c * 32 < Q; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c * 32 + j) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]);
      }
    }
    if (cs > 1) cluster_sync_all();
    else __syncwarp();  // a warp reads only what it wrote
    if (got) {
      constexpr int kAt = 2;  // tokens of a lane whose remote loads are in flight together
      for (int q0 = t0 + (lane >> 3); q0 < t1; q0 += 4 * kAt) {
        float4 sum[kAt];
#pragma unroll
        for (int i = 0; i < kAt; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < cs; ++c) {
          float4 v[kAt];
#pragma unroll
          for (int i = 0; i < kAt; ++i)
            v[i] = ld_cluster_f32x4(part + min(q0 + 4 * i, t1 - 1) * 128 + r4, cs > 1 ? c : rank);
#pragma unroll
          for (int i = 0; i < kAt; ++i)
            sum[i].x += v[i].x, sum[i].y += v[i].y, sum[i].z += v[i].z, sum[i].w += v[i].w;
        }
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
          const int q = q0 + 4 * i;
          if (q >= t1 || p4 >= args.P) continue;  // P is a multiple of 8
          const float gq = args.gq ? args.gq[args.gq_rows ? q : 0] : 1.f;
          const float4 o = make_float4(sum[i].x * g4[0] * gq, sum[i].y * g4[1] * gq,
                                       sum[i].z * g4[2] * gq, sum[i].w * g4[3] * gq);
          if (args.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(args.out) + q * args.ld + p4) = o;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(args.out) + q * args.ld + p4) =
                make_uint2(pack_bf16x2_rn(o.x, o.y), pack_bf16x2_rn(o.z, o.w));
        }
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
    tmem_dealloc(tmem, sa.tmem);
  }
}

// ------------------------------------------------------------------ pair kernel
// A persistent CTA pair per two SMs; a tile is 256 weight rows x TQ tokens (256, or 128 where
// that gives more pairs work). Each CTA holds 128 weight rows of the operand, half of the
// tokens of the other, its rows' scales and all tokens' scales, and accumulates its 128 rows
// x TQ tokens in its own tensor memory.
//
// Tensor memory: two accumulators of TQ columns used in turn and two sets of scale columns.
// For TQ = 256 they do not fit side by side (2 * 256 + 2 * 48 > 512), so the accumulators
// share the columns [160, 256): the epilogue reads those first and then lets the next tile's
// MMAs start, while it goes on with the other 160 columns.
//
// Warp 0: TMA, warp 1: MMA (in the leader) and tensor memory, warps 2-9: epilogue, two warps
// for each quarter of the lanes.
constexpr int kPairThreads = 320;
constexpr int kPairP = 256;                   // weight rows of a tile
constexpr uint32_t kPairSf = 4 * kSfTile;     // scales of 128 rows and one step (NVFP4)
constexpr int kEpiWarps = 8;
constexpr uint32_t kPairEpi = kEpiWarps * 2 * 32 * 32 * 2;
template <int TQ>
struct Pair {
  static constexpr int kStages = TQ == 256 ? 5 : 6;
  static constexpr uint32_t kQBytes = TQ / 2 * 128;
  static constexpr int kSqTiles = TQ / 128;   // token scale tiles
  static constexpr uint32_t kStage = kPBytes + kQBytes + (1 + kSqTiles) * kPairSf;
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + kPairEpi + 256;
  static constexpr bool kShared = TQ == 256;               // accumulators share columns
  static constexpr uint32_t kAcc1 = TQ == 256 ? 160 : 128;  // first column of the second
  static constexpr uint32_t kSfCol = kAcc1 + TQ;           // first scale column
  static constexpr uint32_t kSfSet = 16 + 16 * kSqTiles;
  static_assert(kSmem <= 227 * 1024 && kSfCol + 2 * kSfSet <= 512, "shared and tensor memory");
};

struct PairTile {
  int64_t p0, q0;
};
// Tiles in groups of eight token tiles, so that the tiles in flight at one time form a block
// that shares operands in L2.
template <int TQ>
__device__ __forceinline__ PairTile pair_tile(int t, int p_tiles, int q_tiles) {
  constexpr int kGroup = 8;
  const int per = kGroup * p_tiles;
  const int g = t / per, in = t - g * per;
  const int width = min(kGroup, q_tiles - g * kGroup);
  return {static_cast<int64_t>(in / width) * kPairP, static_cast<int64_t>(g * kGroup + in % width) * TQ};
}

template <Fp4 F, int TQ, bool OUT_F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_fp4_gemm_pair(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_sp, const __grid_constant__ CUtensorMap tm_sq,
                    const __grid_constant__ CUtensorMap tm_ext_p,
                    const __grid_constant__ CUtensorMap tm_ext_q,
                    const __grid_constant__ CUtensorMap tm_out, const Fp4Args args) {
  using C = Pair<TQ>;
  constexpr int S = C::kStages;
  constexpr uint32_t kPairQBytes = C::kQBytes;
  constexpr int kTileStep = kStepCols / kFp4TileCols<F>;  // scale tiles per step: 2 or 4
  constexpr int kMmaTile = 4 / kTileStep;                 // MMAs per scale tile: 2 or 1
  constexpr uint32_t kSfBytes = kTileStep * kSfTile;      // of 128 rows and one step
  constexpr uint32_t kStepTx = 2 * (kPBytes + kPairQBytes + (1 + C::kSqTiles) * kSfBytes);  // both CTAs
  constexpr uint32_t kExtTx = 2 * (kPBytes + kPairQBytes);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* p_s = smem;                          // [S][kPBytes]
  uint8_t* q_s = p_s + S * kPBytes;             // [S][kPairQBytes]
  uint8_t* epi_s = q_s + S * kPairQBytes;       // [8 warps][2][32][32] bf16
  uint8_t* sfp_s = epi_s + kPairEpi;            // [S][kPairSf]
  uint8_t* sfq_s = sfp_s + S * kPairSf;         // [S][kSqTiles kPairSf]: row tiles of kSfBytes
  uint64_t* full = reinterpret_cast<uint64_t*>(sfq_s + S * C::kSqTiles * kPairSf);  // the leader's counts
  uint64_t* empty = full + S;                   // [S] MMAs reading the slot done (both CTAs)
  // of the tile in accumulator 0 or 1 (two of each, so that no waiter is ever two phases behind)
  uint64_t* acc_full = empty + S;               // [2] complete (both CTAs)
  uint64_t* acc_part = acc_full + 2;            // [2] handed over by the epilogue (the leader's)
  uint64_t* mma_drain = acc_part + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int q_tiles = static_cast<int>((args.Q + TQ - 1) / TQ);
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
    for (int h = 0; h < 2; ++h) {
      mbar_init(&acc_full[h], 1);
      mbar_init(&acc_part[h], 2 * kEpiWarps);
    }
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
        const PairTile t = pair_tile<TQ>(first + i * clusters, args.p_tiles, q_tiles);
        const int p0 = static_cast<int>(t.p0) + 128 * rank, q0 = static_cast<int>(t.q0) + TQ / 2 * rank;
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
            tma_load_2d_pair(sfq_s + s * C::kSqTiles * kPairSf, &tm_sq, bar, x, static_cast<int>(t.q0 / 128));
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
      const uint32_t idesc_ext = idesc_bf16_f32(kPairP, TQ, args.ext_mn, false);
      const uint32_t ext_adv = args.ext_mn ? 128u : 2u;
      // descriptors of slot 0; the start-address field counts 16 bytes
      const uint64_t dp0 = smem_desc_sw128(smem_u32(p_s), 16, 1024);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(q_s), 16, 1024);
      const uint64_t dp_ext0 = args.ext_mn ? smem_desc_sw128(smem_u32(p_s), 8192, 1024) : dp0;
      const uint64_t dsp0 = smem_desc_scales(smem_u32(sfp_s)), dsq0 = smem_desc_scales(smem_u32(sfq_s));
      // MMAs of a tile's last step: K may end inside it
      const int tail_mmas = static_cast<int>((args.K - static_cast<int64_t>(args.steps - 1) * kStepCols + 63) / 64);
      int n = 0;
      bool ok = true;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const uint32_t d = tmem + (i & 1) * C::kAcc1;
        // Shared columns: the epilogue has those of tile i - 1 in registers (and, having begun
        // that tile, all of tile i - 2, which used this accumulator). Otherwise: it has all of
        // tile i - 2.
        constexpr int kBack = C::kShared ? 1 : 2;
        if (i >= kBack)
          ok = mbar_wait(&acc_part[(i - kBack) & 1], ((i - kBack) >> 1) & 1u, abort_flag);
        tc_fence_after();
        for (int k = 0; k < total && ok; ++k) {
          const int s = n % S;
          // The scale columns of this step were last read by the MMAs two steps ago (two sets,
          // used in turn), and MMAs of different kinds are not ordered with each other: wait
          // for the completion of step n - 2, or of n - 1 where the kind changes.
          const int before = ext && (k == 0 || k == ext) ? n - 1 : n - 2;
          ok = before >= 0 ? mbar_wait_both(&full[s], (n / S) & 1u, &empty[before % S],
                                            (before / S) & 1u, abort_flag)
                           : mbar_wait(&full[s], (n / S) & 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dq = dq0 + static_cast<uint32_t>(s) * (kPairQBytes >> 4);
          if (k < ext) {
            const uint64_t dp = dp_ext0 + static_cast<uint32_t>(s) * (kPBytes >> 4);
            for (int kk = 0; kk < args.ext_mmas; ++kk)
              umma_bf16_pair(d, dp + kk * ext_adv, dq + kk * 2u, idesc_ext, (k | kk) != 0);
          } else {
            const uint64_t dp = dp0 + static_cast<uint32_t>(s) * (kPBytes >> 4);
            const uint64_t sp = dsp0 + static_cast<uint32_t>(s) * (kPairSf >> 4);
            const uint64_t sq = dsq0 + static_cast<uint32_t>(s) * (C::kSqTiles * kPairSf >> 4);
            const uint32_t sfp = tmem + C::kSfCol + (n & 1) * C::kSfSet, sfq = sfp + 16;
            // scale tile tl and the MMAs that use it
            auto tile = [&](int tl, int mmas) {
              tmem_cp_scales_pair(sfp + tl * 4, sp + tl * (kSfTile >> 4));
#pragma unroll
              for (int h = 0; h < C::kSqTiles; ++h)
                tmem_cp_scales_pair(sfq + (tl * C::kSqTiles + h) * 4, sq + ((h * kSfBytes + tl * kSfTile) >> 4));
#pragma unroll
              for (int sub = 0; sub < kMmaTile; ++sub) {
                const int kk = tl * kMmaTile + sub;
                if (kk < mmas)
                  umma_fp4_pair<F == Fp4::kMx ? 2 : 4>(
                      d, dp + kk * 2u, dq + kk * 2u,
                      idesc_fp4(kPairP, TQ, F == Fp4::kMx, F == Fp4::kMx ? 2 * sub : 0),
                      sfp + tl * 4, sfq + tl * C::kSqTiles * 4, (k | kk) != 0);
              }
            };
            if (k < total - 1 || tail_mmas == 4) {
#pragma unroll
              for (int tl = 0; tl < kTileStep; ++tl) tile(tl, 4);
            } else {
#pragma unroll
              for (int tl = 0; tl < kTileStep; ++tl)
                if (tl * kMmaTile < tail_mmas) tile(tl, tail_mmas);
            }
          }
          umma_commit_pair(&empty[s]);
          if (k == total - 1) umma_commit_pair(&acc_full[i & 1]);
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
    const uint32_t part_bar = cluster_addr(acc_part, 0);  // of accumulator 0
    if (lane == 0) tma_prefetch_desc(&tm_out);
    int chunks = 0;  // stage buffers used
    for (int i = 0; i < my_tiles; ++i) {
      const PairTile t = pair_tile<TQ>(first + i * clusters, args.p_tiles, q_tiles);
      const int64_t p0 = t.p0 + 128 * rank + quarter * 32;
      // this warp's 32-token chunks, those in shared columns first: accumulator 0 shares its
      // chunks 5-7, accumulator 1 its chunks 0-2
      constexpr int kChunks = TQ / 64;
      const int shared0 = (i & 1) ? 0 : 5, own0 = (i & 1) ? 3 : 0;
      const int c0 = C::kShared ? shared0 + 2 * half : 2 * half;
      const int c1 = C::kShared ? (half ? own0 + 2 : shared0 + 1) : 2 * half + 1;
      const int c2 = own0 + (half ? 3 : 0), c3 = own0 + (half ? 4 : 1);
      const int cs[4] = {c0, c1, c2, c3};
      float gq[4], gp[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        gq[j] = 1.f;
        gp[j] = 1.f;
        if (args.gq && j < kChunks) gq[j] = args.gq[args.gq_rows ? min(t.q0 + cs[j] * 32 + lane, args.Q - 1) : 0];
        // rows lane / 4 + 8 j of the quarter (bf16 output), row lane (fp32 output, j = 0)
        const int64_t row = p0 + (OUT_F32 ? lane : (lane >> 2) + 8 * j);
        if (args.gp) gp[j] = args.gp[args.gp_rows ? min(row, args.P - 1) : 0];
      }
      if (!mbar_wait(&acc_full[i & 1], (i >> 1) & 1u, abort_flag)) {
        if (!*abort_flag) record_error(args.err, abort_flag, kErrTimeoutEpilogue);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + (i & 1) * C::kAcc1 + (static_cast<uint32_t>(quarter * 32) << 16);
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
        // Nothing to store: the stage buffers are left alone and not counted, since the waits below
        // count on a bulk group for every use of a buffer.
        if (q >= args.Q || p0 >= args.P) return;
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
        if (elect_one()) {
          tma_store_2d(&tm_out, OUT_F32 ? stage2 : stage2 + (chunks & 1) * 2048, static_cast<int>(p0),
                       static_cast<int>(q));
          bulk_commit_group();
        }
        ++chunks;
      };
      uint32_t v0[32], v1[32];
      const bool both = !C::kShared || half == 0;  // before the hand-over
      fetch(c0, v0);
      if (both) fetch(c1, v1);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(part_bar + (i & 1) * 8);
      emit(0, v0);
      if (!both) {
        fetch(c1, v1);
        tmem_ld_wait();
      }
      emit(1, v1);
      if constexpr (kChunks == 4) {
        fetch(c2, v0);
        tmem_ld_wait();
        emit(2, v0);
        fetch(c3, v1);
        tmem_ld_wait();
        emit(3, v1);
      }
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

template <Fp4 F, int NT>
qlora_status run_split(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                       const Fp4Args& args, bool early, cudaStream_t st) {
  CUtensorMap tp, tq, xp;
  QL_MAP(&tp, kU8, b.codes, b.cols / 2, b.rows, b.cols / 2, 128, kPRows, kSw128);
  QL_MAP(&tq, kU8, a.codes, a.cols / 2, a.rows, a.cols / 2, 128, NT, kSw128);
  xp = tp;
  SplitArgs sa = {};
  if (ext) {
    if (ext->mn_major) QL_MAP(&xp, kBf16Map, ext->p, b.rows, ext->r, b.rows * 2, 64, 64, kSw128);
    else QL_MAP(&xp, kBf16Map, ext->p, ext->r, b.rows, ext->r * 2, 64, kPRows, kSw128);
    sa.t = ext->t;
    sa.t_parts = ext->t_parts;
    sa.t_out = ext->t_out;
    sa.r = ext->r;
    sa.scale = ext->scale;
  }
  sa.early = early;
  // One CTA per SM takes a ring as deep as fits; more than that share SMs in pairs, with half
  // of shared and tensor memory each (NT = 128 leaves no room for a second).
  const int deep = std::min<int>(kSplitMaxSlots, (227 * 1024 - split_smem(NT, 0)) / split_slot_bytes(NT));
  const int half = std::min<int>(kSplitMaxSlots, (113 * 1024 - split_smem(NT, 0)) / split_slot_bytes(NT));
  // as many CTAs a cluster as the SMs take at one time, with two steps each at least: two per
  // SM read 3 to 12 % faster than one (8192 x 28672, one token: 24.7 against 26.8 us)
  const int sms = num_sms(), at_once = half >= 3 ? 2 * sms : sms;
  sa.cs = 1;
  while (sa.cs < 8 && sa.cs * 4 <= args.steps && args.p_tiles * sa.cs * 2 <= at_once) sa.cs *= 2;
  const int64_t ctas = static_cast<int64_t>(args.p_tiles) * sa.cs;
  const bool pairs = ctas > sms && half >= 3;
  sa.slots = pairs ? half : deep;
  sa.tmem = NT + 32 * sa.slots <= 256 ? 256 : 512;
  auto kern = k_fp4_gemm_split<F, NT>;
  const uint32_t smem = split_smem(NT, sa.slots);
  QL_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, split_smem(NT, deep)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sa.cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sa.cs > 1 ? 2 : 1;
  note_launches(1);
  QL_TRY(cudaLaunchKernelEx(&cfg, kern, tp, tq, xp, args, sa));
  return QLORA_OK;
}

template <Fp4 F, int TQ>
qlora_status run_pair(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                      Fp4Args args, cudaStream_t st) {
  CUtensorMap tp, tq, sp, sq, xp, xq, to;
  QL_MAP(&tp, kU8, b.codes, b.cols / 2, b.rows, b.cols / 2, 128, kPRows, kSw128);
  QL_MAP(&tq, kU8, a.codes, a.cols / 2, a.rows, a.cols / 2, 128, TQ / 2, kSw128);
  // scale tiles as rows of 8-byte elements: 64 per tile
  constexpr uint32_t box = kStepCols / kFp4TileCols<F> * 64;
  constexpr CUtensorMapDataType kU64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
  const uint64_t srow = static_cast<uint64_t>(args.ktiles) * 512;
  QL_MAP(&sp, kU64, b.scales, srow / 8, (b.rows + 127) / 128, srow, box, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  QL_MAP(&sq, kU64, a.scales, srow / 8, (a.rows + 127) / 128, srow, box, TQ / 128, CU_TENSOR_MAP_SWIZZLE_NONE);
  xp = tp;
  xq = tq;
  if (ext) {
    if (ext->mn_major) QL_MAP(&xp, kBf16Map, ext->p, b.rows, ext->r, b.rows * 2, 64, 64, kSw128);
    else QL_MAP(&xp, kBf16Map, ext->p, ext->r, b.rows, ext->r * 2, 64, kPRows, kSw128);
    QL_MAP(&xq, kBf16Map, ext->q, 128, a.rows, 256, 64, TQ / 2, kSw128);
  }
  if (args.out_f32)
    QL_MAP(&to, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, args.out, b.rows, a.rows, b.rows * 4, 32, 32,
           CU_TENSOR_MAP_SWIZZLE_NONE);
  else
    QL_MAP(&to, kBf16Map, args.out, b.rows, a.rows, b.rows * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  args.p_tiles = static_cast<int>((b.rows + kPairP - 1) / kPairP);
  const int64_t tiles = static_cast<int64_t>(args.p_tiles) * ((a.rows + TQ - 1) / TQ);
  if (tiles > (int64_t{1} << 30)) {
    set_last_error("the product has too many tiles");
    return QLORA_ERR_SHAPE;
  }
  auto kern = args.out_f32 ? k_fp4_gemm_pair<F, TQ, true> : k_fp4_gemm_pair<F, TQ, false>;
  QL_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pair<TQ>::kSmem));
  // the fewest pairs that take no more rounds than all of them: the others' SMs are left to a
  // kernel beside this one (dA and dB), their share of L2 bandwidth and power to these
  const int64_t pairs = std::max(num_sms() / 2, 1), rounds = (tiles + pairs - 1) / pairs;
  const int grid = 2 * static_cast<int>((tiles + rounds - 1) / rounds);
  QL_TRY(launch_pdl(kern, dim3(grid), dim3(kPairThreads), Pair<TQ>::kSmem, st, tp, tq, sp, sq, xp, xq, to, args));
  return QLORA_OK;
}

template <Fp4 F>
qlora_status run_product(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                         const Fp4Args& args, bool early, cudaStream_t st) {
  if (a.rows > kFp4SplitMaxM) {
    // Narrow tiles where they take no more rounds of the CTA pairs than wide ones, that is,
    // where wide ones leave half of the pairs idle. NVFP4, N = K = 4096: 512 tokens (32 wide or
    // 64 narrow tiles on 74 pairs) 9.9 against 10.7 us wide; 1024 tokens 14.5 against 11.6.
    const int64_t pt = (b.rows + kPairP - 1) / kPairP, pairs = std::max(num_sms() / 2, 1);
    const int64_t wide = (pt * ((a.rows + 255) / 256) + pairs - 1) / pairs;
    const int64_t narrow = (pt * ((a.rows + 127) / 128) + pairs - 1) / pairs;
    return narrow <= wide ? run_pair<F, 128>(a, b, ext, args, st) : run_pair<F, 256>(a, b, ext, args, st);
  }
  if (a.rows <= 32) return run_split<F, 32>(a, b, ext, args, early, st);
  if (a.rows <= 64) return run_split<F, 64>(a, b, ext, args, early, st);
  return run_split<F, 128>(a, b, ext, args, early, st);
}

}  // namespace

qlora_status fp4_product(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                         void* out, bool out_f32, bool early, cudaStream_t st) {
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
  return a.format == QLORA_FP4_MX ? run_product<Fp4::kMx>(a, b, ext, args, early, st)
                                  : run_product<Fp4::kNv>(a, b, ext, args, early, st);
}

}  // namespace qlora
