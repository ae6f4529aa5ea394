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
    if (lane == 0) {
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
    if (lane == 0) {
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

// ------------------------------------------------------------------ host side
constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapDataType kBf16Map = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;

template <Fp4 F, int NT>
qlora_status run_split(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                       Fp4Args args, int cs, cudaStream_t st) {
  CUtensorMap tp, tq, xp, xq;
  QL_MAP(&tp, kU8, b.codes, b.cols / 2, b.rows, b.cols / 2, 128, kPRows, kSw128);
  QL_MAP(&tq, kU8, a.codes, a.cols / 2, a.rows, a.cols / 2, 128, NT, kSw128);
  xp = tp;
  xq = tq;
  if (ext) {
    if (ext->mn_major) QL_MAP(&xp, kBf16Map, ext->p, b.rows, ext->r, b.rows * 2, 64, 64, kSw128);
    else QL_MAP(&xp, kBf16Map, ext->p, ext->r, b.rows, ext->r * 2, 64, kPRows, kSw128);
    QL_MAP(&xq, kBf16Map, ext->q, 128, a.rows, 256, 64, NT, kSw128);
  }
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
qlora_status run_product(const qlora_fp4_matrix& a, const qlora_fp4_matrix& b, const Fp4Ext* ext,
                         const Fp4Args& args, cudaStream_t st) {
  const int64_t M = a.rows;
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
