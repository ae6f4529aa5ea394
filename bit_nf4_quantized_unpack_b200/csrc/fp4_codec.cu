// fp4_codec.cu -- quantization to microscaled 4-bit floating point and reading back.
//
// MXFP4 (blocks of 32 along a row):  e = floor(log2 amax) - 2 clamped to [-127, 127] (-127 for
//   amax = 0), scale byte e + 127, code = e2m1(x 2^-e).
// NVFP4 (blocks of 16): g = 2^e with the smallest e for which top <= 2688 * 2^e, top being the
//   largest magnitude of the row (activations) or of the matrix (weights); g = 1 for top = 0;
//   scale byte c = e4m3(amax / g / 6), code = e2m1(x / g / c), 0 where c = 0.
// e2m1() and e4m3() round to nearest, ties to even, and saturate. With g a power of two the
// only inexact steps are those roundings: x / g is exact, the fp32 quotient amax / 6 is correctly
// rounded, x / (g c) is the rounding of a number within 2^-20 ulp of the real quotient, and
// either lands on a rounding border only when the real quotient does (numerator and border
// times divisor are both fp32 numbers, so a real quotient off the border is off by more than
// half an fp32 ulp). Codes and scales are therefore those of the definition in real arithmetic.
// A block that holds a NaN or an infinity gets the NaN scale and zero codes; its non-finite
// values do not enter top.
//
// Inputs are read by plain loads through pointers that are not __restrict__: they may have been
// written by a kernel that was still running when this one began, which rules out the read-only
// path (__ldg), and nothing may be loaded ahead of griddep_wait_and_release.
#include <cuda_bf16.h>

#include <algorithm>

#include "fp4_device.cuh"

namespace qlora {
namespace {

constexpr int kChunk = 16;  // values per thread and step: 32 bytes of bf16, 64 of fp32
constexpr uint32_t kMag = 0x7FFFFFFFu;
constexpr uint32_t kInf = 0x7F800000u;

// Both bf16 halves of w times 2^64, for values small enough that this is exact.
__device__ __forceinline__ void bf16x2_up64(uint32_t& w) {
  w = pack_bf16x2_rn(__uint_as_float(w << 16) * 0x1p64f, __uint_as_float(w & 0xFFFF0000u) * 0x1p64f);
}

// 16 values as loaded, and their largest magnitude as fp32 bits (kInf or above when one of
// them is not finite: magnitudes order like unsigned integers, NaNs last).
template <bool BF16>
struct Raw16;
template <>
struct Raw16<true> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
    const uint4 a = p[0], b = p[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void scale_2_64() {
#pragma unroll
    for (int i = 0; i < 8; ++i) bf16x2_up64(w[i]);
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);  // two 16-bit maxima
    return max(m & 0xFFFF0000u, m << 16);
  }
};
template <>
struct Raw16<false> {
  float v[16];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = p[i];
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void scale_2_64() {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= 0x1p64f;
  }
  __device__ __forceinline__ float at(int i) const { return v[i]; }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & kMag);
    return m;
  }
};

// The largest finite magnitude, for the rare block whose amax() is not finite.
template <typename R>
__device__ __forceinline__ uint32_t finite_amax(const R& r) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = __float_as_uint(r.at(i)) & kMag;
    if (b < kInf) m = max(m, b);
  }
  return m;
}

// x / d for positive normal d, correctly rounded: the reciprocal's product and one correction
// by its exact remainder (Markstein's method, IBM J. Res. Dev. 34, 1990). (Results below the
// normal range only round to the code 0.)
__device__ __forceinline__ float div_rn(float x, float d, float rcp) {
  const float q = x * rcp;
  return __fmaf_rn(__fmaf_rn(-q, d, x), rcp, q);
}

// 1 / x to one ulp, for x that is neither subnormal nor larger than 2^126.
__device__ __forceinline__ float rcp_1ulp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scale byte of a block from its largest magnitude; g_inv = 1 / gscale (NVFP4).
template <Fp4 F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t am, float g_inv) {
  if (am >= kInf) return kFp4NanScale<F>;
  if (F == Fp4::kMx) {
    const int biased = static_cast<int>(am >> 23) - 2;  // floor(log2) - 2 + 127
    return static_cast<uint32_t>(max(biased, 0));       // zero and subnormal maxima: 2^-127
  }
  return e4m3_bits(div_rn(__uint_as_float(am) * g_inv, 6.f, 1.f / 6.f));
}

// An NVFP4 gscale 2^e and what encoders divide by: their own is 2^64 times as large for a
// tiny one (1 / (g c) would overflow below 2^-118), and so are the values then.
struct Gscale {
  float g, inv, up;
  __device__ __forceinline__ explicit Gscale(int e)
      : g(pow2_f32(e)), inv(pow2_f32(-e)), up(e < -90 ? 0x1p64f : 1.f) {}
  __device__ __forceinline__ float enc() const { return g * up; }
  __device__ __forceinline__ float enc_inv() const { return up == 1.f ? inv : inv * 0x1p-64f; }
};

// What turns a value into the argument of e2m1() under one scale byte c. MX: x * mul. NV: the
// quotient x / (g c) as q = x mul, mul = 1 / (g c) nearly, corrected by its remainder,
// y = q + (x - q g c) mul. c has 4 significant bits, so the remainder is exact although mul is
// off by an ulp or two, and y is the rounding of a number within 2^-20 ulp of the real
// quotient. It is a border of e2m1() (3 bits) just where the quotient is one: elsewhere x and
// the border times g c are different multiples of an ulp of x, which puts the quotient at
// least 8/15 ulp off. What is computed is -q and -y, for the sign of a zero x, and the codes'
// signs are turned at the end.
template <Fp4 F>
struct Encoder {
  float mul, div;  // NV: -1 / (g c), g c; mul = 0 for codes that are all 0
  __device__ __forceinline__ Encoder(uint32_t sb, const Gscale& g) {
    if (F == Fp4::kMx) {
      mul = sb == kFp4NanScale<F> ? 0.f : pow2_f32(127 - static_cast<int>(sb));
    } else {
      const bool none = sb == 0u || sb == kFp4NanScale<F>;
      const float c = none ? 1.f : fp4_scale_value<F>(sb);
      mul = none ? 0.f : -rcp_1ulp(c) * g.enc_inv();
      div = c * g.enc();
    }
  }
  __device__ __forceinline__ bool zero() const { return mul == 0.f; }
  // eight values, v(i), to eight codes
  template <typename V>
  __device__ __forceinline__ uint32_t encode8(V&& v) const {
    float y[8];
    if (F == Fp4::kMx) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v(i) * mul;
      return fp4_pack8(y);
    }
    const uint64_t m2 = f2_pack(mul, mul), d2 = f2_pack(div, div);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t x = f2_pack(v(i), v(i + 1)), q = f2_mul(x, m2);
      f2_unpack(f2_fma(f2_fma(q, d2, x), m2, q), y[i], y[i + 1]);
    }
    return fp4_pack8(y) ^ 0x88888888u;
  }
};

// Codes of 16 values under one scale byte (low nibble first).
template <Fp4 F, typename R>
__device__ __forceinline__ uint2 codes16(R& r, uint32_t sb, const Gscale& g) {
  if (F == Fp4::kNv && g.up != 1.f) r.scale_2_64();  // the same in every thread of a row
  const Encoder<F> e(sb, g);
  if (e.zero()) return make_uint2(0u, 0u);
  return make_uint2(e.encode8([&](int i) { return r.at(i); }),
                    e.encode8([&](int i) { return r.at(8 + i); }));
}

// The scale bytes of four consecutive blocks as one word, valid in the lane that holds the
// first of them (lanes hold 16 values each, in column order; a block is 1 or 2 lanes).
template <Fp4 F>
__device__ __forceinline__ uint32_t gather4(uint32_t sb) {
  constexpr int kStep = kFp4Block<F> / kChunk;
  uint32_t w = sb | __shfl_down_sync(~0u, sb, kStep) << 8;
  w |= __shfl_down_sync(~0u, w, 2 * kStep) << 16;
  return w;
}

// ------------------------------------------------------------------ MXFP4 rows
// A warp takes 512 columns of one row, 16 per lane; neighbouring warps take neighbouring rows,
// whose scale bytes share sectors.
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_quantize_mx(const void* X, uint32_t rows, int64_t cols,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_wait_and_release();
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  for (int64_t seg = blockIdx.y; seg * 512 < cols; seg += gridDim.y) {
    const int64_t col = seg * 512 + lane * kChunk;
    const bool in = col < cols;
    Raw16<BF16> r;
    if (in) r.load(X, row * cols + col);
    else r.zero();
    uint32_t am = r.amax();
    am = max(am, __shfl_xor_sync(~0u, am, 1));
    const uint32_t sb = in ? scale_byte<Fp4::kMx>(am, 1.f) : 0u;
    if (in)
      *reinterpret_cast<uint2*>(codes + (row * cols + col) / 2) = codes16<Fp4::kMx>(r, sb, Gscale(0));
    const uint32_t w = gather4<Fp4::kMx>(sb);
    if ((lane & 7) == 0 && in)
      *reinterpret_cast<uint32_t*>(scales + fp4_scale_offset(row, col / 32, (cols + 127) / 128)) = w;
  }
}

// ------------------------------------------------------------------ NVFP4 rows
// A CTA takes every gridDim.x-th row. The row stays in registers (U chunks a thread) between
// the row maximum and the codes; with one chunk a thread the next row is fetched meanwhile.
// U = 0: rows too long for that are read twice.
template <bool BF16, int U>
__global__ void __launch_bounds__(512)
    k_fp4_quantize_nv(const void* X, uint32_t rows, int64_t cols,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                      float* __restrict__ gscale) {
  griddep_wait_and_release();
  __shared__ uint32_t part[2][16];  // warps' maxima, of even and odd passes
  const int tid = threadIdx.x, nt = blockDim.x;
  const int chunks = static_cast<int>(cols / kChunk), padded = (chunks + 3) & ~3;
  const int64_t ktiles = padded / 4;
  Raw16<BF16> raw[U > 0 ? U : 1], next;
  uint32_t am[U > 0 ? U : 1];
  auto fetch = [&](int64_t row, int u, Raw16<BF16>& r) {
    if (row < rows && tid + u * nt < chunks)
      r.load(X, row * cols + static_cast<int64_t>(tid + u * nt) * kChunk);
    else
      r.zero();
  };
  if constexpr (U == 1) fetch(blockIdx.x, 0, next);
  int pass = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, pass ^= 1) {
    uint32_t top = 0u;
    auto join = [&](const Raw16<BF16>& r) {
      const uint32_t m = r.amax();
      top = max(top, m < kInf ? m : finite_amax(r));
      return m;
    };
    if constexpr (U > 0) {
      if constexpr (U == 1) {
        raw[0] = next;
        fetch(row + gridDim.x, 0, next);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(row, u, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) am[u] = join(raw[u]);
    } else {
      for (int c = tid; c < chunks; c += nt) {
        raw[0].load(X, row * cols + static_cast<int64_t>(c) * kChunk);
        join(raw[0]);
      }
    }
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) part[pass][tid >> 5] = top;
    __syncthreads();  // a warp writes part[pass] again only past the next pass's barrier
    top = __reduce_max_sync(~0u, (tid & 31) < (nt >> 5) ? part[pass][tid & 31] : 0u);  // 16 warps at most
    const Gscale g(nv_gscale_exp(top));
    if (tid == 0) gscale[row] = g.g;
    auto emit = [&](int c, Raw16<BF16>& r, uint32_t m) {
      const bool in = c < chunks;
      const uint32_t sb = in ? scale_byte<Fp4::kNv>(m, g.inv) : 0u;
      if (in)
        *reinterpret_cast<uint2*>(codes + row * (cols / 2) + static_cast<int64_t>(c) * (kChunk / 2)) =
            codes16<Fp4::kNv>(r, sb, g);
      const uint32_t w = gather4<Fp4::kNv>(sb);
      if ((c & 3) == 0 && c < padded)
        *reinterpret_cast<uint32_t*>(scales + fp4_scale_offset(row, c, ktiles)) = w;
    };
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * nt < padded) emit(tid + u * nt, raw[u], am[u]);
    } else {
      for (int c = tid; c - tid < padded; c += nt) {
        if (c < chunks) raw[0].load(X, row * cols + static_cast<int64_t>(c) * kChunk);
        else raw[0].zero();
        emit(c, raw[0], raw[0].amax());
      }
    }
  }
}

// One row by a CTA of 256 threads, in passes of four chunks a thread; a row that fits one pass
// stays in registers between the maximum and the codes.
template <Fp4 F>
__device__ __forceinline__ void quantize_row(const uint16_t* X, int64_t row, int64_t cols,
                                             uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                             float* __restrict__ gscale, uint32_t* part) {
  constexpr int U = 4, NT = 256;
  constexpr int kGroup = 4 * kFp4Block<F> / kChunk;  // chunks of four blocks
  const int tid = threadIdx.x;
  const int chunks = static_cast<int>(cols / kChunk), padded = (chunks + kGroup - 1) / kGroup * kGroup;
  Raw16<true> raw[U];
  auto fetch = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + tid + u * NT;
      if (c < chunks) raw[u].load(X, row * cols + static_cast<int64_t>(c) * kChunk);
      else raw[u].zero();
    }
  };
  fetch(0);
  Gscale g(0);
  if constexpr (F == Fp4::kNv) {
    uint32_t top = 0u;
    for (int base = 0;;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t m = raw[u].amax();
        if (m >= kInf) m = finite_amax(raw[u]);
        top = max(top, m);
      }
      base += U * NT;
      if (base >= chunks) break;
      fetch(base);
    }
    top = __reduce_max_sync(~0u, top);
    if ((tid & 31) == 0) part[tid >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(~0u, part[tid & (NT / 32 - 1)]);
    g = Gscale(nv_gscale_exp(top));
    if (tid == 0) gscale[row] = g.g;
    if (chunks > U * NT) fetch(0);
  }
  for (int base = 0; base < padded; base += U * NT) {
    if (base > 0) fetch(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + tid + u * NT;
      if (base + u * NT >= padded) break;  // the same in every thread
      uint32_t am = raw[u].amax();
      if (F == Fp4::kMx) am = max(am, __shfl_xor_sync(~0u, am, 1));
      const uint32_t sb = c < chunks ? scale_byte<F>(am, g.inv) : 0u;
      if (c < chunks)
        *reinterpret_cast<uint2*>(codes + row * (cols / 2) + static_cast<int64_t>(c) * (kChunk / 2)) =
            codes16<F>(raw[u], sb, g);
      const uint32_t w = gather4<F>(sb);
      if (c % kGroup == 0 && c < padded)
        *reinterpret_cast<uint32_t*>(scales + fp4_scale_offset(row, c * kChunk / kFp4Block<F>, padded / kGroup)) = w;
    }
  }
}

// ------------------------------------------------------------------ few tokens: rows and rank-r product
// One launch for what a few tokens need before their product with the weight, in clusters of
// eight CTAs: X [M, K] in microscaled form, and T = X A with A [K, r] (A_T: stored as [r, K],
// the backward's G = dY B^T). The first ceil(M / 8) clusters quantize one row per CTA. The
// others take 16 tokens, 16 columns of A and 4096 rows of it (512 per CTA, 64 per warp,
// fetched at once: the time is two memory latencies), multiply with mma.sync, and add up
// warps and then CTAs in a fixed order, the CTAs through distributed shared memory. Who reads
// T adds the parts of K above 4096.
constexpr int kPrepThreads = 256;
constexpr int kPrepTok = 16, kPrepCols = 16;
constexpr int kPrepSlice = 512;                    // rows of A per CTA
constexpr int kPrepXPitch = kPrepSlice * 2 + 16;   // bytes; conflict-free for ldmatrix
constexpr int kPrepAPitch = kPrepCols * 2 + 16;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <Fp4 F, bool A_T>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kPrepThreads)
    k_fp4_prep(const uint16_t* X, int M, int64_t K, uint8_t* __restrict__ codes,
               uint8_t* __restrict__ scales, float* __restrict__ gscale, int row_ctas,
               const uint16_t* A, int r, float* __restrict__ T) {
  griddep_wait_and_release();
  __shared__ uint32_t part[16];
  __shared__ __align__(16) uint8_t xs[kPrepTok * kPrepXPitch];
  __shared__ __align__(16) uint8_t as[A_T ? kPrepCols * kPrepXPitch : kPrepSlice * kPrepAPitch];
  __shared__ float mine[kPrepTok * kPrepCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (static_cast<int>(blockIdx.x) < row_ctas) {  // whole clusters, or none
    if (static_cast<int>(blockIdx.x) < M)
      quantize_row<F>(X, blockIdx.x, K, codes, scales, gscale, part);
    return;  // the whole cluster takes this branch: its barrier is not used
  }
  const int jobs_j = (r + kPrepCols - 1) / kPrepCols, jobs_t = (M + kPrepTok - 1) / kPrepTok;
  const int job = (blockIdx.x - row_ctas) / 8, rank = blockIdx.x & 7;
  const int j0 = job % jobs_j * kPrepCols, t0 = job / jobs_j % jobs_t * kPrepTok;
  const int kpart = job / (jobs_j * jobs_t);
  const int64_t k0 = (static_cast<int64_t>(kpart) * 8 + rank) * kPrepSlice;
  const uint32_t xs_s = smem_u32(xs), as_s = smem_u32(as);
#pragma unroll
  for (int u = 0; u < kPrepSlice * kPrepCols / 8 / kPrepThreads; ++u) {
    const int i = tid + u * kPrepThreads;
    if (A_T) {  // 16 rows of 512 columns
      const int j = i / (kPrepSlice / 8), k = i % (kPrepSlice / 8) * 8;
      const bool in = k0 + k < K && j0 + j < r;
      cp_async16(as_s + j * kPrepXPitch + k * 2, in ? A + (j0 + j) * K + k0 + k : A, in);
    } else {    // 512 rows of 16 columns
      const int k = i >> 1, j = (i & 1) * 8;
      const bool in = k0 + k < K && j0 + j < r;
      cp_async16(as_s + k * kPrepAPitch + j * 2, in ? A + (k0 + k) * r + j0 + j : A, in);
    }
  }
#pragma unroll
  for (int u = 0; u < kPrepTok * kPrepSlice / 8 / kPrepThreads; ++u) {
    const int i = tid + u * kPrepThreads, t = i / (kPrepSlice / 8), k = i % (kPrepSlice / 8) * 8;
    const bool in = t0 + t < M && k0 + k < K;
    cp_async16(xs_s + t * kPrepXPitch + k * 2, in ? X + (t0 + t) * K + k0 + k : X, in);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float acc[2][4] = {};
#pragma unroll
  for (int i = 0; i < kPrepSlice / 8 / 16; ++i) {
    const int k = warp * (kPrepSlice / 8) + i * 16;
    uint32_t a[4], b[4];
    ldmatrix_x4(xs_s + (lane & 15) * kPrepXPitch + (k + (lane >> 4) * 8) * 2, a);
    if (A_T)  // matrices: (columns 0-7, k 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
      ldmatrix_x4(as_s + ((lane & 7) + (lane >> 4) * 8) * kPrepXPitch + (k + ((lane >> 3) & 1) * 8) * 2, b);
    else
      ldmatrix_x4_trans(as_s + (k + (lane & 15)) * kPrepAPitch + (lane >> 4) * 16, b);
    mma_16816(acc[0], a, b[0], b[1]);
    mma_16816(acc[1], a, b[2], b[3]);
  }
  __syncthreads();  // the tokens have been read: their memory takes the warps' sums
  float* sums = reinterpret_cast<float*>(xs);  // [8][16 tokens][16]
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sums[warp * 256 + ((lane >> 2) + (e >> 1) * 8) * 16 + h * 8 + (lane & 3) * 2 + (e & 1)] = acc[h][e];
  __syncthreads();
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) v += sums[w * 256 + tid];
  mine[tid] = v;
  cluster_sync_all();
  if (rank == 0) {
    v = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) v += ld_cluster_f32(mine + tid, c);
    const int t = t0 + (tid >> 4), j = j0 + (tid & 15);
    if (t < M && j < r) T[(static_cast<int64_t>(kpart) * M + t) * r + j] = v;
  }
  cluster_sync_all();  // no CTA leaves while its sums are being read
}
static_assert(kPrepTok * kPrepCols == kPrepThreads && 8 * 256 * 4 <= kPrepTok * kPrepXPitch, "sums");

// Few tokens: dA [K, r] = scale X^T G and dB [r, N] = scale T^T dY, G and T fp32 in parts
// [parts][M][r]. A CTA takes 64 columns of X (or of dY) and all of the rank, in passes of 32
// tokens whose successors are fetched meanwhile; a warp 16 x 32 outputs with mma.sync, G (T)
// as three bf16 parts, which hold an fp32 value to its last bit. The first part has sums of its
// own: where one is not finite it is the result, since it has the infinities with their signs, while a
// lower part may be 0 times an infinity or have the other sign. At 128 tokens an FMA version
// was bound by shared memory (12 us for r = 64, K = N = 4096).
constexpr int kGradCols = 64, kGradTok = 32, kGradPitch = 64 * 2 + 16;
__global__ void __launch_bounds__(256)
    k_fp4_small_grads(const uint16_t* X, const uint16_t* dY, int M, int64_t K,
                      int64_t N, const float* G, int g_parts, const float* T,
                      int t_parts, int r, float scale, float* __restrict__ dA, float* __restrict__ dB) {
  griddep_wait_and_release();
  __shared__ __align__(16) uint8_t xs[kGradTok * kGradPitch], vs[3][kGradTok * kGradPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t k_ctas = (K + kGradCols - 1) / kGradCols;
  const bool second = blockIdx.x >= k_ctas;
  const int64_t C = second ? N : K, c0 = (blockIdx.x - (second ? k_ctas : 0)) * kGradCols;
  const uint16_t* src = second ? dY : X;
  const float* val = second ? T : G;
  const int parts = second ? t_parts : g_parts;
  const int lt = tid >> 3, lc = (tid & 7) * 8;  // what this thread stages: token, eight columns
  uint4 w;
  float v[8];
  auto fetch = [&](int m0) {
    const bool in = m0 + lt < M;
    w = make_uint4(0u, 0u, 0u, 0u);
    if (in && c0 + lc < C) w = *reinterpret_cast<const uint4*>(src + (m0 + lt) * C + c0 + lc);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (in && lc < r) {
      const float* p = val + static_cast<int64_t>(m0 + lt) * r + lc;
#pragma unroll 2
      for (int i = 0; i < parts; ++i, p += static_cast<int64_t>(M) * r) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
    }
  };
  const int wc = (warp & 3) * 16, wj = (warp >> 2) * 32;  // this warp's outputs
  const uint32_t xa = smem_u32(xs) + (((lane >> 4) * 8 + (lane & 7)) * kGradPitch + (wc + ((lane >> 3) & 1) * 8) * 2);
  const uint32_t va = smem_u32(vs[0]) + ((lane & 15) * kGradPitch + (wj + (lane >> 4) * 8) * 2);
  float acc[4][4] = {}, low[4][4] = {};  // of the first part, of the others
  fetch(0);
  for (int m0 = 0; m0 < M; m0 += kGradTok) {
    __syncthreads();
    *reinterpret_cast<uint4*>(xs + lt * kGradPitch + lc * 2) = w;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = pack_bf16x2_rn(v[2 * i], v[2 * i + 1]);
        v[2 * i] -= __uint_as_float(q[i] << 16);
        v[2 * i + 1] -= __uint_as_float(q[i] & 0xFFFF0000u);
      }
      *reinterpret_cast<uint4*>(vs[part] + lt * kGradPitch + lc * 2) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    __syncthreads();
    if (m0 + kGradTok < M) fetch(m0 + kGradTok);
    if (wj < r) {
#pragma unroll
      for (int t = 0; t < kGradTok; t += 16) {
        uint32_t a[4];
        ldmatrix_x4_trans(xa + t * kGradPitch, a);
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t b[4];
            ldmatrix_x4_trans(va + part * (kGradTok * kGradPitch) + t * kGradPitch + h * 32, b);
            mma_16816(part ? low[2 * h] : acc[2 * h], a, b[0], b[1]);
            mma_16816(part ? low[2 * h + 1] : acc[2 * h + 1], a, b[2], b[3]);
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const int64_t c = c0 + wc + (lane >> 2) + 4 * e;  // rows lane / 4 and, for e = 2, eight on
      const int j = wj + i * 8 + (lane & 3) * 2;
      if (c >= C || j >= r) continue;
      const float s0 = scale * (isfinite(acc[i][e]) ? acc[i][e] + low[i][e] : acc[i][e]);
      const float s1 = scale * (isfinite(acc[i][e + 1]) ? acc[i][e + 1] + low[i][e + 1] : acc[i][e + 1]);
      if (!second) {
        *reinterpret_cast<float2*>(dA + c * r + j) = make_float2(s0, s1);
      } else {
        dB[j * N + c] = s0;
        dB[(j + 1) * N + c] = s1;
      }
    }
}

// ------------------------------------------------------------------ weights, square blocks
// Largest finite magnitudes, as fp32 bits, of what each CTA reads: *parts[gridDim.x]. One CTA
// per SM, so that who needs the matrix's maximum has few to join, and nothing has to be zero
// before the launch.
constexpr int kAmaxThreads = 1024;
template <bool BF16>
constexpr int kAmaxChunks = BF16 ? 4 : 2;  // per thread, all in flight: 128 bytes
template <bool BF16>
__global__ void __launch_bounds__(kAmaxThreads)
    k_fp4_amax(const void* W, int64_t chunks, uint32_t* __restrict__ parts) {
  griddep_wait_and_release();
  __shared__ uint32_t part[32];
  uint32_t m = 0u;
  constexpr int64_t kBatch = kAmaxThreads * kAmaxChunks<BF16>;
  for (int64_t c0 = blockIdx.x * kBatch + threadIdx.x; c0 < chunks; c0 += gridDim.x * kBatch) {
    Raw16<BF16> r[kAmaxChunks<BF16>];
#pragma unroll
    for (int u = 0; u < kAmaxChunks<BF16>; ++u) {
      if (c0 + u * kAmaxThreads < chunks) r[u].load(W, (c0 + u * kAmaxThreads) * kChunk);
      else r[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kAmaxChunks<BF16>; ++u) {
      const uint32_t a = r[u].amax();
      m = max(m, a < kInf ? a : finite_amax(r[u]));
    }
  }
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = __reduce_max_sync(~0u, part[threadIdx.x]);
    if (threadIdx.x == 0) parts[blockIdx.x] = m;
  }
}

// Transpose of an 8 x 8 square of nibbles, one word per row: swaps 4 x 4, 2 x 2 and single
// nibbles across the diagonal.
__device__ __forceinline__ void transpose_nibbles(uint32_t (&w)[8]) {
#pragma unroll
  for (int s = 4; s >= 1; s >>= 1) {
    const uint32_t mask = s == 4 ? 0x0000FFFFu : s == 2 ? 0x00FF00FFu : 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & s) continue;
      const uint32_t t = (w[i] >> (4 * s) ^ w[i + s]) & mask;
      w[i + s] ^= t;
      w[i] ^= t << (4 * s);
    }
  }
}

// A CTA is one warp (four were 3-10 % slower in bf16, the same in fp32) and takes 32 rows x
// 64 columns of W, a lane 8 x 8 of it (lane = row group * 8 + column
// group), so that squares of 16 and of 32 are whole in the warp: the maxima go through
// shuffles, the transposed codes through an 8 x 8 nibble transpose in registers. The
// transposed copy has the same squares, so it stores the same values.
template <Fp4 F, bool BF16>
__global__ void __launch_bounds__(32)
    k_fp4_quantize_weight(const void* W, int64_t n, int64_t k,
                          const uint32_t* tops, int ntops, uint8_t* __restrict__ codes,
                          uint8_t* __restrict__ scales, float* __restrict__ gscale,
                          uint8_t* __restrict__ t_codes, uint8_t* __restrict__ t_scales) {
  griddep_wait_and_release();
  constexpr int B = kFp4Block<F>;
  const int lane = threadIdx.x, kl = lane & 7, nl = lane >> 3;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 64;
  // NVFP4: from the last rows, which k_fp4_amax left in L2 (fp32 11008 x 4096: 70.9 us, from
  // the first 75.8)
  const int64_t n0 = static_cast<int64_t>(F == Fp4::kNv ? gridDim.y - 1 - blockIdx.y : blockIdx.y) * 32;
  Gscale g(0);
  if (F == Fp4::kNv) {
    uint32_t top = 0u;
    for (int i = lane; i < ntops; i += 32) top = max(top, tops[i]);
    g = Gscale(nv_gscale_exp(__reduce_max_sync(~0u, top)));
    if (blockIdx.x == 0 && blockIdx.y == 0 && lane == 0) *gscale = g.g;
  }
  const int64_t gk = k0 + kl * 8, gn = n0 + nl * 8;
  const bool in = gk < k;  // n is a multiple of 32, k of 32
  // rows of eight values
  uint4 rb[BF16 ? 8 : 1];
  float4 rf[BF16 ? 1 : 16];
  uint32_t am = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (BF16) {
      rb[i] = make_uint4(0u, 0u, 0u, 0u);
      if (in) rb[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + (gn + i) * k + gk);
    } else {
      rf[2 * i] = rf[2 * i + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + (gn + i) * k + gk);
        rf[2 * i] = p[0];
        rf[2 * i + 1] = p[1];
      }
    }
  }
  auto at = [&](int i, int j) -> float {
    if constexpr (BF16) {
      const uint32_t w = j < 2 ? rb[i].x : j < 4 ? rb[i].y : j < 6 ? rb[i].z : rb[i].w;
      return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
    } else {
      const float4 q = rf[2 * i + (j >> 2)];
      return (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
    }
  };
  if constexpr (BF16) {
    constexpr uint32_t kMag2 = 0x7FFF7FFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      am = __vmaxu2(am, __vmaxu2(__vmaxu2(rb[i].x & kMag2, rb[i].y & kMag2),
                                 __vmaxu2(rb[i].z & kMag2, rb[i].w & kMag2)));
    am = max(am & 0xFFFF0000u, am << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(at(i, j)) & kMag);
  }
  am = max(am, __shfl_xor_sync(~0u, am, 1));
  am = max(am, __shfl_xor_sync(~0u, am, 8));
  if (F == Fp4::kMx) {
    am = max(am, __shfl_xor_sync(~0u, am, 2));
    am = max(am, __shfl_xor_sync(~0u, am, 16));
  }
  const uint32_t sb = in ? scale_byte<F>(am, g.inv) : 0u;
  if (F == Fp4::kNv && g.up != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF16) {
        bf16x2_up64(rb[i].x), bf16x2_up64(rb[i].y), bf16x2_up64(rb[i].z), bf16x2_up64(rb[i].w);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          rf[2 * i + h].x *= 0x1p64f, rf[2 * i + h].y *= 0x1p64f, rf[2 * i + h].z *= 0x1p64f, rf[2 * i + h].w *= 0x1p64f;
      }
    }
  }
  const Encoder<F> enc(sb, g);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = enc.encode8([&](int j) { return at(i, j); });
    if (enc.zero()) w[i] = 0u;
    if (in) *reinterpret_cast<uint32_t*>(codes + ((gn + i) * k + gk) / 2) = w[i];
  }
  if (t_codes) {
    transpose_nibbles(w);
    if (in) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint32_t*>(t_codes + ((gk + j) * n + gn) / 2) = w[j];
    }
  }
  // Scale bytes. Lane l writes row l of W (64 / B blocks) and rows l, l + 32 of the transpose
  // (32 / B blocks). Blocks past the edge but inside the last scale tile are 0: lanes outside
  // have sb = 0, and the warp at the edge fills up what no warp covers.
  const int64_t kt = (k / B + 3) / 4, tt = (n / B + 3) / 4;
  const int src = (lane >> 3) * 8;  // the lane that holds (row lane, column group 0)
  if (F == Fp4::kNv) {
    uint32_t v = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) v |= __shfl_sync(~0u, sb, src + 2 * b) << (8 * b);
    *reinterpret_cast<uint32_t*>(scales + fp4_scale_offset(n0 + lane, k0 / 16, kt)) = v;
  } else {
    const uint32_t v = __shfl_sync(~0u, sb, src) | __shfl_sync(~0u, sb, src + 4) << 8;
    *reinterpret_cast<uint16_t*>(scales + fp4_scale_offset(n0 + lane, k0 / 32, kt)) = static_cast<uint16_t>(v);
    if (k0 + 64 >= k && (k0 / 32) % 4 == 0)
      *reinterpret_cast<uint16_t*>(scales + fp4_scale_offset(n0 + lane, k0 / 32 + 2, kt)) = 0;
  }
  if (!t_codes) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = lane + 32 * h, from = row >> 3;  // column group of W's lane 0..7
    if (F == Fp4::kNv) {
      const uint32_t v = __shfl_sync(~0u, sb, from) | __shfl_sync(~0u, sb, from + 16) << 8;
      if (k0 + row < k) {
        *reinterpret_cast<uint16_t*>(t_scales + fp4_scale_offset(k0 + row, n0 / 16, tt)) = static_cast<uint16_t>(v);
        if (n0 + 32 >= n && (n0 / 16) % 4 == 0)
          *reinterpret_cast<uint16_t*>(t_scales + fp4_scale_offset(k0 + row, n0 / 16 + 2, tt)) = 0;
      }
    } else {
      const uint32_t v = __shfl_sync(~0u, sb, from);
      if (k0 + row < k) {
        t_scales[fp4_scale_offset(k0 + row, n0 / 32, tt)] = static_cast<uint8_t>(v);
        if (n0 + 32 >= n)
          for (int64_t b = n0 / 32 + 1; b < tt * 4; ++b) t_scales[fp4_scale_offset(k0 + row, b, tt)] = 0;
      }
    }
  }
}

// ------------------------------------------------------------------ reading back
// A warp takes 1024 columns of one row in strides of 32 lanes; a lane's share of a stride is
// 16 bytes of output. Neighbouring warps take neighbouring rows, whose scale bytes share
// sectors. value = fl32(fl32(code * scale) * gscale); the first product is exact (1 + 3
// mantissa bits), then one rounding to bf16 where asked.
template <Fp4 F, bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_dequant(const uint8_t* codes, const uint8_t* scales,
                  const float* gscale, bool g_per_row, uint32_t rows, int64_t cols,
                  int64_t ktiles, void* __restrict__ out) {
  griddep_wait_and_release();
  constexpr int V = BF16 ? 8 : 4;          // values per lane and stride
  constexpr int U = 1024 / (32 * V);       // strides
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const float g = gscale ? gscale[g_per_row ? row : 0] : 1.f;
  const uint64_t g2 = f2_pack(g, g);
  for (int64_t c0 = static_cast<int64_t>(blockIdx.y) * 1024; c0 < cols; c0 += static_cast<int64_t>(gridDim.y) * 1024) {
    uint32_t w[U], sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = c0 + (u * 32 + lane) * V;
      w[u] = sb[u] = 0u;
      if (col < cols) {
        const uint8_t* src = codes + (row * cols + col) / 2;
        w[u] = BF16 ? *reinterpret_cast<const uint32_t*>(src) : *reinterpret_cast<const uint16_t*>(src);
        sb[u] = scales[fp4_scale_offset(row, col / kFp4Block<F>, ktiles)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = c0 + (u * 32 + lane) * V;
      if (col >= cols) break;
      const float s = fp4_scale_value<F>(sb[u]);
      const uint64_t s2 = f2_pack(s, s);
      float v[V];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 f = e2m1_pair(w[u] >> (8 * j));
        uint64_t x = f2_mul(f2_pack(f.x, f.y), s2);
        if (F == Fp4::kNv || gscale) x = f2_mul(x, g2);  // MXFP4 has none as a rule
        f2_unpack(x, v[2 * j], v[2 * j + 1]);
      }
      if constexpr (BF16)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * cols + col) =
            make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                       pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(out) + row * cols + col) =
            make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

constexpr int64_t kMaxGridY = 65535;

template <bool BF16>
cudaError_t quantize_rows(const void* X, int64_t rows, int64_t cols, int format, uint8_t* codes,
                          uint8_t* scales, float* gscale, cudaStream_t st) {
  if (format == QLORA_FP4_MX) {
    // bf16: two segments a warp where that leaves eight CTAs for each SM (8192 x 11008: 38.3 us
    // against 39.8; 1000 x 4096: 3.8 against 3.2); fp32 is 2 % slower so
    const int64_t segs = (cols + 511) / 512, half = (segs + 1) / 2;
    const bool two = BF16 && (rows + 7) / 8 * half >= 8 * static_cast<int64_t>(num_sms());
    const dim3 grid(static_cast<unsigned>((rows + 7) / 8),
                    static_cast<unsigned>(std::min(two ? half : segs, kMaxGridY)));
    return launch_pdl(k_fp4_quantize_mx<BF16>, grid, dim3(256), 0, st, X,
                      static_cast<uint32_t>(rows), cols, codes, scales);
  }
  // Chunks a thread, while the row fits the registers: two, as more and smaller CTAs cover each
  // other's barriers (bf16 4096 x 4096: 9.1 us, 12.8 with one chunk and 256 threads, 10.3 with
  // four), four where two take more than 512 threads. Up to 1024 columns one, for at least a
  // warp or two (8192 x 1024: 7.3 us; two chunks 9.2).
  const int64_t padded = (cols / kChunk + 3) & ~int64_t{3};
  const int u = padded <= 64 ? 1 : padded <= 1024 ? 2 : padded <= 2048 && BF16 ? 4 : 0;
  const int threads = u == 0 ? 512 : static_cast<int>(((padded + u - 1) / u + 31) / 32 * 32);
  auto kern = u == 1   ? k_fp4_quantize_nv<BF16, 1>
              : u == 2 ? k_fp4_quantize_nv<BF16, 2>
              : u == 4 ? k_fp4_quantize_nv<BF16, BF16 ? 4 : 0>
                       : k_fp4_quantize_nv<BF16, 0>;
  // A CTA a row; as many CTAs as run at one time (32 an SM at most: 8192 x 512 takes 5.4 us, 7.8
  // with 48), each taking several rows, where a row is short (they fetch the next one ahead;
  // 4096 x 1024: 4.4 us against 4.8) and where the 64 registers of fp32 leave room for few CTAs, two
  // from 352 threads on (8192 x 11008: 74 us against 79, 4096 x 16384 48.5 against 53.0;
  // 4096 x 8192, 256 threads: 28.0 against 24.8).
  const bool resident = u == 1 || (u > 0 && !BF16 && threads > 256);
  const int64_t at_once = static_cast<int64_t>(num_sms()) * std::min(32, (u == 1 ? 1536 : 1024) / threads);
  const int64_t grid = resident ? std::min(rows, at_once) : rows;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, st, X,
                    static_cast<uint32_t>(rows), cols, codes, scales, gscale);
}

template <bool BF16>
cudaError_t quantize_weight(const void* W, int64_t n, int64_t k, int format, const Fp4Out& w,
                            const Fp4Out& wt, uint32_t* tops, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((k + 63) / 64), static_cast<unsigned>(n / 32));
  if (format == QLORA_FP4_MX)
    return launch_pdl(k_fp4_quantize_weight<Fp4::kMx, BF16>, grid, dim3(32), 0, st, W, n, k,
                      static_cast<const uint32_t*>(nullptr), 0, w.codes, w.scales, w.gscale, wt.codes,
                      wt.scales);
  const int64_t chunks = n * k / kChunk, batch = kAmaxThreads * kAmaxChunks<BF16>;
  const int ctas = static_cast<int>(std::min<int64_t>({(chunks + batch - 1) / batch, num_sms(), kFp4MaxTops}));
  const cudaError_t e = launch_pdl(k_fp4_amax<BF16>, dim3(ctas), dim3(kAmaxThreads), 0, st, W, chunks, tops);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_fp4_quantize_weight<Fp4::kNv, BF16>, grid, dim3(32), 0, st, W, n, k,
                    static_cast<const uint32_t*>(tops), ctas, w.codes, w.scales, w.gscale, wt.codes,
                    wt.scales);
}

}  // namespace

int64_t fp4_ktiles(int64_t cols, int format) {
  const int64_t b = format == QLORA_FP4_MX ? 32 : 16;
  return (cols / b + 3) / 4;
}

cudaError_t launch_fp4_quantize(const void* X, bool bf16, int64_t rows, int64_t cols, int format,
                                const Fp4Out& out, cudaStream_t st) {
  return bf16 ? quantize_rows<true>(X, rows, cols, format, out.codes, out.scales, out.gscale, st)
              : quantize_rows<false>(X, rows, cols, format, out.codes, out.scales, out.gscale, st);
}

cudaError_t launch_fp4_quantize_weight(const void* W, bool bf16, int64_t n, int64_t k, int format,
                                       const Fp4Out& w, const Fp4Out& wt, void* ws,
                                       cudaStream_t st) {
  uint32_t* tops = static_cast<uint32_t*>(ws);
  return bf16 ? quantize_weight<true>(W, n, k, format, w, wt, tops, st)
              : quantize_weight<false>(W, n, k, format, w, wt, tops, st);
}

int fp4_prep_parts(int64_t K) { return static_cast<int>((K + 8 * kPrepSlice - 1) / (8 * kPrepSlice)); }

cudaError_t launch_fp4_prep(const uint16_t* X, int64_t M, int64_t K, int format, const Fp4Out* out,
                            const uint16_t* A, bool a_t, int r, float* T, cudaStream_t st) {
  const int m = static_cast<int>(M), row_ctas = out ? (m + 7) / 8 * 8 : 0;
  const int jobs = (m + kPrepTok - 1) / kPrepTok * ((r + kPrepCols - 1) / kPrepCols) * fp4_prep_parts(K);
  auto kern = format == QLORA_FP4_MX ? (a_t ? k_fp4_prep<Fp4::kMx, true> : k_fp4_prep<Fp4::kMx, false>)
                                     : (a_t ? k_fp4_prep<Fp4::kNv, true> : k_fp4_prep<Fp4::kNv, false>);
  const Fp4Out o = out ? *out : Fp4Out{};
  return launch_pdl(kern, dim3(row_ctas + 8 * jobs), dim3(kPrepThreads), 0, st, X, m, K, o.codes,
                    o.scales, o.gscale, row_ctas, A, r, T);
}

cudaError_t launch_fp4_small_grads(const uint16_t* X, const uint16_t* dY, int64_t M, int64_t K, int64_t N,
                                   const float* G, int g_parts, const float* T, int t_parts, int r,
                                   float scale, float* dA, float* dB, cudaStream_t st) {
  const int64_t ctas = (K + kGradCols - 1) / kGradCols + (N + kGradCols - 1) / kGradCols;
  return launch_pdl(k_fp4_small_grads, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, st, X, dY,
                    static_cast<int>(M), K, N, G, g_parts, T, t_parts, r, scale, dA, dB);
}

cudaError_t launch_fp4_dequant(const qlora_fp4_matrix& q, bool bf16, void* out, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((q.rows + 7) / 8),
                  static_cast<unsigned>(std::min((q.cols + 1023) / 1024, kMaxGridY)));
  auto kern = q.format == QLORA_FP4_MX
                  ? (bf16 ? k_fp4_dequant<Fp4::kMx, true> : k_fp4_dequant<Fp4::kMx, false>)
                  : (bf16 ? k_fp4_dequant<Fp4::kNv, true> : k_fp4_dequant<Fp4::kNv, false>);
  return launch_pdl(kern, grid, dim3(256), 0, st, q.codes, q.scales, q.gscale, q.gscale_rows > 1,
                    static_cast<uint32_t>(q.rows), q.cols, fp4_ktiles(q.cols, q.format), out);
}

}  // namespace qlora
