// fp4_codec.cu -- quantization to microscaled 4-bit floating point and reading back.
//
// MXFP4 (blocks of 32 along a row):  e = floor(log2 amax) - 2 clamped to [-127, 127] (-127 for
//   amax = 0), scale byte e + 127, code = e2m1(x 2^-e).
// NVFP4 (blocks of 16): g = 2^e with the smallest e for which top <= 2688 * 2^e, top being the
//   largest magnitude of the row (activations) or of the matrix (weights); g = 1 for top = 0;
//   scale byte c = e4m3(amax / g / 6), code = e2m1(x / g / c), 0 where c = 0.
// e2m1() and e4m3() round to nearest, ties to even, and saturate. With g a power of two the
// only inexact steps are those roundings: x / g is exact, and the fp32 quotients amax / 6 and
// x / c are correctly rounded and land on a rounding border only when the real quotient does
// (numerator and border times divisor are both fp32 numbers, so a real quotient off the border
// is off by more than half an fp32 ulp). Codes and scales are therefore those of the
// definition in real arithmetic.
// A block that holds a NaN or an infinity gets the NaN scale and zero codes; its non-finite
// values do not enter top.
#include <cuda_bf16.h>

#include <algorithm>

#include "fp4_device.cuh"

namespace qlora {
namespace {

constexpr int kChunk = 16;  // values per thread and step: 32 bytes of bf16, 64 of fp32

struct Raw16Bf { uint4 a, b; };
struct Raw16F { float4 a, b, c, d; };
template <bool BF16> struct RawOf { using T = Raw16Bf; };
template <> struct RawOf<false> { using T = Raw16F; };

template <bool BF16>
__device__ __forceinline__ typename RawOf<BF16>::T load16(const void* base, int64_t elem) {
  typename RawOf<BF16>::T r;
  if constexpr (BF16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
    r.a = __ldg(p);
    r.b = __ldg(p + 1);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    r.a = __ldg(p);
    r.b = __ldg(p + 1);
    r.c = __ldg(p + 2);
    r.d = __ldg(p + 3);
  }
  return r;
}
__device__ __forceinline__ void expand2(uint32_t w, float* v) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void expand(const Raw16Bf& r, float (&v)[16]) {
  expand2(r.a.x, v), expand2(r.a.y, v + 2), expand2(r.a.z, v + 4), expand2(r.a.w, v + 6);
  expand2(r.b.x, v + 8), expand2(r.b.y, v + 10), expand2(r.b.z, v + 12), expand2(r.b.w, v + 14);
}
__device__ __forceinline__ void expand(const Raw16F& r, float (&v)[16]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
  v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
  v[8] = r.c.x, v[9] = r.c.y, v[10] = r.c.z, v[11] = r.c.w;
  v[12] = r.d.x, v[13] = r.d.y, v[14] = r.d.z, v[15] = r.d.w;
}

// Largest finite magnitude (fp32 bits) of 16 values; bit 31 is set when one is not finite.
__device__ __forceinline__ uint32_t amax16(const float (&v)[16]) {
  uint32_t m = 0u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, finite_mag(v[i], bad));
  return bad ? m | 0x80000000u : m;
}
constexpr uint32_t kMag = 0x7FFFFFFFu;
// Combines two amax16 results.
__device__ __forceinline__ uint32_t amax_join(uint32_t a, uint32_t b) {
  return max(a & kMag, b & kMag) | ((a | b) & 0x80000000u);
}

// Scale byte of a block from its amax16; g_inv = 1 / gscale (NVFP4).
template <Fp4 F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t am, float g_inv) {
  if (am & 0x80000000u) return kFp4NanScale<F>;
  if (F == Fp4::kMx) {
    const int biased = static_cast<int>(am >> 23) - 2;  // floor(log2) - 2 + 127
    return static_cast<uint32_t>(max(biased, 0));       // zero and subnormal maxima: 2^-127
  }
  return e4m3_bits(__fdiv_rn(__uint_as_float(am) * g_inv, 6.f));
}

// Codes of 16 values under one scale byte (low nibble first).
template <Fp4 F>
__device__ __forceinline__ uint2 codes16(const float (&v)[16], uint32_t sb, float g_inv) {
  if (sb == kFp4NanScale<F> || (F == Fp4::kNv && sb == 0u)) return make_uint2(0u, 0u);
  float y[16];
  if (F == Fp4::kMx) {
    const float inv = pow2_f32(127 - static_cast<int>(sb));
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = v[i] * inv;
  } else {
    const float c = fp4_scale_value<F>(sb);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(v[i] * g_inv, c);
  }
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = y[i], hi[i] = y[8 + i];
  return make_uint2(fp4_pack8(lo), fp4_pack8(hi));
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
// A warp takes 512 columns of one row, 16 per lane.
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_quantize_mx(const void* __restrict__ X, int64_t rows, int64_t cols, int segs,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_wait_and_release();
  const int lane = threadIdx.x & 31;
  const int64_t task = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t row = task / segs;
  if (row >= rows) return;
  const int64_t col = (task - row * segs) * 512 + lane * kChunk;
  const bool in = col < cols;
  float v[16] = {};
  if (in) expand(load16<BF16>(X, row * cols + col), v);
  uint32_t am = amax16(v);
  am = amax_join(am, __shfl_xor_sync(~0u, am, 1));
  const uint32_t sb = in ? scale_byte<Fp4::kMx>(am, 1.f) : 0u;
  if (in)
    *reinterpret_cast<uint2*>(codes + (row * cols + col) / 2) = codes16<Fp4::kMx>(v, sb, 1.f);
  const uint32_t w = gather4<Fp4::kMx>(sb);
  if ((lane & 7) == 0 && in)
    *reinterpret_cast<uint32_t*>(
        scales + fp4_scale_offset(row, col / 32, (cols + 127) / 128)) = w;
}

// ------------------------------------------------------------------ NVFP4 rows
// One CTA per row; the row stays in registers (U chunks a thread) between the row maximum
// and the codes. U = 0: rows too long for that are read twice.
template <bool BF16, int U>
__global__ void __launch_bounds__(256)
    k_fp4_quantize_nv(const void* __restrict__ X, int64_t cols, uint8_t* __restrict__ codes,
                      uint8_t* __restrict__ scales, float* __restrict__ gscale) {
  griddep_wait_and_release();
  __shared__ uint32_t part[8];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t row = blockIdx.x;
  const int64_t chunks = cols / kChunk, padded = (chunks + 3) & ~int64_t{3};
  typename RawOf<BF16>::T raw[U > 0 ? U : 1];
  uint32_t top = 0u;
  if constexpr (U > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = tid + static_cast<int64_t>(u) * nt;
      if (c < chunks) raw[u] = load16<BF16>(X, row * cols + c * kChunk);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = tid + static_cast<int64_t>(u) * nt;
      if (c < chunks) {
        float v[16];
        expand(raw[u], v);
        top = max(top, amax16(v) & kMag);
      }
    }
  } else {
    for (int64_t c = tid; c < chunks; c += nt) {
      float v[16];
      expand(load16<BF16>(X, row * cols + c * kChunk), v);
      top = max(top, amax16(v) & kMag);
    }
  }
  top = __reduce_max_sync(~0u, top);
  if ((tid & 31) == 0) part[tid >> 5] = top;
  __syncthreads();
  for (int w = 0; w < (nt >> 5); ++w) top = max(top, part[w]);
  const int e = nv_gscale_exp(top);
  if (tid == 0) gscale[row] = pow2_f32(e);
  const float g_inv = pow2_f32(-e);
  const int64_t ktiles = padded / 4;
  auto emit = [&](int64_t c, const float (&v)[16], bool in) {
    const uint32_t sb = in ? scale_byte<Fp4::kNv>(amax16(v), g_inv) : 0u;
    if (in)
      *reinterpret_cast<uint2*>(codes + (row * cols + c * kChunk) / 2) =
          codes16<Fp4::kNv>(v, sb, g_inv);
    const uint32_t w = gather4<Fp4::kNv>(sb);
    if ((c & 3) == 0 && c < padded)
      *reinterpret_cast<uint32_t*>(scales + fp4_scale_offset(row, c, ktiles)) = w;
  };
  if constexpr (U > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = tid + static_cast<int64_t>(u) * nt;
      if (c - tid >= padded) break;  // the same in every thread
      float v[16] = {};
      if (c < chunks) expand(raw[u], v);
      emit(c, v, c < chunks);
    }
  } else {
    for (int64_t c = tid; c - tid < padded; c += nt) {
      float v[16] = {};
      if (c < chunks) expand(load16<BF16>(X, row * cols + c * kChunk), v);
      emit(c, v, c < chunks);
    }
  }
}

// ------------------------------------------------------------------ weights, square blocks
// Largest finite magnitude of the matrix, as fp32 bits in *top (zero before the launch).
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_amax(const void* __restrict__ W, int64_t chunks, uint32_t* __restrict__ top) {
  griddep_wait_and_release();
  uint32_t m = 0u;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; c < chunks;
       c += stride) {
    float v[16];
    expand(load16<BF16>(W, c * kChunk), v);
    m = max(m, amax16(v) & kMag);
  }
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0 && m) atomicMax(top, m);  // a maximum: no order to depend on
}

// A 64 x 64 tile of W: block scales from the maxima of b x b squares, codes written once
// along the rows and, through shared memory, once along the columns (the transposed copy
// has the same squares, so it stores the same values).
template <Fp4 F, bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_quantize_weight(const void* __restrict__ W, int64_t n, int64_t k,
                          const uint32_t* __restrict__ top, uint8_t* __restrict__ codes,
                          uint8_t* __restrict__ scales, float* __restrict__ gscale,
                          uint8_t* __restrict__ t_codes, uint8_t* __restrict__ t_scales) {
  griddep_wait_and_release();
  constexpr int B = kFp4Block<F>;
  constexpr int NB = 64 / B;               // blocks along a side of the tile
  __shared__ uint32_t part[8][4];          // maxima of 8 rows x 16 columns
  __shared__ uint8_t sbs[4][4];            // scale bytes of the tile's squares
  __shared__ uint8_t tile[64][64 + 4];     // codes, one per byte: [row][column]
  const int tid = threadIdx.x, row = tid >> 2, seg = tid & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * 64, k0 = static_cast<int64_t>(blockIdx.x) * 64;
  float g_inv = 1.f;
  if (F == Fp4::kNv) {
    const int e = nv_gscale_exp(*top);
    g_inv = pow2_f32(-e);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *gscale = pow2_f32(e);
  }
  const int64_t gn = n0 + row, gk = k0 + seg * 16;
  const bool in = gn < n && gk < k;
  float v[16] = {};
  if (in) expand(load16<BF16>(W, gn * k + gk), v);
  uint32_t am = amax16(v);
  am = amax_join(am, __shfl_xor_sync(~0u, am, 4));
  am = amax_join(am, __shfl_xor_sync(~0u, am, 8));
  am = amax_join(am, __shfl_xor_sync(~0u, am, 16));
  if ((tid & 31) < 4) part[tid >> 5][seg] = am;
  __syncthreads();
  if (tid < NB * NB) {
    const int br = tid / NB, bc = tid % NB;
    uint32_t m = 0u;
    for (int i = 0; i < B / 8; ++i)
      for (int j = 0; j < B / 16; ++j) m = amax_join(m, part[br * (B / 8) + i][bc * (B / 16) + j]);
    sbs[br][bc] = static_cast<uint8_t>(scale_byte<F>(m, g_inv));
  }
  __syncthreads();
  const uint2 q = codes16<F>(v, sbs[row / B][seg * 16 / B], g_inv);
  if (in) *reinterpret_cast<uint2*>(codes + (gn * k + gk) / 2) = q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // word of four codes, one per byte
    const uint32_t w16 = ((i & 2) ? q.y : q.x) >> ((i & 1) * 16);
    *reinterpret_cast<uint32_t*>(&tile[row][seg * 16 + i * 4]) =
        (w16 & 0xFu) | (w16 & 0xF0u) << 4 | (w16 & 0xF00u) << 8 | (w16 & 0xF000u) << 12;
  }
  // scale bytes: NB per row of the tile and, transposed, NB per column. Blocks of 16: the
  // tile is one scale tile wide (four blocks); blocks of 32: half of one. Blocks past the
  // edge of W but inside its last scale tile are written as zeros.
  if (tid < 64) {
    const int64_t ktiles = (k / B + 3) / 4;
    if (n0 + tid < n) {
      for (int b = 0; b < NB; ++b) {
        const int64_t blk = k0 / B + b;
        if (blk < ktiles * 4)
          scales[fp4_scale_offset(n0 + tid, blk, ktiles)] = blk * B < k ? sbs[tid / B][b] : 0;
      }
      if (F == Fp4::kMx && k0 + 64 >= k)  // the rest of the last tile's four blocks
        for (int64_t blk = k0 / B + NB; blk < ktiles * 4; ++blk)
          scales[fp4_scale_offset(n0 + tid, blk, ktiles)] = 0;
    }
  } else if (tid < 128 && t_codes) {
    const int c = tid - 64;
    const int64_t ktiles = (n / B + 3) / 4;
    if (k0 + c < k) {
      for (int b = 0; b < NB; ++b) {
        const int64_t blk = n0 / B + b;
        if (blk < ktiles * 4)
          t_scales[fp4_scale_offset(k0 + c, blk, ktiles)] = blk * B < n ? sbs[b][c / B] : 0;
      }
      if (F == Fp4::kMx && n0 + 64 >= n)
        for (int64_t blk = n0 / B + NB; blk < ktiles * 4; ++blk)
          t_scales[fp4_scale_offset(k0 + c, blk, ktiles)] = 0;
    }
  }
  if (!t_codes) return;
  __syncthreads();
  // column c of the tile, 16 rows from r0: eight bytes of the transposed codes
  const int c = tid >> 2, r0 = (tid & 3) * 16;
  if (k0 + c < k && n0 + r0 < n) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 3] |= static_cast<uint32_t>(tile[r0 + i][c]) << (4 * (i & 7));
    *reinterpret_cast<uint2*>(t_codes + ((k0 + c) * n + n0 + r0) / 2) = make_uint2(w[0], w[1]);
  }
}

// ------------------------------------------------------------------ reading back
// A lane takes eight columns of one row. value = fl32(fl32(code * scale) * gscale); the first
// product is exact (1 + 3 mantissa bits), then one rounding to bf16 where asked.
template <Fp4 F, bool BF16>
__global__ void __launch_bounds__(256)
    k_fp4_dequant(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                  const float* __restrict__ gscale, bool g_per_row, int64_t rows, int64_t cols,
                  int64_t ktiles, void* __restrict__ out) {
  griddep_wait_and_release();
  const int64_t per_row = cols / 8, total = rows * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int64_t row = i / per_row, col = (i - row * per_row) * 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const float s = fp4_scale_value<F>(__ldg(scales + fp4_scale_offset(row, col / kFp4Block<F>, ktiles)));
    const float g = gscale ? __ldg(gscale + (g_per_row ? row : 0)) : 1.f;
    uint32_t h[4];
    fp4_unpack8(w, h);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
          "cvt.f32.f16 %1, hi;\n\t}"
          : "=f"(v[2 * j]), "=f"(v[2 * j + 1])
          : "r"(h[j]));
      v[2 * j] = v[2 * j] * s * g;
      v[2 * j + 1] = v[2 * j + 1] * s * g;
    }
    if (BF16) {
      reinterpret_cast<uint4*>(out)[i] =
          make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                     pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

template <bool BF16>
cudaError_t quantize_rows(const void* X, int64_t rows, int64_t cols, int format, uint8_t* codes,
                          uint8_t* scales, float* gscale, cudaStream_t st) {
  if (format == QLORA_FP4_MX) {
    const int segs = static_cast<int>((cols + 511) / 512);
    const int64_t blocks = (rows * segs + 7) / 8;
    return launch_pdl(k_fp4_quantize_mx<BF16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                      st, X, rows, cols, segs, codes, scales);
  }
  const int64_t padded = (cols / kChunk + 3) & ~int64_t{3};
  const int threads = static_cast<int>(std::min<int64_t>(256, (padded + 31) / 32 * 32));
  const int64_t u = (padded + threads - 1) / threads;
  auto kern = u <= 1   ? k_fp4_quantize_nv<BF16, 1>
              : u <= 2 ? k_fp4_quantize_nv<BF16, 2>
              : u <= 4 ? k_fp4_quantize_nv<BF16, 4>
                       : k_fp4_quantize_nv<BF16, 0>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(rows)), dim3(threads), 0, st, X, cols, codes,
                    scales, gscale);
}

template <bool BF16>
cudaError_t quantize_weight(const void* W, int64_t n, int64_t k, int format, const Fp4Out& w,
                            const Fp4Out& wt, uint32_t* top, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((k + 63) / 64), static_cast<unsigned>((n + 63) / 64));
  if (format == QLORA_FP4_MX)
    return launch_pdl(k_fp4_quantize_weight<Fp4::kMx, BF16>, grid, dim3(256), 0, st, W, n, k,
                      static_cast<const uint32_t*>(nullptr), w.codes, w.scales, w.gscale, wt.codes,
                      wt.scales);
  cudaError_t e = cudaMemsetAsync(top, 0, sizeof(uint32_t), st);
  if (e != cudaSuccess) return e;
  const int64_t chunks = n * k / kChunk;
  const int64_t blocks = std::min<int64_t>((chunks + 255) / 256, static_cast<int64_t>(num_sms()) * 8);
  e = launch_pdl(k_fp4_amax<BF16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, W, chunks,
                 top);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_fp4_quantize_weight<Fp4::kNv, BF16>, grid, dim3(256), 0, st, W, n, k,
                    static_cast<const uint32_t*>(top), w.codes, w.scales, w.gscale, wt.codes,
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
  uint32_t* top = static_cast<uint32_t*>(ws);
  return bf16 ? quantize_weight<true>(W, n, k, format, w, wt, top, st)
              : quantize_weight<false>(W, n, k, format, w, wt, top, st);
}

cudaError_t launch_fp4_dequant(const qlora_fp4_matrix& q, bool bf16, void* out, cudaStream_t st) {
  const int64_t total = q.rows * (q.cols / 8);
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, static_cast<int64_t>(num_sms()) * 16);
  auto kern = q.format == QLORA_FP4_MX
                  ? (bf16 ? k_fp4_dequant<Fp4::kMx, true> : k_fp4_dequant<Fp4::kMx, false>)
                  : (bf16 ? k_fp4_dequant<Fp4::kNv, true> : k_fp4_dequant<Fp4::kNv, false>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, q.codes, q.scales,
                    q.gscale, q.gscale_rows > 1, q.rows, q.cols, fp4_ktiles(q.cols, q.format), out);
}

}  // namespace qlora
