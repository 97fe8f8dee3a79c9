// E4M3 with f32 block scales: rows (one scale per 128 inputs), rows through SwiGLU, and weights
// (one scale per 128 x 128 tile).
//
// For the values v of a block, all steps in f32:
//   m = max(max |v|, 2^-100),  scale = m / 448,  code = e4m3(v * (448 / m))
// rounded to nearest even.  448 is the largest E4M3 value; the product of the largest value is
// 448 (1 +- 2^-23), which rounds to 448.  2^-100 keeps 448 / m finite and the scale a normal
// number; a block of zeros gets zero codes.  A NaN in a block, or an infinity, makes every product
// with the block NaN (scale NaN and codes NaN, or scale infinite and codes 0 or NaN).
//
// One pass over the data: a thread holds 16 values of a block (one 32-byte load, or two of 16 bytes where the rows
// start off a 32-byte boundary; one 16-byte store), eight threads a row block, and the block's maximum is a butterfly
// over them.  The SiLU takes the hardware exponential and reciprocal (with the exact ones the arithmetic, not the
// memory, set the time); where a product lies nearer to the border between two codes than that can be off, or a block
// has an up that can outweigh what they lose of a far negative gate, 64 bits decide.
#define MOE_OWN_STATUS
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kRowThreads = 128;
constexpr float kTop = 448.0f;
constexpr float kLeast = 0x1p-100f;

// max(|bits|, floor) of a block's largest |f32| pattern: patterns of magnitudes order like the
// values, with infinities and NaN on top.
__device__ __forceinline__ float block_max(uint32_t abs_bits) {
  return __uint_as_float(max(abs_bits, __float_as_uint(kLeast)));
}

// Four E4M3 codes of four f32 values, nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint4 e4m3x16(const float (&p)[16]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = e4m3x4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}
// The largest magnitude; NaN where there is one (three operands a step).
__device__ __forceinline__ float abs_max16(const float (&v)[16]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 15; i += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[i]), "f"(v[i + 1]));
  asm("max.NaN.abs.f32 %0, %0, %1, %1;" : "+f"(m) : "f"(v[15]));
  return m;
}

// 16 BF16 values; WIDE: from a 32-byte boundary, in one load.
template <bool WIDE>
__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8]) {
  if (WIDE) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// silu(g) u for a BF16 g.  log2(e) = kHi + kLo with 15 bits in kHi: g kHi is exact, and 2^(-g kLo) = 1 - g kLo ln 2
// within 0.8 x 2^-24 while |g| <= 60 (above, e^-g is nothing beside 1).  Then 1 + e^-g is off by 2^-22 (ex2.approx),
// that and two roundings, its reciprocal by 2^-23 more, and two products: 5.4 x 2^-23 together.  Below -60 the value is
// under 2^-81 |u| and less exact, and from -87.5 on it is lost: the reciprocal, under 2^-126, comes as 0.  That is
// nothing beside a block's maximum (less than half of the least code's step), unless |u| is 2^62 times as large as
// the maximum.  The kernel looks for such an up.
constexpr float kEnd = -60.0f, kLost = 0x1p62f;
__device__ __forceinline__ float silu_near(float g, float u) {
  constexpr float kHi = 0x1.7154p+0f, kLoLn2 = 4.8884952e-06f;
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kHi * g));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(e, fmaf(-kLoLn2, g, 1.0f), 1.0f)));
  return g * s * u;
}
// A product's distance from the border between two codes that it is in doubt about: the 20 bits below a code's
// three, off by 5.4 + 5.4 (value and maximum) + 1 (two roundings) times 2^-23 of a mantissa below 2, so 23.6 at most.
// (Below 2^-6, where codes are subnormal, the borders lie elsewhere; such values are taken as they are.)  With 16
// values a lane some 2 % of the warps are in doubt.
constexpr uint32_t kDoubt = 24, kDoubtful = 2 * kDoubt << 12;
__device__ __forceinline__ uint32_t border(float p) {
  return (__float_as_uint(p) << 12) - (0x80000u - kDoubt << 12);   // <= kDoubtful: in doubt
}

// The value in 64 bits (past f32's range an infinity, as it is in f32).  Not inlined: rarely called.
__device__ __noinline__ double silu64(uint16_t gate, uint16_t up) {
  const double g = bf16_bits_to_f32(gate), u = bf16_bits_to_f32(up), h = g / (1.0 + exp(-g)) * u;
  return fabs(h) > (double)0x1.fffffep+127f ? h * INFINITY : h;
}

// Codes in doubt, decided in 64 bits by the block's eight threads (every thread of the warp calls): the maximum
// from the values near it, then the codes.  all, or a value of the block that silu_near may have lost: every value is in doubt,
// and the scale is formed again too.  A product is rounded to f32 by way of an odd last bit, so that the rounding to
// a code decides as one would.
__device__ __noinline__ void settle(const uint16_t* gate, const uint16_t* up, bool have, float most, float f, bool all,
                                    uint4& code, float& scale) {
  uint32_t tops = 0, open = 0;
  int lost = 0;
  if (have)
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const float g = bf16_bits_to_f32(gate[i]), u = bf16_bits_to_f32(up[i]), v = silu_near(g, u);
      lost |= g < kEnd && fabsf(u) >= most * kLost;
      tops |= (uint32_t)(fabsf(v) >= most * (1.0f - 0x1p-19f)) << i;
      open |= (uint32_t)(border(__fmul_rn(v, f)) <= kDoubtful) << i;   // (the kernel's own product)
    }
  __syncwarp();
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) lost |= __shfl_xor_sync(0xFFFFFFFFu, lost, o);
  all |= have && lost;
  if (all) tops = open = 0xFFFFu;
  double m = 0x1p-100;
  bool nan = false;
  for (; tops; tops &= tops - 1) {
    const int i = __ffs(tops) - 1;
    const double h = silu64(gate[i], up[i]);
    nan |= h != h;
    m = fmax(m, fabs(h));
  }
  __syncwarp();
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    m = fmax(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    nan |= __shfl_xor_sync(0xFFFFFFFFu, (int)nan, o) != 0;
  }
  if (nan) m = __longlong_as_double(0x7FF8000000000000ll);
  const double f64 = 448.0 / m;
  for (; open; open &= open - 1) {
    const int i = __ffs(open) - 1;
    const double p = silu64(gate[i], up[i]) * f64;
    float z = __double2float_rz(p);
    if ((double)z != p && p == p) z = __uint_as_float(__float_as_uint(z) | 1u);
    const uint32_t byte = (e4m3x4(z, z, z, z) & 0xFFu) << (8 * (i & 3)), keep = ~(0xFFu << (8 * (i & 3)));
    if (i < 4) code.x = (code.x & keep) | byte;
    else if (i < 8) code.y = (code.y & keep) | byte;
    else if (i < 12) code.z = (code.z & keep) | byte;
    else code.w = (code.w & keep) | byte;
  }
  if (all) scale = (float)(m / 448.0);
  __syncwarp();
}

// Thread u of the flat list handles 16-value chunk u % 8 of block (u / 8) % KB of row u / (8 KB).  Bound by memory
// with enough loads under way, which is a matter of resident threads, and with SwiGLU nearly by the issue slots: 12
// CTAs of 128 an SM (40 registers; ten 157 us), 32-byte loads (of 16 bytes, a warp's touch every sector twice: 3 us
// more), no 64-bit division (16 us).  65787 x 2560 outputs in a graph 148 us (5.7 TB/s, 0.87 of the measured copy),
// called one by one 153 to 180 (outputs made anew, other inputs).  Without SwiGLU in a graph 71 us into expert order
// at 8192 x 5120, k = 8 (6.1 TB/s, 0.93).
template <bool SWIGLU, bool WIDE>
__global__ void __launch_bounds__(kRowThreads, SWIGLU ? 12 : 8) fp8_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int K, int kb, uint64_t kb_inv,
                                                       const int32_t* __restrict__ inv, int k, int64_t limit,
                                                       uint8_t* __restrict__ q, float* __restrict__ scales) {
  asm volatile("griddepcontrol.wait;" ::: "memory");    // launched while the kernel before it may still run
  const int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t blk = u >> 3;
  const int64_t row = kb_inv ? (int64_t)__umul64hi((uint64_t)blk, kb_inv) : blk;   // blk / kb
  const int kblk = (int)(blk - row * kb), c = kblk * 128 + (int)(u & 7) * 16;
  const bool have = row < rows && c < K;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  float largest_up = 0.0f;
  if (have) {
    uint32_t w[8];
    load16<WIDE>(x + row * (SWIGLU ? 2 * (int64_t)K : K) + c, w);
    unpack16(w, v);
    if (SWIGLU) {
      float up[16];
      load16<WIDE>(x + row * 2 * (int64_t)K + K + c, w);
      unpack16(w, up);
      largest_up = abs_max16(up);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = silu_near(v[i], up[i]);
    }
  }
  uint32_t m = __float_as_uint(abs_max16(v));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float most = block_max(m), f = __fdiv_rn(kTop, most);
  float p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = __fmul_rn(v[i], f);
  uint4 code = e4m3x16(p);
  float scale = __fdiv_rn(most, kTop);
  if (SWIGLU) {
    uint32_t doubt = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 16; i += 2) doubt = __vimin3_u32(doubt, border(p[i]), border(p[i + 1]));
    const bool all = have && (!(most < INFINITY) || (most < 0x1p-60f && m != 0));
    const bool look = largest_up >= most * kLost;        // an up may outweigh a gate below kEnd
    if (__any_sync(0xFFFFFFFFu, have && (doubt <= kDoubtful || all || look)))
      settle(x + row * 2 * (int64_t)K + c, x + row * 2 * (int64_t)K + K + c, have, most, f, all, code, scale);
  }
  if (!have) return;
  for (int j = 0; j < k; ++j) {
    const int64_t dst = inv ? __ldg(inv + row * k + j) : row;
    if (dst < 0 || dst >= limit) continue;
    *reinterpret_cast<uint4*>(q + dst * K + c) = code;
    if ((u & 7) == 0) scales[dst * kb + kblk] = scale;
  }
}

// Bound by memory: 6 x 2500 x 5120 in 35.1 us (6.5 TB/s, the measured copy's rate).
// One CTA per tile: thread t holds four 16-value chunks (rows t / 8 + 32 i, chunk t % 8), as loaded until
// the maximum is known: four CTAs fit an SM and cover one another's barrier.
__global__ void __launch_bounds__(256, 4) fp8_tiles_kernel(const uint16_t* __restrict__ w, int N, int K,
                                                           uint8_t* __restrict__ q, float* __restrict__ scales) {
  __shared__ uint32_t s_m[8];
  const int c = blockIdx.x * 128 + (threadIdx.x & 7) * 16;
  const int r0 = blockIdx.y * 128 + (threadIdx.x >> 3);
  const int64_t base = (int64_t)blockIdx.z * N;
  uint4 raw[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    if (r0 + 32 * i < N && c < K) {
      const uint4* p = reinterpret_cast<const uint4*>(w + (base + r0 + 32 * i) * K + c);
      raw[i][0] = __ldg(p);
      raw[i][1] = __ldg(p + 1);
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(bf16x8_abs_max_bits(raw[i][0]), bf16x8_abs_max_bits(raw[i][1])));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_m[i]);
  const float most = block_max(m << 16), f = __fdiv_rn(kTop, most);   // a BF16 pattern is the upper half of its f32's
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + 32 * i < N && c < K) {
      float v[16];
      const uint32_t w8[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                              raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
      unpack16(w8, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], f);
      *reinterpret_cast<uint4*>(q + (base + r0 + 32 * i) * K + c) = e4m3x16(v);
    }
  if (threadIdx.x == 0)
    scales[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = __fdiv_rn(most, kTop);
}

// A launch of the row kernel that may begin while the kernel before it ends.
template <bool SWIGLU>
int launch_rows(const uint16_t* x, int64_t rows, int K, const int32_t* inv, int k, uint8_t* q, float* scales,
                cudaStream_t s) {
  const int kb = (K + 127) / 128;
  // n / kb = the upper half of n * kb_inv for n < 2^35 and kb <= 512 (n kb < 2^64); 0 for kb = 1.
  const uint64_t kb_inv = kb == 1 ? 0 : ~0ull / (uint64_t)kb + 1;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((rows * kb * 8 + kRowThreads - 1) / kRowThreads));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool wide = reinterpret_cast<uintptr_t>(x) % 32 == 0;   // (rows are multiples of 32 bytes)
  cudaError_t err = cudaLaunchKernelEx(&cfg, wide ? fp8_rows_kernel<SWIGLU, true> : fp8_rows_kernel<SWIGLU, false>, x,
                                       rows, K, kb, kb_inv, inv, k, rows * k, q, scales);
  if (err == cudaSuccess) err = cudaGetLastError();
  return err == cudaSuccess ? 1 : -(int)err;
}

}  // namespace

int launch_fp8_quantize(const uint16_t* x, int64_t T, int K, const int32_t* inv, int k, uint8_t* q, float* scales,
                        cudaStream_t s) {
  return launch_rows<false>(x, T, K, inv, k, q, scales, s);
}

int launch_fp8_swiglu_quantize(const uint16_t* gu, int64_t R, int I, uint8_t* q, float* scales, cudaStream_t s) {
  return launch_rows<true>(gu, R, I, nullptr, 1, q, scales, s);
}

int launch_fp8_quantize_weights(const uint16_t* w, int64_t n, int N, int K, uint8_t* q, float* scales,
                                cudaStream_t s) {
  const dim3 grid((K + 127) / 128, (N + 127) / 128, (unsigned)n);
  fp8_tiles_kernel<<<grid, 256, 0, s>>>(w, N, K, q, scales);
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? 1 : -(int)err;
}

}  // namespace moe
