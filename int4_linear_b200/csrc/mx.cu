// Microscaled 4-bit floating point: quantization of fp16 rows to E2M1 codes
// with one scale per block (32 values and E8M0, or 16 and E4M3), and back.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "fq_device.cuh"
#include "fq_host.h"
#include "mx.cuh"

namespace fq {
namespace {

constexpr int kMxThreads = 256;

// Two values to packed E2M1 codes: round to nearest, ties to the even code,
// saturated at 6 (lo in bits 0-3).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Codes of 16 values times inv.
__device__ __forceinline__ void codes16(const __half2* h2, float inv, uint32_t (&q)[2]) {
  q[0] = q[1] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = fmul2(__half22float2(h2[j]), make_float2(inv, inv));
    q[j >> 2] |= e2m1x2(f.x, f.y) << (8 * (j & 3));
  }
}

// Codes of 16 values over d.
__device__ __forceinline__ void codes16_divided(const __half2* h2, float d, uint32_t (&q)[2]) {
  q[0] = q[1] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = __half22float2(h2[j]);
    q[j >> 2] |= e2m1x2(__fdiv_rn(f.x, d), __fdiv_rn(f.y, d)) << (8 * (j & 3));
  }
}

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// One thread per 16 values: 32 bytes in, 8 bytes of codes out, and the scales
// of four blocks leave as one word from the first of the threads that hold
// them (a scale tile keeps a row's four blocks together).  MXFP4 is bound by HBM
// (2 bytes read and 0.53 written per value; 2048 x 16384: 14.0 us, 6.1 TB/s), NVFP4 by its arithmetic, the
// codes' two conversions and the scale's division (0.56 written; 19.4 us, 4.4 TB/s).  One token's row takes 1.4 us.
template <int FMT, typename Index>
__global__ void __launch_bounds__(kMxThreads) mx_quant_kernel(const __half* __restrict__ X, long long ldx, int R,
                                                              int K, const float* __restrict__ g, uint8_t* Q,
                                                              uint8_t* S) {
  constexpr int BLOCK = FMT == FQ_NVFP4 ? 16 : 32;
  pdl_launch_dependents();
  pdl_wait();
  const Index pieces = Index(K) / 16, total = Index(R) * pieces;
  const float gs = FMT == FQ_NVFP4 && g ? *g : 1.0f;
  const float g6 = __fmul_rn(6.0f, gs);
  // K is a multiple of 128: the 8 threads that share a shuffle hold one row
  for (Index e = Index(blockIdx.x) * kMxThreads + threadIdx.x; e < total; e += Index(gridDim.x) * kMxThreads) {
    const Index r = e / pieces, c = e % pieces;
    const uint4* src = reinterpret_cast<const uint4*>(X + static_cast<long long>(r) * ldx + c * 16);
    const uint4 raw[2] = {src[0], src[1]};
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, w[j] & 0x7FFF7FFFu);
    uint32_t mb = max(m2 & 0xFFFFu, m2 >> 16);  // bits of the largest magnitude
    const uint32_t group = 0xFFu << (threadIdx.x & 24);  // the 8 lanes that enter the loop together
    if (FMT == FQ_MXFP4) mb = max(mb, __shfl_xor_sync(group, mb, 1));
    const bool finite = mb < 0x7C00u;
    const float amax = __half2float(__ushort_as_half(static_cast<unsigned short>(mb)));
    uint32_t sb;
    float d = 1.f, inv = 0.f;
    if (FMT == FQ_MXFP4) {
      // every fp16 magnitude is a normal float: its exponent is floor(log2)
      sb = mb ? (__float_as_uint(amax) >> 23) - 2 : 0u;
      inv = __uint_as_float((254u - sb) << 23);
      if (!finite) sb = 0xFFu;
    } else {
      sb = __nv_cvt_float_to_fp8(__fdiv_rn(amax, g6), __NV_SATFINITE, __NV_E4M3);
      d = __fmul_rn(e4m3_value(uint8_t(sb)), gs);
      if (!finite) sb = 0x7Fu;
    }
    uint32_t q[2] = {0, 0};
    const __half2* h2 = reinterpret_cast<const __half2*>(raw);
    if (FMT == FQ_MXFP4) {
      if (finite) codes16(h2, inv, q);
    } else if (finite && d != 0.f) {
      // the codes of the quotients a little below and a little above; where they differ (next to
      // a tie), or the reciprocal may overflow, the division itself decides
      inv = __fdividef(1.0f, d);
      uint32_t up[2];
      codes16(h2, inv * (1.0f - 0x1p-20f), q);
      codes16(h2, inv * (1.0f + 0x1p-20f), up);
      if (q[0] != up[0] || q[1] != up[1] || d < 0x1p-100f) codes16_divided(h2, d, q);
    }
    *reinterpret_cast<uint2*>(Q + static_cast<size_t>(r) * (K / 2) + c * 8) = make_uint2(q[0], q[1]);
    // the scales of four blocks: every thread (E4M3) or every other one (E8M0)
    constexpr int STEP = BLOCK / 16;
    uint32_t word = sb;
#pragma unroll
    for (int b = 1; b < 4; ++b) word |= __shfl_down_sync(group, sb, b * STEP) << (8 * b);
    if ((c & (4 * STEP - 1)) == 0)
      *reinterpret_cast<uint32_t*>(S + mx_scale_offset(int(r), int(c) / STEP, K / BLOCK)) = word;
  }
}

// The upper bytes of the fp16 numbers of four codes (the lower ones are 0).  Magnitudes of codes 0..7: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6, a byte selection by the codes' low bits.  A selector with its top bit set gives the selected
// byte's top bit in all places, so a table whose bytes are odd only then tells the signs.
__device__ __forceinline__ uint32_t e2m1_top_bytes(uint32_t c4) {
  constexpr uint32_t kLow = 0x3E3C3800u, kHigh = 0x46444240u;
  uint32_t sign;  // __byte_perm clears the selectors' top bits
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(c4));
  return __byte_perm(kLow, kHigh, c4 & 0x7777u) | (sign & 0x01010101u) << 7;
}

// One thread per 16 values; bound by HBM (0.53 or 0.56 bytes read and 2 written per value; 16384 x 4096: 31.7 us,
// 5.4 TB/s).
template <int FMT>
__global__ void __launch_bounds__(kMxThreads) mx_dequant_kernel(const uint8_t* __restrict__ Q,
                                                                const uint8_t* __restrict__ S, int R, int K,
                                                                const float* __restrict__ g, __half* __restrict__ X) {
  constexpr int BLOCK = FMT == FQ_NVFP4 ? 16 : 32;
  pdl_launch_dependents();
  pdl_wait();
  const size_t pieces = size_t(K) / 16, total = size_t(R) * pieces;
  const float gs = FMT == FQ_NVFP4 && g ? *g : 1.0f;
  for (size_t e = size_t(blockIdx.x) * kMxThreads + threadIdx.x; e < total; e += size_t(gridDim.x) * kMxThreads) {
    const int r = int(e / pieces), c = int(e % pieces);
    const uint2 w = *reinterpret_cast<const uint2*>(Q + size_t(r) * (K / 2) + size_t(c) * 8);
    const uint32_t sb = S[mx_scale_offset(r, c * 16 / BLOCK, K / BLOCK)];
    float d;
    if (FMT == FQ_MXFP4)
      d = sb == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(sb ? sb << 23 : 0x00400000u);
    else
      d = __fmul_rn(e4m3_value(uint8_t(sb)), gs);
    uint4 out[2];
    __half2* o2 = reinterpret_cast<__half2*>(out);
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // four codes
      const uint32_t c4 = (j < 2 ? w.x : w.y) >> (16 * (j & 1));
      const uint32_t v = e2m1_top_bytes(c4);
      const uint32_t lo = __byte_perm(v, 0, 0x1404), hi = __byte_perm(v, 0, 0x3424);
      const float2 f = fmul2(__half22float2(*reinterpret_cast<const __half2*>(&lo)), make_float2(d, d));
      const float2 g = fmul2(__half22float2(*reinterpret_cast<const __half2*>(&hi)), make_float2(d, d));
      o2[2 * j] = __floats2half2_rn(f.x, f.y);
      o2[2 * j + 1] = __floats2half2_rn(g.x, g.y);
    }
    uint4* dst = reinterpret_cast<uint4*>(X + size_t(r) * K + size_t(c) * 16);
    dst[0] = out[0];
    dst[1] = out[1];
  }
}

// CTAs for `pieces` of 16 values, at most `most`.
int mx_grid(size_t pieces, size_t most) {
  const size_t want = (pieces + kMxThreads - 1) / kMxThreads;
  return int(std::min<size_t>(std::max<size_t>(want, 1), most));
}

fq_status check_mx(int rows, int K, fq_mx_format fmt, const float* g) {
  if (fmt != FQ_MXFP4 && fmt != FQ_NVFP4) return fail(FQ_ERR_UNSUPPORTED, "format %d is not provided", int(fmt));
  FQ_CHECK_ARG(rows >= 1, "rows = %d must be >= 1", rows);
  FQ_CHECK_ARG(K >= kGroup && K <= kMaxK && K % kGroup == 0, "K = %d must be a multiple of 128 in [128, %d]", K,
               kMaxK);
  FQ_CHECK_ARG(!g || fmt == FQ_NVFP4, "FQ_MXFP4 has no tensor scale: g must be NULL");
  FQ_CHECK_ARG(aligned(g, 4), "g must be 4-byte aligned");
  return FQ_OK;
}

}  // namespace
}  // namespace fq

extern "C" {

size_t fq_mx_scale_bytes(int rows, int K, fq_mx_format fmt) {
  if (rows < 1 || K < fq::kGroup || K > fq::kMaxK || K % fq::kGroup || (fmt != FQ_MXFP4 && fmt != FQ_NVFP4)) return 0;
  return (size_t(rows) + fq::kMxTileRows - 1) / fq::kMxTileRows * fq::kMxTileRows * (K / fq::mx_block(fmt));
}

fq_status fq_mx_quant(const uint16_t* X, long long ldx, int R, int K, fq_mx_format fmt, const float* g, uint8_t* Q,
                      uint8_t* S, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_mx(R, K, fmt, g);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(X && Q && S && fq::aligned(X, 16) && fq::aligned(Q, 16) && fq::aligned(S, 16),
               "X, Q and S must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(ldx >= K && ldx % 8 == 0, "ldx = %lld must be a multiple of 8 and at least K = %d", ldx, K);
  const size_t pieces = size_t(R) * (K / 16);
  const dim3 grid(fq::mx_grid(pieces, size_t(fq::sm_count()) * 8)), block(fq::kMxThreads);
  const __half* x = reinterpret_cast<const __half*>(X);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // 32-bit indexes divide faster; the loop's step past the end has to fit as well
  const bool small = pieces < (size_t(1) << 31);
  if (fmt == FQ_MXFP4)
    small ? fq::launch_pdl(fq::mx_quant_kernel<FQ_MXFP4, uint32_t>, grid, block, 0, s, x, ldx, R, K, g, Q, S)
          : fq::launch_pdl(fq::mx_quant_kernel<FQ_MXFP4, uint64_t>, grid, block, 0, s, x, ldx, R, K, g, Q, S);
  else
    small ? fq::launch_pdl(fq::mx_quant_kernel<FQ_NVFP4, uint32_t>, grid, block, 0, s, x, ldx, R, K, g, Q, S)
          : fq::launch_pdl(fq::mx_quant_kernel<FQ_NVFP4, uint64_t>, grid, block, 0, s, x, ldx, R, K, g, Q, S);
  return fq::check_launch("mx_quant_kernel");
}

fq_status fq_mx_dequant(const uint8_t* Q, const uint8_t* S, int R, int K, fq_mx_format fmt, const float* g,
                        uint16_t* X, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_mx(R, K, fmt, g);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(X && Q && S && fq::aligned(X, 16) && fq::aligned(Q, 16) && fq::aligned(S, 16),
               "X, Q and S must be non-NULL and 16-byte aligned");
  // one piece per thread: as many CTAs as fit at once, taking several each, took 40.9 us for 16384 x 4096 instead of 31.7
  const dim3 grid(fq::mx_grid(size_t(R) * (K / 16), size_t(1) << 30)), block(fq::kMxThreads);
  __half* x = reinterpret_cast<__half*>(X);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (fmt == FQ_MXFP4)
    fq::launch_pdl(fq::mx_dequant_kernel<FQ_MXFP4>, grid, block, 0, s, Q, S, R, K, g, x);
  else
    fq::launch_pdl(fq::mx_dequant_kernel<FQ_NVFP4>, grid, block, 0, s, Q, S, R, K, g, x);
  return fq::check_launch("mx_dequant_kernel");
}

}  // extern "C"
