// fp4.cuh - 4-bit microscaled rows: formats, scale layout and the device
// conversions shared by the quantiser and by the kernels that write quantised
// rows themselves.
//
// A value is code * block scale (* row scale). Codes are e2m1 (magnitudes 0,
// 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the lower column in the low nibble.
//   NVFP4: blocks of 16 columns, block scale e4m3, and a power-of-two fp32 row
//          scale rs = 2^(floor(log2 max|row|) - 10), exponent clamped to
//          [-110, 117] (1 for an all-zero row, NaN for a row that is not finite):
//          block scale = e4m3(max|block| / (6 rs)), code = e2m1(x / (block scale * rs)).
//   MXFP4: blocks of 32 columns, block scale 2^(floor(log2 max|block|) - 2) as
//          an e8m0 byte (0 where the exponent would be below -127, 255 = NaN
//          for a block that is not finite), code = e2m1(x / block scale).
// Every rounding is to nearest, ties to even, saturating at the largest code.
// bf16 inputs and power-of-two row scales make each quotient's distance from a
// rounding border either zero or at least 2^-10 (see e2m1_grid), so fp32
// arithmetic gives exactly the codes that exact arithmetic gives.
//
// Block scales lie in the order the tensor core's scale copies read: tiles of
// 128 rows x 4 blocks, 512 bytes each, byte (r % 32) * 16 + (r % 128) / 32 * 4 +
// block % 4; the tiles of 128 rows follow one another along the columns, padded
// to a whole number of 256 columns.
#pragma once

#include <cuda_fp8.h>

#include "ptx.cuh"

namespace cm {

enum Fp4Format : int { kNvfp4 = 0, kMxfp4 = 1 };

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == kNvfp4 ? 16 : 32; }
// 512-byte scale tiles along the columns of 128 rows
__host__ __device__ constexpr int64_t fp4_scale_tiles(int64_t cols, int fmt) {
  return (cols + 255) / 256 * (fmt == kNvfp4 ? 4 : 2);
}
__host__ __device__ constexpr size_t fp4_scale_bytes(int64_t rows, int64_t cols, int fmt) {
  return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>(fp4_scale_tiles(cols, fmt)) * 512;
}
// Byte offset of the scale of (row, block): blocks 4i .. 4i+3 of a row are one aligned 4-byte word.
__host__ __device__ inline size_t fp4_scale_offset(int64_t row, int64_t block, int64_t tiles) {
  return static_cast<size_t>((row >> 7) * tiles + (block >> 2)) * 512 + static_cast<size_t>((row & 31) * 16) +
         static_cast<size_t>(((row >> 5) & 3) * 4) + static_cast<size_t>(block & 3);
}

// A quotient x / (s rs) of a bf16 x by an e4m3 scale and a power of two lies on
// a rounding border of e2m1 (0.25 .. 5) or at least 2^-10 away from every border
// (X 2^a - m D 2^b with integers X < 256, D < 16 and a border m is 0 or at least m / 255 of m D 2^b),
// while its fp32 approximation x * inv, inv a reciprocal good to 2^-22, is off by less than
// 2^-18. Rounding the product to a multiple of 2^-12 (adding and taking off 1.5 * 2^11,
// the first in the fused multiply-add) therefore puts the border cases exactly on
// the border and moves no other one across, without a division per value.
__device__ __forceinline__ float2 e2m1_grid(float2 x, float inv) {
  const float2 c = make_float2(0x1.8p11f, 0x1.8p11f), n = make_float2(-0x1.8p11f, -0x1.8p11f);
  return add2(fma2(x, make_float2(inv, inv), c), n);
}

// Eight values to eight e2m1 codes, value i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 32 bytes of global memory in one load (32-byte aligned).
struct alignas(32) Vec32 {
  uint32_t w[8];
};
__device__ __forceinline__ Vec32 load32(const void *p) {
  Vec32 v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p));
  return v;
}

__device__ __forceinline__ Vec32 load16x2(const void *p) {  // 16-byte aligned
  const uint4 a = static_cast<const uint4 *>(p)[0], b = static_cast<const uint4 *>(p)[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The two bf16 of a word as fp32.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Maximum of the magnitudes of packed bf16 pairs, by their bits (a NaN is above
// infinity, so it is kept): running value in packed form.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t amax_fold(uint32_t m) { return max(m & 0xffffu, m >> 16); }
constexpr uint32_t kBf16Inf = 0x7f80u;  // magnitudes from here up are infinite or NaN

// NVFP4 row scale from the bits of the row's largest magnitude.
__device__ __forceinline__ float nvfp4_row_scale(uint32_t amax) {
  if (amax == 0) return 1.f;
  if (amax >= kBf16Inf) return __uint_as_float(0x7fc00000u);
  const int e = min(max(static_cast<int>(amax >> 7) - 127 - 10, -110), 117);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// 1 / row scale (a power of two: exact), 0 for a row that is not finite, whose
// scales and codes then are 0 while its NaN row scale speaks for it.
__device__ __forceinline__ float nvfp4_row_inv(uint32_t amax) {
  if (amax == 0) return 1.f;
  if (amax >= kBf16Inf) return 0.f;
  const int e = min(max(static_cast<int>(amax >> 7) - 127 - 10, -110), 117);
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// NVFP4 block: e4m3 scale byte of amax / (6 rs) and the factor that takes x to its code's
// grid (0 for a block whose scale is 0). The quotient lies on a rounding border of e4m3 (five
// significant bits) or at least 1 / 255 of it away; the product with 1/6 is good to 2^-23, so
// rounding it to fp16 first (2^-12) puts the former exactly on the border and moves none across.
__device__ __forceinline__ uint32_t nvfp4_block_scale(uint32_t amax, float rs_inv, float *inv) {
  const float m = rs_inv != 0.f ? __uint_as_float(amax << 16) : 0.f;
  const __half2_raw t = __half2(__float2half_rn(m * (rs_inv * (1.f / 6.f))), __half(0.f));
  const uint32_t b = __nv_cvt_halfraw2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3) & 0xffu;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
  *inv = s > 0.f ? rcp_approx(s) * rs_inv : 0.f;
  return b;
}

// MXFP4 block: e8m0 scale byte and 1 / scale (exact; 0 for a block that is not finite).
__device__ __forceinline__ uint32_t mxfp4_block_scale(uint32_t amax, float *inv) {
  if (amax >= kBf16Inf) {
    *inv = 0.f;
    return 255u;
  }
  const int b = max(static_cast<int>(amax >> 7) - 2, 0);
  *inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
  return static_cast<uint32_t>(b);
}

// Scale bytes to fp32.
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3)));
}
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

}  // namespace cm
