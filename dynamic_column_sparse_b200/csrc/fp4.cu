// fp4.cu - rows of bf16 values to 4-bit microscaled codes (the operands of the
// block-scaled product) and back. Formats and scale layout: fp4.cuh.
//
// Quantiser: one warp per row, 16 columns (two 16-byte loads, one 8-byte store)
// per lane and step; the block maxima come from packed 16-bit maxima of the
// bits. NVFP4 needs the row's maximum before its first code and reads the row
// twice, the second time from cache.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.cuh"

namespace cm {
namespace {

template <int FMT>
__global__ void __launch_bounds__(256) quantize_fp4_rows_kernel(const Fp4QuantParams p) {
  if (*(volatile const int *)p.status != kDevOk) return;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int groups = static_cast<int>(p.cols / 16);
  const int64_t tiles = fp4_scale_tiles(p.cols, FMT);
  // groups that carry scale bytes: whole 256-column tiles, the padding written as zero scales
  const int pad_groups = static_cast<int>((p.cols + 255) / 256 * 16);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); row < p.rows;
       row += warps) {
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + row * p.cols);
    float rs_inv = 1.f;
    if (FMT == kNvfp4) {
      uint32_t m = 0;
      for (int g = lane; g < groups; g += 32) {
        const uint4 u[2] = {src[2 * g], src[2 * g + 1]};
        const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = amax_bf16x2(m, w[e]);
      }
      const uint32_t amax = __reduce_max_sync(0xffffffffu, amax_fold(m));
      const float rs = nvfp4_row_scale(amax);
      rs_inv = amax >= kBf16Inf ? 0.f : __frcp_rn(rs);
      if (lane == 0) p.row_scales[row] = rs;
    }
    uint2 *dst = reinterpret_cast<uint2 *>(p.codes + row * (p.cols / 2));
    for (int g0 = 0; g0 < pad_groups; g0 += 32) {
      const int g = g0 + lane;
      const bool live = g < groups;
      uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (live) {
        u[0] = src[2 * g];
        u[1] = src[2 * g + 1];
      }
      const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = amax_bf16x2(m, w[e]);
      uint32_t amax = amax_fold(m);
      float inv;
      uint32_t sb;
      if (FMT == kNvfp4) {
        sb = nvfp4_block_scale(amax, rs_inv, &inv);
      } else {
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        sb = mxfp4_block_scale(amax, &inv);
      }
      if (!live) sb = 0;
      float v[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[2 * e] = FMT == kNvfp4 ? e2m1_grid(bf16_lo(w[e]), inv) : bf16_lo(w[e]) * inv;
        v[2 * e + 1] = FMT == kNvfp4 ? e2m1_grid(bf16_hi(w[e]), inv) : bf16_hi(w[e]) * inv;
      }
      if (live) dst[g] = make_uint2(e2m1x8(v), e2m1x8(v + 8));
      // four blocks' scale bytes to one word, written by the first lane of each four blocks
      constexpr int kLanes = FMT == kNvfp4 ? 1 : 2;  // lanes per block
      uint32_t word = sb;
#pragma unroll
      for (int i = 1; i < 4; ++i) word |= __shfl_down_sync(0xffffffffu, sb, i * kLanes) << (8 * i);
      if ((lane & (4 * kLanes - 1)) == 0 && g < pad_groups)
        *reinterpret_cast<uint32_t *>(p.scales + fp4_scale_offset(row, g / kLanes, tiles)) = word;
    }
  }
}

// 16 columns per thread: one 8-byte code load, one scale byte, two (bf16) or
// four (fp32) 16-byte stores. Every value (two code bits times four scale bits
// times powers of two) is exact in bf16 within its range.
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) dequantize_fp4_rows_kernel(const Fp4QuantParams p, void *out) {
  if (*(volatile const int *)p.status != kDevOk) return;
  const int groups = static_cast<int>(p.cols / 16);
  const int64_t tiles = fp4_scale_tiles(p.cols, FMT);
  const int64_t total = p.rows * groups;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / groups;
    const int g = static_cast<int>(i - row * groups);
    const uint2 c = reinterpret_cast<const uint2 *>(p.codes)[i];
    const uint32_t sb = p.scales[fp4_scale_offset(row, FMT == kNvfp4 ? g : g / 2, tiles)];
    const float s = FMT == kNvfp4 ? e4m3_to_f32(sb) * p.row_scales[row] : e8m0_to_f32(sb);
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t code = ((e < 8 ? c.x : c.y) >> (4 * (e & 7))) & 15u;
      // magnitudes 0, 0.5, then (2 + low bit) * 2^(exponent - 2)
      const uint32_t mag = code & 7u;
      const float a = mag < 2 ? 0.5f * static_cast<float>(mag)
                              : __uint_as_float(((mag >> 1) + 126u) << 23 | (mag & 1u) << 22);
      v[e] = (code & 8u ? -a : a) * s;
    }
    if (F32) {
      float4 *o = reinterpret_cast<float4 *>(out) + i * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
      uint4 *o = reinterpret_cast<uint4 *>(out) + i * 2;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        o[q] = make_uint4(cvt_bf16x2(v[8 * q], v[8 * q + 1]), cvt_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                          cvt_bf16x2(v[8 * q + 4], v[8 * q + 5]), cvt_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    }
  }
}

}  // namespace

cudaError_t launch_quantize_fp4_rows(const Fp4QuantParams &p, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((p.rows + 7) / 8, 148 * 8));
  if (p.fmt == kNvfp4)
    quantize_fp4_rows_kernel<kNvfp4><<<blocks, 256, 0, s>>>(p);
  else
    quantize_fp4_rows_kernel<kMxfp4><<<blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_fp4_rows(const Fp4QuantParams &p, bool f32, void *out, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  const int64_t total = p.rows * (p.cols / 16);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, 148 * 32));
  if (p.fmt == kNvfp4) {
    if (f32) dequantize_fp4_rows_kernel<kNvfp4, true><<<blocks, 256, 0, s>>>(p, out);
    else dequantize_fp4_rows_kernel<kNvfp4, false><<<blocks, 256, 0, s>>>(p, out);
  } else {
    if (f32) dequantize_fp4_rows_kernel<kMxfp4, true><<<blocks, 256, 0, s>>>(p, out);
    else dequantize_fp4_rows_kernel<kMxfp4, false><<<blocks, 256, 0, s>>>(p, out);
  }
  return cudaGetLastError();
}

}  // namespace cm
