// fp4.cu - rows of bf16 values to 4-bit microscaled codes (the operands of the
// block-scaled product) and back. Formats and scale layout: fp4.cuh.
//
// Both are HBM bound. Quantiser: a row is read once and held in registers as bf16 by
// one warp (up to 4096 columns) or by 4 or 16 warps of a CTA, 16 consecutive columns per
// lane and step, so that NVFP4's row maximum costs no second pass; the block maxima
// come from packed 16-bit maxima of the bits, and no value is divided (e2m1_grid).
#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "kernels.cuh"

namespace cm {
namespace {

// W warps per row, NV steps of 16 columns per lane.
template <int FMT, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) quantize_fp4_rows_kernel(const Fp4QuantParams p) {
  constexpr int G = 32 * W, kRows = W == 1 ? 4 : 1;
  constexpr int kLanes = FMT == kNvfp4 ? 1 : 2;  // lanes per block
  __shared__ uint32_t row_max[2][16];
  allow_dependents();  // a product launched behind this kernel sets up meanwhile
  if (__syncthreads_or(*(volatile const int *)p.status != kDevOk)) return;  // all threads alike
  const int t = threadIdx.x % G, lane = threadIdx.x & 31;
  const int groups = static_cast<int>(p.cols / 16);
  const int pad_groups = (groups + 15) / 16 * 16;  // whole 256 columns carry scale bytes
  const int64_t tiles = fp4_scale_tiles(p.cols, FMT);
  const bool wide = (reinterpret_cast<uintptr_t>(p.x) & 31) == 0;
  int slot = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const uint16_t *src = p.x + row * p.cols;
    Vec32 u[NV];
    if (wide) {
#pragma unroll
      for (int v = 0; v < NV; ++v) u[v] = v * G + t < groups ? load32(src + 16 * (v * G + t)) : Vec32{};
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) u[v] = v * G + t < groups ? load16x2(src + 16 * (v * G + t)) : Vec32{};
    }
    uint32_t m[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      uint32_t a = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = amax_bf16x2(a, u[v].w[e]);
      m[v] = amax_fold(a);
    }
    float rs_inv = 1.f;
    if (FMT == kNvfp4) {
      uint32_t amax = m[0];
#pragma unroll
      for (int v = 1; v < NV; ++v) amax = max(amax, m[v]);
      amax = __reduce_max_sync(0xffffffffu, amax);
      if (W > 1) {
        if (lane == 0) row_max[slot][t >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) amax = max(amax, row_max[slot][w]);
        slot ^= 1;
      }
      const float rs = nvfp4_row_scale(amax);
      rs_inv = nvfp4_row_inv(amax);
      if (t == 0) p.row_scales[row] = rs;
    }
    uint2 *dst = reinterpret_cast<uint2 *>(p.codes + row * (p.cols / 2));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = v * G + t;
      float inv;
      uint32_t sb;
      if (FMT == kNvfp4) {
        sb = nvfp4_block_scale(m[v], rs_inv, &inv);
      } else {
        sb = mxfp4_block_scale(max(m[v], __shfl_xor_sync(0xffffffffu, m[v], 1)), &inv);
      }
      if (g < groups) {
        float q[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = u[v].w[e];
          const float2 x = make_float2(bf16_lo(w), bf16_hi(w));
          const float2 d = FMT == kNvfp4 ? e2m1_grid(x, inv) : mul2(x, make_float2(inv, inv));
          q[2 * e] = d.x, q[2 * e + 1] = d.y;
        }
        dst[g] = make_uint2(e2m1x8(q), e2m1x8(q + 8));
      } else {
        sb = 0;
      }
      // one byte per block; a warp's stores to the same four blocks merge into one word
      if ((lane & (kLanes - 1)) == 0 && g < pad_groups)
        p.scales[fp4_scale_offset(row, g / kLanes, tiles)] = static_cast<uint8_t>(sb);
    }
  }
}

// Four e2m1 codes (16 bits) to four bf16: the high and low bytes of the magnitudes
// 0, 0.5 .. 6 by byte permutes with the codes as selectors, then the signs.
__device__ __forceinline__ uint2 e2m1x4_to_bf16(uint32_t c) {
  const uint32_t sel = c & 0x7777u;
  const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel);  // 00 3f 3f 3f | 40 40 40 40
  const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);  // 00 00 80 c0 | 00 40 80 c0
  const uint32_t a = __byte_perm(lo, hi, 0x5140u), b = __byte_perm(lo, hi, 0x7362u);
  return make_uint2(a | (c & 8u) << 12 | (c & 0x80u) << 24, b | (c & 0x800u) << 4 | (c & 0x8000u) << 16);
}

// A thread takes 16 columns of four rows at a time: per row one 8-byte code load, one scale
// byte, one 32-byte (bf16) or four 16-byte (fp32) stores; the rows' loads go out together.
// Every value (two code bits times four scale bits times powers of two) and the
// scale itself are exact in bf16 within its range, so the product is taken there. With a row scale that is no
// power of two, and for fp32 output, code times block scale (exact) times row scale is rounded in fp32
// (4352 x 12288 to bf16: 27 us instead of 24.5; one loop for both kinds of row took 26 for either).
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) dequantize_fp4_rows_kernel(const Fp4QuantParams p, void *out) {
  constexpr int R = 4;
  if (*(volatile const int *)p.status != kDevOk) return;
  const int groups = static_cast<int>(p.cols / 16);
  const int64_t tiles = fp4_scale_tiles(p.cols, FMT);
  const int g = blockIdx.x * 32 + threadIdx.x;
  if (g >= groups) return;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 8;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * 8 + threadIdx.y; row0 < p.rows; row0 += R * step) {
    uint2 c[R];
    uint32_t sb[R];
    float rs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t row = min(row0 + k * step, p.rows - 1);
      c[k] = reinterpret_cast<const uint2 *>(p.codes)[row * groups + g];
      sb[k] = p.scales[fp4_scale_offset(row, FMT == kNvfp4 ? g : g / 2, tiles)];
      rs[k] = FMT == kNvfp4 ? p.row_scales[row] : 1.f;
    }
    // in_bf16: the row scales are powers of two
    auto decode = [&](auto in_bf16) {
      constexpr bool kInBf16 = decltype(in_bf16)::value;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t row = row0 + k * step;
        if (row >= p.rows) break;
        const float bs = FMT == kNvfp4 ? e4m3_to_f32(sb[k]) : e8m0_to_f32(sb[k]);
        const uint32_t s2 = cvt_bf16x2(bs * rs[k], bs * rs[k]);
        const uint2 h[4] = {e2m1x4_to_bf16(c[k].x & 0xffffu), e2m1x4_to_bf16(c[k].x >> 16),
                            e2m1x4_to_bf16(c[k].y & 0xffffu), e2m1x4_to_bf16(c[k].y >> 16)};
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = e & 1 ? h[e >> 1].y : h[e >> 1].x;
          if (kInBf16) w[e] = mul_bf16x2(w[e], s2);
          else if (!F32) w[e] = cvt_bf16x2(bf16_lo(w[e]) * bs * rs[k], bf16_hi(w[e]) * bs * rs[k]);
        }
        const int64_t i = row * groups + g;
        if (F32) {
          float4 *o = reinterpret_cast<float4 *>(out) + i * 4;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            o[q] = make_float4(bf16_lo(w[2 * q]) * bs * rs[k], bf16_hi(w[2 * q]) * bs * rs[k],
                               bf16_lo(w[2 * q + 1]) * bs * rs[k], bf16_hi(w[2 * q + 1]) * bs * rs[k]);
        } else {
          uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + i * 16);
          if (wide) {
            store32(o, w);
          } else {
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
    };
    bool powers = !F32;
#pragma unroll
    for (int k = 0; k < R; ++k) powers = powers && (FMT != kNvfp4 || (__float_as_uint(rs[k]) & 0x7fffffu) == 0);
    if (powers) decode(std::true_type());
    else decode(std::false_type());
  }
}

}  // namespace

namespace {

template <int FMT, int W>
void launch_w(const Fp4QuantParams &p, cudaStream_t s) {
  const int need = static_cast<int>((p.cols / 16 + 32 * W - 1) / (32 * W));
  const int rows = W == 1 ? 4 : 1;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((p.rows + rows - 1) / rows, 148 * (W == 16 ? 4 : 16)));
  const unsigned threads = W == 1 ? 128 : 32 * W;
  if constexpr (W == 1) {  // more warps hold a row of more than two steps only
    if (need <= 1) return quantize_fp4_rows_kernel<FMT, W, 1><<<blocks, threads, 0, s>>>(p);
    if (need <= 2) return quantize_fp4_rows_kernel<FMT, W, 2><<<blocks, threads, 0, s>>>(p);
  }
  if (need <= 4) quantize_fp4_rows_kernel<FMT, W, 4><<<blocks, threads, 0, s>>>(p);
  else if (need <= 6) quantize_fp4_rows_kernel<FMT, W, 6><<<blocks, threads, 0, s>>>(p);
  else quantize_fp4_rows_kernel<FMT, W, 8><<<blocks, threads, 0, s>>>(p);
}

template <int FMT>
void launch_fmt(const Fp4QuantParams &p, cudaStream_t s) {
  if (p.cols <= 4096) launch_w<FMT, 1>(p, s);
  else if (p.cols <= 16384) launch_w<FMT, 4>(p, s);
  else launch_w<FMT, 16>(p, s);
}

}  // namespace

cudaError_t launch_quantize_fp4_rows(const Fp4QuantParams &p, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  if (p.fmt == kNvfp4) launch_fmt<kNvfp4>(p, s);
  else launch_fmt<kMxfp4>(p, s);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_fp4_rows(const Fp4QuantParams &p, bool f32, void *out, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  const unsigned x = static_cast<unsigned>((p.cols / 16 + 31) / 32);
  const int64_t y = std::min<int64_t>((p.rows + 31) / 32, std::max<int64_t>(1, 148 * 32 / x));
  const dim3 grid(x, static_cast<unsigned>(y)), block(32, 8);
  auto kernel = p.fmt == kNvfp4 ? (f32 ? dequantize_fp4_rows_kernel<kNvfp4, true> : dequantize_fp4_rows_kernel<kNvfp4, false>)
                                : (f32 ? dequantize_fp4_rows_kernel<kMxfp4, true> : dequantize_fp4_rows_kernel<kMxfp4, false>);
  kernel<<<grid, block, 0, s>>>(p, out);
  return cudaGetLastError();
}

}  // namespace cm
