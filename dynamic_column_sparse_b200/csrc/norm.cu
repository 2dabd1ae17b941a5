// norm.cu - the norms around a block's layers fused with its gate and residual.
//
// For every row t of sample b:
//   r = res_scale * res + gate[b] * post(y)          post: none, RMS or layer norm (* post_weight)
//   h = pre(r) * weight + bias, * (1 + scale[b]) + shift[b]
// r goes out in the residual stream's type, h as bf16 or as quantised rows
// (e4m3 with a row scale, or 4-bit microscaled: fp4.cuh) for the next
// projection; quantised rows are those of the bf16-rounded h, so they equal
// what the stand-alone quantisers give for the bf16 output. h is computed from
// the unrounded fp32 r.
//
// HBM bound: each row is read once, kept in registers as fp32 and written once;
// the statistics are two-pass in registers (a mean, then squares about it), the
// partial sums of a row's warps joined through shared memory by the pairwise
// rule for means and squares, so no large mean cancels.
//
// A row is held by one warp (up to 1024 columns) or by 4 or 16 warps of one
// CTA, NV groups of 8 columns per thread; column group v * G + t belongs to
// thread t, so every access is 16 bytes per lane and consecutive over a warp.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.cuh"

namespace cm {
namespace {

// Eight columns as they lie in memory, bf16 or fp32.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> raw8(const void *p, int64_t i) {
  Raw8<F32> r;
  const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (F32 ? 4 : 2));
  r.w[0] = s[0];
  if (F32) r.w[F32 ? 1 : 0] = s[1];
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32> &r, float2 *v) {
  if (F32) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[F32].x, r.w[F32].y, r.w[F32].z, r.w[F32].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
  }
}

// Eight values of a vector shared by many rows (weights, gates, scales, shifts), bf16 or fp32.
__device__ __forceinline__ void load8(const void *p, int f32, int64_t i, float2 *v) {
  if (f32)
    unpack8<true>(raw8<true>(p, i), v);
  else
    unpack8<false>(raw8<false>(p, i), v);
}

__device__ __forceinline__ uint4 pack8(const float2 *v) {
  return make_uint4(cvt_bf16x2(v[0].x, v[0].y), cvt_bf16x2(v[1].x, v[1].y), cvt_bf16x2(v[2].x, v[2].y),
                    cvt_bf16x2(v[3].x, v[3].y));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Statistics of one row over its W warps. `slot` alternates between two shared
// buffers, so one barrier per statistic is enough.
template <int W, int NV>
struct RowStats {
  float2 (*buf)[16];        // [2][16]
  const float2 *cols;       // [W]: columns a warp holds, and 1 over that
  float inv_d, eps;
  int nv, warp, lane;
  int slot = 0;

  // The row's mean and 1 / sqrt(variance + eps) (RMS: 0 and the root of the mean square), as the factor and
  // the addend that normalise: x * factor + addend.
  __device__ __forceinline__ float2 norm(const float2 (&r)[NV][4], bool layer) {
    float mean = 0.f, sum = 0.f;
    if (layer) {
      float2 s = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s = add2(s, r[v][e]);
        }
      sum = warp_sum(s.x + s.y);
      mean = sum * cols[warp].y;
    }
    const float2 nm = both(-mean);
    float2 q2 = both(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v < NV - 1 || v < nv) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 d = add2(r[v][e], nm);
          q2 = fma2(d, d, q2);
        }
      }
    float q = warp_sum(q2.x + q2.y);
    if (W > 1) {
      // join the warps: squares about the row's mean = squares about each
      // warp's mean + n_w (mean_w - mean)^2
      if (lane == 0) buf[slot][warp] = make_float2(sum, q);
      __syncthreads();
      float S = 0.f, Q = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) S += buf[slot][w].x;
      const float m = S * inv_d;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 p = buf[slot][w], n = cols[w];
        const float d = fmaf(p.x, n.y, -m);
        Q += fmaf(layer ? n.x * d : 0.f, d, p.y);
      }
      slot ^= 1;
      mean = layer ? m : 0.f;
      q = Q;
    }
    const float f = rsqrtf(fmaf(q, inv_d, eps));
    return make_float2(f, -mean * f);
  }

  // largest bf16 magnitude of the row, as bits
  __device__ __forceinline__ uint32_t amax(uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (W > 1) {
      if (lane == 0) buf[slot][warp].x = __uint_as_float(m);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, __float_as_uint(buf[slot][w].x));
      slot ^= 1;
    }
    return m;
  }
};

// The sample of row t: the last b with offsets[b] <= t, -1 for a row of no sample.
__device__ __forceinline__ int sample_of(const int32_t *off, int B, int64_t t) {
  if (t < off[0] || t >= off[B]) return -1;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int W, int NV, bool R32, bool Y32>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) norm_residual_kernel(const NormParams p) {
  constexpr int G = 32 * W;                   // threads per row
  constexpr int kRows = (W == 1 ? 128 : G) / G;  // rows a CTA works on at a time
  __shared__ float2 buf[2][16];
  __shared__ float2 cols[16];
  if (*(volatile const int *)p.status != kDevOk) return;
  const int t = threadIdx.x % G, warp = t >> 5, lane = t & 31;
  const int D = p.D, ng = D / 8;
  const int nv = t < ng ? (ng - 1 - t) / G + 1 : 0;  // column groups of this thread
  if (threadIdx.x < W) {
    int n = 0;
    for (int v = 0; v < NV; ++v) n += min(max(ng - v * G - static_cast<int>(threadIdx.x) * 32, 0), 32);
    cols[threadIdx.x] = make_float2(8.f * n, n > 0 ? 1.f / (8.f * n) : 0.f);
  }
  __syncthreads();
  RowStats<W, NV> st{buf, cols, 1.f / static_cast<float>(D), p.eps, nv, warp, lane};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  // The next row's loads are issued before the current row's arithmetic: registers hold one
  // row of inputs in flight per thread.
  Raw8<R32> res[NV];
  Raw8<Y32> y[NV];
  const bool has_y = p.y != nullptr;
  auto fetch = [&](int64_t row) {
    if (row >= p.T) return;
    const int64_t base = row * D + t * 8;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v < NV - 1 || v < nv) {  // only a thread's last group may be missing
        res[v] = raw8<R32>(p.res, base + v * G * 8);
        if (has_y) y[v] = raw8<Y32>(p.y, base + v * G * 8);
      }
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G;
  fetch(row);
  for (; row < p.T; row += step) {
    float2 r[NV][4], x[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (has_y) unpack8<Y32>(y[v], r[v]);
      unpack8<R32>(res[v], x[v]);
    }
    fetch(row + step);
    int b = 0;
    if (p.offsets != nullptr) {
      b = sample_of(p.offsets, p.B, row);
      if (b < 0) continue;  // the same for all threads of the row
    }
    const int64_t mod = static_cast<int64_t>(b) * p.ld_mod + t * 8;
    const int64_t base = row * D + t * 8;
    const float2 rs = both(p.res_scale);
    if (has_y) {
      if (p.post_norm != kNormNone) {
        const float2 f = st.norm(r, p.post_norm == kNormLayer);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float2 a[4];
          if (p.post_weight != nullptr && (v < NV - 1 || v < nv)) load8(p.post_weight, 0, (v * G + t) * 8, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[v][e] = fma2(r[v][e], both(f.x), both(f.y));
            if (p.post_weight != nullptr) r[v][e] = mul2(r[v][e], a[e]);
          }
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
          float2 a[4];
          if (p.gate != nullptr) {
            load8(p.gate, p.mod_f32, mod + v * G * 8, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[v][e] = mul2(r[v][e], a[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = fma2(rs, x[v][e], r[v][e]);
        }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v][e] = mul2(rs, x[v][e]);
    }
    if (p.res_out != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
          const int64_t i = base + v * G * 8;
          if (R32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.res_out) + i);
            o[0] = make_float4(r[v][0].x, r[v][0].y, r[v][1].x, r[v][1].y);
            o[1] = make_float4(r[v][2].x, r[v][2].y, r[v][3].x, r[v][3].y);
          } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.res_out) + i) = pack8(r[v]);
          }
        }
    }
    if (p.out == nullptr) continue;
    const float2 f = st.norm(r, p.norm == kNormLayer);
    uint4 h[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v] = make_uint4(0, 0, 0, 0);
      if (v < NV - 1 || v < nv) {
        const int c = (v * G + t) * 8;
        float2 a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v][e] = fma2(r[v][e], both(f.x), both(f.y));
        if (p.weight != nullptr) {
          load8(p.weight, 0, c, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = mul2(r[v][e], a[e]);
        }
        if (p.bias != nullptr) {
          load8(p.bias, 0, c, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = add2(r[v][e], a[e]);
        }
        if (p.scale != nullptr) {
          load8(p.scale, p.mod_f32, mod + v * G * 8, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = fma2(r[v][e], a[e], r[v][e]);
        }
        if (p.shift != nullptr) {
          load8(p.shift, p.mod_f32, mod + v * G * 8, a);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = add2(r[v][e], a[e]);
        }
        h[v] = pack8(r[v]);
      }
    }
    if (p.out_format == kOutBf16) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv)
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + base + v * G * 8) = h[v];
      continue;
    }
    // quantised rows of the bf16 values in h
    uint32_t m[NV];
    uint32_t row_max = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      m[v] = amax_fold(amax_bf16x2(amax_bf16x2(amax_bf16x2(amax_bf16x2(0, h[v].x), h[v].y), h[v].z), h[v].w));
      row_max = max(row_max, m[v]);
    }
    if (p.out_format != kOutMxfp4) row_max = st.amax(row_max);
    if (p.out_format == kOutE4m3) {
      const float amax = __uint_as_float(row_max << 16);
      const float inv = amax > 0.f ? __fdiv_rn(448.f, amax) : 1.f;
      if (t == 0) p.out_row_scales[row] = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
          const uint32_t w[4] = {h[v].x, h[v].y, h[v].z, h[v].w};
          uint32_t o[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t c0 = __nv_cvt_float_to_fp8(__fmul_rn(bf16_lo(w[e]), inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t c1 = __nv_cvt_float_to_fp8(__fmul_rn(bf16_hi(w[e]), inv), __NV_SATFINITE, __NV_E4M3);
            o[e >> 1] |= (c0 | c1 << 8) << (16 * (e & 1));
          }
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + base + v * G * 8) = make_uint2(o[0], o[1]);
        }
      continue;
    }
    const bool nv4 = p.out_format == kOutNvfp4;
    float rs_inv = 1.f;
    if (nv4) {
      const float rs = nvfp4_row_scale(row_max);
      rs_inv = nvfp4_row_inv(row_max);
      if (t == 0) p.out_row_scales[row] = rs;
    }
    const int64_t tiles = fp4_scale_tiles(D, nv4 ? kNvfp4 : kMxfp4);
    const int pad_ng = (D + 255) / 256 * 32;  // column groups that carry scale bytes
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = v * G + t;
      // blocks of 16 or 32 columns: 2 or 4 neighbouring lanes
      uint32_t am = max(m[v], __shfl_xor_sync(0xffffffffu, m[v], 1));
      float inv;
      uint32_t sb;
      if (nv4) {
        sb = nvfp4_block_scale(am, rs_inv, &inv);
      } else {
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        sb = mxfp4_block_scale(am, &inv);
      }
      if (g >= ng) sb = 0;
      const int kl = nv4 ? 2 : 4;  // lanes per block, the first of them writes its scale byte
      if ((lane & (kl - 1)) == 0 && g < pad_ng)
        p.out_scales[fp4_scale_offset(row, g / kl, tiles)] = static_cast<uint8_t>(sb);
      if (g < ng) {
        const uint32_t w[4] = {h[v].x, h[v].y, h[v].z, h[v].w};
        float q[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
          const float2 d = nv4 ? e2m1_grid(u, inv) : mul2(u, both(inv));
          q[2 * e] = d.x, q[2 * e + 1] = d.y;
        }
        static_cast<uint32_t *>(p.out)[row * (D / 8) + g] = e2m1x8(q);
      }
    }
  }
}

template <int W, int NV>
void launch_nv(const NormParams &p, unsigned blocks, cudaStream_t s) {
  const unsigned threads = W == 1 ? 128 : 32 * W;
  if (p.res_f32) {
    if (p.y_f32) norm_residual_kernel<W, NV, true, true><<<blocks, threads, 0, s>>>(p);
    else norm_residual_kernel<W, NV, true, false><<<blocks, threads, 0, s>>>(p);
  } else {
    if (p.y_f32) norm_residual_kernel<W, NV, false, true><<<blocks, threads, 0, s>>>(p);
    else norm_residual_kernel<W, NV, false, false><<<blocks, threads, 0, s>>>(p);
  }
}

template <int W>
cudaError_t launch_w(const NormParams &p, cudaStream_t s) {
  const int need = (p.D / 8 + 32 * W - 1) / (32 * W);
  const int rows = W == 1 ? 4 : 1;
  // resident CTAs, so that each prefetches its next row (W = 16: one or two per SM)
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((p.T + rows - 1) / rows, 148 * (W == 16 ? 2 : 6)));
  switch (need) {
    case 1: launch_nv<W, 1>(p, blocks, s); break;
    case 2: launch_nv<W, 2>(p, blocks, s); break;
    case 3: launch_nv<W, 3>(p, blocks, s); break;
    default: launch_nv<W, 4>(p, blocks, s); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_residual(const NormParams &p, cudaStream_t s) {
  if (p.T <= 0) return cudaSuccess;
  if (p.D <= 32 * 8 * 4) return launch_w<1>(p, s);
  if (p.D <= 128 * 8 * 4) return launch_w<4>(p, s);
  return launch_w<16>(p, s);
}

}  // namespace cm
