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
// A row is held by one warp or by 2 to 16 warps of one CTA, NV groups of 8 columns
// per thread; column group v * G + t belongs to thread t, so every access is 16
// bytes per lane and consecutive over a warp.
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
// Column e of the eight.
template <bool F32>
__device__ __forceinline__ float at8(const Raw8<F32> &r, int e) {
  const uint4 &u = r.w[F32 ? e >> 2 : 0];
  const int i = F32 ? e & 3 : e >> 1;
  const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
  return F32 ? __uint_as_float(w) : e & 1 ? bf16_hi(w) : bf16_lo(w);
}

__device__ __forceinline__ uint4 pack8(const float *v) {
  return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
}

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
  __device__ __forceinline__ float2 norm(const float (&r)[NV][8], bool layer) {
    float mean = 0.f, sum = 0.f;
    if (layer) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e & 1] += r[v][e];
        }
      sum = warp_sum(s[0] + s[1]);
      mean = sum * cols[warp].y;
    }
    float q2[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v < NV - 1 || v < nv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = r[v][e] - mean;
          q2[e & 1] = fmaf(d, d, q2[e & 1]);
        }
      }
    float q = warp_sum(q2[0] + q2[1]);
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

// The sample of a row, the last b with offsets[b] <= row, -1 for a row of no sample. A CTA's
// rows ascend, so the last answer holds up to the sample's end and costs no loads.
struct SampleOf {
  int b = -1;
  int64_t until = INT64_MIN;  // the answer holds for rows below

  __device__ __forceinline__ int operator()(const int32_t *off, int B, int64_t row) {
    if (row >= until) {
      if (row >= off[B]) {
        b = -1, until = INT64_MAX;
      } else if (row < off[0]) {
        b = -1, until = off[0];
      } else {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (off[mid] <= row) lo = mid;
          else hi = mid;
        }
        b = lo, until = off[hi];
      }
    }
    return b;
  }
};

// h = (r * f.x + f.y) * weight + bias, * (1 + scale) + shift, in r. The usual case, scale and
// shift without weight and bias, takes one test.
template <int NV, bool M32>
__device__ __forceinline__ void modulate(float (&r)[NV][8], float2 f, const NormParams &p, int nv, int G, int col,
                                         int64_t mod) {
  const bool plain = p.weight == nullptr && p.bias == nullptr && p.scale != nullptr && p.shift != nullptr;
  if (plain) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v < NV - 1 || v < nv) {
        const Raw8<M32> a = raw8<M32>(p.scale, mod + col + v * G * 8), c = raw8<M32>(p.shift, mod + col + v * G * 8);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          r[v][e] = fmaf(fmaf(r[v][e], f.x, f.y), 1.f + at8<M32>(a, e), at8<M32>(c, e));
      }
    return;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (v < NV - 1 || v < nv) {
      const int c = col + v * G * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] = fmaf(r[v][e], f.x, f.y);
      if (p.weight != nullptr) {
        const Raw8<false> a = raw8<false>(p.weight, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] *= at8<false>(a, e);
      }
      if (p.bias != nullptr) {
        const Raw8<false> a = raw8<false>(p.bias, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] += at8<false>(a, e);
      }
      if (p.scale != nullptr) {
        const Raw8<M32> a = raw8<M32>(p.scale, mod + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] = fmaf(r[v][e], at8<M32>(a, e), r[v][e]);
      }
      if (p.shift != nullptr) {
        const Raw8<M32> a = raw8<M32>(p.shift, mod + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] += at8<M32>(a, e);
      }
    }
}

template <int NV, bool M32>
__device__ __forceinline__ void apply_gate(float (&r)[NV][8], const NormParams &p, int nv, int G, int col, int64_t mod) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (v < NV - 1 || v < nv) {
      const Raw8<M32> a = raw8<M32>(p.gate, mod + col + v * G * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] *= at8<M32>(a, e);
    }
}

// 4-bit codes and block scales of the bf16 row pieces h, whose magnitudes peak at m.
// sf: where the scale of this thread's first block goes.
template <int FMT, int NV>
__device__ __forceinline__ void write_fp4(const uint4 (&h)[NV], const uint32_t (&m)[NV], float rs_inv, uint32_t *codes,
                                          uint8_t *sf, int t, int G, int ng, int pad_ng) {
  constexpr int kLanes = fp4_block(FMT) / 8;  // lanes per block, the first of them writes its scale byte
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int g = v * G + t;
    uint32_t am = max(m[v], __shfl_xor_sync(0xffffffffu, m[v], 1));
    if (kLanes == 4) am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    float inv;
    const uint32_t sb = FMT == kNvfp4 ? nvfp4_block_scale(am, rs_inv, &inv) : mxfp4_block_scale(am, &inv);
    if ((t & (kLanes - 1)) == 0 && g < pad_ng) sf[v * (G / kLanes / 4) * 512] = static_cast<uint8_t>(g < ng ? sb : 0);
    if (g < ng) {
      const uint32_t w[4] = {h[v].x, h[v].y, h[v].z, h[v].w};
      float q[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
        const float2 d = FMT == kNvfp4 ? e2m1_grid(u, inv) : make_float2(u.x * inv, u.y * inv);
        q[2 * e] = d.x, q[2 * e + 1] = d.y;
      }
      codes[v * G] = e2m1x8(q);
    }
  }
}

// CTAs per SM that the registers are held to (80 a thread, 64 with one column group, 128
// with four); the grid is one wave of them, so that every CTA walks its rows with the next
// one in flight. Measured at 20000 rows of 3072 columns: without y four warps of three column groups
// (45.8 us; with 96 registers 47.8, with 72 and larger spills 57.7; six warps of two 55.9), with y six warps of
// two (80.8 us in bf16, 119.5 with an fp32 residual; four warps of three 93 and 139). With y and quantised
// output four warps of three would take 86.4 instead of 98 us, but the sums' order, and with it
// some last bits, would then differ between the output formats.
// The budgets were chosen at that width and hold for all. There the bf16 forms spill nothing, the fp32 one without y 68
// bytes a thread; others spill up to 136 bytes, and 20 to 248 above 8192 columns, where one CTA of 16 warps is all that an
// SM holds. Over the time of the bytes at the copy rate, 61 M values, gated bf16 (fp32 without y): 1536 columns 1.13
// (1.06), 3072 1.09 (1.04), 5120 1.23 (1.35), 8192 1.31 (1.40), 10240 1.48 (1.49), 16384 1.66 (1.59).
constexpr int ctas_per_sm(int W, int NV, bool r32, int y) {
  const int regs = NV == 4 || (NV == 3 && W == 16 && y != 0) ? 128 : NV == 1 || (NV == 2 && y == 0 && !r32) ? 64 : 80;
  const int n = 65536 / (32 * (W == 1 ? 4 : W) * regs);
  return n < 1 ? 1 : n;
}

// What y is.
enum YKind : int { kYNone = 0, kYBf16 = 1, kYF32 = 2 };

template <int W, int NV, bool R32, int Y>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W, ctas_per_sm(W, NV, R32, Y)) norm_residual_kernel(const NormParams p) {
  constexpr bool has_y = Y != kYNone, Y32 = Y == kYF32;
  constexpr int G = 32 * W;                   // threads per row
  constexpr int kRows = (W == 1 ? 128 : G) / G;  // rows a CTA works on at a time
  __shared__ float2 buf[2][16];
  __shared__ float2 cols[16];
  const int t = threadIdx.x % G, warp = t >> 5, lane = t & 31;
  const int D = p.D, ng = D / 8;
  const int nv = t < ng ? (ng - 1 - t) / G + 1 : 0;  // column groups of this thread
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  // The next row's loads go out as soon as this row's inputs are used up, before its last
  // norm: registers hold one row of inputs in flight per thread.
  Raw8<R32> res[NV];
  Raw8<Y32> y[NV];
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
  if (threadIdx.x < W) {
    int n = 0;
    for (int v = 0; v < NV; ++v) n += min(max(ng - v * G - static_cast<int>(threadIdx.x) * 32, 0), 32);
    cols[threadIdx.x] = make_float2(8.f * n, n > 0 ? 1.f / (8.f * n) : 0.f);
  }
  if (__syncthreads_or(*(volatile const int *)p.status != kDevOk)) return;  // all threads alike
  RowStats<W, NV> st{buf, cols, 1.f / static_cast<float>(D), p.eps, nv, warp, lane};
  SampleOf sample;
  for (; row < p.T; row += step) {
    int b = 0;
    if (p.offsets != nullptr) {
      b = sample(p.offsets, p.B, row);
      if (b < 0) {  // the same for all threads of the row
        fetch(row + step);
        continue;
      }
    }
    const int64_t mod = static_cast<int64_t>(b) * p.ld_mod;
    const int64_t base = row * D + t * 8;
    float r[NV][8];
    if (has_y) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] = at8<Y32>(y[v], e);
      if (p.post_norm != kNormNone) {
        const float2 f = st.norm(r, p.post_norm == kNormLayer);
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v < NV - 1 || v < nv) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = fmaf(r[v][e], f.x, f.y);
            if (p.post_weight != nullptr) {
              const Raw8<false> a = raw8<false>(p.post_weight, (v * G + t) * 8);
#pragma unroll
              for (int e = 0; e < 8; ++e) r[v][e] *= at8<false>(a, e);
            }
          }
      }
      if (p.gate != nullptr) {
        if (p.mod_f32)
          apply_gate<NV, true>(r, p, nv, G, t * 8, mod);
        else
          apply_gate<NV, false>(r, p, nv, G, t * 8, mod);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] = fmaf(p.res_scale, at8<R32>(res[v], e), r[v][e]);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] = at8<R32>(res[v], e);
      if (p.res_scale != 1.f) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) r[v][e] *= p.res_scale;
      }
    }
    fetch(row + step);
    if (p.res_out != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv) {
          const int64_t i = base + v * G * 8;
          if (R32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.res_out) + i);
            o[0] = make_float4(r[v][0], r[v][1], r[v][2], r[v][3]);
            o[1] = make_float4(r[v][4], r[v][5], r[v][6], r[v][7]);
          } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.res_out) + i) = pack8(r[v]);
          }
        }
    }
    if (p.out == nullptr) continue;
    const float2 f = st.norm(r, p.norm == kNormLayer);
    if (p.mod_f32)
      modulate<NV, true>(r, f, p, nv, G, t * 8, mod);
    else
      modulate<NV, false>(r, f, p, nv, G, t * 8, mod);
    if (p.out_format == kOutBf16) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < NV - 1 || v < nv)
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + base + v * G * 8) = pack8(r[v]);
      continue;
    }
    // quantised rows of the bf16 values
    uint4 h[NV];
    uint32_t m[NV];
    uint32_t row_max = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v] = v < NV - 1 || v < nv ? pack8(r[v]) : make_uint4(0, 0, 0, 0);
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
    const int pad_ng = (ng + 31) / 32 * 32;  // column groups that carry scale bytes: whole 256 columns
    uint32_t *codes = static_cast<uint32_t *>(p.out) + row * ng + t;
    uint8_t *sf = p.out_scales + fp4_scale_offset(row, t / (nv4 ? 2 : 4), fp4_scale_tiles(D, nv4 ? kNvfp4 : kMxfp4));
    if (nv4) {
      if (t == 0) p.out_row_scales[row] = nvfp4_row_scale(row_max);
      write_fp4<kNvfp4, NV>(h, m, nvfp4_row_inv(row_max), codes, sf, t, G, ng, pad_ng);
    } else {
      write_fp4<kMxfp4, NV>(h, m, 1.f, codes, sf, t, G, ng, pad_ng);
    }
  }
}

template <int W, int NV, bool R32, int Y>
void launch_types(const NormParams &p, cudaStream_t s) {
  const int rows = W == 1 ? 4 : 1;
  const int64_t blocks = std::min<int64_t>((p.T + rows - 1) / rows, 148 * ctas_per_sm(W, NV, R32, Y));
  norm_residual_kernel<W, NV, R32, Y><<<static_cast<unsigned>(blocks), W == 1 ? 128 : 32 * W, 0, s>>>(p);
}

// The kernel takes all but a thread's last column group for granted: each width goes to
// the form whose groups it fills but for the last.
//
// Without y: two or three column groups per thread (one at the smallest widths, four at the largest).
template <bool R32>
void launch_plain(const NormParams &p, cudaStream_t s) {
  const int ng = p.D / 8;
  if (ng <= 32) launch_types<1, 1, R32, kYNone>(p, s);
  else if (ng <= 64) launch_types<1, 2, R32, kYNone>(p, s);
  else if (ng <= 96) launch_types<1, 3, R32, kYNone>(p, s);
  else if (ng <= 128) launch_types<2, 2, R32, kYNone>(p, s);
  else if (ng <= 192) launch_types<2, 3, R32, kYNone>(p, s);
  else if (ng <= 256) launch_types<4, 2, R32, kYNone>(p, s);
  else if (ng <= 384) launch_types<4, 3, R32, kYNone>(p, s);
  else if (ng <= 512) launch_types<8, 2, R32, kYNone>(p, s);
  else if (ng <= 768) launch_types<8, 3, R32, kYNone>(p, s);
  else if (ng <= 1024) launch_types<16, 2, R32, kYNone>(p, s);
  else if (ng <= 1536) launch_types<16, 3, R32, kYNone>(p, s);
  else launch_types<16, 4, R32, kYNone>(p, s);
}

// With y: up to two column groups per thread (three and four at the largest widths).
template <bool R32, int Y>
void launch_gated(const NormParams &p, cudaStream_t s) {
  const int ng = p.D / 8;
  if (ng <= 32) launch_types<1, 1, R32, Y>(p, s);
  else if (ng <= 64) launch_types<1, 2, R32, Y>(p, s);
  else if (ng <= 128) launch_types<2, 2, R32, Y>(p, s);
  else if (ng <= 256) launch_types<4, 2, R32, Y>(p, s);
  else if (ng <= 384) launch_types<6, 2, R32, Y>(p, s);
  else if (ng <= 512) launch_types<8, 2, R32, Y>(p, s);
  else if (ng <= 768) launch_types<12, 2, R32, Y>(p, s);
  else if (ng <= 1024) launch_types<16, 2, R32, Y>(p, s);
  else if (ng <= 1536) launch_types<16, 3, R32, Y>(p, s);
  else launch_types<16, 4, R32, Y>(p, s);
}

}  // namespace

cudaError_t launch_norm_residual(const NormParams &p, cudaStream_t s) {
  if (p.T <= 0) return cudaSuccess;
  if (p.y == nullptr) {
    if (p.res_f32) launch_plain<true>(p, s);
    else launch_plain<false>(p, s);
  } else if (p.res_f32) {
    if (p.y_f32) launch_gated<true, kYF32>(p, s);
    else launch_gated<true, kYBf16>(p, s);
  } else {
    if (p.y_f32) launch_gated<false, kYF32>(p, s);
    else launch_gated<false, kYBf16>(p, s);
  }
  return cudaGetLastError();
}

}  // namespace cm
