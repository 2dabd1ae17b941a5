// heads.cu - a fused q, k, v projection split into heads: RMS norm of every q
// and k head with a weight, rotation by position, and q, k, v written as the
// contiguous [T][h][128] tensors the attention kernels read.
//
// HBM bound: 16 lanes hold one head of 128 columns (8 each, one 16-byte load);
// the same lanes take q, k and v of their (token, head), so three loads are in
// flight per lane and the token's cosines and sines are read once for q and k.
// fp32 throughout, one rounding at the store.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.cuh"

namespace cm {
namespace {

__device__ __forceinline__ void unpack8(const uint4 &u, float *v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
}

// Norm (over the 16 lanes of the head), weight and rotation of 8 columns.
template <bool HALVES>
__device__ __forceinline__ uint4 norm_rotate(const uint4 &u, const float *w, const float *c, const float *n, float eps,
                                             int sub) {
  float v[8];
  unpack8(u, v);
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  const float r = 1.f / sqrtf(q * (1.f / 128.f) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= r * w[e];
  float o[8];
  if (HALVES) {
    // column i < 64 pairs with column i + 64, held 8 lanes away
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float other = __shfl_xor_sync(0xffffffffu, v[e], 8);
      o[e] = sub < 8 ? v[e] * c[e] - other * n[e] : other * n[e] + v[e] * c[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = v[2 * e] * c[e] - v[2 * e + 1] * n[e];
      o[2 * e + 1] = v[2 * e] * n[e] + v[2 * e + 1] * c[e];
    }
  }
  return make_uint4(cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]), cvt_bf16x2(o[4], o[5]), cvt_bf16x2(o[6], o[7]));
}

template <bool HALVES>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const HeadsParams p) {
  if (*(volatile const int *)p.status != kDevOk) return;
  const int sub = threadIdx.x & 15;
  float qw[8], kw[8];
  unpack8(*reinterpret_cast<const uint4 *>(p.q_weight + sub * 8), qw);
  unpack8(*reinterpret_cast<const uint4 *>(p.k_weight + sub * 8), kw);
  const uint32_t total = static_cast<uint32_t>(p.T * p.h);
  const uint32_t step = gridDim.x * 16;
  // all lanes of a warp run the same number of steps (the norm's shuffles are warp-wide)
  for (uint32_t i0 = blockIdx.x * 16 + (threadIdx.x >> 5) * 2; i0 < total; i0 += step) {
    const uint32_t i = i0 + ((threadIdx.x >> 4) & 1);
    const bool live = i < total;
    const uint32_t it = live ? i : total - 1;
    const uint32_t t = it / static_cast<uint32_t>(p.h), hd = it - t * static_cast<uint32_t>(p.h);
    const int64_t hc = static_cast<int64_t>(p.h) * 128;
    const uint16_t *src = p.qkv + static_cast<int64_t>(t) * p.ld + hd * 128 + sub * 8;
    const uint4 q = *reinterpret_cast<const uint4 *>(src);
    const uint4 k = *reinterpret_cast<const uint4 *>(src + hc);
    const uint4 v = *reinterpret_cast<const uint4 *>(src + 2 * hc);
    // angles of this lane's columns: 4 (neighbouring pairs) or 8 (halves)
    constexpr int kA = HALVES ? 8 : 4;
    float c[kA], n[kA];
    const int64_t a0 = static_cast<int64_t>(t) * 64 + (HALVES ? (sub & 7) * 8 : sub * 4);
#pragma unroll
    for (int a = 0; a < kA; a += 4) {
      *reinterpret_cast<float4 *>(c + a) = *reinterpret_cast<const float4 *>(p.cos + a0 + a);
      *reinterpret_cast<float4 *>(n + a) = *reinterpret_cast<const float4 *>(p.sin + a0 + a);
    }
    const uint4 qo = norm_rotate<HALVES>(q, qw, c, n, p.eps, sub);
    const uint4 ko = norm_rotate<HALVES>(k, kw, c, n, p.eps, sub);
    if (live) {
      const int64_t o = static_cast<int64_t>(it) * 128 + sub * 8;
      *reinterpret_cast<uint4 *>(p.q + o) = qo;
      *reinterpret_cast<uint4 *>(p.k + o) = ko;
      *reinterpret_cast<uint4 *>(p.v + o) = v;
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadsParams &p, cudaStream_t s) {
  if (p.T <= 0) return cudaSuccess;
  const int64_t total = p.T * p.h;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((total + 15) / 16, 148 * 64));
  if (p.halves)
    qk_norm_rope_kernel<true><<<blocks, 256, 0, s>>>(p);
  else
    qk_norm_rope_kernel<false><<<blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace cm
