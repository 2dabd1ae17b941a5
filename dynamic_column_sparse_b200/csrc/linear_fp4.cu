// linear_fp4.cu - product of 4-bit microscaled rows on the block-scaled tensor
// core path (tcgen05.mma kind::mxf4nvf4, fp32 accumulators in TMEM):
//   out[t][n] = act(rx[t] rw[n] sum_k x[t][k] w[n][k] + bias[n])
// with x [T][K] and w [N][K] as codes, block scales and (NVFP4) row scales.
//
// Persistent, one CTA per SM, one 128 x 128 output tile at a time, tiles walked
// weight-slice fastest so a row block of x is read from HBM once while the
// weights stay in L2. Warp 0 fills a ring of stages of 256 columns: both code tiles
// by TMA (128-byte swizzle), both tiles' block scales by bulk copies of their
// consecutive 512-byte scale tiles. Warp 1 copies a stage's scales to TMEM and
// issues its four MMAs. Warps 2-5 drain one accumulator (scales, bias,
// activation, rounding, TMA stores through swizzled shared memory) while the
// other is being filled.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace cm {
namespace {

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int *status, volatile int *abort_flag) {
  const bool ok = mbar_wait(bar, parity, status, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

struct LinCfg {
  static constexpr int kStages = 5;
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = 128 * 128;
  static constexpr uint32_t kSfBytes = 2048;  // 128 rows x 256 columns of scales (MXFP4 uses half)
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + 2 * kSfBytes;
  static constexpr uint32_t kOutBytes = 4096;  // 32 rows x 128 bytes, two per epilogue warp
  static constexpr uint32_t kOutOff = kStages * kStageBytes;
  static constexpr uint32_t kColOff = kOutOff + 8 * kOutBytes;  // [2][2][128] fp32 row scales of w, bias
  static constexpr uint32_t kBarOff = kColOff + 2 * 2 * 128 * 4;
  static constexpr uint32_t kSmem = 1024 + kBarOff + 256;
  static constexpr uint32_t kSfCol = 256;  // TMEM columns past the two accumulators
};

// GELU, tanh form, as u * sigmoid(2 z) with the exact exponential identity
// (1 + tanh z) / 2 = 1 / (1 + e^(-2z)); relative error a few 2^-22.
__device__ __forceinline__ float gelu_exact(float u) {
  const float z2 = 1.5957691216057308f * fmaf(0.044715f * u, u * u, u);  // 2 sqrt(2/pi) (...)
  return __fdividef(u, 1.f + exp2_approx(-1.4426950408889634f * z2));
}

template <int FMT>
__global__ void __launch_bounds__(192, 1)
    linear_fp4_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_out, const LinearFp4Params p) {
  using C = LinCfg;
  constexpr int S = C::kStages;
  constexpr bool S16 = FMT == kNvfp4;
  constexpr int kAtoms = S16 ? 4 : 2;  // 512-byte scale tiles per stage and operand
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align_up<1024>(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *empty = full + S;
  uint64_t *acc_full = empty + S;      // [2]
  uint64_t *acc_empty = acc_full + 2;  // [2]
  uint64_t *col_bar = acc_empty + 2;   // the epilogue's per-column values of a tile are in place
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(col_bar + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (*(volatile int *)p.status != kDevOk) return;
  const int tiles_m = (p.T + 127) / 128, tiles_n = (p.N + 127) / 128;
  const int ntiles = tiles_m * tiles_n;
  const int nk = (p.K + 255) / 256;
  const int64_t sf_tiles = static_cast<int64_t>(nk) * kAtoms;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 128);
    }
    mbar_init(col_bar, 128);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    int kg = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      const int mt = tile / tiles_n, nt = tile - mt * tiles_n;
      for (int kb = 0; kb < nk; ++kb, ++kg) {
        const int s = kg % S;
        if (!wait_warp(&empty[s], ((kg / S) & 1) ^ 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t *st = smem + s * C::kStageBytes;
          mbar_arrive_expect_tx(&full[s], C::kABytes + C::kBBytes + 2 * kAtoms * 512);
          tma_load_2d(st, &tm_x, &full[s], kb * 128, mt * 128);
          tma_load_2d(st + C::kABytes, &tm_w, &full[s], kb * 128, nt * 128);
          bulk_load(st + C::kABytes + C::kBBytes, p.sx + (mt * sf_tiles + kb * kAtoms) * 512, kAtoms * 512, &full[s]);
          bulk_load(st + C::kABytes + C::kBBytes + C::kSfBytes, p.sw + (nt * sf_tiles + kb * kAtoms) * 512,
                    kAtoms * 512, &full[s]);
        }
        __syncwarp();
      }
    }
    if (!ok)  // gave up: let the copies in flight land before the CTA's shared memory goes away
      for (int f = max(kg - S, 0); f < kg; ++f) mbar_drain(&full[f % S], (f / S) & 1);
  } else if (warp == 1) {
    int kg = 0, tl = 0;
    bool ok = true;
    const uint32_t sfa = tmem + C::kSfCol, sfb = sfa + 16;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x, ++tl) {
      const int ab = tl & 1;
      if (!wait_warp(&acc_empty[ab], ((tl >> 1) & 1) ^ 1, p.status, abort_flag)) break;
      tc_fence_after();
      for (int kb = 0; kb < nk; ++kb, ++kg) {
        const int s = kg % S;
        if (!wait_warp(&full[s], (kg / S) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a0 = smem_u32(smem + s * C::kStageBytes);
          const uint32_t b0 = a0 + C::kABytes, f0 = b0 + C::kBBytes, g0 = f0 + C::kSfBytes;
#pragma unroll
          for (int j = 0; j < kAtoms; ++j) {
            tmem_cp_scales(sfa + 4 * j, sdesc_plain(f0 + 512 * j));
            tmem_cp_scales(sfb + 4 * j, sdesc_plain(g0 + 512 * j));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int j = S16 ? kk : kk >> 1;
            umma_fp4<S16>(tmem + ab * 128, sdesc_sw128(a0 + kk * 32, 16, 1024), sdesc_sw128(b0 + kk * 32, 16, 1024),
                          idesc_fp4(128, 128, S16, S16 ? 0 : (kk & 1) * 2), sfa + 4 * j, sfb + 4 * j,
                          (kb | kk) != 0);
          }
          umma_commit(&empty[s]);
          if (kb == nk - 1) umma_commit(&acc_full[ab]);
        }
        __syncwarp();
      }
    }
  } else {
    const int quad = warp & 3;  // TMEM lanes this warp may read
    const int e = threadIdx.x - 64;
    uint8_t *stage = smem + C::kOutOff + (warp - 2) * 2 * C::kOutBytes;
    float *cols = reinterpret_cast<float *>(smem + C::kColOff);
    int tl = 0, buf = 0;
    for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x, ++tl) {
      const int mt = tile / tiles_n, nt = tile - mt * tiles_n;
      const int ab = tl & 1;
      // this tile's per-column factors and biases (double-buffered by tile), this thread's row factor
      float *rw = cols + ab * 256, *bs = rw + 128;
      const int n = nt * 128 + e;
      rw[e] = S16 && n < p.N ? p.rw[n] : 1.f;
      bs[e] = p.bias != nullptr && n < p.N ? bf16_bits_to_f32(p.bias[n]) : 0.f;
      const int row = mt * 128 + quad * 32 + lane;
      const float rx = S16 && row < p.T ? p.rx[row] : 1.f;
      mbar_arrive(col_bar);
      if (!wait_warp(col_bar, tl & 1, p.status, abort_flag)) break;
      if (!wait_warp(&acc_full[ab], (tl >> 1) & 1, p.status, abort_flag)) break;
      tc_fence_after();
      const int chunk = p.out_f32 ? 32 : 64;  // columns of one 128-byte store row
      for (int c0 = 0; c0 < 128; c0 += chunk) {
        uint8_t *dst = stage + buf * C::kOutBytes;
        if (lane == 0) bulk_wait_read<1>();  // the store that used this buffer has read it
        __syncwarp();
        for (int c1 = 0; c1 < chunk; c1 += 32) {
          float v[32];
          tmem_ld32(tmem + ab * 128 + (static_cast<uint32_t>(quad * 32) << 16) + c0 + c1, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = fmaf(v[i], rx * rw[c0 + c1 + i], bs[c0 + c1 + i]);
            if (p.gelu) v[i] = gelu_exact(v[i]);
          }
          if (p.out_f32) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4 *>(dst + sw128_offset(lane, q)) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4 *>(dst + sw128_offset(lane, c1 / 8 + q)) =
                  make_uint4(cvt_bf16x2(v[8 * q], v[8 * q + 1]), cvt_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                             cvt_bf16x2(v[8 * q + 4], v[8 * q + 5]), cvt_bf16x2(v[8 * q + 6], v[8 * q + 7]));
          }
        }
        if (c0 + chunk >= 128) {  // the accumulator is read out
          tc_fence_before();
          mbar_arrive(&acc_empty[ab]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (nt * 128 + c0 < p.N && mt * 128 + quad * 32 < p.T)
            tma_store_2d(&tm_out, dst, nt * 128 + c0, mt * 128 + quad * 32);
          bulk_commit();
        }
        buf ^= 1;
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_linear_fp4(const LinearFp4Params &p, const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                              const CUtensorMap &tm_out, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>((p.T + 127) / 128) * ((p.N + 127) / 128);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(tiles, sms));
  auto kernel = p.fmt == kNvfp4 ? linear_fp4_kernel<kNvfp4> : linear_fp4_kernel<kMxfp4>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LinCfg::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, 192, LinCfg::kSmem, s>>>(tm_x, tm_w, tm_out, p);
  return cudaGetLastError();
}

}  // namespace cm
