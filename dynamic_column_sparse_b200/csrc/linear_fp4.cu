// linear_fp4.cu - product of 4-bit microscaled rows on the block-scaled tensor
// core path (tcgen05.mma kind::mxf4nvf4, fp32 accumulators in TMEM):
//   out[t][n] = act(rx[t] rw[n] sum_k x[t][k] w[n][k] + bias[n])
// with x [T][K] and w [N][K] as codes, block scales and (NVFP4) row scales.
//
// Persistent, one CTA per SM. Two forms: a CTA pair (cta_group::2) on a 256 x
// 256 output tile, each CTA holding 128 rows of x, 128 rows of w and 128 rows of
// the result; and one CTA on a 128 x 128 tile where the larger tiles would leave SMs
// idle. Tiles are walked weight-slice fastest, so a row block of x is read
// from HBM once while the weights stay in L2.
//
// Warp 0 fills a ring of stages of 256 columns with TMA: code tiles
// (128-byte swizzle) and the block scales' 512-byte tiles. Warp 1 (of the leading CTA)
// copies scales to TMEM and issues the MMAs. The scale columns are a ring of
// their own, one slot per scale tile, filled one slot ahead of the MMAs: with a
// copy and its MMAs back to back the tensor core idled more than half the time
// (546 of 1240 cycles per stage busy, ncu). Warps 2-9 drain one accumulator (scales,
// bias, activation, rounding, TMA stores through swizzled shared memory) while
// the other is being filled. At 256 columns the two accumulators share 64 TMEM
// columns, which leaves 64 for the scales: the shared columns are drained first and the next
// tile's MMAs wait for them only.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace cm {
namespace {

// CG CTAs per tile; BN tile columns; 128 * CG tile rows.
template <int CG, int BN>
struct LinCfg {
  static constexpr int kStages = CG == 2 ? 5 : 5;
  static constexpr int kBRows = BN / CG;  // rows of w a CTA loads
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = kBRows * 128;
  static constexpr uint32_t kSaBytes = 2048, kSbBytes = BN / 128 * 2048;  // MXFP4 uses half
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr uint32_t kOutBytes = 4096;  // 32 rows x 128 bytes, one per epilogue warp
  static constexpr uint32_t kOutOff = kStages * kStageBytes;
  static constexpr uint32_t kColOff = kOutOff + 8 * kOutBytes;  // [BN] row scale of w and bias, bf16 each
  static constexpr uint32_t kBarOff = kColOff + BN * 4;
  static constexpr uint32_t kSmem = 1024 + kBarOff + 256;
  static constexpr uint32_t kAcc1 = BN == 256 ? 192 : BN;        // TMEM column of the second accumulator
  static constexpr uint32_t kSfCol = kAcc1 + BN;                 // scale slots: 4 columns of x, BN / 32 of w
  static constexpr uint32_t kSfCols = 4 + BN / 32;
  static constexpr int kSfSlots = 5;
  static_assert(kSfCol + kSfSlots * kSfCols <= 512, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory");
};

// Bounded wait of a whole warp, which leaves it together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, int *status, volatile int *abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const bool ok = mbar_wait(bar, parity, status, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// GELU, tanh form, as u * sigmoid(2 z) by the identity (1 + tanh z) / 2 =
// 1 / (1 + e^(-2z)); relative error a few 2^-22.
__device__ __forceinline__ float gelu_sigmoid(float u) {
  const float z2 = 1.5957691216057308f * fmaf(0.044715f * u, u * u, u);  // 2 sqrt(2/pi) (...)
  return __fdividef(u, 1.f + exp2_approx(-1.4426950408889634f * z2));
}

// 64 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float *v) {
  tmem_ld32_async(taddr, v);
  tmem_ld32_async(taddr + 32, v + 32);
  tmem_wait_ld_regs(v);
  reg_fence32(v + 32);
}

template <int FMT, int CG, int BN>
__global__ void __launch_bounds__(320, 1)
    linear_fp4_kernel(const __grid_constant__ LinearFp4Maps m, const LinearFp4Params p) {
  using C = LinCfg<CG, BN>;
  constexpr int S = C::kStages;
  constexpr bool S16 = FMT == kNvfp4;
  constexpr int kAtoms = S16 ? 4 : 2;       // scale tiles per stage and 128 rows
  constexpr int kPerAtom = 4 / kAtoms;      // MMAs (64 columns of K) per scale tile
  constexpr uint32_t kTx = CG * (C::kABytes + C::kBBytes + kAtoms * 512 * (1 + BN / 128));
  constexpr int kEpiArrivals = 8 * CG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align_up<1024>(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *empty = full + S;
  uint64_t *acc_full = empty + S;      // [2]
  uint64_t *acc_empty = acc_full + 2;  // [2]
  uint64_t *shared_empty = acc_empty + 2;  // the columns both accumulators share are drained
  uint64_t *col_bar = shared_empty + 1;    // the epilogue warps of this CTA
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(col_bar + 1);
  uint32_t *go = tmem_slot + 1;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int tiles_m = (p.T + 128 * CG - 1) / (128 * CG), tiles_n = (p.N + BN - 1) / BN;
  const int ntiles = tiles_m * tiles_n;
  const int first = static_cast<int>(blockIdx.x) / CG, step = static_cast<int>(gridDim.x) / CG;
  const int nk = (p.K + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kEpiArrivals);
    }
    mbar_init(shared_empty, kEpiArrivals / 2);
    mbar_init(col_bar, 8);
    *abort_flag = 0;
    *go = *(volatile int *)p.status == kDevOk;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's
  // both CTAs of a pair go by the leader's reading of the status word
  const bool run = (CG == 2 ? cluster_load(cluster_addr(go, 0)) : *go) != 0;

  if (!run) {
  } else if (warp == 0) {
    const uint32_t lead = elect_lane();
    int s = 0, kg = 0;
    uint32_t ph = 1;  // parity of the wait for an empty stage
    bool ok = true;
    for (int tile = first; tile < ntiles && ok; tile += step) {
      const int mt = tile / tiles_n, nt = tile - mt * tiles_n;
      const int xr = mt * CG + rank;  // this CTA's 128 rows of x
      for (int kb = 0; kb < nk; ++kb, ++kg) {
        if (!wait_warp(&empty[s], ph, p.status, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t *a = smem + s * C::kStageBytes, *b = a + C::kABytes, *sa = b + C::kBBytes, *sb = sa + C::kSaBytes;
        if (CG == 1 || rank == 0) mbar_arrive_expect_tx_lead(&full[s], kTx, lead);
        const uint32_t bar = CG == 2 ? cluster_addr(&full[s], 0) : smem_u32(&full[s]);
        tma_load_2d_lead<CG>(a, &m.x, bar, kb * 128, xr * 128, lead);
        tma_load_2d_lead<CG>(b, &m.w, bar, kb * 128, nt * BN + rank * C::kBRows, lead);
        tma_load_3d_lead<CG>(sa, &m.sx, bar, 0, kb * kAtoms, xr, lead);
        tma_load_3d_lead<CG>(sb, &m.sw, bar, 0, kb * kAtoms, nt * (BN / 128), lead);
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    if (!ok && rank == 0)  // gave up: let the copies in flight land before the shared memory goes away
      for (int f = max(kg - S, 0); f < kg; ++f) mbar_drain(&full[f % S], (f / S) & 1);
  } else if (warp == 1 && rank == 0) {
    const uint32_t lead = elect_lane();
    const int my_tiles = first < ntiles ? (ntiles - 1 - first) / step + 1 : 0;
    int left = my_tiles * nk;          // stages not yet looked at
    const uint64_t desc_ab = sdesc_sw128(smem_u32(smem), 16, 1024), desc_sf = sdesc_plain(smem_u32(smem));
    constexpr uint32_t kSfOff = C::kABytes + C::kBBytes;
    uint32_t sf = C::kSfCol;           // columns of the next scale slot
    // copies scale tile j of stage s into the next slot; returns the slot's columns
    auto copy_scales = [&](int s, int j) {
      const uint64_t d = desc_sf + static_cast<uint64_t>((s * C::kStageBytes + kSfOff + 512 * j) >> 4);
      const uint32_t at = sf;
      tmem_cp_scales<CG>(tmem + at, d, lead);
#pragma unroll
      for (int i = 0; i < BN / 128; ++i)
        tmem_cp_scales<CG>(tmem + at + 4 + 4 * i, d + ((C::kSaBytes + i * kAtoms * 512) >> 4), lead);
      sf = at + C::kSfCols == C::kSfCol + C::kSfSlots * C::kSfCols ? C::kSfCol : at + C::kSfCols;
      return tmem + at;
    };
    int s = 0;
    uint32_t ph = 0;
    bool ok = left > 0 && wait_warp(&full[0], 0, p.status, abort_flag);
    uint32_t next = 0;
    if (ok) {
      tc_fence_after();
      next = copy_scales(0, 0);
    }
    for (int tl = 0; tl < my_tiles && ok; ++tl) {
      const int ab = tl & 1;
      const uint32_t acc = tmem + ab * C::kAcc1;
      ok = wait_warp(&acc_empty[ab], ((tl >> 1) & 1) ^ 1, p.status, abort_flag);
      if (BN == 256 && ok && tl > 0) ok = wait_warp(shared_empty, (tl - 1) & 1, p.status, abort_flag);
      tc_fence_after();
      for (int kb = 0; kb < nk && ok; ++kb) {
        const uint64_t da = desc_ab + static_cast<uint64_t>((s * C::kStageBytes) >> 4), db = da + (C::kABytes >> 4);
        const int s1 = s + 1 == S ? 0 : s + 1;
        const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph;
        --left;
#pragma unroll
        for (int j = 0; j < kAtoms; ++j) {
          const uint32_t sa = next;
          if (j + 1 < kAtoms) {
            next = copy_scales(s, j + 1);
          } else if (left > 0) {
            ok = wait_warp(&full[s1], ph1, p.status, abort_flag);
            if (!ok) break;
            tc_fence_after();
            next = copy_scales(s1, 0);
          }
#pragma unroll
          for (int q = 0; q < kPerAtom; ++q) {
            const int kk = j * kPerAtom + q;
            umma_fp4<S16, CG>(acc, da + kk * 2, db + kk * 2, idesc_fp4(128 * CG, BN, S16, q * 2), sa, sa + 4,
                              (kb | kk) != 0, lead);
          }
        }
        if (!ok) break;
        umma_commit_lead<CG>(&empty[s], lead);
        if (kb == nk - 1) umma_commit_lead<CG>(&acc_full[ab], lead);
        s = s1, ph = ph1;
      }
    }
  } else if (warp >= 2) {
    // two warps per lane quadrant, each half of the tile's columns
    constexpr int kCols = BN / 2, kChunks = kCols / 64;
    const int quad = warp & 3;  // TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;
    const int e = threadIdx.x - 64;
    uint8_t *stage = smem + C::kOutOff + (warp - 2) * C::kOutBytes;
    uint32_t *cols = reinterpret_cast<uint32_t *>(smem + C::kColOff);
    int tl = 0;
    // a drained accumulator (or its shared columns) goes back to the leader's MMA warp
    auto release = [&](uint64_t *bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster_relaxed(cluster_addr(bar, 0));
        else
          mbar_arrive(bar);
      }
    };
    for (int tile = first; tile < ntiles; tile += step, ++tl) {
      const int mt = tile / tiles_n, nt = tile - mt * tiles_n;
      const int ab = tl & 1;
      const int row0 = (mt * CG + rank) * 128 + quad * 32;
      // this row's factor; this thread's column: row scale of w above, bias below, both bf16
      const float rx = S16 && row0 + lane < p.T ? p.rx[row0 + lane] : 1.f;
      const int n = nt * BN + e;
      uint32_t col = 0x3f800000u;
      if (e < BN && n < p.N) {
        if (S16) col = static_cast<uint32_t>(f32_to_bf16_bits(p.rw[n])) << 16;
        if (p.bias != nullptr) col |= p.bias[n];
      }
      // the warps have read the previous tile's column values; put this tile's in place
      if (lane == 0) mbar_arrive(col_bar);
      if (!wait_warp(col_bar, 0, p.status, abort_flag)) break;
      if (e < BN) cols[e] = col;
      __syncwarp();
      if (lane == 0) mbar_arrive(col_bar);
      if (!wait_warp(col_bar, 1, p.status, abort_flag)) break;
      if (!wait_warp(&acc_full[ab], (tl >> 1) & 1, p.status, abort_flag)) break;
      tc_fence_after();
      // The columns both accumulators share are the last 64 of the first one and the
      // first 64 of the second: held by the warps of one half, which drain them first.
      const bool has_shared = BN == 256 && half == (ab ^ 1);
      for (int i = 0; i < kChunks; ++i) {
        const int c0 = half * kCols + (BN == 256 && ab == 0 && half == 1 ? kChunks - 1 - i : i) * 64;
        float v[64];
        tmem_ld64(tmem + ab * C::kAcc1 + (static_cast<uint32_t>(quad * 32) << 16) + c0, v);
        if (has_shared && i == 0) release(shared_empty);
        if (i == kChunks - 1) release(&acc_empty[ab]);
        // Every lane reads every column's values, a shared-memory wavefront for each
        // word: with fp32 values these reads were the longest part of the epilogue.
#pragma unroll
        for (int g = 0; g < 64; g += 16) {
          uint4 w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4 *>(cols + c0 + g + 4 * q);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t w0 = q & 1 ? w[q >> 1].z : w[q >> 1].x, w1 = q & 1 ? w[q >> 1].w : w[q >> 1].y;
            float2 &u = *reinterpret_cast<float2 *>(v + g + 2 * q);
            const float2 o = make_float2(bf16_lo(w0), bf16_lo(w1));
            u = S16 ? fma2(u, mul2(make_float2(rx, rx), make_float2(bf16_hi(w0), bf16_hi(w1))), o)
                    : make_float2(u.x + o.x, u.y + o.y);
          }
        }
        if (p.gelu) {
#pragma unroll
          for (int q = 0; q < 64; ++q) v[q] = gelu_sigmoid(v[q]);
        }
        const int x0 = nt * BN + c0;
        auto store = [&](int x) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (x < p.N && row0 < p.T) tma_store_2d(&m.out, stage, x, row0);
            bulk_commit();
          }
        };
        auto free_buffer = [&]() {  // the warp's last store has read the buffer
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        };
        if (p.out_f32) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            free_buffer();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4 *>(stage + sw128_offset(lane, q)) = make_float4(
                  v[32 * hf + 4 * q], v[32 * hf + 4 * q + 1], v[32 * hf + 4 * q + 2], v[32 * hf + 4 * q + 3]);
            store(x0 + 32 * hf);
          }
        } else {
          free_buffer();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(stage + sw128_offset(lane, q)) =
                make_uint4(cvt_bf16x2(v[8 * q], v[8 * q + 1]), cvt_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                           cvt_bf16x2(v[8 * q + 4], v[8 * q + 5]), cvt_bf16x2(v[8 * q + 6], v[8 * q + 7]));
          store(x0);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // neither CTA's memory goes away while the other still uses it
  tc_fence_after();
  if (warp == 1) {
    if (CG == 2)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

template <int CG, int BN>
cudaError_t launch_form(const LinearFp4Params &p, LinearFp4Maps m, int sms, cudaStream_t s) {
  using C = LinCfg<CG, BN>;
  const int64_t tiles = static_cast<int64_t>((p.T + 128 * CG - 1) / (128 * CG)) * ((p.N + BN - 1) / BN);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(tiles, sms / CG)) * CG;
  auto kernel = p.fmt == kNvfp4 ? linear_fp4_kernel<kNvfp4, CG, BN> : linear_fp4_kernel<kMxfp4, CG, BN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(320);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, m, p);
}

}  // namespace

cudaError_t launch_linear_fp4(const LinearFp4Params &p, const LinearFp4Maps &m, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return m.pair ? launch_form<2, 256>(p, m, sms, s) : launch_form<1, 128>(p, m, sms, s);
}

// The form whose waves over 148 SMs are fewer: a wave of pair tiles takes about as
// long as one of single tiles.
bool linear_fp4_pair(int64_t T, int64_t N) {
  const int64_t pair = ((T + 255) / 256) * ((N + 255) / 256), single = ((T + 127) / 128) * ((N + 127) / 128);
  return (pair + 73) / 74 < (single + 147) / 148;
}

}  // namespace cm
