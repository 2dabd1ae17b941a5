// linear_fp4.cu - product of 4-bit microscaled rows on the block-scaled tensor
// core path (tcgen05.mma kind::mxf4nvf4, fp32 accumulators in TMEM):
//   out[t][n] = act(rx[t] rw[n] sum_k x[t][k] w[n][k] + bias[n])
// with x [T][K] and w [N][K] as codes, block scales and (NVFP4) row scales.
//
// Persistent, one CTA per SM. Three forms: a CTA pair (cta_group::2) on a 256 x
// 256 output tile, each CTA holding 128 rows of x, 128 rows of w and 128 rows of
// the result; and one CTA on a 128 x 256 or 128 x 128 tile where larger tiles would leave SMs
// idle (linear_fp4_form chooses; a fourth form, below, takes a few rows). Tiles are walked weight-slice
// fastest, so a row block of x is read from HBM once while the weights stay in L2.
//
// Warp 0 fills a ring of stages of 256 columns with TMA: code tiles
// (128-byte swizzle) and the block scales' 512-byte tiles. Warp 1 (of the leading CTA)
// copies scales to TMEM and issues the MMAs. What bounded it first was the issuing: inside a
// one-lane branch every tcgen05 instruction took 100 to 150 cycles, against about 21 for a
// scale copy and 33 for an MMA when the whole warp computes the operands and the elected lane is the
// instruction's predicate (4352 x 9216 x 3072: 149.8 -> 70.6 us). The scale columns are a ring of
// their own, one slot per scale tile, filled one slot ahead of the MMAs. Warps 2-9 drain one
// accumulator (scales, bias, activation, rounding, TMA stores through swizzled shared memory) while
// the other is being filled. At 256 columns the two accumulators share 64 TMEM
// columns, which leaves 64 for the scales: the shared columns are drained first and the next
// tile's MMAs wait for them only.
// What bounds it now is shared memory, then power: a stage's 38 KB written and 32 KB read by
// the MMAs take 547 cycles at 128 bytes each (544 measured with K = 12288; the tensor pipe needs 512),
// an epilogue about 2000 more, and the chip runs it at its power cap (4.3 to 4.8 PFLOP/s sustained).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace cm {
namespace {

// CG CTAs per tile; BN tile columns; 128 * CG tile rows.
template <int CG, int BN>
struct LinCfg {
  static constexpr int kStages = CG == 1 && BN == 256 ? 3 : 5;
  static constexpr int kBRows = BN / CG;  // rows of w a CTA loads
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = kBRows * 128;
  static constexpr uint32_t kSaBytes = 2048, kSbBytes = BN / 128 * 2048;  // MXFP4 uses half
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr uint32_t kOutBytes = 4096;  // 32 rows x 128 bytes, one per epilogue warp
  static constexpr uint32_t kOutOff = kStages * kStageBytes;
  static constexpr uint32_t kColOff = kOutOff + 8 * kOutBytes;  // [BN] row scale of w and bias, bf16 each
  static constexpr uint32_t kBiasOff = kColOff + BN * 4;        // [BN] the same with row scales of 1
  static constexpr uint32_t kScaleOff = kBiasOff + BN * 4;      // [BN] row scale of w, fp32
  static constexpr uint32_t kFlagOff = kScaleOff + BN * 4;      // [8] warps whose columns have scales that bf16 does not hold
  static constexpr uint32_t kBarOff = kFlagOff + 32;
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
// 1 / (1 + e^(-2z)). The error is a few 2^-22 of |u|. Relative to the result it grows in the negative tail, where
// the exponent's rounding (a few 2^-24 of 2 |z|) is the result's: to about 2^-15 at 2 |z| = 87, the last fp32 holds.
__device__ __forceinline__ float gelu_sigmoid(float u) {
  const float z2 = 1.5957691216057308f * fmaf(0.044715f * u, u * u, u);  // 2 sqrt(2/pi) (...)
  return __fdividef(u, 1.f + exp2_approx(-1.4426950408889634f * z2));
}

// A sum (at most 2^39, in steps of 2^-20) times a row scale of x and one of w. The scales' product may leave
// fp32's range where the result does not (zero times an infinity above all). So x's scale is brought nearer to
// one by a power of two that the sum takes up (split_scale: the scale, the sum's factor), and a product that
// overflows all the same becomes the largest number, with which every sum but zero still overflows.
__device__ __forceinline__ bool far_from_one(float rx) { return fabsf(rx) >= 0x1p11f || fabsf(rx) < 0x1p-30f; }
__device__ __forceinline__ float2 split_scale(float rx) {
  if (fabsf(rx) >= 0x1p11f) return make_float2(rx * 0x1p-24f, 0x1p24f);
  if (fabsf(rx) < 0x1p-30f) return make_float2(rx * 0x1p40f, 0x1p-40f);
  return make_float2(rx, 1.f);
}
__device__ __forceinline__ float scaled(float sum, float2 f, float rw) {
  float m = f.x * rw;
  if (fabsf(m) == INFINITY) m = copysignf(FLT_MAX, m);
  return sum * f.y * m;
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
    wait_for_primary();  // this kernel is complete only when the one before it is
  } else if (warp == 0) {
    const uint32_t lead = elect_lane();
    // loads of stage kg (K block kb of a tile) into slot s: w's, or x's
    auto load_w = [&](int s, int kb, int nt) {
      uint8_t *b = smem + s * C::kStageBytes + C::kABytes, *sb = b + C::kBBytes + C::kSaBytes;
      if (CG == 1 || rank == 0) mbar_arrive_expect_tx_lead(&full[s], kTx, lead);
      const uint32_t bar = CG == 2 ? cluster_addr(&full[s], 0) : smem_u32(&full[s]);
      tma_load_2d_lead<CG>(b, &m.w, bar, kb * 128, nt * BN + rank * C::kBRows, lead);
      tma_load_3d_lead<CG>(sb, &m.sw, bar, 0, kb * kAtoms, nt * (BN / 128), lead);
    };
    auto load_x = [&](int s, int kb, int mt) {
      uint8_t *a = smem + s * C::kStageBytes, *sa = a + C::kABytes + C::kBBytes;
      const int xr = mt * CG + rank;  // this CTA's 128 rows of x
      const uint32_t bar = CG == 2 ? cluster_addr(&full[s], 0) : smem_u32(&full[s]);
      tma_load_2d_lead<CG>(a, &m.x, bar, kb * 128, xr * 128, lead);
      tma_load_3d_lead<CG>(sa, &m.sx, bar, 0, kb * kAtoms, xr, lead);
    };
    // w does not wait for the quantiser of x that this kernel may have been launched behind: the ring's
    // first turn loads it ahead
    int ahead = 0;
    for (int tile = first; tile < ntiles && ahead < S; tile += step)
      for (int kb = 0; kb < nk && ahead < S; ++kb, ++ahead) load_w(ahead, kb, tile % tiles_n);
    wait_for_primary();
    int s = 0, kg = 0;
    uint32_t ph = 1;  // parity of the wait for an empty stage
    bool ok = true;
    for (int tile = first; tile < ntiles && ok; tile += step) {
      const int mt = tile / tiles_n, nt = tile - mt * tiles_n;
      for (int kb = 0; kb < nk; ++kb, ++kg) {
        if (kg >= ahead) {
          if (!wait_warp(&empty[s], ph, p.status, abort_flag)) {
            ok = false;
            break;
          }
          load_w(s, kb, nt);
        }
        load_x(s, kb, mt);
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    if (!ok && rank == 0)  // gave up: let the copies in flight land before the shared memory goes away
      for (int f = max(kg - S, 0); f < kg; ++f) mbar_drain(&full[f % S], (f / S) & 1);
  } else if (warp == 1 && rank == 0) {
    const uint32_t lead = elect_lane();
    const int my_tiles = first < ntiles ? (ntiles - 1 - first) / step + 1 : 0;
    int left = my_tiles * nk;          // stages not yet looked at
    const uint64_t desc_ab = sdesc_sw128(smem_u32(smem), 16, 1024), desc_sf = sdesc_plain(smem_u32(smem), 128);
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
    uint32_t *biases = reinterpret_cast<uint32_t *>(smem + C::kBiasOff);
    float *scales = reinterpret_cast<float *>(smem + C::kScaleOff);
    uint32_t *flags = reinterpret_cast<uint32_t *>(smem + C::kFlagOff);
    int tl = 0;
    wait_for_primary();  // the row scales of x
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
      // this row's factor; this thread's column: row scale of w above, bias below, both bf16, which holds
      // the quantiser's powers of two and NaN
      float rx = S16 && row0 + lane < p.T ? p.rx[row0 + lane] : 1.f;
      const int n = nt * BN + e;
      float rw = 1.f;
      uint32_t bias = 0;
      if (e < BN && n < p.N) {
        if (S16) rw = p.rw[n];
        if (p.bias != nullptr) bias = p.bias[n];
      }
      const bool odd = S16 && __any_sync(0xffffffffu, (__float_as_uint(rw) & 0xffffu) != 0);
      // the warps have read the previous tile's column values; put this tile's in place
      if (lane == 0) mbar_arrive(col_bar);
      if (!wait_warp(col_bar, 0, p.status, abort_flag)) break;
      if (e < BN) {
        cols[e] = bias | static_cast<uint32_t>(f32_to_bf16_bits(rw)) << 16;
        if (S16) biases[e] = bias | 0x3f800000u, scales[e] = rw;
      }
      if (S16 && lane == 0) flags[warp - 2] = odd;
      __syncwarp();
      if (lane == 0) mbar_arrive(col_bar);
      if (!wait_warp(col_bar, 1, p.status, abort_flag)) break;
      // in a tile with other scales, and in a warp with scales far from one, both are applied ahead of the rest
      bool ahead = false;
      if (S16) {
        const uint4 f0 = reinterpret_cast<const uint4 *>(flags)[0], f1 = reinterpret_cast<const uint4 *>(flags)[1];
        ahead = (f0.x | f0.y | f0.z | f0.w | f1.x | f1.y | f1.z | f1.w) != 0 || __any_sync(0xffffffffu, far_from_one(rx));
      }
      const uint32_t *colp = ahead ? biases : cols;
      const float rxs = rx;
      if (ahead) rx = 1.f;
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
        // Two roundings more, where the scales need it only: 86 instead of 63 us at 12000 x 9216 x 256, 55
        // instead of 46 at 4352 x 12288 x 1024, 56.5 instead of 52.5 at 4352 x 9216 x 3072.
        if (S16 && ahead) {
          const float2 f = split_scale(rxs);
#pragma unroll
          for (int q = 0; q < 64; q += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(scales + c0 + q);
            v[q] = scaled(v[q], f, w.x), v[q + 1] = scaled(v[q + 1], f, w.y);
            v[q + 2] = scaled(v[q + 2], f, w.z), v[q + 3] = scaled(v[q + 3], f, w.w);
          }
        }
        // Every lane reads every column's values, a shared-memory wavefront for each
        // word: with fp32 values these reads were the longest part of the epilogue.
#pragma unroll
        for (int g = 0; g < 64; g += 16) {
          uint4 w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4 *>(colp + c0 + g + 4 * q);
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

// ------------------------------------------------------------------ a few rows

// Products with at most 8 rows, and few enough columns to quantise them anew in every CTA
// (16 of a row per thread and step, at most kRowItems steps): one launch and no workspace.
// Bound by reading w once, in practice by launch and pipeline latency: 1 x 18432 x 3072
// NVFP4 moves 32 MB (4.9 us at the copy rate).
//
// Warps 2-9 quantise x into shared memory while warp 0 already fills the ring with w;
// then warps 4 and 8, whose TMEM lanes hold the rows, are the epilogue. Only one 8-row
// swizzle atom of x exists per stage: the descriptors' stride between 8-row groups is 0, so
// all 128 rows of the instruction read it (and the scale copies likewise); rows from the
// eighth on repeat the first eight, and none but the T first is stored.
constexpr int kRowMax = 8, kRowItems = 2;

constexpr int kRowStagesMax = kRowItems * 16;  // one row of as many columns: 8192

struct RowCfg {
  static constexpr int kStages = 5;
  static constexpr uint32_t kWBytes = 128 * 128, kSwBytes = 2048;
  static constexpr uint32_t kStageBytes = kWBytes + kSwBytes;
  static constexpr uint32_t kXBytes = 1024, kSxBytes = 512;  // x per 256 columns: codes; scales, 128 bytes per tile
  static constexpr uint32_t kXOff = kStages * kStageBytes;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr uint32_t smem(int nk) { return 1024 + kXOff + nk * (kXBytes + kSxBytes) + 2 * 128 * 8 + kBarBytes; }
  static constexpr uint32_t kSfCol = 256, kSfCols = 8;
  static constexpr int kSfSlots = 5;
};

template <int FMT>
__global__ void __launch_bounds__(320, 1)
    linear_fp4_rows_kernel(const __grid_constant__ LinearFp4Maps m, const LinearFp4Params p) {
  using C = RowCfg;
  constexpr int S = C::kStages;
  constexpr bool S16 = FMT == kNvfp4;
  constexpr int kAtoms = S16 ? 4 : 2, kPerAtom = 4 / kAtoms;
  constexpr uint32_t kTx = C::kWBytes + kAtoms * 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align_up<1024>(smem_raw);
  const int nk = (p.K + 255) / 256;
  uint8_t *xs = smem + C::kXOff;                    // codes, 1 KB per 256 columns
  uint8_t *sx = xs + nk * C::kXBytes;               // scales, 128 bytes per scale tile
  float2 *cols = reinterpret_cast<float2 *>(sx + nk * C::kSxBytes);  // [2][128]: row scale of w and bias
  uint64_t *full = reinterpret_cast<uint64_t *>(cols + 2 * 128);
  uint64_t *empty = full + S;
  uint64_t *acc_full = empty + S;      // [2]
  uint64_t *acc_empty = acc_full + 2;  // [2]
  uint64_t *x_ready = acc_empty + 2;
  uint32_t *row_max = reinterpret_cast<uint32_t *>(x_ready + 1);  // [8] bits of the rows' largest magnitudes
  uint32_t *tmem_slot = row_max + kRowMax;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (__syncthreads_or(*(volatile int *)p.status != kDevOk)) return;  // all threads alike
  const int ntiles = (p.N + 127) / 128;
  const int first = blockIdx.x, step = gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 2);
    }
    mbar_init(x_ready, 256);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < kRowMax) row_max[threadIdx.x] = 0;
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's

  if (warp == 0) {
    const uint32_t lead = elect_lane();
    int s = 0, kg = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int tile = first; tile < ntiles && ok; tile += step) {
      for (int kb = 0; kb < nk; ++kb, ++kg) {
        if (!wait_warp(&empty[s], ph, p.status, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t *b = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx_lead(&full[s], kTx, lead);
        tma_load_2d_lead<1>(b, &m.w, smem_u32(&full[s]), kb * 128, tile * 128, lead);
        tma_load_3d_lead<1>(b + C::kWBytes, &m.sw, smem_u32(&full[s]), 0, kb * kAtoms, tile, lead);
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    if (!ok)  // gave up: let the copies in flight land before the shared memory goes away
      for (int f = max(kg - S, 0); f < kg; ++f) mbar_drain(&full[f % S], (f / S) & 1);
  } else if (warp == 1) {
    const uint32_t lead = elect_lane();
    const int my_tiles = first < ntiles ? (ntiles - 1 - first) / step + 1 : 0;
    const uint64_t desc_w = sdesc_sw128(smem_u32(smem), 16, 1024), desc_x = sdesc_sw128(smem_u32(xs), 16, 0);
    const uint64_t desc_sw = sdesc_plain(smem_u32(smem) + C::kWBytes, 128), desc_sx = sdesc_plain(smem_u32(sx), 0);
    int s = 0;
    uint32_t ph = 0, sf = C::kSfCol;
    bool ok = wait_warp(x_ready, 0, p.status, abort_flag);
    for (int tl = 0; tl < my_tiles && ok; ++tl) {
      const int ab = tl & 1;
      ok = wait_warp(&acc_empty[ab], ((tl >> 1) & 1) ^ 1, p.status, abort_flag);
      tc_fence_after();
      for (int kb = 0; kb < nk && ok; ++kb) {
        ok = wait_warp(&full[s], ph, p.status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t st = static_cast<uint64_t>((s * C::kStageBytes) >> 4);
#pragma unroll
        for (int j = 0; j < kAtoms; ++j) {
          tmem_cp_scales<1>(tmem + sf, desc_sx + (kb * C::kSxBytes + j * 128) / 16, lead);
          tmem_cp_scales<1>(tmem + sf + 4, desc_sw + st + j * 32, lead);
#pragma unroll
          for (int q = 0; q < kPerAtom; ++q) {
            const int kk = j * kPerAtom + q;
            umma_fp4<S16, 1>(tmem + ab * 128, desc_x + kb * (C::kXBytes / 16) + kk * 2, desc_w + st + kk * 2,
                             idesc_fp4(128, 128, S16, q * 2), tmem + sf, tmem + sf + 4, (kb | kk) != 0, lead);
          }
          sf = sf + C::kSfCols == C::kSfCol + C::kSfSlots * C::kSfCols ? C::kSfCol : sf + C::kSfCols;
        }
        umma_commit_lead<1>(&empty[s], lead);
        if (kb == nk - 1) umma_commit_lead<1>(&acc_full[ab], lead);
        if (++s == S) s = 0, ph ^= 1;
      }
    }
  } else {
    // quantise: item i is 16 columns of a row; the columns up to a whole 256 are zeros
    const int t = threadIdx.x - 64, groups = p.K / 16, per_row = nk * 16, items = p.T * per_row;
    Vec32 u[kRowItems];
    uint32_t am[kRowItems];
#pragma unroll
    for (int v = 0; v < kRowItems; ++v) {
      const int i = v * 256 + t, r = i / per_row, g = i - r * per_row;
      u[v] = i < items && g < groups ? load16x2(p.x + static_cast<int64_t>(r) * p.K + g * 16) : Vec32{};
    }
#pragma unroll
    for (int v = 0; v < kRowItems; ++v) {
      uint32_t a = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = amax_bf16x2(a, u[v].w[e]);
      am[v] = amax_fold(a);
      const int i = v * 256 + t;
      if (S16 && i < items) atomicMax(&row_max[i / per_row], am[v]);
    }
    if (S16) asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
    for (int v = 0; v < kRowItems; ++v) {
      const int i = v * 256 + t;
      if (v * 256 + (t & ~31) >= items) break;  // whole warps leave together (per_row is even: pairs of lanes share a row)
      const int r = i / per_row, g = i - r * per_row;
      float inv;
      uint32_t sb;
      if (S16) {
        sb = nvfp4_block_scale(am[v], nvfp4_row_inv(i < items ? row_max[r] : 0), &inv);
      } else {
        sb = mxfp4_block_scale(max(am[v], __shfl_xor_sync(0xffffffffu, am[v], 1)), &inv);
      }
      if (i < items) {
        float q[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t w = u[v].w[e];
          const float2 x = make_float2(bf16_lo(w), bf16_hi(w));
          const float2 d = S16 ? e2m1_grid(x, inv) : make_float2(x.x * inv, x.y * inv);
          q[2 * e] = d.x, q[2 * e + 1] = d.y;
        }
        const int st = g >> 4, c = g & 15;
        *reinterpret_cast<uint2 *>(xs + st * C::kXBytes + sw128_offset(r, c >> 1) + (c & 1) * 8) =
            make_uint2(e2m1x8(q), e2m1x8(q + 8));
        // scale of a block: byte block % 4 of the row's 16 bytes in its scale tile
        const int blk = S16 ? c : c >> 1;
        if (S16 || (g & 1) == 0)
          sx[st * C::kSxBytes + (blk >> 2) * 128 + r * 16 + (blk & 3)] = static_cast<uint8_t>(g < groups ? sb : 0);
      }
    }
    fence_async_smem();
    mbar_arrive(x_ready);
    if ((warp & 3) == 0) {  // TMEM lanes 0-31; warp 4 takes the first 64 columns, warp 8 the others
      const int half = warp >> 3;
      bool ok = wait_warp(x_ready, 0, p.status, abort_flag);
      const float rx = S16 && lane < p.T ? nvfp4_row_scale(row_max[lane & 7]) : 1.f;
      const float2 f = split_scale(rx);
      const bool far = S16 && __any_sync(0xffffffffu, far_from_one(rx));
      int tl = 0;
      for (int tile = first; tile < ntiles && ok; tile += step, ++tl) {
        const int ab = tl & 1, n0 = tile * 128 + half * 64;
        float2 *cw = cols + ab * 128 + half * 64;
#pragma unroll
        for (int c = lane; c < 64; c += 32) {
          float2 col = make_float2(1.f, 0.f);
          if (n0 + c < p.N) {
            if (S16) col.x = p.rw[n0 + c];
            if (p.bias != nullptr) col.y = bf16_lo(p.bias[n0 + c]);
          }
          cw[c] = col;
        }
        __syncwarp();
        ok = wait_warp(&acc_full[ab], (tl >> 1) & 1, p.status, abort_flag);
        if (!ok) break;
        tc_fence_after();
        float v[64];
        tmem_ld64(tmem + ab * 128 + half * 64, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ab]);
        if (far) {
#pragma unroll
          for (int q = 0; q < 64; ++q) v[q] = scaled(v[q], f, cw[q].x) + cw[q].y;
        } else {
#pragma unroll
          for (int q = 0; q < 64; ++q) v[q] = fmaf(v[q], rx * cw[q].x, cw[q].y);
        }
        if (p.gelu) {
#pragma unroll
          for (int q = 0; q < 64; ++q) v[q] = gelu_sigmoid(v[q]);
        }
        if (lane < p.T) {
          const int64_t o = static_cast<int64_t>(lane) * p.N + n0;
#pragma unroll
          for (int q = 0; q < 64; q += 8) {
            if (n0 + q >= p.N) break;  // N is a multiple of 8
            if (p.out_f32) {
              float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + o + q);
              d[0] = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
              d[1] = make_float4(v[q + 4], v[q + 5], v[q + 6], v[q + 7]);
            } else {
              *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + o + q) =
                  make_uint4(cvt_bf16x2(v[q], v[q + 1]), cvt_bf16x2(v[q + 2], v[q + 3]),
                             cvt_bf16x2(v[q + 4], v[q + 5]), cvt_bf16x2(v[q + 6], v[q + 7]));
            }
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Shared-memory limit of a kernel, raised once per device.
template <auto Kernel>
cudaError_t allow_smem(uint32_t bytes, int dev) {
  static std::atomic<bool> done[64];
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int FMT, int CG, int BN>
cudaError_t launch_form(const LinearFp4Params &p, const LinearFp4Maps &m, int dev, int sms, cudaStream_t s) {
  using C = LinCfg<CG, BN>;
  const int64_t tiles = static_cast<int64_t>((p.T + 128 * CG - 1) / (128 * CG)) * ((p.N + BN - 1) / BN);
  const cudaError_t e = allow_smem<linear_fp4_kernel<FMT, CG, BN>>(C::kSmem, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  // behind its own quantiser: set up while that runs
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, sms / CG)) * CG);
  cfg.blockDim = dim3(320);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.x != nullptr ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_fp4_kernel<FMT, CG, BN>, m, p);
}

template <int FMT>
cudaError_t launch_rows(const LinearFp4Params &p, const LinearFp4Maps &m, int dev, int sms, cudaStream_t s) {
  const int nk = (p.K + 255) / 256;
  const cudaError_t e = allow_smem<linear_fp4_rows_kernel<FMT>>(RowCfg::smem(kRowStagesMax), dev);
  if (e != cudaSuccess) return e;
  linear_fp4_rows_kernel<FMT><<<std::min((p.N + 127) / 128, sms), 320, RowCfg::smem(nk), s>>>(m, p);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_fmt(const LinearFp4Params &p, const LinearFp4Maps &m, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  switch (m.form) {
    case kLinearRows: return launch_rows<FMT>(p, m, dev, sms, s);
    case kLinearPair: return launch_form<FMT, 2, 256>(p, m, dev, sms, s);
    case kLinearWide: return launch_form<FMT, 1, 256>(p, m, dev, sms, s);
    default: return launch_form<FMT, 1, 128>(p, m, dev, sms, s);
  }
}

}  // namespace

cudaError_t launch_linear_fp4(const LinearFp4Params &p, const LinearFp4Maps &m, cudaStream_t s) {
  return p.fmt == kNvfp4 ? launch_fmt<kNvfp4>(p, m, s) : launch_fmt<kMxfp4>(p, m, s);
}

// A few rows of bf16 x are quantised in the product's kernel (kRowItems per thread at most): 1
// x 18432 x 3072 takes 8.5 us in a graph, 1 x 3072 x 3072 8.2 (two launches 12.9 and 8.6), and a
// call costs the host 5 us less; at 8 rows of 3072 the quantiser in every CTA would take 2.5 us
// more than its own launch. Otherwise the form of
// the least estimated time on 148 SMs: waves x (time of a tile's ends + time of its
// K / 256 stages), in units of 10 ns, fitted to measurements of NVFP4 products (MXFP4 goes by them too). It takes the
// shortest of each row but one: 1024 x 3072 x 3072 runs as pairs, 4% longer than wide tiles would (us):
//                            single    wide     pair
//     333 x 12288 x 3072       13.7    12.6     16.4
//    1024 x  3072 x 3072       12.2    10.4     10.8
//    4352 x  9216 x 3072       71.9    66.0     54.6
//    4352 x  3072 x 12288      86.4    87.9     60.9
//     512 x  3072 x 12288      18.6    29.2     21.6
//   10000 x   256 x 256         6.5     6.1      7.1
LinearFp4Form linear_fp4_form(int64_t T, int64_t N, int64_t K, bool quantised) {
  const int64_t nk = (K + 255) / 256;
  if (!quantised && T <= kRowMax && T * nk * 16 <= 256 * kRowItems) return kLinearRows;
  const int64_t m1 = (T + 127) / 128, m2 = (T + 255) / 256, n1 = (N + 127) / 128, n2 = (N + 255) / 256;
  const int64_t single = (m1 * n1 + 147) / 148 * (95 + 27 * nk), wide = (m1 * n2 + 147) / 148 * (140 + 50 * nk),
                pair = 90 + (m2 * n2 + 73) / 74 * (130 + 36 * nk);
  if (pair < single && pair < wide) return kLinearPair;
  return wide < single ? kLinearWide : kLinearSingle;
}

}  // namespace cm
