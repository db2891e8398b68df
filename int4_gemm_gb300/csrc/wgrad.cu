// Weight gradient of routed experts from 8-bit activation checkpoints:
//   dW[e] (+)= sum over the rows r of expert e of d_y[r]^T x[row_token[r]],
//   x = bf16(codes * scales) (E4M3, one scale per row and 128 columns; exact
//   for the power-of-two scales of a checkpoint), bf16 d_y, FP32 sums.
//
// The contraction runs over rows, along which neither operand is contiguous:
// d_y is [r][n] and x is [r][k], so both enter the tensor cores MN-major, as
// they lie.  A first kernel restores x once per token into the workspace (the
// codes are read once, not once per 256 columns of N and per routed copy);
// the second is a grouped bf16 GEMM on CTA pairs:
//   tile     256 (n) x 256 (k) per pair, 128 n rows and 128 k columns of the
//            operands per CTA, 64 rows r per stage (32 KB per CTA);
//   warp 0   TMA producer: two 64 x 64 boxes of d_y, and of x sixteen
//            four-row gathers per 64 columns through row_token (or two boxes
//            when the checkpoint is in row order);
//   warp 1   even CTA: four tcgen05.mma kind::f16 (256 x 256 x 16) per stage
//            into one of two 256-column TMEM slots; odd CTA: tells the even
//            one that its half of the stage has landed.  In a group's last
//            stage both first clear the rows behind the group (they belong to
//            the next expert, whose values may be infinite);
//   warps 2..9  epilogue: TMEM to dW.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q4 {
namespace {

// ------------------------------------------------------------------ restore
constexpr int kRestoreThreads = 256;

// 16 codes per thread: x[t, c .. c + 16) = bf16(code * scale), row pitch KP.
__global__ void __launch_bounds__(kRestoreThreads)
    wgrad_restore_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t tokens,
                         int64_t K, int64_t KP, __nv_bfloat16* __restrict__ x) {
  pdl_wait();
  const uint32_t per_row = (uint32_t)(K / 16);
  const int64_t KB = (K + 127) / 128;
  for (int64_t t = blockIdx.y; t < tokens; t += gridDim.y) {
    for (uint32_t v = blockIdx.x * kRestoreThreads + threadIdx.x; v < per_row; v += gridDim.x * kRestoreThreads) {
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes + t * K) + v);
      const float s = __ldg(scales + t * KB + v / 8);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t h;  // two E4M3 codes as f16 (exact)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      uint4* out = reinterpret_cast<uint4*>(x + t * KP + (int64_t)v * 16);
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// ------------------------------------------------------------------ GEMM
constexpr int kRows = 64;                          // rows r per stage
constexpr int kHalf = 128;                         // n rows, and k columns, of one CTA's operands
constexpr int kTile = 256;                         // pair tile, both ways
constexpr int kStages = 6;
constexpr uint32_t kPanelBytes = kRows * 128;      // 64 rows x 64 bf16, 128-byte swizzle
constexpr uint32_t kOperandBytes = 2 * kPanelBytes;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kSlots = 2;
constexpr int kEpiWarp0 = 2, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024 /*align*/ + 256 /*barriers*/;
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(kSlots * kTile <= 512, "TMEM columns");

struct Smem {
  uint64_t full[kStages];       // this CTA's copies of the stage landed
  uint64_t pair_full[kStages];  // even CTA: the odd CTA's did, its rows behind the group are clear
  uint64_t empty[kStages];      // the stage's MMAs are done (both CTAs)
  uint64_t slot_full[kSlots];   // the slot holds a tile (both CTAs)
  uint64_t slot_empty[kSlots];  // even CTA: every epilogue warp of the pair has read it
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) <= 256, "barrier block");

struct Params {
  int64_t R, N, K, tokens;
  const int32_t* row_token;
  const int32_t* offsets;
  void* dw;
  int num_n, num_k, tiles, bf16, accumulate;
  KernelCtl ctl;
};

// tcgen05.mma kind::f16: FP32 accumulator (bits 4-5 = 1), bf16 A and B (1 in
// bits 7-9 and 10-12), both MN-major (bits 15 and 16), N / 8 in bits 17-22,
// M / 16 in bits 24-28.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);

__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
      : "memory");
}

// MN-major operand at rows 16 s of its stage: 64 x 8 atoms of 1024 bytes (8
// rows of 128 bytes), 8-row groups 1024 bytes apart (stride offset), 64-wide
// panels kPanelBytes apart (leading offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t s) {
  return smem_desc(addr + s * 16 * 128, kPanelBytes, 1024, 2);
}

__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int32_t x, const int32_t (&r)[4],
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

// Arrive on a peer's mbarrier with everything this thread has seen visible to
// the cluster (the cleared rows of the odd CTA's stage among it).
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Clears rows [from, 64) of the stage's four panels (the whole warp).
__device__ __forceinline__ void clear_rows(uint8_t* stage, int from, int lane) {
  const int words = (kRows - from) * 8;  // 16-byte words per panel
  for (int p = 0; p < 4; ++p) {
    uint4* dst = reinterpret_cast<uint4*>(stage + p * kPanelBytes + from * 128);
    for (int i = lane; i < words; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();  // the tensor cores read what these threads wrote
  __syncwarp();
}

// The bounded wait, with one answer for the whole warp: a lane that gave up
// takes the others along.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const KernelCtl& ctl, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, ctl, abort_flag)) != 0;
}

struct Tile {
  int e, n0, k0;
  int64_t lo;
  int rows;
};
__device__ __forceinline__ Tile tile_of(const Params& p, int t) {
  Tile o;
  const int per = p.num_n * p.num_k;
  o.e = t / per;
  const int r = t - o.e * per;
  o.n0 = (r % p.num_n) * kTile;
  o.k0 = (r / p.num_n) * kTile;
  o.lo = min(max((int64_t)__ldg(p.offsets + o.e), (int64_t)0), p.R);
  const int64_t hi = min((int64_t)__ldg(p.offsets + o.e + 1), p.R);
  o.rows = hi > o.lo ? (int)(hi - o.lo) : 0;
  return o;
}

__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_x,
                      const Params p) {
  extern __shared__ uint8_t smem_raw[];
  pdl_wait();  // operands may come from the previous kernel
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem* sm = reinterpret_cast<Smem*>(smem + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();  // 0: issues the pair's MMAs
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->pair_full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&sm->slot_full[s]), 1);
      mbar_init(smem_u32(&sm->slot_empty[s]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&sm->mma_done), 1);
    sm->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_y);
    prefetch_tmap(&tmap_x);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sm->tmem_base), kSlots * kTile);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier_sync();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort_flag = &sm->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t stage = 0, phase = 0;
    int issued[kStages];
    uint32_t issued_phase[kStages];
    for (int s = 0; s < kStages; ++s) issued[s] = 0, issued_phase[s] = 0;
    bool alive = true;
    for (int t = cid; t < p.tiles && alive; t += ncl) {
      const Tile w = tile_of(p, t);
      for (int r0 = 0; r0 < w.rows; r0 += kRows) {
        // lane l gathers rows 4 (l % 16) .. of panel l / 16; rows behind the
        // group repeat its last one (cleared before use)
        int32_t tok[4];
        if (p.row_token) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = min(r0 + (lane & 15) * 4 + i, w.rows - 1);
            tok[i] = min(max(__ldg(p.row_token + w.lo + r), 0), (int32_t)(p.tokens - 1));
          }
        }
        if (!warp_wait(smem_u32(&sm->empty[stage]), phase ^ 1, p.ctl, abort_flag)) {
          alive = false;
          break;
        }
        const uint32_t y = smem_u32(smem + stage * kStageBytes), x = y + kOperandBytes;
        const uint32_t full = smem_u32(&sm->full[stage]);
        const int32_t row = (int32_t)w.lo + r0;
        if (lane == 0) {
          mbar_arrive_expect_tx(full, kStageBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tma_load_2d(y + i * kPanelBytes, &tmap_y, (w.n0 + rank * kHalf + i * 64) * 2, row, full);
        }
        __syncwarp();
        const int x0 = (w.k0 + rank * kHalf) * 2;
        if (p.row_token) {
          const int i = lane >> 4;
          tma_gather4(x + i * kPanelBytes + (lane & 15) * 512, &tmap_x, x0 + i * 128, tok, full);
        } else if (lane < 2) {
          tma_load_2d(x + lane * kPanelBytes, &tmap_x, x0 + lane * 128, row, full);
        }
        issued[stage] = 1;
        issued_phase[stage] = phase;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    // drain: every copy this warp issued has landed before the CTA exits
    if (lane == 0) {
      KernelCtl drain = p.ctl;
      for (int s = 0; s < kStages; ++s)
        if (issued[s]) mbar_wait(smem_u32(&sm->full[s]), issued_phase[s], drain, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    uint32_t stage = 0, phase = 0;
    if (rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      uint32_t done = 0;
      bool alive = true;
      for (int t = cid; t < p.tiles && alive; t += ncl) {
        const Tile w = tile_of(p, t);
        if (w.rows == 0) continue;
        const uint32_t slot = done % kSlots, sphase = (done / kSlots) & 1;
        if (!warp_wait<true>(smem_u32(&sm->slot_empty[slot]), sphase ^ 1, p.ctl, abort_flag)) break;
        ++done;
        const uint32_t d = tmem + slot * kTile;
        for (int r0 = 0; r0 < w.rows; r0 += kRows) {
          if (!warp_wait(smem_u32(&sm->full[stage]), phase, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          uint8_t* st = smem + stage * kStageBytes;
          if (w.rows - r0 < kRows) clear_rows(st, w.rows - r0, lane);
          if (!warp_wait<true>(smem_u32(&sm->pair_full[stage]), phase, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          __syncwarp();
          tc_fence_after();
          if (lane == 0) {
            const uint32_t y = smem_u32(st), x = y + kOperandBytes;
#pragma unroll
            for (uint32_t s = 0; s < kRows / 16; ++s)
              mma_bf16_pair(d, operand_desc(y, s), operand_desc(x, s), r0 != 0 || s != 0 ? 1u : 0u);
            tc_commit_pair_mc(smem_u32(&sm->empty[stage]), 3);  // the stage is free in both CTAs
          }
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
        if (alive && lane == 0) tc_commit_pair_mc(smem_u32(&sm->slot_full[slot]), 3);
        __syncwarp();
      }
      // all MMAs this thread issued are complete before TMEM is released
      if (lane == 0) {
        tc_commit_pair_mc(smem_u32(&sm->mma_done), 1);
        KernelCtl drain = p.ctl;
        mbar_wait(smem_u32(&sm->mma_done), 0, drain, nullptr);
      }
    } else {
      // ---------------------------------------------------------- relay (odd CTA)
      const uint32_t leader_pair_full = mapa_shared(smem_u32(&sm->pair_full[0]), 0);
      bool alive = true;
      for (int t = cid; t < p.tiles && alive; t += ncl) {
        const Tile w = tile_of(p, t);
        for (int r0 = 0; r0 < w.rows; r0 += kRows) {
          if (!warp_wait(smem_u32(&sm->full[stage]), phase, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          if (w.rows - r0 < kRows) clear_rows(smem + stage * kStageBytes, w.rows - r0, lane);
          if (lane == 0) mbar_arrive_cluster_release(leader_pair_full + stage * 8);
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                  // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;   // column half of the slot
    const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16) + h * 128;
    const uint32_t leader_slot_empty = mapa_shared(smem_u32(&sm->slot_empty[0]), 0);
    uint32_t done = 0;
    for (int t = cid; t < p.tiles; t += ncl) {
      const Tile w = tile_of(p, t);
      const int64_t n = w.n0 + rank * kHalf + q * 32 + lane;
      const int64_t k0 = w.k0 + h * 128;
      const uint32_t slot = done % kSlots, sphase = (done / kSlots) & 1;
      if (w.rows) {
        ++done;
        if (!warp_wait(smem_u32(&sm->slot_full[slot]), sphase, p.ctl, abort_flag)) break;
        tc_fence_after();
      } else if (p.accumulate) {
        continue;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // 16 columns at a time
        uint32_t r[16];
        if (w.rows) {
          __syncwarp();
          tmem_ld_32x32b_x16(t_lane + slot * kTile + c * 16, r);
          tmem_ld_wait();
          if (c == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_slot_empty + slot * 8);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = 0u;
        }
        const int64_t k = k0 + c * 16;
        if (n >= p.N || k >= p.K) continue;  // K is a multiple of 16
        const int64_t at = ((int64_t)w.e * p.N + n) * p.K + k;
        if (p.bf16) {
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dw) + at);
          out[0] = make_uint4(o[0], o[1], o[2], o[3]);
          out[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
          float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.dw) + at);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float4 v = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                   __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
            if (p.accumulate) {
              const float4 old = out[j];
              v.x += old.x, v.y += old.y, v.z += old.z, v.w += old.w;
            }
            out[j] = v;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_barrier_sync();  // the pair's MMAs are complete in both CTAs
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kSlots * kTile);
  }
  // no CTA leaves while its peer may still arrive on its barriers
  cluster_barrier_sync();
}

// The restored rows are padded to whole tiles of columns, so that no gather
// reaches past them; what the padding holds only meets columns that are not
// stored.
int64_t padded_k(int64_t K) { return ceil_div(K, kTile) * kTile; }

}  // namespace

size_t wgrad_workspace_bytes(int64_t tokens, int64_t N, int64_t K) {
  (void)N;
  return (size_t)tokens * (size_t)padded_k(K) * sizeof(__nv_bfloat16);
}

q4_status launch_wgrad(const WgradArgs& a, cudaStream_t stream) {
  const int64_t KP = padded_k(a.K);
  __nv_bfloat16* x = static_cast<__nv_bfloat16*>(a.ws);
  Params p = {};
  p.R = a.R, p.N = a.N, p.K = a.K, p.tokens = a.tokens;
  p.row_token = a.row_token, p.offsets = a.offsets;
  p.dw = a.dw, p.bf16 = a.w_dtype == Q4_BF16, p.accumulate = a.accumulate;
  const int64_t num_n = ceil_div(a.N, kTile), num_k = ceil_div(a.K, kTile);
  if (num_n * num_k > INT32_MAX / 2 / a.E) return Q4_ERR_UNSUPPORTED_SHAPE;
  p.num_n = (int)num_n, p.num_k = (int)num_k, p.tiles = (int)(a.E * num_n * num_k);
  p.ctl = KernelCtl{device_status_ptr(), wait_budget_ns()};

  CUtensorMap ty, tx;
  q4_status st = make_tmap_2d_u8(&ty, a.dy, a.N * 2, a.R, a.ldy * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_2d_u8(&tx, x, KP * 2, a.tokens, KP * 2, 128, a.row_token ? 1 : kRows, true);
  if (st != Q4_OK) return st;

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return Q4_ERR_CUDA;
  static int max_pairs[64] = {0};
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (!max_pairs[dev]) {  // persistent: as many pairs as are resident at once
    Q4_CUDA_TRY(cudaFuncSetAttribute(wgrad_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    int n = 0;
    cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, wgrad_pair_kernel, &cfg) != cudaSuccess || n <= 0) n = num_sms() / 2;
    max_pairs[dev] = std::min(n, num_sms() / 2);
  }

  const unsigned gx = (unsigned)ceil_div(a.K / 16, kRestoreThreads);
  const unsigned gy = (unsigned)std::min<int64_t>(a.tokens, 65535);
  st = launch_pdl(wgrad_restore_kernel, dim3(gx, gy), kRestoreThreads, 0, stream, a.codes, a.scales, a.tokens, a.K,
                  KP, x);
  if (st != Q4_OK) return st;
  cfg.gridDim = dim3(2u * (unsigned)std::min(p.tiles, max_pairs[dev]), 1, 1);
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, wgrad_pair_kernel, ty, tx, p));
  return Q4_OK;
}

}  // namespace q4
