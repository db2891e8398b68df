// Weight gradient of routed experts from 8-bit activation checkpoints:
//   dW[e] (+)= sum over the rows r of expert e of d_y[r]^T x[row_token[r]],
//   x = bf16(codes * scales) (E4M3, one scale per row and 128 columns; exact
//   for the power-of-two scales of a checkpoint), bf16 d_y, FP32 sums.
//
// The contraction runs over rows, along which neither operand is contiguous:
// d_y is [r][n] and x is [r][k], so both enter the tensor cores MN-major, as
// they lie.  A first kernel restores x into the workspace in the order of the
// routed rows; the second is a grouped bf16 GEMM on CTA pairs:
//   tile     256 (n) x 256 (k) per pair, 128 n rows and 128 k columns of the
//            operands per CTA, 64 rows r per stage (32 KB per CTA);
//   warp 0   TMA producer: two 64 x 64 boxes of each operand per stage;
//   warp 1   even CTA: four tcgen05.mma kind::f16 (256 x 256 x 16) per stage
//            into one of two 256-column TMEM slots; odd CTA: tells the even
//            one that its half of the stage has landed.  In a group's last
//            stage both first clear the rows behind the group (they belong to
//            the next expert, whose values may be infinite);
//   warps 2..9  epilogue: TMEM through 128-byte swizzled rows in shared memory
//            to dW by TMA stores (adds, when accumulating), clipped at the
//            edges of the expert's matrix.
// Restoring once per token and letting the producer gather rows (four-row TMA
// gathers, 32 per stage) moved 0.4 GB less and was slower: 2453 us against
// 1087 us with rows in order (64 experts of 2048 x 7168, 32768 rows).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q4 {
namespace {

// ------------------------------------------------------------------ restore
constexpr int kRestoreThreads = 256;

// 8 codes per thread and row: x[r, c .. c + 8) = bf16(code * scale) of token
// row_token[r], for the rows that belong to an expert; kRestoreRows rows at a
// time, their loads in flight together.
constexpr int kRestoreRows = 4;

__global__ void __launch_bounds__(kRestoreThreads)
    wgrad_restore_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t tokens,
                         int64_t K, const int32_t* __restrict__ row_token, const int32_t* __restrict__ last, int64_t R,
                         __nv_bfloat16* __restrict__ x) {
  pdl_wait();
  const uint32_t v = blockIdx.x * kRestoreThreads + threadIdx.x;
  if (v >= (uint32_t)(K / 8)) return;
  const int64_t KB = (K + 127) / 128, rows = min((int64_t)__ldg(last), R);
  for (int64_t r0 = (int64_t)blockIdx.y * kRestoreRows; r0 < rows; r0 += (int64_t)gridDim.y * kRestoreRows) {
    uint2 c[kRestoreRows];
    float s[kRestoreRows];
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i) {
      const int64_t r = min(r0 + i, rows - 1);
      const int64_t t = row_token ? min(max((int64_t)__ldg(row_token + r), (int64_t)0), tokens - 1) : r;
      c[i] = __ldg(reinterpret_cast<const uint2*>(codes + t * K) + v);
      s[i] = __ldg(scales + t * KB + v / 16);
    }
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h;  // two E4M3 codes as f16 (exact)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)((j < 2 ? c[i].x : c[i].y) >> (16 * (j & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s[i], f.y * s[i]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (r0 + i < rows)
        reinterpret_cast<uint4*>(x + (r0 + i) * K)[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------------ GEMM
constexpr int kRows = 64;                          // rows r per stage
constexpr int kHalf = 128;                         // n rows, and k columns, of one CTA's operands
constexpr int kTile = 256;                         // pair tile, both ways
constexpr int kStages = 5;
constexpr uint32_t kPanelBytes = kRows * 128;      // 64 rows x 64 bf16, 128-byte swizzle
constexpr uint32_t kOperandBytes = 2 * kPanelBytes;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kSlots = 2;
constexpr int kEpiWarp0 = 2, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kOutBytes = 32 * 128;           // 32 rows of 128 bytes: one TMA store of an epilogue warp
constexpr uint32_t kOutTotal = 2 * kEpiWarps * kOutBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kOutTotal + 1024 /*align*/ + 256 /*barriers*/;
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
  int64_t R, N, K;
  const int32_t* offsets;
  int num_n, num_k, tiles, accumulate;
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

// A 32-row box of 128-byte rows from shared memory to dW[z], or added to it
// (each element by one box, so sums do not depend on an order).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z,
                                             bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most kLeft of this thread's store groups still read their shared memory.
template <int kLeft>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// Arrive on a peer's mbarrier with everything this thread has seen visible to
// the cluster: the cleared rows of the odd CTA's stage.  Only after a clear:
// as the arrival of every stage it cost 1.1 us a stage and held the whole
// kernel there (64 x 2048 x 7168, 32768 rows in order: 1764 us).
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

template <typename W>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_w, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  pdl_wait();  // operands may come from the previous kernel
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_smem = smem + kStages * kStageBytes;
  Smem* sm = reinterpret_cast<Smem*>(out_smem + kOutTotal);
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
    prefetch_tmap(&tmap_w);
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
          for (int i = 0; i < 2; ++i) {
            tma_load_2d(y + i * kPanelBytes, &tmap_y, (w.n0 + rank * kHalf + i * 64) * 2, row, full);
            tma_load_2d(x + i * kPanelBytes, &tmap_x, (w.k0 + rank * kHalf + i * 64) * 2, row, full);
          }
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
          const bool part = w.rows - r0 < kRows;
          if (part) clear_rows(smem + stage * kStageBytes, w.rows - r0, lane);
          if (lane == 0) {
            if (part)
              mbar_arrive_cluster_release(leader_pair_full + stage * 8);
            else
              mbar_arrive_cluster(leader_pair_full + stage * 8);
          }
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
    uint8_t* buf = out_smem + (warp - kEpiWarp0) * 2 * kOutBytes;
    constexpr int kCols = 128 / (int)sizeof(W);  // columns of one store
    uint32_t done = 0, stores = 0;
    for (int t = cid; t < p.tiles; t += ncl) {
      const Tile w = tile_of(p, t);
      const int n0 = w.n0 + rank * kHalf + q * 32;
      const int k0 = w.k0 + h * 128;
      const uint32_t slot = done % kSlots, sphase = (done / kSlots) & 1;
      if (w.rows) {
        ++done;
        if (!warp_wait(smem_u32(&sm->slot_full[slot]), sphase, p.ctl, abort_flag)) break;
        tc_fence_after();
      } else if (p.accumulate) {
        continue;
      }
#pragma unroll
      for (int c = 0; c < 128 / kCols; ++c, ++stores) {
        uint8_t* line = buf + (stores & 1) * kOutBytes;
        if (lane == 0) tma_store_wait_read<1>();  // the store before the last has read this buffer
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i) {  // 16 columns at a time
          uint32_t r[16];
          if (w.rows) {
            tmem_ld_32x32b_x16(t_lane + slot * kTile + c * kCols + i * 16, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = 0u;
          }
          constexpr int kWords = (int)sizeof(W);  // 16-byte words of 16 columns
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            uint4 o;
            if constexpr (sizeof(W) == 4) {
              o = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            } else {
              uint32_t b[4];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * j + 2 * m]),
                                                               __uint_as_float(r[8 * j + 2 * m + 1]));
                b[m] = *reinterpret_cast<const uint32_t*>(&v);
              }
              o = make_uint4(b[0], b[1], b[2], b[3]);
            }
            *reinterpret_cast<uint4*>(line + lane * 128 + (((i * kWords + j) ^ (lane & 7)) << 4)) = o;
          }
        }
        if (w.rows && c == 128 / kCols - 1) {  // the slot's columns of this warp are all read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader_slot_empty + slot * 8);
        }
        fence_proxy_async_smem();  // the TMA store reads what these threads wrote
        __syncwarp();
        const int k = k0 + c * kCols;
        if (lane == 0) {
          if (n0 < p.N && k < p.K) tma_store_3d(&tmap_w, smem_u32(line), k, n0, w.e, p.accumulate != 0);
          tma_store_commit();  // a group per buffer use, empty past the edge: the wait above counts groups
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // written before the CTA exits
    __syncwarp();
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

}  // namespace

// The restored rows.
size_t wgrad_workspace_bytes(int64_t R, int64_t N, int64_t K) {
  (void)N;
  return (size_t)R * (size_t)K * sizeof(__nv_bfloat16);
}

namespace {

template <typename W>
q4_status launch_typed(const WgradArgs& a, cudaStream_t stream) {
  __nv_bfloat16* x = static_cast<__nv_bfloat16*>(a.ws);
  Params p = {};
  p.R = a.R, p.N = a.N, p.K = a.K;
  p.offsets = a.offsets;
  p.accumulate = a.accumulate;
  const int64_t num_n = ceil_div(a.N, kTile), num_k = ceil_div(a.K, kTile);
  if (num_n * num_k > INT32_MAX / 2 / a.E) return Q4_ERR_UNSUPPORTED_SHAPE;
  p.num_n = (int)num_n, p.num_k = (int)num_k, p.tiles = (int)(a.E * num_n * num_k);
  p.ctl = KernelCtl{device_status_ptr(), wait_budget_ns()};

  CUtensorMap ty, tx, tw;
  q4_status st = make_tmap_2d_u8(&ty, a.dy, a.N * 2, a.R, a.ldy * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_2d_u8(&tx, x, a.K * 2, a.R, a.K * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_3d(&tw, sizeof(W) == 4 ? Q4_F32 : Q4_BF16, a.dw, a.K, a.N, a.E, a.K, a.N * a.K, 128 / sizeof(W), 32,
                    1, true);
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
    Q4_CUDA_TRY(cudaFuncSetAttribute(wgrad_pair_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    int n = 0;
    cfg.gridDim = dim3((unsigned)(num_sms() / 2 * 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, wgrad_pair_kernel<W>, &cfg) != cudaSuccess || n <= 0) n = num_sms() / 2;
    max_pairs[dev] = std::min(n, num_sms() / 2);
  }

  const int64_t gx = ceil_div(a.K / 8, kRestoreThreads);
  const int64_t gy = std::min<int64_t>(ceil_div(a.R, kRestoreRows), 65535);
  st = launch_pdl(wgrad_restore_kernel, dim3((unsigned)gx, (unsigned)gy), kRestoreThreads, 0, stream, a.codes,
                  a.scales, a.tokens, a.K, a.row_token, a.offsets + a.E, a.R, x);
  if (st != Q4_OK) return st;
  cfg.gridDim = dim3(2u * (unsigned)std::min(p.tiles, max_pairs[dev]), 1, 1);
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, wgrad_pair_kernel<W>, ty, tx, tw, p));
  return Q4_OK;
}

}  // namespace

q4_status launch_wgrad(const WgradArgs& a, cudaStream_t stream) {
  return a.w_dtype == Q4_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace q4
