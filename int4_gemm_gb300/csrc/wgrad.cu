// Weight gradient of routed experts from 8-bit activation checkpoints:
//   dW[e] (+)= sum over the rows r of expert e of d_y[r]^T x[row_token[r]],
//   x = bf16(codes * scales) (E4M3, one scale per row and 128 columns; exact
//   for the power-of-two scales of a checkpoint), bf16 d_y, FP32 sums.
//
// The contraction runs over rows, along which neither operand is contiguous:
// d_y is [r][n] and x is [r][k], so both enter the tensor cores MN-major, as
// they lie.  A first kernel restores x into the workspace in the order of the
// routed rows, and there lays out each expert's last rows, those behind its
// last multiple of 64, once more with zeros behind them, x's and d_y's: the
// rows that follow belong to the next expert, whose values may be infinite.
// The second is a grouped bf16 GEMM on CTA pairs:
//   tile     256 (n) x 256 (k) per pair, 128 n rows and 128 k columns of the
//            operands per CTA, 64 rows r per stage (32 KB per CTA);
//   warp 0   TMA producer: two 64 x 64 boxes of each operand per stage; the
//            bytes of both CTAs are counted on the even one's mbarrier;
//   warp 1   even CTA: four tcgen05.mma kind::f16 (256 x 256 x 16) per stage
//            into one of two 256-column TMEM slots;
//   warps 2..9  epilogue: TMEM through 128-byte swizzled rows in shared memory
//            to dW by TMA stores (adds, when accumulating), clipped at the
//            edges of the expert's matrix.
// 64 experts of 2048 x 7168, bf16 dW, the restoring (98 us) included: 726
// us with 512 rows each (1326 TFLOP/s), 756 us with 27 to 1933; 2 experts of
// 16384 rows, where few outputs are written: 551 us (1747).  Between the two
// stand the stores: without them the first takes 645 us.
// Measured and not kept, same sizes: restoring once per token and gathering
// rows in the producer (four-row TMA gathers, 32 per stage), 2453 us; codes
// converted on their way into the stage by eight or sixteen more warps, 1636
// and 1244 us; clusters of two pairs that share d_y by multicast, 795 us (and
// 744 instead of 635); clearing the rows behind a group in shared memory, which
// the odd CTA has to release to the cluster, 0.5 us per expert and tile; the odd
// CTA's arrival passed on by a warp of it, 738 us (and 625 instead of 570); a
// warp's whole part of a slot in registers before its first store, 762 us; the
// next expert's rows brought into L2 while an expert's tiles run, 729 us (FP32:
// 883 instead of 898).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q4 {
namespace {

// Lets the next kernel in the stream start once every block of this one has come
// here or exited.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ restore
constexpr int kRestoreThreads = 256;
constexpr int kRows = 64;         // rows r per stage of the GEMM
constexpr int kRestoreUnits = 4;  // groups of 8 columns of a thread, whose loads are in flight together

// 8 codes (two words) as bf16(code * s).
__device__ __forceinline__ uint4 restore8(uint2 c, float s) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h;  // two E4M3 codes as f16 (exact)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)((j < 2 ? c.x : c.y) >> (16 * (j & 1)))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    o[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct RestoreArgs {
  const uint8_t* codes;
  const float* scales;
  int64_t tokens, K;
  const int32_t* row_token;
  const int32_t* offsets;
  int64_t R;
  int E;
  const __nv_bfloat16* dy;
  int64_t N, ldy;
  __nv_bfloat16 *x, *x_tail, *y_tail;  // [R, K], [E * kRows, K], [E * kRows, N]
};

// First row and number of rows of expert e.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int64_t R, int e, int64_t& lo, int& rows) {
  lo = min(max((int64_t)__ldg(offsets + e), (int64_t)0), R);
  const int64_t hi = min((int64_t)__ldg(offsets + e + 1), R);
  rows = hi > lo ? (int)(hi - lo) : 0;
}

// Rows (blockIdx.y, threadIdx.y): those of every expert first, then each
// expert's kRows tail rows.  A thread takes kRestoreUnits groups of 8 columns of
// its row, threads apart, so that finding the row costs little beside the
// conversions (one group of four rows: 31 us instead of 25 for 8192 rows of
// 7168).  Bound by the writes: 32768 rows of 7168 and 64 tails in 98 us, 5.6 TB/s.
__global__ void __launch_bounds__(kRestoreThreads, 8)
    wgrad_restore_kernel(const RestoreArgs a, int64_t rows_out) {
  pdl_wait();
  // the product may set up its barriers and tensor memory beside this kernel's
  // last blocks; it waits for them before it reads (16 of 520 x 1024, 2000 rows:
  // 16.4 -> 15.5 us)
  pdl_release();
  const uint32_t v0 = blockIdx.x * blockDim.x * kRestoreUnits + threadIdx.x;
  const uint32_t xu = (uint32_t)(a.K / 8), yu = (uint32_t)(a.N / 8);
  const int64_t KB = (a.K + 127) / 128;
  for (int64_t b = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; b < rows_out; b += (int64_t)gridDim.y * blockDim.y) {
    const bool tail = b >= a.R;
    int64_t from = b, to = b;  // source row and row written
    int64_t end = min((int64_t)__ldg(a.offsets + a.E), a.R);
    if (tail) {
      to = b - a.R;
      int64_t lo;
      int rows;
      expert_rows(a.offsets, a.R, (int)(to / kRows), lo, rows);
      if (rows % kRows == 0) continue;  // no tail
      from = lo + rows / kRows * kRows + to % kRows;
      end = lo + rows;
    } else if (from >= end) {
      continue;
    }
    const bool have = from < end;
    int64_t t = 0;
    if (have) t = a.row_token ? min(max((int64_t)__ldg(a.row_token + from), (int64_t)0), a.tokens - 1) : from;
    const uint2* src = reinterpret_cast<const uint2*>(a.codes + t * a.K);
    const float* scale = a.scales + t * KB;
    uint4* dst = reinterpret_cast<uint4*>((tail ? a.x_tail : a.x) + to * a.K);
    uint2 c[kRestoreUnits];
    float s[kRestoreUnits];
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
      const uint32_t v = v0 + i * blockDim.x;
      c[i] = make_uint2(0u, 0u);
      s[i] = 0.f;
      if (have && v < xu) {
        c[i] = __ldg(src + v);
        s[i] = __ldg(scale + v / 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
      const uint32_t v = v0 + i * blockDim.x;
      if (v < xu) dst[v] = restore8(c[i], s[i]);
    }
    if (!tail) continue;
    const uint4* ysrc = reinterpret_cast<const uint4*>(a.dy + from * a.ldy);
    uint4* ydst = reinterpret_cast<uint4*>(a.y_tail + to * a.N);
    for (uint32_t v = blockIdx.x * blockDim.x + threadIdx.x; v < yu; v += gridDim.x * blockDim.x)
      ydst[v] = have ? __ldg(ysrc + v) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------------ GEMM
constexpr int kHalf = 128;                         // n rows, and k columns, of one CTA's operands
constexpr int kTile = 256;                         // pair tile, both ways
// Six stages and one store buffer per epilogue warp: with five and two, 835 us
// for 760 (64 experts of 2048 x 7168, 512 rows each, bf16; FP32: 1095 for 904).
constexpr int kStages = 6;
constexpr uint32_t kPanelBytes = kRows * 128;      // 64 rows x 64 bf16, 128-byte swizzle
constexpr uint32_t kOperandBytes = 2 * kPanelBytes;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kSlots = 2;
constexpr int kEpiWarp0 = 2, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kOutBytes = 32 * 128;           // 32 rows of 128 bytes: one TMA store of an epilogue warp
constexpr uint32_t kOutTotal = kEpiWarps * kOutBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kOutTotal + 1024 /*align*/ + 256 /*barriers*/;
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(kSlots * kTile <= 512, "TMEM columns");

struct Smem {
  uint64_t full[kStages];       // even CTA: both CTAs' copies of the stage landed
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
  int E, splits, num_n, num_k, tiles, accumulate;
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
// (each element by one box, so sums do not depend on an order; this addition
// takes subnormal numbers as zero).
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
// This thread's stores have read their shared memory.
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The bounded wait, with one answer for the whole warp: a lane that gave up
// takes the others along.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const KernelCtl& ctl, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, ctl, abort_flag)) != 0;
}

// A box into this CTA's shared memory whose bytes are counted on an mbarrier of
// the pair, given by its shared::cluster address.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

struct Tile {
  int e, z, n0, k0;  // expert, matrix of the output, first n and k
  int64_t lo;        // the expert's first row
  int rows;          // its rows, and the part [begin, end) of them to sum
  int begin, end;
};
__device__ __forceinline__ Tile tile_of(const Params& p, int t) {
  Tile o;
  const int per = p.num_n * p.num_k;
  o.z = t / per;
  const int r = t - o.z * per;
  o.n0 = (r % p.num_n) * kTile;
  o.k0 = (r / p.num_n) * kTile;
  o.e = o.z;
  if (p.splits > 1) {
    const int split = o.z / p.E;
    o.e = o.z - split * p.E;
    expert_rows(p.offsets, p.R, o.e, o.lo, o.rows);
    const int stages = (o.rows + kRows - 1) / kRows;
    o.begin = (int)((int64_t)stages * split / p.splits) * kRows;
    o.end = min((int)((int64_t)stages * (split + 1) / p.splits) * kRows, o.rows);
  } else {
    expert_rows(p.offsets, p.R, o.e, o.lo, o.rows);
    o.begin = 0;
    o.end = o.rows;
  }
  return o;
}

template <typename W>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_pair_kernel(const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_yt, const __grid_constant__ CUtensorMap tmap_xt,
                      const __grid_constant__ CUtensorMap tmap_w, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_smem = smem + kStages * kStageBytes;
  Smem* sm = reinterpret_cast<Smem*>(out_smem + kOutTotal);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();  // 0: issues the pair's MMAs
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
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
    prefetch_tmap(&tmap_yt);
    prefetch_tmap(&tmap_xt);
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
  pdl_wait();  // from here on global memory: operands come from the previous kernel
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort_flag = &sm->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t leader_full = mapa_shared(smem_u32(&sm->full[0]), 0);
    uint32_t stage = 0, phase = 0;
    int issued[kStages];
    uint32_t issued_phase[kStages];
    for (int s = 0; s < kStages; ++s) issued[s] = 0, issued_phase[s] = 0;
    bool alive = true;
    for (int t = cid; t < p.tiles && alive; t += ncl) {
      const Tile w = tile_of(p, t);
      for (int r0 = w.begin; r0 < w.end; r0 += kRows) {
        if (!warp_wait(smem_u32(&sm->empty[stage]), phase ^ 1, p.ctl, abort_flag)) {
          alive = false;
          break;
        }
        const uint32_t y = smem_u32(smem + stage * kStageBytes), x = y + kOperandBytes;
        const uint32_t full = leader_full + stage * 8;
        const bool tail = w.rows - r0 < kRows;
        const int32_t row = tail ? w.e * kRows : (int32_t)w.lo + r0;
        const CUtensorMap* ym = tail ? &tmap_yt : &tmap_y;
        const CUtensorMap* xm = tail ? &tmap_xt : &tmap_x;
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm->full[stage]), 2 * kStageBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tma_load_2d_pair(y + i * kPanelBytes, ym, (w.n0 + rank * kHalf + i * 64) * 2, row, full);
            tma_load_2d_pair(x + i * kPanelBytes, xm, (w.k0 + rank * kHalf + i * 64) * 2, row, full);
          }
        }
        issued[stage] = 1;
        issued_phase[stage] = phase;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    // drain: every copy of the pair has landed before its CTAs exit (they leave
    // together).  The odd CTA sees no count of its own: where it gave up, it
    // leaves its copies a time far beyond any copy's.
    if (!alive) {
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) __nanosleep(1000);
    }
    if (lane == 0 && rank == 0) {
      KernelCtl drain = p.ctl;
      for (int s = 0; s < kStages; ++s)
        if (issued[s]) mbar_wait(smem_u32(&sm->full[s]), issued_phase[s], drain, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t stage = 0, phase = 0;
      // ---------------------------------------------------------- MMA issuer
      uint32_t done = 0;
      bool alive = true;
      for (int t = cid; t < p.tiles && alive; t += ncl) {
        const Tile w = tile_of(p, t);
        if (w.begin >= w.end) continue;
        const uint32_t slot = done % kSlots, sphase = (done / kSlots) & 1;
        if (!warp_wait<true>(smem_u32(&sm->slot_empty[slot]), sphase ^ 1, p.ctl, abort_flag)) break;
        ++done;
        const uint32_t d = tmem + slot * kTile;
        for (int r0 = w.begin; r0 < w.end; r0 += kRows) {
          if (!warp_wait<true>(smem_u32(&sm->full[stage]), phase, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t y = smem_u32(smem + stage * kStageBytes), x = y + kOperandBytes;
#pragma unroll
            for (uint32_t s = 0; s < kRows / 16; ++s)
              mma_bf16_pair(d, operand_desc(y, s), operand_desc(x, s), r0 != w.begin || s != 0 ? 1u : 0u);
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
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                  // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;   // column half of the slot
    const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16) + h * 128;
    const uint32_t leader_slot_empty = mapa_shared(smem_u32(&sm->slot_empty[0]), 0);
    uint8_t* line = out_smem + (warp - kEpiWarp0) * kOutBytes;
    constexpr int kCols = 128 / (int)sizeof(W);  // columns of one store
    uint32_t done = 0;
    for (int t = cid; t < p.tiles; t += ncl) {
      const Tile w = tile_of(p, t);
      const int n0 = w.n0 + rank * kHalf + q * 32;
      const int k0 = w.k0 + h * 128;
      const uint32_t slot = done % kSlots, sphase = (done / kSlots) & 1;
      const bool some = w.begin < w.end;
      if (some) {
        ++done;
        if (!warp_wait(smem_u32(&sm->slot_full[slot]), sphase, p.ctl, abort_flag)) break;
        tc_fence_after();
      } else if (p.accumulate) {
        continue;
      }
#pragma unroll
      for (int c = 0; c < 128 / kCols; ++c) {
        if (lane == 0) tma_store_wait_read();  // the last store has read the buffer
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i) {  // 16 columns at a time
          uint32_t r[16];
          if (some) {
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
        if (some && c == 128 / kCols - 1) {  // the slot's columns of this warp are all read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader_slot_empty + slot * 8);
        }
        fence_proxy_async_smem();  // the TMA store reads what these threads wrote
        __syncwarp();
        const int k = k0 + c * kCols;
        if (lane == 0) {
          if (n0 < p.N && k < p.K) tma_store_3d(&tmap_w, smem_u32(line), k, n0, w.z, p.accumulate != 0);
          tma_store_commit();
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

namespace {

// dW = the sum of its splits' parts in their order (added to what it holds,
// when accumulating); 4 elements per thread.
constexpr int kJoinThreads = 256;

template <typename W>
__global__ void __launch_bounds__(kJoinThreads)
    wgrad_join_kernel(const float4* __restrict__ parts, int splits, int64_t n4, int accumulate, W* __restrict__ dw) {
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  if (i >= n4) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (sizeof(W) == 4)
    if (accumulate) sum = reinterpret_cast<const float4*>(dw)[i];
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 v = __ldg(parts + s * n4 + i);
    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
  }
  if constexpr (sizeof(W) == 4) {
    reinterpret_cast<float4*>(dw)[i] = sum;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
    reinterpret_cast<uint2*>(dw)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                 *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// Where the tiles leave more than half of the CTA pairs idle and the experts'
// rows are many, the rows are split, so that tiles times splits fill the pairs,
// and the parts are joined by another launch (about 5 us, worth 16 stages).
int split_count(int64_t R, int64_t N, int64_t K, int E) {
  if (E <= 0 || N <= 0 || K <= 0) return 1;
  const int64_t tiles = E * ceil_div(N, kTile) * ceil_div(K, kTile), stages = R / E / kRows;
  const int64_t splits = std::min<int64_t>({num_sms() / 2 / tiles, stages / 4, 64});
  return splits >= 2 && stages - stages / splits >= 16 ? (int)splits : 1;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

// The restored rows, the tails of x and d_y, the parts of split sums.
size_t wgrad_workspace_bytes(int64_t R, int64_t N, int64_t K, int E) {
  const int splits = split_count(R, N, K, E);
  return align256((size_t)R * K * 2) + align256((size_t)E * kRows * K * 2) + align256((size_t)E * kRows * N * 2) +
         (splits > 1 ? (size_t)splits * E * N * K * sizeof(float) : 0);
}

namespace {

// dw: [splits * E, N, K].
template <typename W>
q4_status launch_typed(const WgradArgs& a, W* dw, int splits, cudaStream_t stream) {
  RestoreArgs r = {a.codes, a.scales, a.tokens, a.K, a.row_token, a.offsets, a.R, a.E};
  r.dy = static_cast<const __nv_bfloat16*>(a.dy), r.N = a.N, r.ldy = a.ldy;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  r.x = reinterpret_cast<__nv_bfloat16*>(ws);
  ws += align256((size_t)a.R * a.K * 2);
  r.x_tail = reinterpret_cast<__nv_bfloat16*>(ws);
  ws += align256((size_t)a.E * kRows * a.K * 2);
  r.y_tail = reinterpret_cast<__nv_bfloat16*>(ws);
  Params p = {};
  p.R = a.R, p.N = a.N, p.K = a.K;
  p.offsets = a.offsets;
  p.E = a.E, p.splits = splits;
  p.accumulate = splits == 1 && a.accumulate;
  const int64_t num_n = ceil_div(a.N, kTile), num_k = ceil_div(a.K, kTile);
  if (num_n * num_k > INT32_MAX / 2 / a.E / splits) return Q4_ERR_UNSUPPORTED_SHAPE;
  p.num_n = (int)num_n, p.num_k = (int)num_k, p.tiles = (int)(splits * a.E * num_n * num_k);
  p.ctl = KernelCtl{device_status_ptr(), wait_budget_ns()};

  CUtensorMap ty, tx, yt, xt, tw;
  q4_status st = make_tmap_2d_u8(&ty, a.dy, a.N * 2, a.R, a.ldy * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_2d_u8(&tx, r.x, a.K * 2, a.R, a.K * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_2d_u8(&yt, r.y_tail, a.N * 2, (uint64_t)a.E * kRows, a.N * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_2d_u8(&xt, r.x_tail, a.K * 2, (uint64_t)a.E * kRows, a.K * 2, 128, kRows, true);
  if (st != Q4_OK) return st;
  st = make_tmap_3d(&tw, sizeof(W) == 4 ? Q4_F32 : Q4_BF16, dw, a.K, a.N, (uint64_t)splits * a.E, a.K, a.N * a.K, 128 / sizeof(W), 32,
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

  const int64_t rows_out = a.R + (int64_t)a.E * kRows, units = a.K / 8;
  const int64_t per_row = std::min<int64_t>(kRestoreThreads, ceil_div(ceil_div(units, kRestoreUnits), 32) * 32);
  const int64_t rows_per = kRestoreThreads / per_row;
  st = launch_pdl(wgrad_restore_kernel,
                  dim3((unsigned)ceil_div(units, per_row * kRestoreUnits),
                       (unsigned)std::min<int64_t>(ceil_div(rows_out, rows_per), 65535)),
                  dim3((unsigned)per_row, (unsigned)rows_per), 0, stream, r, rows_out);
  if (st != Q4_OK) return st;
  cfg.gridDim = dim3(2u * (unsigned)std::min(p.tiles, max_pairs[dev]), 1, 1);
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, wgrad_pair_kernel<W>, ty, tx, yt, xt, tw, p));
  return Q4_OK;
}

}  // namespace

q4_status launch_wgrad(const WgradArgs& a, cudaStream_t stream) {
  const int splits = split_count(a.R, a.N, a.K, a.E);
  if (splits == 1)
    return a.w_dtype == Q4_F32 ? launch_typed(a, static_cast<float*>(a.dw), 1, stream)
                               : launch_typed(a, static_cast<__nv_bfloat16*>(a.dw), 1, stream);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  float* parts = reinterpret_cast<float*>(ws + align256((size_t)a.R * a.K * 2) + align256((size_t)a.E * kRows * a.K * 2) +
                                          align256((size_t)a.E * kRows * a.N * 2));
  q4_status st = launch_typed(a, parts, splits, stream);
  if (st != Q4_OK) return st;
  const int64_t n4 = a.E * a.N * a.K / 4;
  const unsigned grid = (unsigned)ceil_div(n4, kJoinThreads);
  if (a.w_dtype == Q4_F32)
    return launch_pdl(wgrad_join_kernel<float>, grid, kJoinThreads, 0, stream, reinterpret_cast<const float4*>(parts),
                      splits, n4, (int)a.accumulate, static_cast<float*>(a.dw));
  return launch_pdl(wgrad_join_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, stream,
                    reinterpret_cast<const float4*>(parts), splits, n4, 0, static_cast<__nv_bfloat16*>(a.dw));
}

}  // namespace q4
