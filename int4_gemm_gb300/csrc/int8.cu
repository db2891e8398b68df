// Product of 8-bit integers with one scale per row of either operand:
//   C[m, n] = sa[m] sb[n] sum over k of qa[m, k] qb[n, k]
// with exact 32-bit integer sums.
//
// It runs on this GPU's f16 tensor cores, which are far faster than its
// integer ones: an 8-bit integer is an f16 number, a product of two (at most
// 2^14) and the FP32 sum of 1024 of them (at most 2^24) are exact, and every
// 1024 columns the sum is added to a 32-bit integer.  The weights are the M
// operand of the MMA, its rows the tensor memory's lanes:
//   warp 0       TMA producer: 128 columns of the weight rows and of the tokens
//                per stage, as 8-bit codes;
//   warps 4..    converters, groups of four that take turns of 64 columns:
//                a thread reads its weight row's 64 codes and stores them as f16
//                in tensor memory, the MMA's A operand; the tokens' codes go to
//                shared memory as f16, swizzled, the B operand.  (With both
//                operands in shared memory its 128 bytes per clock would bound
//                the product: 96 KB per 64 columns of a 256 x 256 tile instead of
//                64 KB.)
//   warp 1       MMA issuer: two halves of the tile's tokens one after another,
//                each into one of three accumulator slots, so that a slot is read
//                while the next ones are filled;
//   last eight   promotion: slot -> 32-bit integers in registers, then scales and
//                stores.
// Large products run on CTA pairs (256 weight rows x 256 tokens, cta_group::2),
// the others on single CTAs (128 weight rows x 16 to 128 tokens) whose K range is
// split over a cluster where there are few tiles; the integer sums then meet in
// distributed shared memory.
//
// Measured: 8192 x 28672 x 8192 2030 us (1895 TFLOP/s: the tensor pipe, at the rate of
// a library product in bf16), 4096 x 4864 x 4096 98.8 us (1653 TFLOP/s), 256 x 8192 x 8192
// 38.5 us (891 TFLOP/s: the conversion, 268 ns per 64 columns of a 128-token tile), 1 x
// 8192 x 8192 17.6 us (3.8 TB/s: 9.9 us of reading at the copy rate, the rest start, join
// and stores).
#include <algorithm>
#include <atomic>
#include <cstddef>

#include "common.cuh"
#include "elem.cuh"
#include "int8_plan.h"
#include "internal.h"

namespace q4 {
namespace {

// ------------------------------------------------------------------ product
constexpr int kSegmentK = 512;    // columns of half a run: a run's sums, of 1024 columns, are exact in FP32
constexpr int kConvSlots = 4;     // slots of converted weights and tokens
constexpr int kAccSlots = 3;      // accumulator slots of kHalf tokens
constexpr int kMaxStages = 12;
constexpr uint32_t kWeightBytes = kRows * kStageK;
constexpr int kConvWarp0 = 4, kPromWarps = 8;
// Registers per thread after the launch, which gives every thread the same: the
// warps that issue copies and MMAs, the converters, the promotion (Cut::prom_regs).
constexpr int kIssueRegs = 48, kConvRegs = 64;
constexpr uint32_t kSmemTotal = 232448;
constexpr uint32_t kSmemRing = kSmemTotal - 1024 /*align*/ - 512 /*barriers*/;

struct Smem {
  uint64_t full[kMaxStages];        // the stage's codes landed
  uint64_t empty[kMaxStages];       // the converters have read it
  uint64_t conv_full[kConvSlots];   // converted (on a pair's even CTA: the odd CTA's part too, by its relay)
  uint64_t conv_empty[kConvSlots];  // its MMAs are done
  uint64_t acc_full[kAccSlots];
  uint64_t acc_empty[kAccSlots];    // (pair: on the even CTA, by both)
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) <= 512, "barrier block");

struct Params {
  int64_t M, N, K;
  const float *sa, *sb;
  void* C;
  int c_dtype;
  int num_m, num_n, splits;  // tiles of tokens and weight rows; K parts (cluster size, single CTAs)
  KernelCtl ctl;
};

// tcgen05.mma kind::f16: FP32 accumulator (bits 4-5 = 1), f16 A and B (0), both
// K-major, N / 8 in bits 17-22, M / 16 in bits 24-28.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t M, uint32_t N) { return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24); }

template <bool kPair>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair)
    tc_commit_pair_mc(bar, 3);
  else
    tc_commit(bar);
}

// The bounded wait, with one answer for the whole warp.
template <bool kCluster>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const KernelCtl& ctl, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, ctl, abort_flag)) != 0;
}

// One lane of a converged warp.  Its branch is known to be taken by one thread, so
// that the operands of MMAs in it can stay in uniform registers: behind a test of
// the lane number every MMA took 180 clocks to issue instead of 60.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <int kRegs>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 16 consecutive TMEM columns of the warp's 32 lanes from registers
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Four 8-bit integers as f16, exactly: the byte b = q + 128 below the exponent of
// 1024 is 1024 + b, and 1152 less is q.
__device__ __forceinline__ uint2 int8x4_to_f16(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 offset = __half2half2(__ushort_as_half(0x6480));
  const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), offset);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), offset);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A lane's scales of a tile: its weight row's, and those of the tokens lane, lane +
// 32, ...  Single CTAs load them when the tile begins, behind whose sums their way
// from memory hides (256 x 8192 x 8192 40.1 -> 38.6 us, 1 x 128 x 128 4.35 -> 4.10);
// pairs, which have no registers for them until the sums are complete, then.
template <int kCols>
struct Scales {
  float weight, token[(kCols + 31) / 32];
  __device__ __forceinline__ void load(const Params& p, int64_t m0, int64_t n, int cols, int lane) {
    weight = n < p.N ? __ldg(p.sb + n) : 0.f;
#pragma unroll
    for (int i = 0; i < (kCols + 31) / 32; ++i) token[i] = i * 32 + lane < cols ? __ldg(p.sa + m0 + i * 32 + lane) : 0.f;
  }
};

// Tokens m0 .. m0 + cols - 1 of one weight row n per lane: 32 consecutive outputs
// of a token per store.  The tokens' scales come from the lanes that loaded them.
template <int kCols, typename C>
__device__ __forceinline__ void store_columns_as(C* out, const Params& p, int64_t m0, int64_t n, int cols, const Scales<kCols>& scales,
                                                 const int (&v)[kCols]) {
  out += m0 * p.N + n;
#pragma unroll
  for (int j = 0; j < kCols; ++j) {
    const float s = __shfl_sync(0xffffffffu, scales.token[j / 32], j & 31);
    if (n < p.N && j < cols) out[0] = to_elem<C>((float)v[j] * s * scales.weight);
    out += p.N;
  }
}

// The same for one CTA's share of a tile whose K parts lie in the shared memory of
// the cluster's kParts CTAs, part[weight row][token]: groups of four tokens of one
// weight row per lane, `first`, first + step and so on (a warp's at most 32 tokens;
// lane l has the scale of the l-th).  A load from another CTA takes some 1000
// clocks, so several are in flight.
template <int kParts, typename C>
__device__ __forceinline__ void join_columns_as(const Params& p, uint32_t row_smem, int64_t m0, int64_t n, int cols, int first,
                                                int step, float token_scale, float weight_scale) {
  constexpr int kFlight = 8 / kParts;
  C* out = static_cast<C*>(p.C) + m0 * p.N + n;
  for (int c0 = 4 * first, at = 0; c0 < cols; c0 += 4 * step * kFlight, at += 4 * kFlight) {
    int x[kFlight][kParts][4];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int c = c0 + 4 * step * f;
      if (c >= cols) break;
#pragma unroll
      for (int r = 0; r < kParts; ++r)
        asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[f][r][0]), "=r"(x[f][r][1]), "=r"(x[f][r][2]), "=r"(x[f][r][3])
                     : "r"(mapa_shared(row_smem + 4 * c, (uint32_t)r)));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int v = 0;
#pragma unroll
        for (int r = 0; r < kParts; ++r) v += x[f][r][i];
        const int c = c0 + 4 * step * f + i;
        const float s = __shfl_sync(0xffffffffu, token_scale, at + 4 * f + i);
        if (c < cols && n < p.N) out[c * p.N] = to_elem<C>((float)v * s * weight_scale);
      }
  }
}
template <int kParts>
__device__ __forceinline__ void join_columns(const Params& p, uint32_t row_smem, int64_t m0, int64_t n, int cols, int first,
                                             int step, float token_scale, float weight_scale) {
  if (p.c_dtype == Q4_BF16)
    join_columns_as<kParts, __nv_bfloat16>(p, row_smem, m0, n, cols, first, step, token_scale, weight_scale);
  else
    join_columns_as<kParts, float>(p, row_smem, m0, n, cols, first, step, token_scale, weight_scale);
}

// What a CTA holds of a tile: kHalf tokens per accumulator slot, kHalves slots.
template <bool kPair, int kHalf, int kHalves>
struct Cut {
  static constexpr int width = kHalf * kHalves;            // tokens of a tile
  static constexpr int own = kPair ? width / 2 : width;    // of which this CTA holds
  static constexpr int box = kPair ? kHalf / 2 : kHalf;    // tokens of one copy
  static constexpr uint32_t stage_bytes = kWeightBytes + own * kStageK;
  // columns per conversion: with few tokens two panels, whose MMAs are short, so
  // that the waits and commits around them count half (1 token x 8192 x 8192: 21.5
  // us with one)
  static constexpr int panels = kHalf <= 64 ? 2 : 1;
  static constexpr int per_stage = kStageK / (panels * kPanel);  // conversions per stage
  static constexpr int segment = kSegmentK / (panels * kPanel);  // conversions per half run
  static constexpr uint32_t panel_bytes = own * 128;
  static constexpr uint32_t f16_bytes = panels * panel_bytes;  // converted tokens per slot
  static constexpr uint32_t acc_columns = kHalf <= 64 ? 64 : 128;
  static constexpr uint32_t tmem_a = kAccSlots * acc_columns;  // first column of the converted weights
  static constexpr uint32_t a_columns = panels * kPanel / 2;
  static_assert(tmem_a + kConvSlots * a_columns <= 512, "TMEM columns");
  // groups of four converter warps: more where small accumulators leave registers
  // for them, since the weights' way through a group takes 800 clocks per chunk
  // whatever the tokens, and HBM brings 64 columns in 350
  static constexpr int groups = kHalf > 64 ? 2 : kHalves == 1 ? 4 : 3;
  static constexpr int conv_slots = own > 128 ? 2 : groups == 3 ? 3 : kConvSlots;
  static constexpr int fit = (kSmemRing - conv_slots * f16_bytes) / stage_bytes;
  static constexpr int stages = fit < kMaxStages ? fit : kMaxStages;
  static constexpr int prom_warp0 = kConvWarp0 + 4 * groups;
  static constexpr int threads = (prom_warp0 + kPromWarps) * 32;
  static constexpr int prom_regs = kHalf <= 64 ? 96 : 152;
  static constexpr int launch_regs = 65536 / threads / 8 * 8;
  static_assert(kIssueRegs + groups * kConvRegs + 2 * prom_regs <= (1 + groups + 2) * launch_regs, "registers");
  // a group that has waited for its conversion slot knows that the chunks up to
  // conv_slots before its own are done, so that neither of its two waits can take
  // an older phase of the barrier for its own
  static_assert(conv_slots >= groups && stages * per_stage >= conv_slots, "phases");
  static_assert(stages >= 3 && f16_bytes % 1024 == 0 && stage_bytes % 1024 == 0, "shared memory");
};

template <bool kPair, int kHalf, int kHalves>
__global__ void __launch_bounds__((Cut<kPair, kHalf, kHalves>::threads), 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_t, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem* sm = reinterpret_cast<Smem*>(smem + kSmemRing);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  using T = Cut<kPair, kHalf, kHalves>;
  uint8_t* f16_smem = smem + T::stages * T::stage_bytes;
  const int units = kPair ? gridDim.x >> 1 : gridDim.x / p.splits;
  const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x / p.splits;
  const int tiles = p.num_m * p.num_n;
  const int KB = (int)((p.K + kStageK - 1) / kStageK);
  const int kb0 = kPair ? 0 : (int)((int64_t)KB * rank / p.splits);  // this CTA's stages
  const int kb1 = kPair ? KB : (int)((int64_t)KB * (rank + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 4 * T::per_stage);
    }
    for (int s = 0; s < kConvSlots; ++s) {
      mbar_init(smem_u32(&sm->conv_full[s]), kPair && rank == 0 ? 5 : 4);
      mbar_init(smem_u32(&sm->conv_empty[s]), 1);
    }
    for (int s = 0; s < kAccSlots; ++s) {
      mbar_init(smem_u32(&sm->acc_full[s]), 1);
      mbar_init(smem_u32(&sm->acc_empty[s]), kPair ? 8 : 4);
    }
    mbar_init(smem_u32(&sm->mma_done), 1);
    sm->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_t);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(&sm->tmem_base), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&sm->tmem_base), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_barrier_sync();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  pdl_wait();  // from here on global memory: operands come from the previous kernel
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort_flag = &sm->abort;
  auto tile_mn = [&](int t, int64_t& m0, int64_t& n0) {
    const Tile at = tile_at(t, T::width, p.num_m, p.num_n);
    m0 = (int64_t)at.m * T::width;
    n0 = (int64_t)at.n * (kPair ? 2 * kRows : kRows) + (kPair ? rank * kRows : 0);
  };

  if (warp < kConvWarp0) {
    registers_down<kIssueRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t stage = 0, phase = 0, count = 0;
      bool alive = true;
      for (int t = unit; t < tiles && alive; t += units) {
        int64_t m0, n0;
        tile_mn(t, m0, n0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!warp_wait<false>(smem_u32(&sm->empty[stage]), phase ^ 1, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          if (lane == 0) {
            const uint32_t dst = smem_u32(smem + stage * T::stage_bytes), full = smem_u32(&sm->full[stage]);
            mbar_arrive_expect_tx(full, T::stage_bytes);
            tma_load_2d(dst, &tmap_w, kb * kStageK, (int32_t)n0, full);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              tma_load_2d(dst + kWeightBytes + h * T::box * kStageK, &tmap_t, kb * kStageK,
                          (int32_t)m0 + h * kHalf + (kPair ? rank * T::box : 0), full);
          }
          ++count;
          if (++stage == T::stages) stage = 0, phase ^= 1;
        }
      }
      // drain: every copy has landed before the CTA exits
      if (lane == 0) {
        KernelCtl drain = p.ctl;
        constexpr uint32_t S = T::stages;
        for (uint32_t g = count > S ? count - S : 0u; g < count; ++g)
          mbar_wait(smem_u32(&sm->full[g % S]), (g / S) & 1, drain, nullptr);
      }
      __syncwarp();
    } else if (warp == 1 && (!kPair || rank == 0)) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = mma_desc(kPair ? 2 * kRows : kRows, kHalf);
      constexpr uint32_t half_bytes = T::panel_bytes / kHalves;
      const uint64_t desc0 = smem_desc(smem_u32(f16_smem), 16, 1024, 2);  // 128-byte swizzle, 8-row groups 1024 bytes apart
      const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0), bar0 = smem_u32(&sm->conv_full[0]);
      const uint32_t acc_full0 = smem_u32(&sm->acc_full[0]), acc_empty0 = smem_u32(&sm->acc_empty[0]);
      constexpr uint32_t kToEmpty = offsetof(Smem, conv_empty) - offsetof(Smem, conv_full);
      // the issue path counts: a 64-column chunk's MMAs run for 512 clocks (256 x 256),
      // and every uniform operation in front of them takes some ten
      uint32_t slot = 0, phase = 0;
      uint32_t acc[2] = {0, 0}, next_acc = 0, next_phase = 1;  // each half's slot; the next one, parity of its wait
      bool alive = true;
      auto chunk_wait = [&]() {
        alive = warp_wait<kPair>(bar0 + slot * 8, phase, p.ctl, abort_flag);
        tc_fence_after();
        return alive;
      };
      auto next_chunk = [&]() {
        __syncwarp();
        if (++slot == T::conv_slots) slot = 0, phase ^= 1;
      };
      // one half's MMAs of the chunk in `slot`; the first of a run overwrite
      auto half = [&](int h, bool first) {
        const uint64_t b = desc0 + (slot * T::f16_bytes + h * half_bytes) / 16;
        const uint32_t d = tmem_u + acc[h] * T::acc_columns, a = tmem_u + T::tmem_a + slot * T::a_columns;
#pragma unroll
        for (uint32_t k = 0; k < T::panels * kPanel / 16; ++k)
          mma_f16<kPair>(d, a + k * 8, b + k / 4 * (T::panel_bytes / 16) + k % 4 * 2, idesc, !first || k != 0 ? 1u : 0u);
      };
      for (int t = unit; t < tiles && alive; t += units) {
        int seg = 0;
        for (int left = T::per_stage * (kb1 - kb0); left > 0 && alive; left -= T::segment, ++seg) {
          const int n = min(left, T::segment);  // chunks of this segment
          // the second half's runs begin one segment apart from the first's, so
          // that their slots are read at different times
          const bool begins[2] = {seg % 2 == 0, seg % 2 == 1 || seg == 0};
          const bool ends[2] = {seg % 2 == 1 || left <= T::segment, seg % 2 == 0 || left <= T::segment};
          if (!chunk_wait()) break;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            if (begins[h]) {
              if (!warp_wait<kPair>(acc_empty0 + next_acc * 8, next_phase, p.ctl, abort_flag)) {
                alive = false;
                break;
              }
              tc_fence_after();
              acc[h] = next_acc;
              if (++next_acc == kAccSlots) next_acc = 0, next_phase ^= 1;
            }
            if (elect_one()) {
              half(h, begins[h]);
              if (n == 1 && ends[h]) commit<kPair>(acc_full0 + acc[h] * 8);
              if (h == kHalves - 1) commit<kPair>(bar0 + kToEmpty + slot * 8);
            }
            __syncwarp();
          }
          if (!alive) break;
          next_chunk();
#pragma unroll 1
          for (int i = 1; i < n; ++i) {
            if (!chunk_wait()) break;
            if (elect_one()) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h) {
                half(h, false);
                if (i == n - 1 && ends[h]) commit<kPair>(acc_full0 + acc[h] * 8);  // the run is complete
              }
              commit<kPair>(bar0 + kToEmpty + slot * 8);
            }
            next_chunk();
          }
        }
      }
      // every MMA (of this thread, the same one throughout) is complete before TMEM
      // is released
      if (elect_one()) {
        if constexpr (kPair)
          tc_commit_pair_mc(smem_u32(&sm->mma_done), 1);
        else
          tc_commit(smem_u32(&sm->mma_done));
      }
      __syncwarp();
      KernelCtl drain = p.ctl;
      mbar_wait(smem_u32(&sm->mma_done), 0, drain, nullptr);
      __syncwarp();
    } else if (kPair && warp == 1) {
      // ---------------------------------------------------------- relay (odd CTA)
      // hands over the tokens' f16 in this CTA's shared memory, which the even CTA's
      // MMAs read (an arrival with .release.cluster: 8192 x 28672 x 8192 3478 us instead
      // of 2050)
      const uint32_t leader_full = mapa_shared(smem_u32(&sm->conv_full[0]), 0);
      uint32_t slot = 0, phase = 0;
      bool alive = true;
      for (int t = unit; t < tiles && alive; t += units) {
        for (int i = 0; i < T::per_stage * (kb1 - kb0); ++i) {
          if (!warp_wait<false>(smem_u32(&sm->conv_full[slot]), phase, p.ctl, abort_flag)) {
            alive = false;
            break;
          }
          if (lane == 0) mbar_arrive_cluster_smem(leader_full + slot * 8);
          if (++slot == T::conv_slots) slot = 0, phase ^= 1;
        }
      }
      __syncwarp();
    }
  } else if (warp < T::prom_warp0) {
    // ------------------------------------------------------------ converters
    registers_down<kConvRegs>();
    const int group = (warp - kConvWarp0) >> 2, q = warp & 3;
    static_assert(T::groups % T::per_stage == 0, "a group takes the same part of its stages");
    constexpr int kStep = T::groups / T::per_stage;  // a group takes every kStep-th stage
    const int sub = group % T::per_stage;            // which of its parts
    uint32_t at_stage = group / T::per_stage;        // stages since the start
    int tile = unit, kb = kb0 + group / T::per_stage;
    bool alive = true;
    for (;;) {
      while (kb >= kb1 && tile < tiles) kb -= kb1 - kb0, tile += units;
      if (tile >= tiles || !alive) break;
      {
        const uint32_t stage = at_stage % T::stages, phase = (at_stage / T::stages) & 1;
        const uint32_t chunk = T::per_stage * at_stage + sub, slot = chunk % T::conv_slots;
        if (!warp_wait<kPair>(smem_u32(&sm->conv_empty[slot]), ((chunk / T::conv_slots) & 1) ^ 1, p.ctl, abort_flag) ||
            !warp_wait<false>(smem_u32(&sm->full[stage]), phase, p.ctl, abort_flag)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint8_t* raw = smem + stage * T::stage_bytes;
        // this thread's weight row: 64 codes per panel, two halves of 16 TMEM columns
        constexpr int kPieces = T::panels * 4;  // of 16 codes
        {
          const int r = q * 32 + lane;
          const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + T::tmem_a + slot * T::a_columns;
#pragma unroll
          for (int j0 = 0; j0 < kPieces; j0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = *reinterpret_cast<const uint4*>(raw + r * kStageK + (((sub * kPieces + j0 + j) ^ (r & 7)) << 4));
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              uint32_t o[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4& x = v[j + i / 4];
                const uint2 f = int8x4_to_f16((i & 3) == 0 ? x.x : (i & 3) == 1 ? x.y : (i & 3) == 2 ? x.z : x.w);
                o[2 * i] = f.x;
                o[2 * i + 1] = f.y;
              }
              tmem_st_x16(at + (j0 + j) * 8, o);
            }
          }
        }
        // tokens: a warp takes 8 rows of four 16-code pieces at a time, four times
        // in flight
        const int r0 = q * 8 + (lane & 7), j = lane >> 3;
        constexpr int kTurns = (T::own + 31) / 32, kFlight = kTurns < 4 ? kTurns : 4;
#pragma unroll
        for (int pan = 0; pan < T::panels; ++pan) {
          const uint8_t* from = raw + kWeightBytes + r0 * kStageK + (((sub * kPieces + pan * 4 + j) ^ (lane & 7)) << 4);
          uint8_t* to = f16_smem + slot * T::f16_bytes + pan * T::panel_bytes + r0 * 128;
#pragma unroll
          for (int u = 0; u < kTurns; u += kFlight) {
            uint4 x[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
              if (T::own >= 32 || q * 8 < T::own) x[i] = *reinterpret_cast<const uint4*>(from + (u + i) * 32 * kStageK);
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
              if (T::own < 32 && q * 8 >= T::own) continue;
              const uint2 f0 = int8x4_to_f16(x[i].x), f1 = int8x4_to_f16(x[i].y), f2 = int8x4_to_f16(x[i].z), f3 = int8x4_to_f16(x[i].w);
              *reinterpret_cast<uint4*>(to + (u + i) * 32 * 128 + (((2 * j) ^ (lane & 7)) << 4)) = make_uint4(f0.x, f0.y, f1.x, f1.y);
              *reinterpret_cast<uint4*>(to + (u + i) * 32 * 128 + (((2 * j + 1) ^ (lane & 7)) << 4)) = make_uint4(f2.x, f2.y, f3.x, f3.y);
            }
          }
        }
        tmem_st_wait();
        fence_proxy_async_smem();  // the tensor cores read what these threads wrote
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm->empty[stage]));
          mbar_arrive(smem_u32(&sm->conv_full[slot]));
        }
        at_stage += kStep, kb += kStep;
      }
    }
  } else {
    // ------------------------------------------------------------ promotion + store
    registers_up<T::prom_regs>();
    const int q = warp & 3;                     // TMEM lane quarter this warp may access
    const int h = (warp - T::prom_warp0) >> 2;  // half of the tile's tokens
    const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t leader_empty = kPair ? mapa_shared(smem_u32(&sm->acc_empty[0]), 0) : smem_u32(&sm->acc_empty[0]);
    const int segs = (T::per_stage * (kb1 - kb0) + T::segment - 1) / T::segment;
    const int runs = h == 0 ? (segs + 1) / 2 : 1 + segs / 2;
    uint32_t begun = 0;  // runs begun before this tile, in the order in which they take slots
    bool alive = h < kHalves;
    const bool split = !kPair && p.splits > 1;
    // of a split tile: its weight row's scale, and one of the tokens that the warp joins
    const int join_first = 2 * rank + h, join_step = 2 * p.splits;
    float token_scale = 0.f, weight_scale = 0.f;
    if (split) {
      int64_t m0, n0;
      tile_mn(unit, m0, n0);
      const int64_t n = n0 + q * 32 + lane, m = m0 + 4 * (join_first + join_step * (lane >> 2)) + (lane & 3);
      weight_scale = n < p.N ? __ldg(p.sb + n) : 0.f;
      token_scale = m < p.M ? __ldg(p.sa + m) : 0.f;
    }
    int sum[kHalf];
    for (int t = unit; t < tiles && alive; t += units) {
      int64_t m0, n0;
      tile_mn(t, m0, n0);
      m0 += h * kHalf;
      const int64_t n = n0 + q * 32 + lane;
      const int cols = (int)min((int64_t)kHalf, p.M - m0);
      Scales<kHalf> scales;
      if (!kPair && !split) scales.load(p, m0, n, cols, lane);
#pragma unroll
      for (int j = 0; j < kHalf; ++j) sum[j] = 0;
      for (int run = 0; run < runs; ++run) {
        // two runs begin with a tile's first segment, one with every other
        const uint32_t g = begun + (kHalves == 1 ? run : run == 0 ? h : 2 * run + 1 - h), a = g % kAccSlots;
        if (!warp_wait<kPair>(smem_u32(&sm->acc_full[a]), (g / kAccSlots) & 1, p.ctl, abort_flag)) {
          alive = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kHalf / 16; ++c) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(t_lane + a * T::acc_columns + c * 16, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c * 16 + j] += __float2int_rn(__uint_as_float(r[j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair)
            mbar_arrive_cluster(leader_empty + a * 8);
          else
            mbar_arrive(leader_empty + a * 8);
        }
      }
      begun += kHalves == 1 ? (segs + 1) / 2 : segs + 1;
      if (!alive) break;
      if (!split) {
        if (kPair) scales.load(p, m0, n, cols, lane);
        if (p.c_dtype == Q4_BF16)
          store_columns_as<kHalf>(static_cast<__nv_bfloat16*>(p.C), p, m0, n, cols, scales, sum);
        else
          store_columns_as<kHalf>(static_cast<float*>(p.C), p, m0, n, cols, scales, sum);
      }
    }
    if (split) {
      // the cluster's parts of one tile meet in shared memory, which no copy and no
      // MMA uses any more (this CTA's are complete: the last sums were read)
      int64_t m0, n0;
      tile_mn(unit, m0, n0);
      constexpr int kPitch = T::width + 4;
      const uint32_t row = smem_u32(smem) + (uint32_t)((q * 32 + lane) * kPitch * 4);
      if (h < kHalves) {
#pragma unroll
        for (int j = 0; j < kHalf; j += 4)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (uint32_t)((h * kHalf + j) * 4)), "r"(sum[j]),
                       "r"(sum[j + 1]), "r"(sum[j + 2]), "r"(sum[j + 3])
                       : "memory");
      }
      cluster_barrier_sync();  // every part is there
      const int cols = (int)min((int64_t)T::width, p.M - m0);
      if (!*abort_flag) {
        const int64_t n = n0 + q * 32 + lane;
        if (p.splits == 2)
          join_columns<2>(p, row, m0, n, cols, join_first, join_step, token_scale, weight_scale);
        else
          join_columns<4>(p, row, m0, n, cols, join_first, join_step, token_scale, weight_scale);
      }
      cluster_barrier_sync();  // no CTA leaves while another reads its part
    }
  }
  // (the promotion warps of a split tile meet the cluster's others above; what
  // follows is short enough for every warp's registers)
  if (!kPair && p.splits > 1 && warp < T::prom_warp0) {
    cluster_barrier_sync();
    cluster_barrier_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_barrier_sync();  // the pair's MMAs are complete in both CTAs
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
  if (kPair) cluster_barrier_sync();  // no CTA leaves while its peer may still arrive on its barriers
}

template <bool kPair, int kHalf, int kHalves>
q4_status launch_plan(const Plan& s, const int8_t* qa, const int8_t* qb, const Params& p, cudaStream_t stream) {
  using T = Cut<kPair, kHalf, kHalves>;
  const auto kernel = int8_gemm_kernel<kPair, kHalf, kHalves>;
  CUtensorMap tw, tt;
  q4_status st;
  if ((st = make_tmap_2d_u8(&tw, qb, p.K, p.N, p.K, kStageK, kRows, true)) != Q4_OK) return st;
  if ((st = make_tmap_2d_u8(&tt, qa, p.K, p.M, p.K, kStageK, T::box, true)) != Q4_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return Q4_ERR_CUDA;
  // CTAs that are resident at once (single CTAs: one per SM), 0 before the device's
  // first call; written once all is set up, since calls come from several threads
  static std::atomic<int> resident[64];
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(T::threads, 1, 1);
  cfg.dynamicSmemBytes = kSmemTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)(kPair ? 2 : s.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int ctas = resident[dev].load(std::memory_order_acquire);
  if (!ctas) {
    Q4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal));
    ctas = num_sms();
    if (kPair) {  // persistent: as many pairs as are resident at once
      int n = 0;
      cfg.gridDim = dim3((unsigned)(ctas / 2 * 2), 1, 1);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) n = ctas / 2;
      ctas = 2 * std::min(n, ctas / 2);
    }
    resident[dev].store(ctas, std::memory_order_release);
  }
  const int tiles = s.num_m * s.num_n;
  const int grid = kPair ? 2 * std::min(tiles, ctas / 2) : s.splits > 1 ? tiles * s.splits : std::min(tiles, ctas);
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, tw, tt, p));
  return Q4_OK;
}

}  // namespace

q4_status launch_int8_gemm(const int8_t* qa, const float* sa, const int8_t* qb, const float* sb, int64_t M, int64_t N, int64_t K,
                           void* C, int c_dtype, cudaStream_t stream) {
  const Plan s = plan_of(M, N, K, num_sms());
  Params p = {};
  p.M = M; p.N = N; p.K = K;
  p.sa = sa; p.sb = sb; p.C = C; p.c_dtype = c_dtype;
  p.num_m = s.num_m; p.num_n = s.num_n; p.splits = s.splits;
  p.ctl = KernelCtl{device_status_ptr(), wait_budget_ns()};
  if (s.pair) return launch_plan<true, 128, 2>(s, qa, qb, p, stream);
  if (s.width == 16) return launch_plan<false, 16, 1>(s, qa, qb, p, stream);
  if (s.width == 32) return launch_plan<false, 32, 1>(s, qa, qb, p, stream);
  if (s.width == 64) return launch_plan<false, 64, 1>(s, qa, qb, p, stream);
  return launch_plan<false, 64, 2>(s, qa, qb, p, stream);
}

}  // namespace q4
