// What kernels that hold whole rows share (the norm, its gradient, the INT8
// quantizer): rows spread over threads, their reduction, and a ring of rows in
// shared memory.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "ring_rows.h"

namespace q4 {
namespace {

// 8 of the 128 columns of a block, held by one of 16 lanes: with 128-bit accesses
// (kVec) columns 8 l .. 8 l + 7 of lane l, otherwise l, l + 16, ..., 16-bit
// elements one per word.  Columns past the block's end are zero.
template <typename T, bool kVec>
struct Piece {
  static constexpr bool packed = kVec && sizeof(T) == 2;
  static constexpr int words = packed ? 4 : 8;
  uint32_t w[words];

  // cols <= 0: no column.
  __device__ __forceinline__ void load(const T* p, int l, int cols) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < words / 4; ++i) {
        const uint4 v = 8 * l < cols ? reinterpret_cast<const uint4*>(p + 8 * l)[i] : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if (cols >= 128) {  // no test per element
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = one(p + l + 16 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = l + 16 * i < cols ? one(p + l + 16 * i) : 0u;
    }
  }
  static __device__ __forceinline__ uint32_t one(const T* p) {
    if constexpr (sizeof(T) == 2)
      return *reinterpret_cast<const unsigned short*>(p);
    else
      return __float_as_uint(*p);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (packed) {
      const float2 v = unpack2<T>(w[i / 2]);
      return i & 1 ? v.y : v.x;
    } else if constexpr (sizeof(T) == 2) {
      return unpack2<T>(w[i]).x;
    } else {
      return __uint_as_float(w[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, int l, int cols, const float (&f)[8]) {
    if constexpr (kVec) {
      if (8 * l >= cols) return;
      uint4* out = reinterpret_cast<uint4*>(p + 8 * l);
      if constexpr (sizeof(T) == 4) {
        out[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        out[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      } else {
        out[0] = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
      }
    } else if (cols >= 128) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[l + 16 * i] = to_elem<T>(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (l + 16 * i < cols) p[l + 16 * i] = to_elem<T>(f[i]);
    }
  }
  // Eight codes: bytes 0..3 in c.x, 4..7 in c.y.
  static __device__ __forceinline__ void store_codes(uint8_t* p, int l, int cols, uint2 c) {
    if constexpr (kVec) {
      if (8 * l < cols) *reinterpret_cast<uint2*>(p + 8 * l) = c;
    } else if (cols >= 128) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[l + 16 * i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (l + 16 * i < cols) p[l + 16 * i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
  }
};

// The low byte of v f rounded to the nearest integer (even at ties), |v f| < 2^22:
// adding 1.5 * 2^23 leaves the integer in the low bits of the sum.
__device__ __forceinline__ uint32_t int8_bits(float v, float f) { return __float_as_uint(fmaf(v, f, 12582912.f)); }
__device__ __forceinline__ uint2 int8x8(const float (&v)[8], float f) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __byte_perm(int8_bits(v[4 * i], f), int8_bits(v[4 * i + 1], f), 0x0040);
    const uint32_t hi = __byte_perm(int8_bits(v[4 * i + 2], f), int8_bits(v[4 * i + 3], f), 0x0040);
    o[i] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(o[0], o[1]);
}

// The weights of a piece (columns c + ...), T or FP32; all 1 without weights.
template <typename T, bool kVec>
__device__ __forceinline__ void load_weights(const void* w, bool w32, int c, int l, int cols, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w32) {
    Piece<float, kVec> p;
    p.load(static_cast<const float*>(w) + c, l, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = p.at(i);
  } else {
    Piece<T, kVec> p;
    p.load(static_cast<const T*>(w) + c, l, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = p.at(i);
  }
}

// The larger of two, and NaN where one of them is (fmaxf drops it): a NaN among a
// row's values reaches its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (sum, largest) over the `group` threads that hold a row, in every one of them.
// Groups of more than a warp are whole warps of a block that comes here together;
// buf alternates between two buffers from row to row, so that one barrier per row
// is enough.
struct Exchange {
  __align__(16) float2 part[2][32];
};
// Groups of a block that the exchange has room for: up to four warps each take four
// slots, up to eight eight, larger ones all of them; within a warp there is no exchange.
constexpr int most_groups(int group) { return group <= 32 ? 64 : group <= 128 ? 8 : group <= 256 ? 4 : 1; }
// Before the first row: parts that no warp writes are zero.
__device__ __forceinline__ void exchange_init(Exchange& ex) {
  if (threadIdx.x < 64) ex.part[threadIdx.x >> 5][threadIdx.x & 31] = make_float2(0.f, 0.f);
}
template <bool kTop>
__device__ __forceinline__ float2 group_reduce(float sum, float top, int group, Exchange& ex, int buf) {
  if (group >= 32) {
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (kTop) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 16));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (kTop) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (group > 32) {
    const int lane = threadIdx.x & 31, warps = group >> 5, warp = threadIdx.x >> 5;
    const int slots = warps <= 4 ? 4 : 8, first = warp / warps * slots;
    if (lane == 0) ex.part[buf][warps <= 8 ? first + warp % warps : warp] = make_float2(sum, top);
    __syncthreads();
    if (warps <= 8) {  // few enough for every thread to add them up
      const float4* part = reinterpret_cast<const float4*>(ex.part[buf] + first);
      float4 v[4];
      v[0] = part[0], v[1] = part[1];
      v[2] = v[3] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slots == 8) v[2] = part[2], v[3] = part[3];
      sum = ((v[0].x + v[0].z) + (v[1].x + v[1].z)) + ((v[2].x + v[2].z) + (v[3].x + v[3].z));
      if (kTop) top = max_nan(max_nan(max_nan(v[0].y, v[0].w), max_nan(v[1].y, v[1].w)), max_nan(max_nan(v[2].y, v[2].w), max_nan(v[3].y, v[3].w)));
    } else {
      const float2 v = ex.part[buf][lane];
      sum = v.x, top = v.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (kTop) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
    }
  }
  return make_float2(sum, top);
}

// Threads of a block for kC pieces per thread.
constexpr int max_threads(int C) { return C == 1 ? 1024 : 512; }

// Which row and columns a thread holds: `group` threads per row, the block's
// groups one row each, piece i of thread t the 128-column block t / 16 + i *
// (group / 16).
struct Place {
  int l, t, group, per_block, sub, stride;
  __device__ __forceinline__ explicit Place(int group_)
      : l(threadIdx.x & 15), t(threadIdx.x % group_), group(group_), per_block(blockDim.x / group_), sub(threadIdx.x / group_),
        stride(group_ >> 4) {}
  __device__ __forceinline__ int block(int i) const { return (t >> 4) + i * stride; }
  __device__ __forceinline__ int at(int i) const { return block(i) * 128; }
  // columns of piece i of a row of H (0: a row that is not there)
  __device__ __forceinline__ int cols(int i, int H) const { return min(128, H - at(i)); }
  // Whether C pieces of every thread lie inside a row of H.
  __device__ __forceinline__ bool whole(int C, int H) const { return C * stride * 128 == H; }
};

// ------------------------------------------------------------------ rows through shared memory
constexpr int kMaxRing = 8;
// A ring of stages, each the block's next per_block rows of up to three matrices.
struct Ring {
  uint64_t full[kMaxRing];
  int abort;
};
struct RingArgs {
  int stages, edge;  // edge: rows at either end that are read in place
  uint32_t stage_bytes, row_bytes;
  KernelCtl ctl;
};

__device__ __forceinline__ void ring_init(Ring& ring, const RingArgs& r, Exchange& ex) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < r.stages; ++s) mbar_init(smem_u32(&ring.full[s]), 1);
    ring.abort = 0;
    fence_mbar_init();
  }
  exchange_init(ex);
  __syncthreads();
}

// Bytes of a row in a stage.
template <bool kVec>
__host__ __device__ constexpr uint32_t staged_row(uint32_t row_bytes) {
  return kVec ? row_bytes : window_bytes(row_bytes);
}

// One thread: rows base .. of the matrices into stage s, but for those that are read
// in place.
template <bool kVec, int kMats>
__device__ __forceinline__ void ring_fill(Ring& ring, const RingArgs& r, uint32_t smem, int s, const void* const (&mat)[kMats],
                                          const int64_t (&pitch)[kMats], int64_t base, int64_t rows, int per_block) {
  if (base >= rows) return;
  const uint32_t bar = smem_u32(&ring.full[s]), staged = staged_row<kVec>(r.row_bytes);
  const uint32_t dst = smem + s * r.stage_bytes;
  if constexpr (kVec) {
    const int n = (int)min((int64_t)per_block, rows - base);
    int mats = 0;
    for (int m = 0; m < kMats; ++m) mats += mat[m] != nullptr;
    mbar_arrive_expect_tx(bar, (uint32_t)(mats * n) * staged);
    for (int m = 0; m < kMats; ++m) {
      if (!mat[m]) continue;
      const uint8_t* src = static_cast<const uint8_t*>(mat[m]) + base * pitch[m];
      const uint32_t to = dst + (uint32_t)(m * per_block) * staged;
      if (pitch[m] == r.row_bytes)
        bulk_load(to, src, (uint32_t)n * staged, bar);
      else
        for (int i = 0; i < n; ++i) bulk_load(to + i * staged, src + i * pitch[m], staged, bar);
    }
  } else {
    const CopiedRows c = copied_rows(base, per_block, rows, r.edge);
    const int n = c.end - c.begin;
    const uint32_t first = dst + (uint32_t)c.begin * staged;
    base += c.begin;
    uint32_t bytes = 0;
    for (int turn = 0; turn < 2; ++turn) {  // the bytes first, then the copies
      if (turn) mbar_arrive_expect_tx(bar, bytes);
      for (int m = 0; m < kMats; ++m) {
        if (!mat[m]) continue;
        for (int i = 0; i < n; ++i) {
          const Window w = window_of(reinterpret_cast<uintptr_t>(mat[m]) + (base + i) * pitch[m], r.row_bytes);
          if (turn)
            bulk_load(first + (uint32_t)(m * per_block + i) * staged, reinterpret_cast<const void*>(w.begin), w.size, bar);
          else
            bytes += w.size;
        }
      }
    }
  }
}

// Whether a stage's phase is over, so that it may be filled again (it is not where a
// wait ran out).
__device__ __forceinline__ bool ring_over(Ring& ring, int stage, uint32_t phase) {
  return mbar_try_wait(smem_u32(&ring.full[stage]), phase);
}
// After the last row: where a wait ran out, the block stays for as long again, so that
// copies still on their way end before its memory is another's.
__device__ __forceinline__ void ring_end(Ring& ring, const RingArgs& r) {
  if (threadIdx.x == 0 && *static_cast<volatile int*>(&ring.abort)) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 <= r.ctl.wait_ns) {
    }
  }
}

// A row of a matrix in its stage.
template <bool kVec, typename T>
__device__ __forceinline__ const T* ring_row(const uint8_t* stage, const RingArgs& r, int m, const Place& pl, const void* mat,
                                             int64_t pitch, int64_t row) {
  const uint8_t* p = stage + (uint32_t)(m * pl.per_block + pl.sub) * staged_row<kVec>(r.row_bytes);
  if (!kVec) p += (reinterpret_cast<uintptr_t>(mat) + row * pitch) & 15;
  return reinterpret_cast<const T*>(p);
}

// The weights of a thread's pieces as they were loaded, 16-bit ones packed (as
// FP32 in shared memory, from where every row took them, 20 to 30% slower).  FP32
// weights of 16-bit rows are read from global memory every time.
template <typename T, bool kVec, int kC>
struct HeldWeights {
  Piece<T, kVec> w[kC];
  const void* p;
  bool held;
  __device__ __forceinline__ HeldWeights(const void* weight, int w_dtype, const Place& pl, int H)
      : p(weight), held(!weight || sizeof(T) == 4 || w_dtype != Q4_F32) {
    constexpr uint32_t kOne = sizeof(T) == 4 ? 0x3f800000u : std::is_same<T, __half>::value ? 0x3c003c00u : 0x3f803f80u;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (weight && held) {
        w[i].load(static_cast<const T*>(weight) + pl.at(i), pl.l, pl.cols(i, H));
      } else {
#pragma unroll
        for (int j = 0; j < Piece<T, kVec>::words; ++j) w[i].w[j] = kOne;
      }
    }
  }
  template <bool kHeld>
  __device__ __forceinline__ void get(const Place& pl, int H, int i, float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = w[i].at(j);
    if (!kHeld && !held) load_weights<T, kVec>(p, true, pl.at(i), pl.l, pl.cols(i, H), f);
  }
};

// How rows are spread: kC pieces per thread, threads per row and per block, blocks,
// and the ring's stages (0: none) and bytes.
struct Shape {
  int C, group, threads, grid, stages;
  uint32_t stage_bytes;
};
constexpr uint32_t kRingTotal = 216 * 1024;  // of an SM's shared memory
// Rows of `blocks` 128-column blocks, C pieces per thread, at most (where a row
// takes no more) most_threads threads.
inline Shape spread(int blocks, int C, int most_threads) {
  Shape s = {};
  s.C = C;
  const int halves = (int)ceil_div(blocks, C);  // groups of 16 lanes
  s.group = halves == 1 ? 16 : (halves + 1) / 2 * 32;
  s.threads = std::max(1, most_threads / s.group) * s.group;
  return s;
}

// Blocks per SM that the ring kernels are compiled for: single elements need many
// warps (the norm; the gradient keeps its rows in registers instead: 9973 x 1411 bf16,
// at the time, 42.3 us with two blocks, 58.7 with three, 46.2 with three that read
// their rows twice, 67.5 with one); of aligned rows, whose threads hold 32 elements,
// three blocks would spill (34 us instead of 26 for 4096 x 7168 to INT8).
__host__ __device__ constexpr int resident_blocks(bool vec, int threads, bool gradient) {
  return threads > 256 ? 1 : vec || gradient ? 2 : 3;
}

// Rows go through the ring where its blocks have a turn each, aligned ones of the norm
// where every other block has (bf16, ring and straight: norm 256 x 8192 6.1 and 7.1 us,
// 600 x 8192 10.1 and 14.2, 1000 x 4096 7.5 and 12.1, but of one turn in four 256 x 4096
// 4.0 and 3.4; single elements 500 x 2047 4.8 and 4.1, 1500 x 2047 10.0 and 10.8;
// gradient 700 x 4096 13.8 and 15.7, 2000 x 2048 12.0 and 15.6, 400 x 4096 12.9 and 11.0).
inline Shape shape_of(int64_t rows, int64_t H, int mats, int size, bool vec, bool gradient) {
  const int blocks = (int)ceil_div(H, 128);
  const int64_t sms = num_sms();
  if (blocks <= (vec ? 128 : 32)) {
    Shape s = spread(blocks, !vec ? 2 : blocks >= 16 ? 4 : blocks >= 4 ? 2 : 1, 256);
    const int per_block = s.threads / s.group;
    const uint32_t row_bytes = (uint32_t)(H * size);
    s.stage_bytes = (uint32_t)(mats * per_block) * (vec ? staged_row<true>(row_bytes) : staged_row<false>(row_bytes));
    int resident = resident_blocks(vec, s.threads, gradient);
    while (resident > 1 && 2 * s.stage_bytes > kRingTotal / resident) --resident;
    s.stages = (int)std::min<int64_t>(kMaxRing, kRingTotal / resident / s.stage_bytes);
    s.grid = (int)std::min<int64_t>(ceil_div(rows, per_block), sms * resident);
    if (s.stages >= 2 && ceil_div(rows, per_block) * (vec && !gradient ? 2 : 1) >= sms * resident) return s;
  }
  int C = 1;
  const int most = rows <= 2 * sms ? 64 : 16;  // blocks of 128 columns that one piece per thread takes
  if (blocks > most) C = blocks > 128 ? 8 : 4;
  Shape s = spread(blocks, C, 128);
  s.grid = (int)std::min<int64_t>(ceil_div(rows, s.threads / s.group), sms * std::max(1, 1024 / s.threads));
  return s;
}

template <typename F>
q4_status by_pieces(int C, F&& f) {
  if (C == 1) return f(std::integral_constant<int, 1>());
  if (C == 2) return f(std::integral_constant<int, 2>());
  if (C == 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 8>());
}

// The kernel's shared memory is allowed once per device (calls come from several
// threads).
template <typename Kernel>
q4_status allow_smem(Kernel kernel, std::atomic<int> (&ready)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return Q4_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    Q4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingTotal));
    ready[dev].store(1, std::memory_order_release);
  }
  return Q4_OK;
}

RingArgs ring_of(const Shape& s, bool vec, int64_t row_bytes) {
  return RingArgs{s.stages, vec ? 0 : edge_rows((uint32_t)row_bytes), s.stage_bytes, (uint32_t)row_bytes,
                  KernelCtl{device_status_ptr(), wait_budget_ns()}};
}

}  // namespace
}  // namespace q4
